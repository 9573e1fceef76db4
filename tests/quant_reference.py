"""The 8-bit KV cache in 64-bit numpy, one sequence and block at a time: the format, the
quantising append, and attention over what is stored.  Shares no code with the package."""
from __future__ import annotations

import numpy as np

BLOCK = 16
E_MIN, E_MAX = -64, 64


def _code_values() -> np.ndarray:
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = -x if c & 128 else x
    v[0x7f] = v[0xff] = np.nan
    return v


VALUES = _code_values()          # value of each e4m3 code


def e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (ties to even, clamped to +-448, non-finite to NaN), as float64."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    a = np.minimum(np.abs(np.where(ok, x, 0.0)), 448.0)
    _, k = np.frexp(a)
    step = np.exp2(np.maximum(k - 1, -6) - 3.0)
    y = np.copysign(np.minimum(np.rint(a / step) * step, 448.0), x)
    return np.where(ok, y, np.nan)


def half_step(x: np.ndarray) -> np.ndarray:
    """Half the spacing of the e4m3 values around x: the largest rounding error."""
    _, k = np.frexp(np.minimum(np.abs(x), 448.0))
    return np.exp2(np.maximum(k - 1, -6) - 4.0)


def exponent(amax: float) -> int:
    """The smallest e in [E_MIN, E_MAX] with amax <= 448 * 2^e (E_MAX when none is)."""
    for e in range(E_MIN, E_MAX):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def finite_amax(x: np.ndarray) -> float:
    a = np.abs(x[np.isfinite(x)])
    return float(a.max()) if a.size else 0.0


class Sequence:
    """One KV head of one tensor of one sequence: code values [rows, D], exponents [blocks]."""

    def __init__(self, rows: int, D: int):
        self.v = np.full((rows, D), np.nan)      # value of each code
        self.e = np.zeros((rows + BLOCK - 1) // BLOCK, dtype=np.int64)

    def append(self, x: np.ndarray, start: int, exponents=None):
        """Rows x [n, D] at positions start, start + 1, ...  exponents: the block exponents to
        use in place of the rule's (for inputs known up to rounding)."""
        n = x.shape[0]
        at = start
        while at < start + n:
            blk, j0 = divmod(at, BLOCK)
            end = min(start + n, (blk + 1) * BLOCK)
            part = x[at - start:end - start]
            e = exponent(finite_amax(part)) if exponents is None else int(exponents[blk])
            if j0:
                e = max(e, int(self.e[blk]))
                if e > self.e[blk]:
                    rows = slice(blk * BLOCK, at)
                    self.v[rows] = e4m3(self.v[rows] * 2.0 ** float(self.e[blk] - e))
            self.v[at:end] = e4m3(part * 2.0 ** float(-e))
            self.e[blk] = e
            at = end

    def stored(self, lo: int, hi: int) -> np.ndarray:
        pos = np.arange(lo, hi)
        return self.v[lo:hi] * np.exp2(self.e[pos // BLOCK].astype(np.float64))[:, None]


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray) -> np.ndarray:
    """softmax(q k^T) v in 64 bits: q [G, D], k and v [n, D]; zeros when n == 0."""
    if k.shape[0] == 0:
        return np.zeros_like(q)
    s = q @ k.T
    w = np.exp(s - s.max(axis=1, keepdims=True))
    return (w / w.sum(axis=1, keepdims=True)) @ v


def attend_tolerance(q: np.ndarray, k: np.ndarray, v: np.ndarray) -> float:
    """Bound on an fp32 evaluation's error: a score sums D products in fp32 along at most 40
    roundings in sequence (each up to 2^-24 of the sum of magnitudes), a weight's relative
    error is twice the score's, weights carry at least 16 bits, and the output is an average
    of values of magnitude at most max |v|."""
    if k.shape[0] == 0:
        return 0.0
    s_err = 40 * 2.0 ** -24 * float((np.abs(q) @ np.abs(k).T).max())
    return (2 * s_err + 2.0 ** -16) * float(np.abs(v).max())
