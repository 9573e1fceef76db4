"""The 4-bit KV cache in 64-bit numpy: the format, coding and decoding of 32 channels, the
producer's formulas.  Shares no code with the package."""
from __future__ import annotations

import numpy as np

TOP, NAN = 0xA7, 0xFF
# the scale of each byte 0 .. TOP: an f16 number of three mantissa bits, no sign
SCALES = np.array([c * 2.0 ** -17 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 18)
                   for c in range(TOP + 1)])


def code_group(x: np.ndarray):
    """Scale bytes [...] and codes 1 .. 15 [..., 32] of values [..., 32]."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x).all(-1)
    x = np.where(ok[..., None], x, 0.0)
    amax = np.abs(x).max(-1)
    byte = np.minimum(np.searchsorted(7.5 * SCALES, amax), TOP)   # first with amax <= 7.5 s
    s = SCALES[byte][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.where(s > 0, np.floor(np.abs(x) / s + 0.5), 0.0)   # ties away from zero
    n = np.copysign(np.minimum(n, 7.0), x)
    return np.where(ok, byte, NAN), (n + 8).astype(np.int64)


def encode(k: np.ndarray, v: np.ndarray) -> np.ndarray:
    """Rows uint8 [..., planes, 272] of K and V [..., KVH, D]."""
    lead = k.shape[:-2]
    out = np.empty((*lead, k.shape[-2] * k.shape[-1] // 256, 272), dtype=np.uint8)
    for t, x in enumerate((k, v)):
        byte, u = code_group(x.reshape(*lead, -1, 8, 32))
        u = u.reshape(*lead, -1, 256)
        out[..., 128 * t:128 * t + 128] = u[..., 0::2] | (u[..., 1::2] << 4)
        out[..., 256 + 8 * t:264 + 8 * t] = byte
    return out


def decode(rows: np.ndarray, D: int):
    """K and V float64 [..., KVH, D] of rows uint8 [..., planes, 272]."""
    got = []
    for t in range(2):
        c = rows[..., 128 * t:128 * t + 128].astype(np.int64)
        u = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], 8, 32)
        b = rows[..., 256 + 8 * t:264 + 8 * t]
        s = np.where(b <= TOP, SCALES[np.minimum(b, TOP)], np.nan)
        got.append(((u - 8.0) * s[..., None]).reshape(*rows.shape[:-2], -1, D))
    return got


def norm_rope(x, w, pos, pairs, theta):
    """rope(x / rms(x) * w) of x [n, heads, D] at positions pos [n], in 64 bits (w None: no weight and
    no rotation)."""
    x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    if w is None:
        return x
    x = x * w
    D = x.shape[-1]
    a = pos[:, None, None] * theta ** (-2.0 * np.arange(pairs) / D)
    lo, hi = x[..., :pairs].copy(), x[..., D // 2:D // 2 + pairs].copy()
    x[..., :pairs] = lo * np.cos(a) - hi * np.sin(a)
    x[..., D // 2:D // 2 + pairs] = hi * np.cos(a) + lo * np.sin(a)
    return x


def bf16(x: np.ndarray) -> np.ndarray:
    """Finite values away from the ends of the range rounded to fp32 and from there to bf16, each to
    nearest even (the fp32 step counts where it ends on a tie)."""
    x = np.asarray(x).astype(np.float32).astype(np.float64)
    _, e = np.frexp(x)
    unit = np.exp2(e - 8.0)
    return np.rint(x / unit) * unit


def bf16_doubt(x: np.ndarray, rel: float) -> np.ndarray:
    """Whether a relative error of `rel` may change the bf16 number that x rounds to."""
    return bf16(x * (1 + rel)) != bf16(x * (1 - rel))
