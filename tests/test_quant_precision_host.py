"""The bound that the GPU tests hold the 8-bit decode kernel's weights to: a plain evaluation with
the kernel's roundings keeps it; weights of 16 or 11 bits and a position lost at either end
do not."""
import numpy as np
import pytest

from tests import quant_reference as ref
from tests.quant_precision import attend_and_bound


def case(rng, L, D, exact_scores):
    k = ref.e4m3(rng.standard_normal((L, D)) * 60) * 2.0 ** -6
    v = ref.e4m3(rng.standard_normal((L, D)) * 60) * 2.0 ** -6
    q = np.zeros((8, D))
    if exact_scores:
        q[:, 7] = [2.0, -2.0, 1.0, -1.0, 4.0, -4.0, 2.0, 0.5]
    else:
        q[:] = rng.standard_normal((8, D)) * 2 / np.sqrt(D)
    return q, k, v


def rounded(x, bits):
    """x to `bits` significant bits, to nearest."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


def evaluate(q, k, v, bits=22, drop=None):
    """fp32 scores and exponentials; the numerator's weights of `bits` bits; positions `drop` lost."""
    keep = np.ones(k.shape[0], bool)
    if drop is not None:
        keep[drop] = False
    k, v = k[keep], v[keep]
    x = (q.astype(np.float32) @ k.T.astype(np.float32)) * np.float32(np.log2(np.e))
    p = np.exp2((x - np.ceil(x.max(axis=1, keepdims=True))).astype(np.float64) + 12).astype(np.float32)
    return rounded(p.astype(np.float64), bits) @ v / p.sum(axis=1, dtype=np.float64)[:, None]


def kept(seed, L, D, exact_scores, **kw):
    q, k, v = case(np.random.default_rng(seed), L, D, exact_scores)
    o, bound = attend_and_bound(q, k, v, exact_scores)
    return bool(np.all(np.abs(evaluate(q, k, v, **kw) - o) <= bound))


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("exact_scores", [True, False])
def test_plain_evaluation_keeps_the_bound(D, exact_scores):
    for L in (1, 2, 3, 16, 17, 33, 100, 700, 2049):
        assert kept(L, L, D, exact_scores), L


@pytest.mark.parametrize("D", [256, 512])
def test_weights_of_16_bits_do_not(D):
    for L in (2, 3, 16, 17, 33):
        assert not kept(L, L, D, True, bits=16), L


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("exact_scores", [True, False])
def test_weights_of_one_f16_do_not(D, exact_scores):
    for L in (2, 3, 17, 33):
        assert not kept(L, L, D, exact_scores, bits=11), L


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("exact_scores", [True, False])
def test_a_lost_position_does_not(D, exact_scores):
    for L in (2, 17, 100, 700, 2049):
        for drop in (0, L - 1, L // 2):
            assert not kept(L, L, D, exact_scores, drop=drop), (L, drop)
