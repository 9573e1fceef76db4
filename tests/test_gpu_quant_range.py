"""8-bit decode attention where scores are far beyond what fp32 resolves to a unit, and where
queries and key scales lie at the ends of their ranges.

Only one channel of q is not zero, so a score is one product and exact to its last rounding, the
same in every position that holds the same key.  The positions that win do so by a sixth of their
score and more: every other weight is zero, the winners' are equal, and the output is the mean of
their values.  Tolerance: weights carry 22 bits, the sums of at most 3 values, 1 / l and the last
product one rounding each, together below 2^-20 of the largest value.
"""
import numpy as np
import pytest
import torch

from tests import quant_reference as ref
from tests.test_gpu_quant import E4M3, GEO, filled, run_decode

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

CHANNEL = 7
CODE = {float(v): c for c, v in enumerate(ref.VALUES) if np.isfinite(v)}


def batch(layer, many):
    """Lengths of segments in one piece, in several, and split over many units; `many`: enough
    segments for the smaller units."""
    lens = [17, 700, 5000, 1]
    if many:
        B = 24 if layer == "sliding" else 80
        lens += [(37 * i) % 150 + 1 for i in range(B - len(lens))]
    return lens


class RandomCache:
    """Random codes and value scales 2^(2 spread) apart, contiguous or paged."""

    def __init__(self, geo, B, S, paged, seed, spread):
        self.KVH, self.D, self.B, self.S, self.paged = geo["KVH"], geo["D"], B, S, paged
        nblk = (S + 15) // 16
        self.table = None
        shape, sshape = (B, S, self.KVH, self.D), (B, nblk, self.KVH)
        if paged:
            table = np.random.default_rng(seed).permutation(B * nblk + 2)[:B * nblk].reshape(B, nblk)
            self.table = torch.from_numpy(table.astype(np.int32)).cuda()
            shape, sshape = (B * nblk + 2, 16, self.KVH, self.D), (B * nblk + 2, self.KVH)
        rng = np.random.default_rng(seed)
        self.codes, self.scales = [], []
        for t in range(2):
            g = torch.Generator(device="cuda").manual_seed(seed * 2 + t)
            self.codes.append((torch.randn(shape, generator=g, device="cuda") * 60).to(E4M3))
            e = rng.integers(-spread, spread + 1, sshape) - 6
            self.scales.append(torch.tensor(np.exp2(e.astype(np.float64)), device="cuda").float())

    @property
    def args(self):
        return (*self.codes, *self.scales)


def one_channel_keys(cache, lens, q7, exponent, seed):
    """Keys whose channel 7 decides: winners (up to three per sequence and head, in blocks of
    their own) and losers, in the order of the sign of q7.  One winner's block has twice the
    scale and half the codes.  Returns the positions of the largest score, [b][h], by what is
    stored (a scale above 2^64 counts as 2^64)."""
    rng = np.random.default_rng(seed)
    S, KVH = cache.S, cache.KVH
    best = 256.0 if q7 > 0 else 128.0
    losers = [x for x in CODE if (16 <= x <= 208 if q7 > 0 else 160 <= x <= 448)]
    nblk = (S + 15) // 16
    values = np.zeros((cache.B, nblk * 16, KVH))
    exps = np.full((cache.B, nblk, KVH), exponent)
    for b, L in enumerate(lens):
        for h in range(KVH):
            values[b, :S, h] = rng.choice(losers, S)
            blocks = rng.permutation((L + 15) // 16)[:rng.integers(1, 4)]
            at = sorted(int(min(16 * k + rng.integers(0, 16), L - 1)) for k in blocks)
            values[b, at, h] = best
            if len(blocks) > 1:             # the same keys, coded another way
                k = at[0] // 16
                exps[b, k, h] += 1
                values[b, 16 * k:16 * k + 16, h] /= 2
    score = values * np.exp2(np.minimum(exps, ref.E_MAX).astype(float)).repeat(16, 1) * np.sign(q7)
    won = [[np.flatnonzero(score[b, :L, h] == score[b, :L, h].max()) for h in range(KVH)]
           for b, L in enumerate(lens)]
    order = sorted(CODE)
    as_codes = np.array([CODE[x] for x in order], np.uint8)[np.searchsorted(order, values)]
    as_codes, scales = torch.from_numpy(as_codes).cuda(), torch.from_numpy(np.exp2(exps.astype(float))).cuda()
    codes = cache.codes[0].view(torch.uint8)
    if cache.paged:
        codes[cache.table.long(), :, :, CHANNEL] = as_codes.view(cache.B, nblk, 16, KVH)
        cache.scales[0][cache.table.long()] = scales.float()
    else:
        codes[..., CHANNEL] = as_codes[:, :S]
        cache.scales[0].copy_(scales)
    return won


def check_winners(cache, out, won):
    G = out.shape[1] // cache.KVH
    got = out.double().cpu().numpy()
    for b in range(len(won)):
        for h in range(cache.KVH):
            at = torch.from_numpy(won[b][h]).cuda()
            if cache.paged:
                pages = cache.table[b].long()[at // 16]
                codes, scales = cache.codes[1].view(torch.uint8)[pages, at % 16, h], cache.scales[1][pages, h]
            else:
                codes, scales = cache.codes[1].view(torch.uint8)[b, at, h], cache.scales[1][b, at // 16, h]
            v = ref.VALUES[codes.cpu().numpy()] * scales.double().cpu().numpy()[:, None]
            worst = float(np.abs(got[b, h * G:(h + 1) * G] - v.mean(0)).max() / np.abs(v).max())
            assert worst <= 2.0 ** -20, (b, h, won[b][h])


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_beyond_fp32_units(layer, many, sign):
    """Scores of 2^25 to 2^100 at the winners, of either sign, over value scales 2^24 apart: as
    fp32 tells them apart, and finite."""
    geo, lens = GEO[layer], batch(layer, many)
    for i, (score, exponent) in enumerate([(2.0 ** 25, 0), (6e7, 20), (1e8, 0), (2.0 ** 27, 40),
                                           (1.5e9, 64), (2.0 ** 60, 20), (2.0 ** 100, 64)]):
        cache = RandomCache(geo, len(lens), max(lens), many, 301 + i, 12)
        q = torch.zeros((len(lens), geo["H"], geo["D"]), dtype=torch.bfloat16, device="cuda")
        q7 = sign * score / (256.0 if sign > 0 else 128.0) * 2.0 ** -exponent
        q[..., CHANNEL] = q7
        won = one_channel_keys(cache, lens, q7, exponent, 311 + i)
        out = run_decode(cache, q, lens, 0, out_dtype=torch.float32)
        assert int(torch.isfinite(out).logical_not().sum()) == 0, (score, exponent)
        check_winners(cache, out, won)


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_queries_and_key_scales_at_opposite_ends(layer, many, sign):
    """The largest queries with the smallest key scales, and tiny queries with the largest: the
    scores are finite fp32 numbers, whatever their factors' sizes."""
    geo, lens = GEO[layer], batch(layer, many)
    for i, (q7, exponent) in enumerate([(1.5 * 2.0 ** 127, -64), (2.0 ** 126, -63), (2.0 ** 115, -20),
                                        (2.0 ** -62, 63), (2.0 ** -61, 62)]):
        cache = RandomCache(geo, len(lens), max(lens), many, 321 + i, 12)
        q = torch.zeros((len(lens), geo["H"], geo["D"]), dtype=torch.bfloat16, device="cuda")
        q[..., CHANNEL] = sign * q7
        won = one_channel_keys(cache, lens, sign * q7, exponent, 331 + i)
        out = run_decode(cache, q, lens, 0, out_dtype=torch.float32)
        assert int(torch.isfinite(out).logical_not().sum()) == 0, (q7, exponent)
        check_winners(cache, out, won)


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("small", [False, True])
def test_query_elements_far_below_their_heads_largest(layer, small):
    """The head's largest element meets zero codes, so that the others decide.  Down to 2^-31 of
    it they count exactly: attend_tolerance.  Below, each is off by at most 2^-39 of the largest,
    a score by that times the sum of |k|, a weight by twice as much."""
    geo, lens = GEO[layer], [200, 1500]
    cache = filled(geo, 2, 1500, False, seed=341, spread=1)
    cache.codes[0].view(torch.uint8)[..., CHANNEL] = 0
    g = torch.Generator(device="cuda").manual_seed(342)
    q = torch.rand((2, geo["H"], geo["D"]), generator=g, device="cuda") * 0.25 + 0.125
    q = torch.where(torch.rand(q.shape, generator=g, device="cuda") < 0.5, -q, q).bfloat16()
    if small:
        q = q * 2.0 ** -4
    q[..., CHANNEL] = 2.0 ** 28
    out = run_decode(cache, q, lens, 0, out_dtype=torch.float32).double().cpu().numpy()
    G, qd = geo["H"] // geo["KVH"], q.double().cpu().numpy()
    for b, L in enumerate(lens):
        for h in range(cache.KVH):
            cache.ref[0][b][h].v[:, CHANNEL] = 0.0
            k, v = (cache.ref[t][b][h].stored(0, L) for t in range(2))
            heads = qd[b, h * G:(h + 1) * G]
            tol = ref.attend_tolerance(heads, k, v)
            if small:
                tol += 2 * 2.0 ** (28 - 39) * float(np.abs(k).sum(1).max() * np.abs(v).max())
            worst = float(np.abs(out[b, h * G:(h + 1) * G] - ref.attend(heads, k, v)).max())
            assert worst <= tol, (b, h)
