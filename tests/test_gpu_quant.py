"""GPU tests of the 8-bit KV cache (gqa_append_quant, gqa_read_quant,
gqa_prepare_decode_quant, gqa_decode_quant and their paged forms) against the 64-bit
reference in quant_reference.py.

Append: inputs are bf16 and scales are powers of two, so each code is one exact division
and one rounding; codes and scales must be equal.  Read: a code times a power of two is
exact in bf16 and fp32.  Producer: the kernel's fp32 values carry a relative error of a few
2^-24 of the largest (4e-6 on heads of unit RMS and weights up to 2), so a stored value lies within half a step
of the exact one plus that.  Decode: quant_reference.attend_tolerance, plus half a bf16
step for bf16 outputs.
"""
import numpy as np
import pytest
import torch

import decode_attention_gb300 as gqa
import oracle
from decode_attention_gb300 import inputs
from tests import quant_reference as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

GEO = {"sliding": inputs.SLIDING, "global": inputs.GLOBAL}
ROPE = {"sliding": (oracle.SLIDING_ROPE_PAIRS, oracle.SLIDING_ROPE_THETA),
        "global": (oracle.GLOBAL_ROPE_PAIRS, oracle.GLOBAL_ROPE_THETA)}
FILL = 0x35          # byte of rows that nothing may write
E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Cache:
    """An 8-bit cache on the GPU, contiguous or paged (pages in a random order), every byte and
    scale at a fill value, and its reference: one Sequence per (b, head, tensor)."""

    def __init__(self, geo, B, S, paged, seed=0):
        self.KVH, self.D, self.B, self.S, self.paged = geo["KVH"], geo["D"], B, S, paged
        nblk = (S + 15) // 16
        if paged:
            table = np.random.default_rng(seed).permutation(B * nblk + 2)[:B * nblk].reshape(B, nblk)
            self.host_table, self.P = table.astype(np.int32), B * nblk + 2
            self.table = i32(self.host_table)
            shape, sshape = (self.P, 16, self.KVH, self.D), (self.P, self.KVH)
        else:
            self.table = None
            shape, sshape = (B, S, self.KVH, self.D), (B, nblk, self.KVH)
        self.codes = [torch.full(shape, FILL, dtype=torch.uint8, device="cuda").view(E4M3) for _ in "kv"]
        self.scales = [torch.full(sshape, 3.0, device="cuda") for _ in "kv"]
        self.ref = [[[ref.Sequence(S, self.D) for _ in range(self.KVH)] for _ in range(B)] for _ in "kv"]
        for r in (r for x in self.ref for y in x for r in y):
            r.v[:] = ref.VALUES[FILL]
            r.e[:] = 1                       # the exponent field of the fill scale, 3.0
        self.written = np.zeros((B, S), dtype=bool)

    @property
    def args(self):
        return (*self.codes, *self.scales)

    def host(self, t):
        """(codes uint8 [B, S, KVH, D], scales [B, blocks, KVH]) of tensor t by position."""
        c, s = self.codes[t].view(torch.uint8).cpu().numpy(), self.scales[t].cpu().numpy()
        if self.paged:
            c = c[self.host_table].reshape(self.B, -1, self.KVH, self.D)[:, :self.S]
            s = s[self.host_table]
        return c, s

    def append(self, k_new, v_new, off, lens):
        """The call under test and the reference's own append."""
        a = (k_new, v_new, i32(off))
        if self.paged:
            gqa.gqa_append_quant_paged(*a, self.table, i32(lens), *self.args)
        else:
            gqa.gqa_append_quant(*a, i32(lens), *self.args)
        for t, x in enumerate((k_new, v_new)):
            x = x.double().cpu().numpy()
            for b in range(self.B):
                n = off[b + 1] - off[b]
                if n <= 0 or lens[b] < n or lens[b] > self.S:
                    continue
                self.written[b, lens[b] - n:lens[b]] = True
                for h in range(self.KVH):
                    self.ref[t][b][h].append(x[off[b]:off[b + 1], h], lens[b] - n)

    def check(self):
        torch.cuda.synchronize()
        for t in range(2):
            c, s = self.host(t)
            for b in range(self.B):
                w = self.written[b]
                assert np.all(c[b][~w] == FILL), "a row that was not appended changed"
                blocks = sorted(set(np.flatnonzero(w) // 16))
                rest = [i for i in range(s.shape[1]) if i not in blocks]
                assert np.all(s[b][rest] == 3.0)
                for h in range(self.KVH):
                    r = self.ref[t][b][h]
                    assert np.array_equal(s[b, blocks, h], np.exp2(r.e[blocks].astype(np.float64)))
                    assert np.array_equal(ref.VALUES[c[b][w, h]], r.v[w], equal_nan=True)
        if self.paged:
            used = set(self.host_table.ravel().tolist())
            for p in set(range(self.P)) - used:
                assert torch.all(self.codes[0].view(torch.uint8)[p] == FILL)


def rows(gen, shape, spread=0):
    """bf16 rows; with spread > 0 each (row, head) is scaled by 2^u, u uniform in +-spread."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if spread:
        x = x * torch.exp2((2 * torch.rand(shape[:-1], generator=gen, device="cuda") - 1) * spread)[..., None]
    return x.to(torch.bfloat16)


# ---------------------------------------------------------------------------- append

@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("spread", [0, 12])
def test_append_chunks(layer, paged, spread):
    """Chunks that start and end anywhere in a block, sequences without new tokens, a cache
    whose length is no whole number of blocks, filled to its last row."""
    geo, S = GEO[layer], 77
    gen = torch.Generator(device="cuda").manual_seed(11 + spread)
    have = [0, 1, 15, 16, 17, 40, 0, 76]
    cache = Cache(geo, len(have), S, paged, seed=3)
    for new in (have, [1, 0, 1, 16, 3, 37, 0, 1], [15, 30, 0, 1, 57, 0, 77, 0]):
        lens = have if new is have else [a + n for a, n in zip(have, new)]
        off = np.concatenate([[0], np.cumsum(new)]).tolist()
        n = (max(1, off[-1]), geo["KVH"], geo["D"])
        cache.append(rows(gen, n, spread), rows(gen, n, spread), off, lens)
        have = lens
    cache.check()


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_append_values_at_the_ends_of_the_range(layer):
    """Zeros, subnormals, the largest bf16, infinities and NaN, in rows of their own and mixed;
    a scale that grows by the whole range; values exactly at a scale's border."""
    geo = GEO[layer]
    KVH, D = geo["KVH"], geo["D"]
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = rows(gen, (64, KVH, D))
    x[0:16] = 0
    x[16, :, 3] = float("inf")
    x[17, :, 4] = float("-inf")
    x[18, :, 5] = float("nan")
    x[19] = float("nan")
    x[20] = float("inf")
    x[32] = 1e-39                      # subnormal
    x[33, :, 0] = 3.3e38
    x[34:48] = x[34:48] * 1e-20
    x[48:63] = 1.75 * 2.0 ** -3        # 448 * 2^-11 exactly
    x[63] = 1.7578125 * 2.0 ** -3      # the next bf16
    cache = Cache(geo, 1, 64, False)
    for lo, hi in ((0, 33), (33, 34), (34, 63), (63, 64)):
        cache.append(x[lo:hi], x[lo:hi].neg(), [0, hi - lo], [hi])
    cache.check()


def test_append_skips_what_does_not_fit():
    """Offsets outside [0, N], decreasing offsets, lengths below the new tokens or above the
    capacity, and a bad page: nothing of those is written, the rest is."""
    geo, S = GEO["sliding"], 48
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = rows(gen, (40, 16, 256))
    for paged in (False, True):
        off, lens = [0, 10, 20, 18, 28, 50, 40], [9, 49, 30, 20, 40, 35]
        #   b: 0 too short, 1 too long, 2 decreasing, 3 fine (18..28), 4 beyond N, 5 decreasing
        cache = Cache(geo, 6, S, paged)
        if paged:
            gqa.gqa_append_quant_paged(x, x, i32(off), cache.table, i32(lens), *cache.args)
        else:
            gqa.gqa_append_quant(x, x, i32(off), i32(lens), *cache.args)
        for t in range(2):
            for h in range(16):
                cache.ref[t][3][h].append(x[18:28, h].double().cpu().numpy(), 10)
        cache.written[3, 10:20] = True
        cache.check()
    cache = Cache(geo, 1, S, True)
    table = cache.table.clone()
    table[0, 1] = cache.P
    gqa.gqa_append_quant_paged(x, x, i32([0, 40]), table, i32([40]), *cache.args)
    for t in range(2):
        for h in range(16):
            cache.ref[t][0][h].append(x[:, h].double().cpu().numpy(), 0)
    cache.written[0, :16] = cache.written[0, 32:40] = True
    cache.check()


# ---------------------------------------------------------------------------- read

def filled(geo, B, S, paged, seed, spread=3, nan_rows=True):
    """A Cache whose bytes are random codes (NaN codes among them when nan_rows) with random
    scales; its reference holds the same."""
    cache = Cache(geo, B, S, paged, seed)
    rng = np.random.default_rng(seed)
    for t in range(2):
        g = torch.Generator(device="cuda").manual_seed(seed * 2 + t)
        c = (torch.randn(cache.codes[t].shape, generator=g, device="cuda") * 60).to(E4M3)
        cache.codes[t].view(torch.uint8).copy_(c.view(torch.uint8))
        e = rng.integers(-spread, spread + 1, cache.scales[t].shape) - 6
        cache.scales[t].copy_(torch.tensor(np.exp2(e.astype(np.float64))))
        hc, hs = cache.host(t)
        for b in range(B):
            for h in range(cache.KVH):
                cache.ref[t][b][h].v = ref.VALUES[hc[b, :, h]]
                cache.ref[t][b][h].e = np.log2(hs[b, :, h]).astype(np.int64)
    return cache


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read_back(layer, paged, dtype):
    geo = GEO[layer]
    lens, S = [0, 1, 16, 33, 61, 70, -3], 61       # 70 and -3 are clamped
    cache = filled(geo, len(lens), S, paged, seed=21)
    cap = 64 if paged else S
    for window, out_rows in ((0, 61), (20, 61), (0, 30), (5, 70)):
        outs = [torch.full((len(lens), out_rows, cache.KVH, cache.D), 7.0, dtype=dtype, device="cuda")
                for _ in "kv"]
        if paged:
            got = gqa.gqa_read_quant_paged(*cache.args, cache.table, i32(lens), window, *outs)
        else:
            got = gqa.gqa_read_quant(*cache.args, i32(lens), window, *outs)
        assert got[0] is outs[0] and got[1] is outs[1]
        for t in range(2):
            o = outs[t].double().cpu().numpy()
            for b, L in enumerate(lens):
                L = min(max(L, 0), cap)
                lo, hi = max(0, L - window) if window else 0, min(L, out_rows, S)
                lo = min(lo, out_rows)
                for h in range(cache.KVH):
                    if hi > lo:
                        assert np.array_equal(o[b, lo:hi, h], cache.ref[t][b][h].stored(lo, hi))
                top = min(L, out_rows)
                assert np.all(o[b, :lo] == 7.0) and np.all(o[b, max(top, lo):] == 7.0)


def test_read_defaults_and_bad_page():
    geo = GEO["global"]
    cache = filled(geo, 2, 48, True, seed=22)
    table = cache.table.clone()
    table[1, 1] = -1
    k, v = gqa.gqa_read_quant_paged(*cache.args, table, i32([48, 48]), 0, out_dtype=torch.float32)
    assert tuple(k.shape) == (2, 48, 4, 512) and k.dtype == torch.float32
    assert torch.all(v[1, 16:32] == 0)             # new outputs start at zero
    for t, o in ((0, k), (1, v)):
        for b, r in ((0, slice(0, 48)), (1, slice(0, 16)), (1, slice(32, 48))):
            want = np.stack([cache.ref[t][b][h].stored(r.start, r.stop) for h in range(4)], 1)
            assert np.array_equal(o[b, r].double().cpu().numpy(), want)


# ---------------------------------------------------------------------------- producer

def producer_inputs(geo, B, seed, gain=1.0):
    raw = inputs.raw_projections(B, geo["H"], geo["KVH"], geo["D"], seed, device="cuda")
    return raw


def producer_exact(layer, raw, lens):
    n_rot, theta = ROPE[layer]
    bits = inputs.bf16_bits
    return oracle.prepare_decode_f64(bits(raw["q_raw"]), bits(raw["k_raw"]), bits(raw["v_raw"]),
                                     bits(raw["w_q"]), bits(raw["w_k"]), np.asarray(lens), n_rot, theta)


PRODUCER_ERR = 4e-6


def check_producer(layer, cache, raw, lens, q_out):
    """After the call on a cache whose reference holds the state before it: the stored token
    within half a step (plus the fp32 error) of the exact value, earlier rows re-coded for the
    stored scale, the scale the rule's for an amax within the error, other rows untouched."""
    rq, rk, rv = producer_exact(layer, raw, lens)
    got_q = q_out.double().cpu().numpy()
    for b, L in enumerate(lens):
        if L >= 1:
            step = np.exp2(np.floor(np.log2(np.maximum(np.abs(rq[b]), 1e-30))) - 8)
            assert np.all(np.abs(got_q[b] - rq[b]) <= step + PRODUCER_ERR)
    for t, exact in ((0, rk), (1, rv)):
        c, s = cache.host(t)
        for b, L in enumerate(lens):
            if L < 1 or L > cache.S:
                continue
            blk, slot = divmod(L - 1, 16)
            for h in range(cache.KVH):
                r, x = cache.ref[t][b][h], exact[b, h]
                amax = float(np.abs(x).max())
                fits = {ref.exponent(amax - PRODUCER_ERR), ref.exponent(amax + PRODUCER_ERR)}
                if slot:
                    fits = {max(e, int(r.e[blk])) for e in fits}
                e = int(np.log2(s[b, blk, h]))
                assert s[b, blk, h] == 2.0 ** e and e in fits
                forced = np.array(r.e)
                forced[blk] = e
                r.append(x[None], L - 1, forced)
                old = slice(blk * 16, L - 1)
                assert np.array_equal(ref.VALUES[c[b, old, h]], r.v[old], equal_nan=True)
                y = ref.VALUES[c[b, L - 1, h]]
                scaled = x * 2.0 ** -e
                near = np.maximum(ref.half_step(scaled), ref.half_step(y))
                assert np.all(np.abs(y - scaled) <= near + PRODUCER_ERR * 2.0 ** -e)
                r.v[L - 1] = y


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
def test_producer(layer, paged):
    geo, S = GEO[layer], 77
    lens = [0, 1, 2, 16, 17, 40, 64, 77, 78, 31]      # 0: no token; 78: past a contiguous cache
    cache = filled(geo, len(lens), S, paged, seed=31, spread=2)
    before = [cache.host(t) for t in range(2)]
    raw = producer_inputs(geo, len(lens), 32)
    q_out = torch.full((len(lens), 32, geo["D"]), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (raw["q_raw"], raw["k_raw"], raw["v_raw"], raw["w_q"], raw["w_k"])
    call_lens = [min(L, 77) if paged else L for L in lens]
    if paged:
        table = cache.table.clone()
        table[9, 1] = cache.P + 3                     # sequence 9's token has a bad page
        gqa.gqa_prepare_decode_quant_paged(*args, table, i32(call_lens), q_out, *cache.args)
    else:
        gqa.gqa_prepare_decode_quant(*args, i32(call_lens), q_out, *cache.args)
    torch.cuda.synchronize()
    assert torch.all(q_out[0] == 7.0)
    check_lens = list(call_lens)
    if paged:
        check_lens[9] = 0
    for t in range(2):                                # rows outside the token's block never change
        c, s = cache.host(t)
        for b, L in enumerate(check_lens):
            keep = np.ones(S, dtype=bool)
            if 1 <= L <= S:
                keep[(L - 1) // 16 * 16:L] = False
            assert np.array_equal(c[b][keep], before[t][0][b][keep])
            blocks = [i for i in range(s.shape[1]) if not (1 <= L <= S and i == (L - 1) // 16)]
            assert np.array_equal(s[b][blocks], before[t][1][b][blocks])
    if paged:
        q_check = q_out.clone()
        q_check[9] = 0
        raw9 = {k: v.clone() for k, v in raw.items()}
        check_producer(layer, cache, raw9, check_lens, q_check)
    else:
        check_producer(layer, cache, raw, check_lens, q_out)


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_producer_codes_of_many_tokens(layer):
    """First tokens of blocks: codes and scales are those of the 64-bit values, except where one
    lies within 2^-28 (of its row's largest) of a border between two codes.  The producer's sine
    and cosine are good to 2^-30, which a rotation counts at most sqrt(2) times, 1 / rms and
    the products to 2^-40, and the angles and the 64-bit reference's own to 2^-38 at 2000."""
    geo, B, S = GEO[layer], 256, 2000
    lens = [1 + 16 * int(x) for x in np.random.default_rng(33).integers(0, S // 16, B)]
    cache = [torch.zeros((B, S, geo["KVH"], geo["D"]), dtype=torch.uint8, device="cuda").view(E4M3)
             for _ in "kv"]
    scales = [torch.zeros((B, S // 16, geo["KVH"]), device="cuda") for _ in "kv"]
    raw = producer_inputs(geo, B, 34)
    q_out = torch.empty((B, 32, geo["D"]), dtype=torch.bfloat16, device="cuda")
    gqa.gqa_prepare_decode_quant(raw["q_raw"], raw["k_raw"], raw["v_raw"], raw["w_q"], raw["w_k"],
                                 i32(lens), q_out, *cache, *scales)
    at = torch.tensor(lens, device="cuda") - 1
    every = torch.arange(B, device="cuda")
    for t, x in enumerate(producer_exact(layer, raw, lens)[1:]):
        got = ref.VALUES[cache[t].view(torch.uint8)[every, at].cpu().numpy()]
        s = scales[t][every, at // 16].double().cpu().numpy()
        amax = np.abs(x).max(-1)
        low, high = ([[ref.exponent(a * f) for a in row] for row in amax] for f in (1 - 2.0 ** -28, 1 + 2.0 ** -28))
        assert np.all((s == np.exp2(np.array(low, float))) | (s == np.exp2(np.array(high, float))))
        scaled, room = x / s[..., None], (amax / s)[..., None] * 2.0 ** -28
        below, above = ref.e4m3(scaled - room), ref.e4m3(scaled + room)
        assert np.mean(below != above) < 1e-5
        assert np.all((got == below) | (got == above))


# ---------------------------------------------------------------------------- decode

def expected(cache, q, lens, window, b, h, G):
    L = min(max(int(lens[b]), 0), cache.ref[0][b][h].v.shape[0])
    lo = max(0, L - window) if window else 0
    k, v = cache.ref[0][b][h].stored(lo, L), cache.ref[1][b][h].stored(lo, L)
    return ref.attend(q[b, h * G:(h + 1) * G], k, v), ref.attend_tolerance(q[b, h * G:(h + 1) * G], k, v)


def check_decode(cache, q, lens, window, out, skip=()):
    G = q.shape[1] // cache.KVH
    got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
    for b in range(len(lens)):
        if b in skip:
            continue
        for h in range(cache.KVH):
            want, tol = expected(cache, qd, lens, window, b, h, G)
            y = got[b, h * G:(h + 1) * G]
            bound = tol + (np.abs(want) * 2.0 ** -8 if out.dtype == torch.bfloat16 else 0.0)
            worst = float(np.max(np.abs(y - want) - bound))
            assert worst <= 0 or np.array_equal(y, want), f"b={b} h={h}: {worst:.3e} beyond the bound"


def queries(geo, B, seed, gain=0.25):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((B, geo["H"], geo["D"]), generator=g, device="cuda") * gain).to(torch.bfloat16)


def run_decode(cache, q, lens, window, table=None, **kw):
    if cache.paged:
        return gqa.gqa_decode_quant_paged(q, *cache.args, cache.table if table is None else table,
                                          i32(lens), window, **kw)
    return gqa.gqa_decode_quant(q, *cache.args, i32(lens), window, **kw)


def poison(cache, lens, window):
    """NaN codes in every row outside the attended ranges, nonsense in the scales of blocks that
    hold none of them."""
    for t in range(2):
        c = cache.codes[t].view(torch.uint8)
        for b, L in enumerate(lens):
            lo = max(0, L - window) if window else 0
            for pos in list(range(0, lo)) + list(range(L, cache.S)):
                if cache.paged:
                    c[int(cache.host_table[b, pos // 16]), pos % 16] = 0x7f
                else:
                    c[b, pos] = 0x7f
            for blk in range((cache.S + 15) // 16):
                if blk * 16 >= L or (blk + 1) * 16 <= lo:
                    where = int(cache.host_table[b, blk]) if cache.paged else (b, blk)
                    cache.scales[t][where] = float("nan")


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("window", [0, 100])
def test_decode_lengths_and_masks(layer, paged, window):
    geo = GEO[layer]
    lens, S = [0, 1, 15, 16, 17, 31, 99, 100, 101, 113, 128, 129, 255, 300, 333], 333
    cache = filled(geo, len(lens), S, paged, seed=41)
    poison(cache, lens, window)
    q = queries(geo, len(lens), 42)
    for dtype in (torch.float32, torch.bfloat16):
        out = run_decode(cache, q, lens, window, out_dtype=dtype)
        check_decode(cache, q, lens, window, out)
        assert torch.all(out[0] == 0)
    assert gqa.gqa_device_status() == 0


@pytest.mark.parametrize("layer,lens,window", [("sliding", [5000, 1, 1024, 1025, 2047], 1024),
                                               ("sliding", [4096, 777], 0),
                                               ("global", [6000, 3, 2049], 0),
                                               ("global", [9000], 4097)])
@pytest.mark.parametrize("paged", [False, True])
def test_decode_long(layer, lens, window, paged):
    """Long enough that segments are split over many CTAs and merged."""
    geo = GEO[layer]
    cache = filled(geo, len(lens), max(lens), paged, seed=43)
    q = queries(geo, len(lens), 44)
    out = run_decode(cache, q, lens, window, out_dtype=torch.float32)
    check_decode(cache, q, lens, window, out)
    again = run_decode(cache, q, lens, window, out_dtype=torch.float32)
    assert torch.equal(out, again), "results are bit-reproducible"


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("spread", [0, 12])
def test_decode_scales_far_apart(layer, spread):
    """Blocks whose scales differ by up to 2^(2 spread); and scales of zero taken as 2^-64."""
    geo, lens = GEO[layer], [700, 45]
    cache = filled(geo, 2, 700, False, seed=45, spread=spread)
    # keys keep moderate scales so that scores stay finite and spread over positions
    cache.scales[0].fill_(2.0 ** -6)
    for b in range(2):
        for h in range(cache.KVH):
            cache.ref[0][b][h].e[:] = -6
    cache.scales[1][1, 0] = 0.0
    for h in range(cache.KVH):
        cache.ref[1][1][h].e[0] = -64
    q = queries(geo, 2, 46)
    out = run_decode(cache, q, lens, 0, out_dtype=torch.float32)
    check_decode(cache, q, lens, 0, out)


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("lens", [[700], [5000, 1200, 17]])
def test_decode_scales_at_both_ends(layer, lens):
    """One block of values near 2^68 among blocks of zeros (whose scale is 2^-64): the zeros'
    weights vanish beside 2^128, their share of the normaliser (1% to 13%) does not."""
    geo, KVH, D = GEO[layer], GEO[layer]["KVH"], GEO[layer]["D"]
    cache = Cache(geo, len(lens), max(lens), False)
    for t in range(2):
        cache.codes[t].zero_()
        cache.scales[t].fill_(2.0 ** -64)
    q = torch.zeros((len(lens), geo["H"], D), dtype=torch.bfloat16, device="cuda")
    q[..., 3] = 10.5                                        # scores 10.5 at one position, else 0
    for b, L in enumerate(lens):
        at = (L - 1) // 2
        cache.codes[0].view(torch.uint8)[b, at, :, 3] = 0x38     # 1.0
        cache.codes[1].view(torch.uint8)[b, at, :, ::2] = 0x7e   # 448
        cache.scales[0][b, at // 16] = 1.0
        cache.scales[1][b, at // 16] = 2.0 ** 60
        for h in range(KVH):
            for t in range(2):
                r = cache.ref[t][b][h]
                r.v[:] = 0.0
                r.e[:] = -64
                r.e[at // 16] = 60 if t else 0
            cache.ref[0][b][h].v[at, 3] = 1.0
            cache.ref[1][b][h].v[at, ::2] = 448.0
    out = run_decode(cache, q, lens, 0, out_dtype=torch.float32)
    check_decode(cache, q, lens, 0, out)


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_decode_queries_of_any_size(layer):
    """Heads of zeros, tiny, large and mixed-magnitude queries; scores that are all far below
    zero."""
    geo, lens = GEO[layer], [200]
    cache = filled(geo, 1, 200, False, seed=47, spread=1)
    q = queries(geo, 1, 48)
    q[0, 0] = 0
    q[0, 1] = q[0, 1] * 1e-30
    q[0, 2] = q[0, 2] * 64
    q[0, 3, ::2] = q[0, 3, ::2] * 2.0 ** -20
    out = run_decode(cache, q, lens, 0, out_dtype=torch.float32)
    check_decode(cache, q, lens, 0, out)
    # every key has one channel of the same sign and the query the other: scores near -1e4
    c = cache.codes[0].view(torch.uint8)
    c[..., 7] = 0x7e                                  # 448
    cache.scales[0].fill_(1.0)
    for h in range(cache.KVH):
        r = cache.ref[0][0][h]
        r.v[:, 7] = 448.0
        r.e[:] = 0
    q = queries(geo, 1, 49, gain=2.0 ** -6)
    q[..., 7] = -24.0
    out = run_decode(cache, q, lens, 0, out_dtype=torch.float32)
    check_decode(cache, q, lens, 0, out)


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_decode_nan_inside_the_range(layer):
    """A NaN key or value that is attended makes its KV head's outputs NaN, and no other."""
    geo, lens = GEO[layer], [40, 40]
    G = geo["H"] // geo["KVH"]
    for t in range(2):
        cache = filled(geo, 2, 40, False, seed=50)
        cache.codes[t].view(torch.uint8)[0, 13, 2, 9] = 0x7f
        q = queries(geo, 2, 51)
        out = run_decode(cache, q, lens, 0, out_dtype=torch.float32)
        bad = torch.isnan(out)
        if t == 0:
            assert torch.all(bad[0, 2 * G:3 * G])
        else:
            assert torch.all(bad[0, 2 * G:3 * G, 9])
        bad[0, 2 * G:3 * G] = False
        assert not torch.any(bad)
        check_decode(cache, q, lens, 0, out, skip=(0,))


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_decode_bad_pages_and_lengths(layer):
    """A page id outside [0, P) among the attended pages: that sequence is NaN and the status
    says so; outside the window it is not looked at.  Lengths are clamped."""
    geo = GEO[layer]
    lens = [300, 300, 300, 40]
    cache = filled(geo, 4, 320, True, seed=52)
    table = cache.table.clone()
    table[0, 3] = cache.P
    table[1, 18] = -1
    table[2, 2] = -7                                   # before the window
    q = queries(geo, 4, 53)
    window = 200
    assert gqa.gqa_device_status() == 0
    out = run_decode(cache, q, lens, window, table, out_dtype=torch.float32)
    check_decode(cache, q, lens, window, out, skip=(1,))
    assert torch.all(torch.isnan(out[1]))
    assert gqa.gqa_device_status() == gqa.GQA_DEVICE_BAD_PAGE
    out = run_decode(cache, q, lens, 0, table, out_dtype=torch.float32)
    assert torch.all(torch.isnan(out[:3]))
    check_decode(cache, q, lens, 0, out, skip=(0, 1, 2))
    assert gqa.gqa_device_status() == gqa.GQA_DEVICE_BAD_PAGE
    out = run_decode(cache, q, [321, -4, 300, 40], 0, out_dtype=torch.float32)
    check_decode(cache, q, [320, 0, 300, 40], 0, out)
    assert gqa.gqa_device_status() == gqa.GQA_DEVICE_BAD_LENGTH


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_decode_whole_batch(layer):
    """256 sequences of lengths 0 .. 255 (every plan lane), some checked."""
    geo = GEO[layer]
    lens = [(i * 37) % 256 for i in range(256)]
    cache = filled(geo, 256, 255, True, seed=54)
    q = queries(geo, 256, 55)
    out = run_decode(cache, q, lens, 64, out_dtype=torch.float32)
    check_decode(cache, q, lens, 64, out, skip=[b for b in range(256) if b % 9])
    for b in range(256):
        assert lens[b] or torch.all(out[b] == 0)


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_workspace_of_the_caller_streams_and_graph(layer):
    """Two graphs with workspaces of their own, replayed on two streams at once, equal the plain
    calls; a workspace that is too small is refused."""
    geo = GEO[layer]
    H, KVH, D = geo["H"], geo["KVH"], geo["D"]
    lens = [900, 33, 1500]
    caches = [filled(geo, 3, 1500, p, seed=60 + p) for p in (False, True)]
    qs = [queries(geo, 3, 62 + i) for i in range(2)]
    want = [run_decode(c, q, lens, 1024, out_dtype=torch.float32) for c, q in zip(caches, qs)]
    wss = [gqa.new_workspace(3, 1504, H, KVH, D, 1024) for _ in range(2)]
    outs = [torch.zeros_like(w) for w in want]
    seq = i32(lens)
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for c, q, ws, out, s in zip(caches, qs, wss, outs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            if c.paged:
                gqa.gqa_decode_quant_paged(q, *c.args, c.table, seq, 1024, out=out, workspace=ws)
            else:
                gqa.gqa_decode_quant(q, *c.args, seq, 1024, out=out, workspace=ws)
        graphs.append(g)
    for _ in range(5):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert all(gqa.gqa_device_status(ws) == 0 for ws in wss)
    with pytest.raises(gqa.GQAError) as err:
        gqa.gqa_decode_quant(qs[0], *caches[0].args, seq, 1024, workspace=wss[0][:4096])
    assert err.value.status == gqa.GQA_ERR_WORKSPACE


# ---------------------------------------------------------------------------- together

@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
def test_prompt_then_steps(layer, paged):
    """A ragged prompt, then decode steps, each a producer and an attention call back to back
    on one stream: every step's output matches attention over what is stored, and the read-back
    returns it."""
    geo, S = GEO[layer], 64
    G = geo["H"] // geo["KVH"]
    window = 24 if layer == "sliding" else 0
    gen = torch.Generator(device="cuda").manual_seed(70)
    lens = np.array([13, 1, 31, 40])
    cache = Cache(geo, 4, S, paged, seed=71)
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    shape = (off[-1], geo["KVH"], geo["D"])
    cache.append(rows(gen, shape), rows(gen, shape), off, lens.tolist())
    for step in range(6):
        lens = lens + 1
        raw = producer_inputs(geo, 4, 80 + step)
        q_out = torch.empty((4, 32, geo["D"]), dtype=torch.bfloat16, device="cuda")
        args = (raw["q_raw"], raw["k_raw"], raw["v_raw"], raw["w_q"], raw["w_k"])
        seq = i32(lens)
        if paged:
            gqa.gqa_prepare_decode_quant_paged(*args, cache.table, seq, q_out, *cache.args)
            out = gqa.gqa_decode_quant_paged(q_out, *cache.args, cache.table, seq, window,
                                             out_dtype=torch.float32)
            k, v = gqa.gqa_read_quant_paged(*cache.args, cache.table, seq, 0, out_dtype=torch.float32)
        else:
            gqa.gqa_prepare_decode_quant(*args, seq, q_out, *cache.args)
            out = gqa.gqa_decode_quant(q_out, *cache.args, seq, window, out_dtype=torch.float32)
            k, v = gqa.gqa_read_quant(*cache.args, seq, 0, out_dtype=torch.float32)
        check_producer(layer, cache, raw, lens.tolist(), q_out)
        check_decode(cache, q_out, lens, window, out)
        for t, got in enumerate((k, v)):
            got = got.double().cpu().numpy()
            for b in range(4):
                for h in range(geo["KVH"]):
                    assert np.array_equal(got[b, :lens[b], h], cache.ref[t][b][h].stored(0, lens[b]))
    assert G * geo["KVH"] == 32 and gqa.gqa_device_status() == 0


def test_matches_the_bf16_core_on_exact_values():
    """Values that both caches hold exactly: the 8-bit and the bf16 attention calls agree within
    their fp32 errors."""
    for layer in ("sliding", "global"):
        geo, lens = GEO[layer], [1300, 40]
        cache = filled(geo, 2, 1300, False, seed=90, spread=1)
        k, v = gqa.gqa_read_quant(*cache.args, i32(lens), 0)
        q = queries(geo, 2, 91)
        a = run_decode(cache, q, lens, geo["window"], out_dtype=torch.float32)
        b = gqa.gqa_decode(q, k, v, i32(lens), geo["window"], out_dtype=torch.float32)
        check_decode(cache, q, lens, geo["window"], a)
        assert float((a - b).abs().max()) <= 1e-3 * float(v.abs().max())


# ---------------------------------------------------------------------------- refusals

def test_binding_refusals_and_empty_batches():
    """Wrong types, layouts, shapes and devices raise before anything is enqueued; an empty batch
    or append is a no-op."""
    geo = GEO["sliding"]
    c, p = Cache(geo, 2, 40, False), Cache(geo, 2, 40, True)
    gen = torch.Generator(device="cuda").manual_seed(95)
    x, q, lens, off = rows(gen, (8, 16, 256)), queries(geo, 2, 96), i32([4, 4]), i32([0, 4, 8])
    k, v, ks, vs = c.args
    wide = torch.zeros(2, 40, 16, 512, device="cuda").to(E4M3)[..., ::2]
    bad_caches = [(k.view(torch.uint8), v, ks, vs), (k, v[:1].clone(), ks, vs), (k, v, ks[:, :2].clone(), vs),
                  (k, v, ks.double(), vs), (k, v, ks, vs.cpu()), (wide, wide, ks, vs), (k, v, ks[0], vs[0]),
                  (None, v, ks, vs), (k, v, ks, None)]
    raw = producer_inputs(geo, 2, 97)
    head = (raw["q_raw"], raw["k_raw"], raw["v_raw"], raw["w_q"], raw["w_k"])
    q_out = torch.empty_like(q)
    for bad in bad_caches:
        with pytest.raises(ValueError):
            gqa.gqa_decode_quant(q, *bad, lens, 0)
        with pytest.raises(ValueError):
            gqa.gqa_append_quant(x, x, off, lens, *bad)
        with pytest.raises(ValueError):
            gqa.gqa_read_quant(*bad, lens, 0)
        with pytest.raises(ValueError):
            gqa.gqa_prepare_decode_quant(*head, lens, q_out, *bad)
    with pytest.raises(ValueError):
        gqa.gqa_decode_quant(q.float(), *c.args, lens, 0)
    with pytest.raises(ValueError):
        gqa.gqa_decode_quant(q, *c.args, lens.long(), 0)
    with pytest.raises(ValueError):
        gqa.gqa_decode_quant(q, *c.args, i32([4]), 0)
    with pytest.raises(ValueError):
        gqa.gqa_decode_quant(q, *c.args, lens, 0, out=torch.empty(2, 32, 512, device="cuda"))
    with pytest.raises(TypeError):
        gqa.gqa_decode_quant(q, *c.args, lens, 0, out=torch.empty(2, 32, 256, device="cuda").half())
    with pytest.raises(ValueError):
        gqa.gqa_append_quant(x, x[:4].clone(), off, lens, *c.args)
    with pytest.raises(ValueError):
        gqa.gqa_append_quant(x, x, i32([0, 8]), lens, *c.args)
    with pytest.raises(ValueError):
        gqa.gqa_append_quant(x[:, ::2], x[:, ::2], off, lens, *c.args)
    with pytest.raises(ValueError):
        gqa.gqa_read_quant(*c.args, lens, 0, k_out=torch.empty(2, 40, 16, 256, device="cuda"))
    with pytest.raises(ValueError):
        gqa.gqa_prepare_decode_quant(head[0], head[1], None, *head[3:], lens, q_out, *c.args)
    with pytest.raises(ValueError):
        gqa.gqa_decode_quant_paged(q, *p.args, None, lens, 0)
    with pytest.raises(ValueError):
        gqa.gqa_decode_quant_paged(q, *p.args, p.table[:1].clone(), lens, 0)
    with pytest.raises(gqa.GQAError):
        gqa.gqa_decode_quant(q, *c.args, lens, -1)
    gqa.gqa_append_quant(x[:0], x[:0], i32([0, 0, 0]), lens, *c.args)      # no tokens
    e = [t[:0] for t in c.args]
    assert gqa.gqa_decode_quant(q[:0], *e, lens[:0], 0).shape == (0, 32, 256)
    gqa.gqa_append_quant(x, x, off[:1], lens[:0], *e)
    torch.cuda.synchronize()
    c.check()                                                             # nothing was written
    p.check()
