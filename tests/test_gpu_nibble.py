"""GPU tests of what writes and reads the 4-bit KV cache (gqa_append_nibble, gqa_read_nibble,
gqa_prepare_tokens_nibble) and of the producer for many tokens (gqa_prepare_tokens), contiguous and
paged, against the 64-bit reference in nibble_reference.py.

Append: scales and codes are exact functions of bf16 inputs, so whole caches are compared byte for
byte, rows that nothing may write among them.  Read: exact in both types.  Producer, bf16: half a step
of bf16 (2^-9 of a value's binade, 2^-8 of the value at most) plus the fp32 arithmetic's error: a sum
of D squares in fp32 (8 or 16 along a lane, 5 levels of lanes, halved by the root), root, quotient,
weight and rotation are within 16 roundings of 2^-24 of the head's largest magnitude, the angle's cos
and sin within 2^-24 of a value each.  Producer, 4 bits: codes equal, but for 32 channels where an
error of 2^-27 could change a bf16 number.
"""
import numpy as np
import pytest
import torch

import decode_attention_gb300 as gqa
import oracle
from decode_attention_gb300 import inputs
from tests import nibble_reference as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

GEO = {"sliding": inputs.SLIDING, "global": inputs.GLOBAL}
ROPE = {"sliding": (oracle.SLIDING_ROPE_PAIRS, oracle.SLIDING_ROPE_THETA),
        "global": (oracle.GLOBAL_ROPE_PAIRS, oracle.GLOBAL_ROPE_THETA)}
FILL = 0x5A          # byte of rows that nothing may write


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def offsets(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int64)


class Cache:
    """A cache on the GPU, contiguous or paged (pages in a random order, two spare), every byte at a
    fill value, and what it should hold: `want`, rows by position [B, S, planes, 272]."""

    def __init__(self, geo, B, S, paged, seed=0):
        self.KVH, self.D, self.B, self.S, self.paged = geo["KVH"], geo["D"], B, S, paged
        self.planes = self.KVH * self.D // 256
        nblk = (S + 15) // 16
        if paged:
            self.P = B * nblk + 2
            self.host_table = np.random.default_rng(seed).permutation(self.P)[:B * nblk].reshape(B, nblk).astype(np.int32)
            self.table = i32(self.host_table)
            shape = (self.P, self.planes, 16, 272)
        else:
            self.table = None
            shape = (B, self.planes, S, 272)
        self.kv = torch.full(shape, FILL, dtype=torch.uint8, device="cuda")
        self.want = np.full((B, nblk * 16 if paged else S, self.planes, 272), FILL, dtype=np.uint8)

    @property
    def pages(self):
        return (self.table,) if self.paged else ()

    def fn(self, name):
        return getattr(gqa, name + ("_paged" if self.paged else ""))

    def set_rows(self, rows):
        """Rows [B, S, planes, 272] written past every call."""
        self.want[:, :rows.shape[1]] = rows
        r = torch.tensor(self.want, device="cuda").transpose(1, 2)           # [B, planes, S, 272]
        if self.paged:
            r = r.reshape(self.B, self.planes, -1, 16, 272).transpose(1, 2)
            self.kv[self.table.long()] = r
        else:
            self.kv.copy_(r)

    def note(self, k, v, off, lens, capacity=None):
        """What an append of k, v [N, KVH, D] should do; the positions written."""
        rows = ref.encode(k, v)
        for b in range(self.B):
            n = off[b + 1] - off[b]
            if n > 0 and lens[b] >= n and lens[b] <= (self.want.shape[1] if capacity is None else capacity):
                self.want[b, lens[b] - n:lens[b]] = rows[off[b]:off[b + 1]]

    def host(self):
        r = self.kv.cpu().numpy()
        if not self.paged:
            return r.transpose(0, 2, 1, 3)
        return r[self.host_table].transpose(0, 1, 3, 2, 4).reshape(self.want.shape)

    def check(self, doubtful=None):
        got = self.host()
        if doubtful is None:
            assert np.array_equal(got, self.want)
        else:
            assert np.array_equal(np.where(doubtful, 0, got), np.where(doubtful, 0, self.want))
        if self.paged:
            spare = sorted(set(range(self.P)) - set(self.host_table.ravel().tolist()))
            assert torch.all(self.kv[spare] == FILL)


def rows(gen, n, geo, spread=0):
    x = torch.randn((n, geo["KVH"], geo["D"]), generator=gen, device="cuda")
    if spread:
        s = (2 * torch.rand((n, geo["KVH"], geo["D"] // 32, 1), generator=gen, device="cuda") - 1) * spread
        x = (x.view(n, geo["KVH"], -1, 32) * torch.exp2(s)).view_as(x)
    return x.to(torch.bfloat16)


def f64(x):
    return x.double().cpu().numpy()


# ---------------------------------------------------------------------------- append, read

NEW = [[0, 1, 15, 16, 17, 40, 0, 76], [1, 0, 1, 16, 3, 37, 0, 1], [15, 30, 0, 1, 57, 0, 77, 0]]


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("spread", [0, 14])
def test_append_chunks(layer, paged, spread):
    """Chunks that start and end anywhere in a page, sequences without new tokens, a cache whose
    length is no whole number of pages, filled to its last row; groups of very unlike sizes."""
    geo = GEO[layer]
    gen = torch.Generator(device="cuda").manual_seed(11 + spread)
    cache = Cache(geo, 8, 77, paged, seed=3)
    have = np.zeros(8, dtype=np.int64)
    for new in NEW:
        have = have + new
        off = offsets(new)
        k, v = (rows(gen, off[-1], geo, spread) for _ in "kv")
        cache.fn("gqa_append_nibble")(k, v, i32(off), *cache.pages, i32(have), cache.kv)
        cache.note(f64(k), f64(v), off, have)
        cache.check()


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_append_values_at_the_ends_of_the_range(layer):
    """Zeros of both signs, subnormals, ties, values around the largest and far beyond it, infinities
    and NaN of both signs."""
    geo = GEO[layer]
    special = torch.tensor([0.0, -0.0, 1e-40, -1e-40, 2.0 ** -18, 2.0 ** -17, -(2.0 ** -14), 449.0, 450.0, 452.0,
                            -450.0, 1e5, -3e38, 0.5, 1.5, -2.5, 7.5, -7.5, 60.0, 1e-3], dtype=torch.bfloat16)
    gen = torch.Generator().manual_seed(4)
    n = 24
    x = special[torch.randint(len(special), (n, geo["KVH"], geo["D"]), generator=gen)]
    x[::3] *= 0.0                                  # all zeros
    x[1::3, :, ::2] = x[1::3, :, 1::2] * 0.01      # groups without the largest
    y = x.clone()
    y[2, :, 5] = float("nan")
    y[5, :, 250] = float("inf")
    y[8, 0, 0] = -float("inf")
    y[11, :, 31:33] = -float("nan")
    cache = Cache(geo, 1, n, False)
    off, lens = offsets([n]), np.array([n])
    k, v = y.cuda(), x.flip(0).contiguous().cuda()
    gqa.gqa_append_nibble(k, v, i32(off), i32(lens), cache.kv)
    cache.note(f64(k), f64(v), off, lens)
    cache.check()
    for dtype in (torch.bfloat16, torch.float32):
        ko, vo = gqa.gqa_read_nibble(cache.kv, i32(lens), 0, out_dtype=dtype)
        wk, wv = ref.decode(cache.want, geo["D"])
        assert np.array_equal(f64(ko), wk, equal_nan=True) and np.array_equal(f64(vo), wv, equal_nan=True)
    assert np.isnan(wk).sum() > 0


@pytest.mark.parametrize("paged", [False, True])
def test_every_scale_and_tie(paged):
    """For every scale: the largest magnitude that takes it, the next bf16 number, and all ties
    between codes."""
    geo = GEO["sliding"]
    need = np.concatenate([ref.SCALES * 7.5, ref.bf16(ref.SCALES * 7.5 * (1 + 2.0 ** -7))])
    need = need[need > 0]
    x = np.zeros((len(need), 32))
    x[:, 0] = need
    s = ref.SCALES[ref.code_group(ref.bf16(x))[0]]
    x[:, 1:15] = s[:, None] * (np.arange(14) - 6.5)
    x[:, 15:29] = -x[:, 1:15] * (1 + 2.0 ** -8)
    x = torch.tensor(x).to(torch.bfloat16)
    n = (len(need) * 32 + 4095) // 4096
    k = torch.zeros(n * 4096, dtype=torch.bfloat16)
    k[:x.numel()] = x.flatten()
    k = k.view(n, 16, 256).cuda()
    cache = Cache(geo, 1, n, paged)
    cache.fn("gqa_append_nibble")(k, -k, i32([0, n]), *cache.pages, i32([n]), cache.kv)
    cache.note(f64(k), f64(-k), [0, n], [n])
    cache.check()


@pytest.mark.parametrize("paged", [False, True])
def test_append_skips_what_does_not_fit(paged):
    """Offsets outside [0, N], a length below the number of new tokens, above the capacity or
    negative, a page out of range: nothing else changes."""
    geo = GEO["global"]
    B, S = 6, 48
    cache = Cache(geo, B, S, paged, seed=9)
    gen = torch.Generator(device="cuda").manual_seed(5)
    N = 40
    k, v = (rows(gen, N, geo) for _ in "kv")
    off = np.array([0, 5, 12, 20, 28, 35, 60])       # the last sequence reaches past N
    lens = np.array([4, 7, S + 1, -3, 20, 48])       # 4 < 5 new tokens; S + 1 and -3 no lengths
    if paged:
        cache.host_table = cache.host_table.copy()
        table = cache.host_table.copy()
        table[4, 0] = cache.P
        table[4, 2] = -1
        cache.table = i32(table)
    cache.fn("gqa_append_nibble")(k, v, i32(off), *cache.pages, i32(lens), cache.kv)
    for b in (1, 4):
        got = ref.encode(f64(k), f64(v))[off[b]:off[b + 1]]
        pos = np.arange(lens[b] - len(got), lens[b])
        keep = ~((b == 4) & paged & (pos < 16))
        cache.want[b, pos[keep]] = got[keep]
    cache.check()


def test_empty_calls():
    geo = GEO["sliding"]
    cache = Cache(geo, 2, 20, False)
    none = torch.empty((0, geo["KVH"], geo["D"]), dtype=torch.bfloat16, device="cuda")
    gqa.gqa_append_nibble(none, none, i32([0, 0, 0]), i32([0, 0]), cache.kv)
    cache.check()
    q = torch.empty((0, 32, geo["D"]), dtype=torch.bfloat16, device="cuda")
    gqa.gqa_prepare_tokens_nibble(q, none, none, q.new_zeros(256), q.new_zeros(256), i32([0, 0, 0]), i32([3, 0]),
                                  q.clone(), cache.kv)
    cache.check()
    empty = torch.empty((0, 16, 20, 272), dtype=torch.uint8, device="cuda")
    ko, vo = gqa.gqa_read_nibble(empty, i32([]), 0)
    assert ko.shape == vo.shape == (0, 20, 16, 256)
    assert gqa.gqa_decode_nibble(q, empty, i32([]), 0).shape == (0, 32, 256)


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("window", [0, 1, 33])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read(layer, paged, window, dtype):
    """All bytes that a row may hold, lengths from none to the capacity and outside of it, outputs
    of more and of fewer rows; rows outside the range stay as they were."""
    geo = GEO[layer]
    lens = [0, 1, 16, 50, 77, 78, -1, 2000]
    S = 78
    cache = Cache(geo, len(lens), S, paged, seed=2)
    cache.set_rows(np.random.default_rng(8).integers(0, 256, (len(lens), S, cache.planes, 272), dtype=np.uint8))
    wk, wv = ref.decode(cache.want, geo["D"])
    full = cache.want.shape[1]
    for out_rows in (40, 100):
        outs = [torch.full((len(lens), out_rows, geo["KVH"], geo["D"]), 3.0, dtype=dtype, device="cuda")
                for _ in "kv"]
        got = cache.fn("gqa_read_nibble")(cache.kv, *cache.pages, i32(lens), window, *outs)
        assert got[0] is outs[0] and got[1] is outs[1]
        for o, w in zip(outs, (wk, wv)):
            want = np.full(o.shape, 3.0)
            for b, L in enumerate(lens):
                L = min(max(L, 0), full)
                lo, hi = max(0, L - window) if window else 0, min(L, out_rows)
                want[b, lo:max(lo, hi)] = w[b, lo:max(lo, hi)]
            assert np.array_equal(f64(o), want, equal_nan=True)
    ko, _ = cache.fn("gqa_read_nibble")(cache.kv, *cache.pages, i32(lens), 0, out_rows=9, out_dtype=dtype)
    assert ko.shape[1] == 9 and torch.all(ko[0] == 0)
    if paged:
        bad = cache.host_table.copy()
        bad[4, 1], bad[4, 2] = -1, cache.P
        o = torch.full((len(lens), S, geo["KVH"], geo["D"]), 3.0, dtype=dtype, device="cuda")
        gqa.gqa_read_nibble_paged(cache.kv, i32(bad), i32(lens), 0, o, o.clone())
        want = np.full(o.shape[1:], 3.0)
        want[:16], want[48:77] = wk[4, :16], wk[4, 48:77]
        assert np.array_equal(f64(o[4]), want, equal_nan=True)


# ---------------------------------------------------------------------------- producer

class Tokens:
    """Raw projections of a ragged batch, and the formulas' q, k, v in 64 bits."""

    def __init__(self, layer, new, lens, seed, keqv=False):
        geo = GEO[layer]
        self.H, self.KVH, self.D, self.layer = geo["H"], geo["KVH"], geo["D"], layer
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.off, self.lens = offsets(new), np.asarray(lens)
        N = max(1, self.off[-1])
        make = lambda h, s: (s * torch.randn((N, h, self.D), generator=gen, device="cuda")).to(torch.bfloat16)  # noqa: E731
        self.q, self.k, self.v = make(self.H, 2.0), make(self.KVH, 30.0), None if keqv else make(self.KVH, 0.02)
        w = lambda: (1 + 0.5 * torch.randn(self.D, generator=gen, device="cuda")).to(torch.bfloat16)  # noqa: E731
        self.wq, self.wk = w(), w()
        self.q_out = torch.full_like(self.q, 3.0)
        self.pos = np.concatenate([np.arange(L - n, L) for n, L in zip(new, lens)] or [[0]])

    @property
    def args(self):
        return self.q, self.k, self.v, self.wq, self.wk, i32(self.off)

    def exact(self):
        pairs, theta = ROPE[self.layer]
        v = self.k if self.v is None else self.v
        n = self.off[-1]
        return (ref.norm_rope(f64(self.q)[:n], f64(self.wq), self.pos, pairs, theta),
                ref.norm_rope(f64(self.k)[:n], f64(self.wk), self.pos, pairs, theta),
                ref.norm_rope(f64(v)[:n], None, self.pos, pairs, theta))


def near(got, want):
    """Half a bf16 step of each value, and 20 roundings of fp32 of the head's largest."""
    got = f64(got)
    _, e = np.frexp(want)
    tol = np.exp2(e - 9.0) + 20 * 2.0 ** -24 * np.abs(want).max(-1, keepdims=True)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


PRODUCED = dict(new=[3, 0, 1, 16, 70, 0, 8], lens=[3, 5, 90, 31, 70, 0, 81])
FAR = dict(new=[2, 1, 5], lens=[262144, 200001, 131073])


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("form", ["contiguous", "paged", "ring", "keqv", "keqv_paged"])
def test_producer(layer, form):
    """Ragged tokens into a bf16 cache.  The ring keeps the last rows of sequences with more new
    tokens than it has; every other row stays as it was."""
    if layer == "sliding" and "keqv" in form:
        pytest.skip("values = keys on global layers only")
    t = Tokens(layer, **PRODUCED, seed=21, keqv="keqv" in form)
    KVH, D, B = t.KVH, t.D, len(t.lens)
    rows_, paged = 24 if form == "ring" else 88, form.endswith("paged")
    q, k, v = t.exact()
    if paged:
        nblk = 6
        table = np.random.default_rng(1).permutation(B * nblk + 2)[:B * nblk].reshape(B, nblk)
        table[3, 1] = -1                     # positions 16 .. 31 of sequence 3 have no page
        table[4, 0] = B * nblk + 2
        caches = [torch.full((B * nblk + 2, 16, KVH, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        gqa.gqa_prepare_tokens_paged(*t.args, i32(table), i32(t.lens), t.q_out,
                                     None if "keqv" in form else caches[0], caches[1])
    else:
        caches = [torch.full((B, rows_, KVH, D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        gqa.gqa_prepare_tokens(*t.args, i32(t.lens), t.q_out, None if "keqv" in form else caches[0], caches[1],
                               ring=form == "ring")
    near(t.q_out, q)
    for c, want in zip(caches, (k, v)):
        written = torch.zeros(c.shape[:2], dtype=torch.bool)
        if c is caches[0] and "keqv" in form:
            assert torch.all(c == 3.0)
            continue
        for b in range(B):
            for i in range(t.off[b], t.off[b + 1]):
                pos = t.pos[i]
                if paged:
                    o, r = table[b, pos // 16], pos % 16
                    if not 0 <= o < B * nblk + 2:
                        continue
                elif form == "ring":
                    o, r = b, pos % rows_
                    if pos < t.lens[b] - rows_:
                        continue
                else:
                    o, r = b, pos
                    if pos >= rows_:
                        continue
                near(c[o, r], want[i])
                written[o, r] = True
        assert torch.all(c[~written.cuda()] == 3.0)


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_producer_at_far_positions(layer):
    """Positions up to the longest cache, in a ring."""
    t = Tokens(layer, **FAR, seed=22)
    caches = [torch.zeros((3, 8, t.KVH, t.D), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    gqa.gqa_prepare_tokens(*t.args, i32(t.lens), t.q_out, *caches, ring=True)
    q, k, v = t.exact()
    near(t.q_out, q)
    for b in range(3):
        for i in range(t.off[b], t.off[b + 1]):
            near(caches[0][b, t.pos[i] % 8], k[i])
            near(caches[1][b, t.pos[i] % 8], v[i])


def test_producer_skips_sequences_that_do_not_fit():
    t = Tokens("sliding", [4, 3, 2, 5], [4, 3, 2, 5], seed=23)
    off, lens = t.off.copy(), t.lens.copy()
    lens[1] = 2                     # fewer positions than new tokens
    off[4] = 40                     # past N
    cache = Cache(GEO["sliding"], 4, 8, False)
    gqa.gqa_prepare_tokens_nibble(t.q, t.k, t.v, t.wq, t.wk, i32(off), i32(lens), t.q_out, cache.kv)
    q, k, v = t.exact()
    near(t.q_out[:4], q[:4])
    near(t.q_out[7:9], q[7:9])
    assert torch.all(t.q_out[4:7] == 3.0) and torch.all(t.q_out[9:] == 3.0)
    got = cache.host()
    assert np.all(got[1] == FILL) and np.all(got[3] == FILL)
    assert np.all(got[0, 4:] == FILL) and not np.any(np.all(got[0, :4] == FILL, axis=-1))


def check_codes(t, cache, capacity):
    _, k, v = t.exact()
    kept = t.off[-1]
    cache.note(ref.bf16(k), ref.bf16(v), t.off, t.lens, capacity)
    doubt = np.zeros(cache.want.shape, dtype=bool)
    for b in range(cache.B):
        for i in range(t.off[b], t.off[b + 1]):
            for which, x in ((0, k), (1, v)):
                d = ref.bf16_doubt(x[i], 2.0 ** -27).reshape(-1, 8, 32).any(-1)      # [planes, groups]
                doubt[b, t.pos[i], :, 128 * which:128 * which + 128] |= np.repeat(d, 16, -1)
                doubt[b, t.pos[i], :, 256 + 8 * which:264 + 8 * which] |= d
    assert doubt.mean() < 1e-3 and kept > 0
    cache.check(doubt)


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
def test_producer_into_4_bits(layer, paged):
    t = Tokens(layer, **PRODUCED, seed=24)
    cache = Cache(GEO[layer], len(t.lens), 96, paged, seed=6)
    cache.fn("gqa_prepare_tokens_nibble")(*t.args, *cache.pages, i32(t.lens), t.q_out, cache.kv)
    near(t.q_out, t.exact()[0])
    check_codes(t, cache, 96)


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_one_token_per_sequence_into_4_bits(layer):
    """The decode step's form, the whole batch at positions up to the longest cache's last."""
    B = 5
    lens = [1, 2, 17, 40, 33]
    t = Tokens(layer, [1] * B, lens, seed=25)
    cache = Cache(GEO[layer], B, 40, False)
    gqa.gqa_prepare_tokens_nibble(*t.args, i32(t.lens), t.q_out, cache.kv)
    check_codes(t, cache, 40)


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_raw_values_that_are_not_finite(layer):
    """A NaN or an infinity in a head's raw key makes that head's key NaN and nothing else; zeros
    stay zeros."""
    t = Tokens(layer, [4], [4], seed=26)
    t.k[0, 1, 7], t.v[1, 0, 3], t.k[2, 0, 5] = float("nan"), float("inf"), -float("inf")
    t.v[3] = 0.0
    cache = Cache(GEO[layer], 1, 4, False)
    gqa.gqa_prepare_tokens_nibble(*t.args, i32(t.lens), t.q_out, cache.kv)
    k, v = (x.double().cpu().numpy()[0] for x in gqa.gqa_read_nibble(cache.kv, i32([4]), 0))
    nan = np.isnan(k).any(-1)
    assert nan.sum() == 2 and nan[0, 1] and nan[2, 0] and np.isnan(k[0, 1]).all()
    # (an infinite square sum gives x / inf = 0 for the finite ones and NaN for the infinite one)
    assert np.isnan(k[2, 0, 5 // 32 * 32:5 // 32 * 32 + 32]).all()
    assert np.isnan(v).any(-1).sum() == 1 and np.isnan(v[1, 0, :32]).all()
    assert np.all(v[3] == 0)


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_one_token_agrees_with_the_decode_steps_producer(layer):
    """gqa_prepare_decode on the same tokens: both round the same fp32 formulas, so they differ by one
    bf16 step at most."""
    lens = [1, 7, 30, 12]
    t = Tokens(layer, [1] * 4, lens, seed=27)
    one, many = ([torch.zeros((4, 32, t.KVH, t.D), dtype=torch.bfloat16, device="cuda") for _ in "kv"] for _ in "om")
    gqa.gqa_prepare_tokens(*t.args, i32(lens), t.q_out, *many)
    q = torch.empty_like(t.q)
    gqa.gqa_prepare_decode(t.q, t.k, t.v, t.wq, t.wk, i32(lens), q, *one)
    for a, b in zip([q, *one], [t.q_out, *many]):
        a, b = f64(a), f64(b)
        _, e = np.frexp(np.maximum(np.abs(a), np.abs(b)))
        head = np.abs(a).max(-1, keepdims=True)
        assert np.all(np.abs(a - b) <= np.exp2(e - 8.0) + 40 * 2.0 ** -24 * head)


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_many_tokens(layer):
    """More tokens than CTAs, long and short sequences: every token's q and codes."""
    B = 9
    new = [300, 1, 2, 77, 0, 513, 64, 65, 1000]
    lens = [n + 3 * i for i, n in enumerate(new)]
    t = Tokens(layer, new, lens, seed=28)
    cache = Cache(GEO[layer], B, 1024, True, seed=8)
    gqa.gqa_prepare_tokens_nibble_paged(*t.args, cache.table, i32(lens), t.q_out, cache.kv)
    near(t.q_out, t.exact()[0])
    check_codes(t, cache, 1024)
