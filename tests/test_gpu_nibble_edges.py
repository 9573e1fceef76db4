"""GPU tests of the 4-bit cache's calls where rounding decides: scores of thousands, whose largest has
all the weight; codes at the longest cache's last positions, of the largest batch, and of values
next to a border between codes; batches that are mostly padding; keys given as values.

Every test counts what it compares.
"""
import numpy as np
import pytest
import torch

import decode_attention_gb300 as gqa
from tests import nibble_reference as nib
from tests.quant_precision import attend_and_bound

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from tests.test_gpu_nibble import GEO, ROPE, Cache, Tokens, check_codes, f64, i32, near  # noqa: E402
from tests.test_gpu_nibble_decode import check, filled, queries, run  # noqa: E402

LENS = [1, 40, 333]


def one_channel_keys(cache, channel, order, seed):
    """Sets a channel of every key to a code of its own, random or rising with the position, times 1/4."""
    rng = np.random.default_rng(seed)
    r = cache.want.copy()
    B, S = r.shape[:2]
    u = rng.integers(1, 16, (B, S, cache.KVH))
    if order == "rising":
        for b, L in enumerate(LENS):
            u[b, :L].sort(axis=0)
    per = cache.D // 256
    byte, shift, c = channel % 256 // 2, 4 * (channel % 2), channel % 256
    planes = np.arange(cache.KVH) * per + channel // 256
    r[:, :, planes, byte] = (r[:, :, planes, byte] & (0xF0 >> shift)) | (u << shift)
    r[:, :, planes, 256 + c // 32] = 104      # 2^-2
    cache.set_rows(r)
    cache.k, cache.v = nib.decode(cache.want, cache.D)
    assert np.array_equal(cache.k[..., channel], (u - 8) / 4)


@pytest.mark.parametrize("layer,channel", [("sliding", 9), ("sliding", 254), ("global", 9), ("global", 509)])
@pytest.mark.parametrize("order", ["random", "rising"])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1.0, 40.0, 1e3, 4e3, 1e4, 2.4e4, 1e6, 1e8, 1e20, 1e30, 1e37])
def test_one_channel_decides(layer, channel, order, size):
    """One channel of q is set, so a score is one exact product, rounded twice (by log2 e and its product):
    2^-23 of it.  Equal scores stay equal.  From size 1000 on others are 250 apart or more, which rounding
    moves by 2^-22 of their size, 2^-18 of their distance at most: the positions of the largest share the weight.
    Below, attend_and_bound, and 2^-32 of the largest for each weight that is rounded to nothing."""
    geo = GEO[layer]
    cache = filled(geo, 3, 333, False, 41)
    one_channel_keys(cache, channel, order, 42)
    q = torch.zeros((3, geo["H"], geo["D"]), dtype=torch.bfloat16, device="cuda")
    q[..., channel] = size
    q[:, 1::2, channel] *= -1
    out = f64(run(cache, q, LENS, 0, out_dtype=torch.float32))
    qd, G = f64(q), geo["H"] // geo["KVH"]
    compared = 0
    for b, L in enumerate(LENS):
        for h in range(geo["KVH"]):
            qh, k, v = qd[b, h * G:(h + 1) * G], cache.k[b, :L, h], cache.v[b, :L, h]
            if size < 1000:
                want, bound = attend_and_bound(qh, k, v, True)
                bound = bound + L * 2.0 ** -32 * np.abs(v).max()
            else:
                s = qh @ k.T
                w = (s == s.max(axis=1, keepdims=True)).astype(np.float64)
                w /= w.sum(axis=1, keepdims=True)
                want = w @ v
                # weights to 22 bits, chains of sums as in attend_and_bound
                bound = (2.0 ** -20 + 2 * ((L + 15) // 16 / 2 + 8) * 2.0 ** -24) * (w @ np.abs(v))
            assert np.all(np.abs(out[b, h * G:(h + 1) * G] - want) <= bound), (b, h)
            compared += G
    assert compared == 3 * geo["H"]


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("size", [100.0, 300.0, 1000.0])
def test_scores_of_thousands(layer, size):
    """All channels set.  Where the largest score is clear of the others by 60 and twice the bound of
    their fp32 sums (40 roundings of the sum of magnitudes), the output is its position's value, and of
    the others' at most 333 e^-60 < 2^-78 (log2 of it is 8.4 - 86.5)."""
    geo = GEO[layer]
    cache = filled(geo, 3, 333, True, 43)
    q = queries(geo, 3, 44, size)
    out, qd, G = f64(run(cache, q, LENS, 0, out_dtype=torch.float32)), f64(q), geo["H"] // geo["KVH"]
    compared = 0
    for b, L in enumerate(LENS):
        for h in range(geo["KVH"]):
            qh, k, v = qd[b, h * G:(h + 1) * G], cache.k[b, :L, h], cache.v[b, :L, h]
            s = qh @ k.T
            err = 40 * 2.0 ** -24 * (np.abs(qh) @ np.abs(k).T).max(axis=1)
            top = np.sort(s, axis=1)
            clear = np.ones(G, bool) if L == 1 else top[:, -1] - top[:, -2] > 60 + 2 * err
            want = v[s.argmax(axis=1)]
            bound = 2.0 ** -19 * np.abs(want) + 2.0 ** -78 * np.abs(v).max()
            over = (np.abs(out[b, h * G:(h + 1) * G] - want) - bound)[clear]
            assert over.max(initial=0.0) <= 0, (b, h, over.max())
            compared += clear.sum()
    assert compared >= 0.8 * 3 * geo["H"]


# ---------------------------------------------------------------------------- codes

def expected_rows(t):
    """Rows of every token [N, planes, 272], and where 2^-27 may change one."""
    _, k, v = t.exact()
    rows = nib.encode(nib.bf16(k), nib.bf16(v))
    doubt = np.zeros(rows.shape, dtype=bool)
    for which, x in ((0, k), (1, v)):
        d = nib.bf16_doubt(x, 2.0 ** -27).reshape(len(x), -1, 8, 32).any(-1)
        doubt[..., 128 * which:128 * which + 128] = np.repeat(d, 16, -1)
        doubt[..., 256 + 8 * which:264 + 8 * which] = d
    return rows, doubt


FAR = dict(new=[40, 17, 33], lens=[262144, 200001, 131073])


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_codes_at_far_positions(layer):
    """Positions up to the longest cache's last.  Only the pages of the new tokens exist, and of those
    not the first: the others' entries are out of range."""
    t = Tokens(layer, **FAR, seed=31)
    planes = t.KVH * t.D // 256
    table = np.full((3, 16384), -1, dtype=np.int32)
    for b in range(3):
        blocks = np.unique(t.pos[t.off[b]:t.off[b + 1]] // 16)
        table[b, blocks] = 0
    table[0, (262144 - 40) // 16] = -1
    n = int((table >= 0).sum())
    table[table >= 0] = np.random.default_rng(32).permutation(n)
    pages = torch.full((n, planes, 16, 272), 0x5A, dtype=torch.uint8, device="cuda")
    gqa.gqa_prepare_tokens_nibble_paged(*t.args, i32(table), i32(t.lens), t.q_out, pages)
    near(t.q_out, t.exact()[0])
    rows, doubt = expected_rows(t)
    got, written = pages.cpu().numpy(), np.zeros((n, 16), dtype=bool)
    for b in range(3):
        for i in range(t.off[b], t.off[b + 1]):
            page, slot = table[b, t.pos[i] // 16], t.pos[i] % 16
            if page >= 0:
                written[page, slot] = True
                assert np.array_equal(np.where(doubt[i], 0, got[page, :, slot]), np.where(doubt[i], 0, rows[i])), (b, i)
    assert written.sum() == 90 - 8 and doubt.mean() < 1e-3
    assert np.all(got.transpose(0, 2, 1, 3)[~written] == 0x5A)


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_codes_at_the_end_of_the_longest_contiguous_cache(layer):
    t = Tokens(layer, [70], [262144], seed=33)
    kv = torch.full((1, t.KVH * t.D // 256, 262144, 272), 0x5A, dtype=torch.uint8, device="cuda")
    gqa.gqa_prepare_tokens_nibble(*t.args, i32(t.lens), t.q_out, kv)
    rows, doubt = expected_rows(t)
    got = kv[0, :, -70:].transpose(0, 1).cpu().numpy()
    assert np.array_equal(np.where(doubt, 0, got), np.where(doubt, 0, rows)) and doubt.mean() < 1e-3
    assert torch.all(kv[0, :, :-70] == 0x5A)


def test_codes_of_the_largest_batch():
    """256 sequences of one new token each; those of length 97 do not fit."""
    t = Tokens("global", [1] * 256, [1 + 5 * b % 97 for b in range(256)], seed=66)
    cache = Cache(GEO["global"], 256, 96, True, seed=3)
    gqa.gqa_prepare_tokens_nibble_paged(*t.args, cache.table, i32(t.lens), t.q_out, cache.kv)
    near(t.q_out, t.exact()[0])
    rows, doubt = expected_rows(t)
    skip = np.zeros(cache.want.shape, dtype=bool)
    fits = [b for b in range(256) if t.lens[b] <= 96]
    for b in fits:
        cache.want[b, t.lens[b] - 1], skip[b, t.lens[b] - 1] = rows[b], doubt[b]
    assert 200 < len(fits) < 256 and doubt.mean() < 1e-3
    cache.check(skip)


@pytest.mark.parametrize("paged", [False, True])
def test_keys_as_values(paged):
    """A layer without a value projection: k_raw is v_raw too, normed without weight or rotation."""
    t = Tokens("global", [3, 0, 1, 16, 70], [3, 5, 90, 31, 70], seed=34, keqv=True)
    cache = Cache(GEO["global"], 5, 96, paged, seed=6)
    cache.fn("gqa_prepare_tokens_nibble")(t.q, t.k, t.k, t.wq, t.wk, i32(t.off), *cache.pages, i32(t.lens), t.q_out,
                                          cache.kv)
    check_codes(t, cache, 96)


BORDER, LEAST = 2.0 ** -23, 2.0 ** -26   # relative distances of a value from a border


def border_vectors(layer, keys, pos, wk, gen):
    """Random raw head vectors of which one value lies between LEAST and BORDER of itself from a border
    of bf16 that is one of its codes or of their scale, by the formulas in 64 bits: raw [n, D] on the GPU
    and the index into pos of each.  (Not values that a rotation leaves below an eighth of what it adds up:
    an error of 2^-30 of that is 2^-27 of them, below LEAST.)"""
    D = GEO[layer]["D"]
    pairs, theta = ROPE[layer]
    M = (1 << 26) // D
    raw = torch.randn((M, D), generator=gen, device="cuda").to(torch.bfloat16)
    which = torch.arange(M, device="cuda") % len(pos)
    y = raw.double()
    y /= (y.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    parts = y.abs()
    if keys:
        y *= wk.double()
        a = torch.tensor(pos, dtype=torch.float64, device="cuda")[:, None] * theta ** (
            -2.0 * torch.arange(pairs, dtype=torch.float64, device="cuda") / D)
        c, s = a.cos()[which], a.sin()[which]
        lo, hi = y[:, :pairs].clone(), y[:, D // 2:D // 2 + pairs].clone()
        y[:, :pairs], y[:, D // 2:D // 2 + pairs] = lo * c - hi * s, hi * c + lo * s
        parts = y.abs()
        parts[:, :pairs] = parts[:, D // 2:D // 2 + pairs] = lo.abs() + hi.abs()
    unit = torch.exp2(torch.frexp(y)[1].double() - 8)            # a step of bf16
    off = y.abs() / unit
    off = ((off - off.floor() - 0.5).abs() * unit / y.abs())     # relative distance from a border
    vec, ch = torch.nonzero((off < BORDER) & (off > LEAST) & (8 * y.abs() > parts), as_tuple=True)
    group = y.view(M, -1, 32)[vec, ch // 32].cpu().numpy()
    at = (ch % 32).cpu().numpy()[:, None] == np.arange(32)
    ends = [nib.code_group(nib.bf16(np.where(at, group * (1 + d * 2 * BORDER), group))) for d in (-1, 1)]
    differ = (ends[0][0] != ends[1][0]) | (ends[0][1] != ends[1][1]).any(-1)
    vec = torch.unique(vec[torch.tensor(differ, device="cuda")])
    return raw[vec], which[vec].cpu().numpy()


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("keys", [False, True])
@pytest.mark.parametrize("far", [False, True])
def test_values_next_to_a_border_between_codes(layer, keys, far):
    """Every key (or value) head has a value within two units of 2^-24 of a border between two codes, on
    either side, which fp32's own error may cross: the codes are those of the formulas in 64 bits."""
    geo, n = GEO[layer], 24
    L = 262144 if far else n
    t = Tokens(layer, [n], [L], seed=35)
    slots, gen = geo["KVH"], torch.Generator(device="cuda").manual_seed(36)
    have = np.zeros(n, dtype=int)
    to = t.k if keys else t.v
    for _ in range(60):
        raw, which = border_vectors(layer, keys, t.pos, t.wk, gen)
        for x, i in zip(raw, which):
            if have[i] < slots:
                to[i, have[i]] = x
                have[i] += 1
        if have.min() == slots:
            break
    assert have.min() == slots
    nblk = L // 16 + 1
    table = np.full((1, nblk), -1, dtype=np.int32)
    first = (L - n) // 16
    table[0, first:] = np.arange(nblk - first)
    pages = torch.zeros((nblk - first, geo["KVH"] * geo["D"] // 256, 16, 272), dtype=torch.uint8, device="cuda")
    gqa.gqa_prepare_tokens_nibble_paged(*t.args, i32(table[:, :16384]), i32([L]), t.q_out, pages)
    rows, doubt = expected_rows(t)
    got = pages.transpose(1, 2).reshape(-1, *rows.shape[1:]).cpu().numpy()[(L - n) % 16:][:n]
    wrong = (got != rows) & ~doubt
    assert not wrong.any(), (wrong.any(-1).sum(), "planes differ")
    # (the fp32 number that such a value rounds to changes in one place in some 14 of where it may lie, and a vector's
    # values of one mantissa lie alike: most heads are compared whole)
    heads = doubt.reshape(n, geo["KVH"], -1, 272)[..., slice(256, 264) if keys else slice(264, 272)].any((-1, -2))
    assert heads.mean() < 1 / 3


# ---------------------------------------------------------------------------- padding

@pytest.mark.parametrize("layer,lens", [("sliding", [1024] + [0] * 15), ("sliding", [0] * 7 + [1500]),
                                        ("sliding", [0, 400, 0, 0]), ("sliding", [0] * 255 + [700]),
                                        ("global", [8192] + [0] * 31), ("global", [0, 0, 2048, 0]),
                                        ("global", [0] * 40 + [20000, 3] + [0] * 60), ("global", [0] * 5)])
@pytest.mark.parametrize("paged", [False, True])
def test_batches_that_are_mostly_padding(layer, lens, paged):
    """Few sequences beside empty ones, whose rows are zeros; the same sequences alone, within the same
    tolerance; the same call twice, the same bits."""
    geo = GEO[layer]
    there = [b for b, L in enumerate(lens) if L]
    cache = filled(geo, max(1, len(there)), max(16, *lens), paged, 64)
    B, q = len(lens), queries(geo, len(lens), 65)
    own = [lens[b] for b in there]
    if paged:
        table = torch.full((B, cache.table.shape[1]), -1, dtype=torch.int32, device="cuda")
        table[there] = cache.table[:len(there)]
        args = (cache.kv, table)
    else:
        kv = torch.full((B, *cache.kv.shape[1:]), 0xFF, dtype=torch.uint8, device="cuda")
        kv[there] = cache.kv[:len(there)]
        args = (kv,)
    outs = [cache.fn("gqa_decode_nibble")(q, *args, i32(lens), geo["window"], out_dtype=torch.float32) for _ in range(2)]
    assert torch.equal(*outs)
    empty = [b for b in range(B) if not lens[b]]
    assert torch.all(outs[0][empty] == 0)
    if there:
        check(cache, q[there], own, geo["window"], outs[0][there])
        check(cache, q[there], own, geo["window"], run(cache, q[there].contiguous(), own, geo["window"], out_dtype=torch.float32))
    assert gqa.gqa_device_status() == 0
