"""GPU tests of gqa_decode_nibble[_paged] and of the 4-bit cache's calls together.

The reference is softmax(q k^T) v in 64 bits on the values that the cache's bytes stand for.  Tolerance
of an fp32 result: quant_reference.attend_tolerance, an fp32 evaluation whose weights carry at
least 16 bits; of a bf16 result, half a step of bf16 (2^-9 of its binade's top) more.
"""
import contextlib
import time

import numpy as np
import pytest
import torch

import decode_attention_gb300 as gqa
from decode_attention_gb300 import inputs
from tests import nibble_reference as nib
from tests.quant_precision import attend_and_bound
from tests.quant_reference import attend, attend_tolerance

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from tests.test_gpu_nibble import GEO, Cache, Tokens, check_codes, f64, i32, offsets, rows  # noqa: E402


def queries(geo, B, seed, size=0.25):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (size * torch.randn((B, geo["H"], geo["D"]), generator=g, device="cuda")).to(torch.bfloat16)


def filled(geo, B, S, paged, seed, poison=None, window=0):
    """A cache of random codes with scales around 1/3, so that values are of unit size.  poison: lengths;
    rows outside [L - window, L) get scale bytes and codes of 0xff."""
    cache = Cache(geo, B, S, paged, seed)
    rng = np.random.default_rng(seed)
    full = cache.want.shape[1]
    r = np.empty((B, full, cache.planes, 272), dtype=np.uint8)
    u = rng.integers(1, 16, (B, full, cache.planes, 512), dtype=np.uint8)
    r[..., :256] = u[..., 0::2] | (u[..., 1::2] << 4)
    r[..., 256:] = rng.integers(100, 110, (B, full, cache.planes, 16), dtype=np.uint8)
    for b, L in enumerate(poison if poison is not None else []):
        L = min(max(L, 0), full)
        r[b, L:] = 0xFF
        if window:
            r[b, :max(0, L - window)] = 0xFF
    cache.set_rows(r)
    cache.k, cache.v = nib.decode(cache.want, geo["D"])
    return cache


def run(cache, q, lens, window, **kw):
    return cache.fn("gqa_decode_nibble")(q, cache.kv, *cache.pages, i32(lens), window, **kw)


def check(cache, q, lens, window, out, skip=()):
    got, qd = f64(out), f64(q)
    G = q.shape[1] // cache.KVH
    for b, L in enumerate(lens):
        if b in skip:
            continue
        L = min(max(L, 0), cache.want.shape[1])
        lo = max(0, L - window) if window else 0
        for h in range(cache.KVH):
            k, v = cache.k[b, lo:L, h], cache.v[b, lo:L, h]
            qh = qd[b, h * G:(h + 1) * G]
            want = attend(qh, k, v)
            tol = attend_tolerance(qh, k, v)
            if out.dtype == torch.bfloat16:
                tol = tol + np.exp2(np.frexp(np.abs(want) + tol)[1] - 9.0)
            err = np.abs(got[b, h * G:(h + 1) * G] - want)
            assert np.all(err <= tol), (b, h, L, float(err.max()))


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 255, 256, 300]


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("window", [0, 1, 16, 50])
def test_lengths_and_windows(layer, paged, window):
    """Every place of a first and a last position within a page; all rows that are not attended are
    NaN; 32- and 16-bit results."""
    geo = GEO[layer]
    cache = filled(geo, len(LENS), 300, paged, 31, poison=LENS, window=window)
    q = queries(geo, len(LENS), 32)
    for dtype in (torch.float32, torch.bfloat16):
        out = run(cache, q, LENS, window, out_dtype=dtype)
        check(cache, q, LENS, window, out)
        assert torch.all(out[0] == 0)
    assert gqa.gqa_device_status() == 0


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("S", [1, 5, 16, 37])
def test_short_caches(layer, S):
    """A contiguous cache of odd length, filled to its last row, at the end of its memory."""
    geo = GEO[layer]
    lens = [S, max(S - 1, 0), S]
    cache = filled(geo, 3, S, False, 33, poison=lens)
    q = queries(geo, 3, 34)
    check(cache, q, lens, 0, run(cache, q, lens, 0, out_dtype=torch.float32))


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
def test_uneven_batches(layer, paged):
    """Long, short and empty sequences side by side: pieces in several units, dynamic chunks."""
    geo = GEO[layer]
    lens = [3, 2914, 130, 0, 1371, 40, 5000, 1, 640, 77, 16, 500] + [33 + 7 * i for i in range(20)]
    cache = filled(geo, len(lens), 5000, paged, 35)
    q = queries(geo, len(lens), 36)
    flush = torch.zeros(256 << 20, dtype=torch.uint8, device="cuda")
    for window in (0, 1024):
        outs = []
        for _ in range(4):
            flush.add_(1)
            outs.append(run(cache, q, lens, window, out_dtype=torch.float32))
        check(cache, q, lens, window, outs[0], skip=[b for b in range(len(lens)) if b > 11 and b % 4])
        assert all(torch.equal(o, outs[0]) for o in outs[1:]), "the same call twice"
        half = run(cache, q, lens, window)
        assert torch.equal(half, outs[0].to(torch.bfloat16))


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_largest_batch(layer):
    geo = GEO[layer]
    lens = [(i * 37) % 200 for i in range(256)]
    cache = filled(geo, 256, 200, True, 37, poison=lens)
    q = queries(geo, 256, 38)
    for window in (0, 30):
        out = run(cache, q, lens, window, out_dtype=torch.float32)
        check(cache, q, lens, window, out, skip=[b for b in range(256) if b % 5])


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
def test_precision(layer, paged):
    """Scores of a few units, where many positions carry weight: the bound of quant_precision, which
    holds weights to 20 bits."""
    geo = GEO[layer]
    lens = [2, 3, 16, 17, 33, 100, 1, 700, 2049]
    cache = filled(geo, len(lens), 2049, paged, 39)
    H, KVH, D = geo["H"], geo["KVH"], geo["D"]
    g = torch.Generator(device="cuda").manual_seed(40)
    q = (torch.randn((len(lens), H, D), generator=g, device="cuda") * 1.5 / D ** 0.5).bfloat16()
    for window in (0, 64):
        out, qd, G = f64(run(cache, q, lens, window, out_dtype=torch.float32)), f64(q), H // KVH
        for b, L in enumerate(lens):
            lo = max(0, L - window) if window else 0
            for h in range(KVH):
                o, bound = attend_and_bound(qd[b, h * G:(h + 1) * G], cache.k[b, lo:L, h], cache.v[b, lo:L, h], False)
                assert np.max(np.abs(out[b, h * G:(h + 1) * G] - o) - bound) <= 0, (b, h, L, window)


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 40.0, 1e4, 1e8, 1e20, 1e30])
def test_scores_of_any_size(layer, size):
    """Queries from vanishing to scores near fp32's end.  One channel of q is set, so that scores are
    exact products and the largest wins by whole units (or, tiny, all weigh the same)."""
    geo = GEO[layer]
    lens = [1, 40, 333]
    cache = filled(geo, 3, 333, False, 41)
    q = torch.zeros((3, geo["H"], geo["D"]), dtype=torch.bfloat16, device="cuda")
    q[..., 9] = size
    q[:, 1::2, 9] *= -1
    out = f64(run(cache, q, lens, 0, out_dtype=torch.float32))
    qd, G = f64(q), geo["H"] // geo["KVH"]
    for b, L in enumerate(lens):
        for h in range(geo["KVH"]):
            qh, k, v = qd[b, h * G:(h + 1) * G], cache.k[b, :L, h], cache.v[b, :L, h]
            want = attend(qh, k, v)
            # a score is one exact product and its product with log2 e, rounded: 2^-23 of it; it moves
            # a weight by as much, unless the next score is further away than any rounding
            s = np.abs(qh @ k.T).max()
            gap = np.diff(np.unique(qh[0] @ k.T)).min() if L > 1 and np.unique(k[:, 9]).size > 1 else 1.0
            if s * 2.0 ** -22 > 1e-3 and gap < 1000 + s * 2.0 ** -20:
                continue
            tol = min(s * 2.0 ** -22, 1e-3) * np.abs(v).max() * 2 + 2.0 ** -16 * np.abs(v).max()
            assert np.abs(out[b, h * G:(h + 1) * G] - want).max() <= tol, (b, h, size)


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("same_sign", [False, True])
def test_largest_queries_over_the_smallest_keys(layer, same_sign):
    """Queries around 2^127, of one sign or both (their sum is beyond fp32), over keys of the smallest
    scale: scores of some 2^110 to 2^120, finite, and 2^90 apart, so that one position of a head has all
    the weight."""
    geo = GEO[layer]
    lens = [1, 30, 200]
    cache = filled(geo, 3, 200, False, 55)
    r = cache.want.copy()
    r[..., 256:264] = 1
    cache.set_rows(r)
    cache.k, cache.v = nib.decode(cache.want, geo["D"])
    g = torch.Generator(device="cuda").manual_seed(56)
    q = torch.rand((3, geo["H"], geo["D"]), generator=g, device="cuda") + 0.9
    if not same_sign:
        q *= torch.sign(torch.rand(q.shape, generator=g, device="cuda") - 0.5)
    q = (q * 2.0 ** 126).to(torch.bfloat16)
    out, qd, G = f64(run(cache, q, lens, 0, out_dtype=torch.float32)), f64(q), geo["H"] // geo["KVH"]
    for b, L in enumerate(lens):
        for h in range(geo["KVH"]):
            s = qd[b, h * G:(h + 1) * G] @ cache.k[b, :L, h].T
            top = np.sort(s, axis=1)
            # (the rounding of D products in fp32, at most 2^-24 of each for 40 roundings in sequence, and
            # of the codes' offset of 8, up to 8 / 3 of them, may change the order of what is nearer)
            clear = np.ones(G, bool) if L == 1 else top[:, -1] - top[:, -2] > 2.0 ** -16 * np.abs(qd[b, h * G:(h + 1) * G]).sum(1) * 7 * 2.0 ** -17
            want = cache.v[b, s.argmax(1), h]
            assert np.isfinite(out[b]).all()
            assert np.abs(out[b, h * G:(h + 1) * G] - want)[clear].max(initial=0) <= 2.0 ** -16 * np.abs(want).max()
            assert L > 1 or clear.all()


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_scales_at_the_ends(layer):
    """Values of the smallest and the largest scales side by side, in K and in V."""
    geo = GEO[layer]
    lens = [50, 200]
    cache = filled(geo, 2, 200, False, 43)
    r = cache.want.copy()
    rng = np.random.default_rng(44)
    r[..., 264:] = rng.choice([0, 1, 7, 8, 60, 120, 160, nib.TOP], r[..., 264:].shape)
    r[..., 256:264] = rng.choice([0, 1, 8, 60, 100], r[..., 256:264].shape)
    r[1, ::3, :, 256:264] = nib.TOP
    cache.set_rows(r)
    cache.k, cache.v = nib.decode(cache.want, geo["D"])
    q = queries(geo, 2, 45, 2e-3)
    check(cache, q, lens, 0, run(cache, q, lens, 0, out_dtype=torch.float32))


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_values_that_are_not_numbers(layer):
    """NaN in an attended key: its head's outputs; in a value: its 32 channels of that head; NaN in a
    query: its own head alone."""
    geo = GEO[layer]
    H, KVH, D = geo["H"], geo["KVH"], geo["D"]
    G = H // KVH
    lens = [40, 40, 40, 40]
    cache = filled(geo, 4, 40, False, 46)
    r = cache.want.copy()
    r[0, 11, 0, 256 + 3] = 0xFF            # K of head 0
    r[1, 39, 0, 264 + 1] = 0xFF            # V of head 0, channels 32 .. 63
    cache.set_rows(r)
    cache.k, cache.v = nib.decode(cache.want, D)
    q = queries(geo, 4, 47)
    q[2, 5, 8] = float("nan")
    out = f64(run(cache, q, lens, 0, out_dtype=torch.float32))
    nan = np.isnan(out)
    want = np.zeros_like(nan)
    want[0, :G] = True
    want[1, :G, 32:64] = True
    want[2, 5] = True
    assert np.array_equal(nan, want)
    check(cache, q, lens, 0, run(cache, q, lens, 0, out_dtype=torch.float32), skip=(0, 1, 2))


def test_bad_pages_and_lengths():
    """A page out of range on an attended position: that sequence NaN, the others as ever, a status
    bit; past the attended range it is not looked at.  A bad length is clamped and reported."""
    for layer in ("sliding", "global"):
        geo = GEO[layer]
        lens = [60, 60, 60, 100, -5]
        cache = filled(geo, 5, 64, True, 48)
        ws = gqa.new_workspace(5, 64, geo["H"], geo["KVH"], geo["D"], 0)
        good = cache.host_table.copy()
        bad = good.copy()
        bad[0, 2], bad[1, 0] = cache.P, -1
        q = queries(geo, 5, 49)
        out = gqa.gqa_decode_nibble_paged(q, cache.kv, i32(bad), i32(lens), 20, out_dtype=torch.float32, workspace=ws)
        torch.cuda.synchronize()
        assert torch.isnan(out[0]).all()
        assert gqa.gqa_device_status(ws) == gqa.GQA_DEVICE_BAD_PAGE | gqa.GQA_DEVICE_BAD_LENGTH
        check(cache, q, lens, 20, out, skip=(0,))      # (sequence 1 attends 40 .. 59, sequence 3 is clamped to 64)
        assert torch.all(out[4] == 0)
        out = gqa.gqa_decode_nibble_paged(q, cache.kv, i32(good), i32([60] * 5), 20, workspace=ws)
        torch.cuda.synchronize()
        assert gqa.gqa_device_status(ws) == 0 and not torch.isnan(out).any()


def test_offsets_past_32_bits():
    """A contiguous cache of over 4 GB: the last sequence's rows lie beyond 2^32 bytes."""
    geo, S, B = GEO["sliding"], 262144, 4
    kv = torch.randint(0x11, 0x100, (B, 16, S, 272), dtype=torch.uint8, device="cuda")
    kv[..., 256:] = 104
    assert kv.numel() > 1 << 32
    lens = [5, 0, 1, S]
    q = queries(geo, B, 51)
    k, v = (rows(torch.Generator(device="cuda").manual_seed(s), 3, geo) for s in (52, 53))
    gqa.gqa_append_nibble(k, v, i32([0, 0, 0, 0, 3]), i32(lens), kv)
    got = gqa.gqa_decode_nibble(q, kv, i32(lens), 1024, out_dtype=torch.float32)
    tail = kv[3, :, S - 1024:].transpose(0, 1).cpu().numpy()
    assert np.array_equal(tail[-3:], nib.encode(f64(k), f64(v)))
    kd, vd = nib.decode(tail, 256)
    qd = f64(q)
    for h in range(16):
        a = (qd[3, 2 * h:2 * h + 2], kd[:, h], vd[:, h])
        assert np.abs(f64(got)[3, 2 * h:2 * h + 2] - attend(*a)).max() <= attend_tolerance(*a)
    ko, _ = gqa.gqa_read_nibble(kv, i32([0, 0, 0, S]), 2, torch.zeros((B, S, 16, 256), dtype=torch.bfloat16, device="cuda"),
                                torch.zeros((B, S, 16, 256), dtype=torch.bfloat16, device="cuda"))
    assert np.array_equal(f64(ko[3, -2:]), kd[-2:]) and torch.all(ko[:3] == 0)


# ---------------------------------------------------------------------------- together

@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
def test_prompts_then_steps(layer, paged):
    """Prompts of several lengths through the producer, then decode steps of one token each: cache and
    attention against the formulas from the raw projections on."""
    geo = GEO[layer]
    new = [40, 1, 17, 0, 64]
    window = 32 if layer == "sliding" else 0
    cache = Cache(geo, 5, 80, paged, seed=7)
    t = Tokens(layer, new, new, seed=61)
    cache.fn("gqa_prepare_tokens_nibble")(*t.args, *cache.pages, i32(t.lens), t.q_out, cache.kv)
    check_codes(t, cache, 80)
    lens = np.array(new)
    for s in range(3):
        lens = lens + 1
        t = Tokens(layer, [1] * 5, lens, seed=62 + s)
        cache.fn("gqa_prepare_tokens_nibble")(*t.args, *cache.pages, i32(lens), t.q_out, cache.kv)
        check_codes(t, cache, 80)
        out = run(cache, t.q_out, lens, window, out_dtype=torch.float32)
        cache.want = cache.host()
        cache.k, cache.v = nib.decode(cache.want, geo["D"])
        check(cache, t.q_out, lens, window, out)
        # what is read back is what was attended
        ko, vo = cache.fn("gqa_read_nibble")(cache.kv, *cache.pages, i32(lens), 0, out_dtype=torch.float32)
        for b, L in enumerate(lens):
            assert np.array_equal(f64(ko)[b, :L], cache.k[b, :L]) and np.array_equal(f64(vo)[b, :L], cache.v[b, :L])


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_draft_tokens_through_multi_query_decode(layer):
    """gqa_prepare_tokens ahead of gqa_decode_mq: T tokens each, attention by the formulas."""
    geo, T, B, S = GEO[layer], 4, 3, 64
    lens = [20, 4, 61]
    t = Tokens(layer, [T] * B, lens, seed=71)
    g = torch.Generator(device="cuda").manual_seed(72)
    caches = [torch.randn((B, S, t.KVH, t.D), generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]
    gqa.gqa_prepare_tokens(*t.args, i32(lens), t.q_out, *caches)
    q = (t.q_out * 0.1).to(torch.bfloat16).view(B, T, 32, t.D)
    out = f64(gqa.gqa_decode_mq(q, *caches, i32(lens), geo["window"], out_dtype=torch.float32))
    k, v = (f64(c) for c in caches)
    G = 32 // t.KVH
    for b in range(B):
        for j in range(T):
            L = lens[b] - T + j + 1
            for h in range(t.KVH):
                a = (f64(q)[b, j, h * G:(h + 1) * G], k[b, :L, h], v[b, :L, h])
                assert np.abs(out[b, j, h * G:(h + 1) * G] - attend(*a)).max() <= attend_tolerance(*a)


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_captured_step(layer):
    """Producer and attention of a step captured in a graph and replayed on new inputs and lengths."""
    geo, B, S = GEO[layer], 3, 900
    lens = np.array([5, 300, 899])
    cache = filled(geo, B, S, True, 81)
    t = Tokens(layer, [1] * B, lens, seed=82)
    ws = gqa.new_workspace(B, S, geo["H"], geo["KVH"], geo["D"], 0)
    seq, off, out = i32(lens), i32(range(B + 1)), torch.empty((B, 32, geo["D"]), device="cuda")

    def step():
        gqa.gqa_prepare_tokens_nibble_paged(t.q, t.k, t.v, t.wq, t.wk, off, cache.table, seq, t.q_out, cache.kv)
        gqa.gqa_decode_nibble_paged(t.q_out, cache.kv, cache.table, seq, geo["window"], out=out, workspace=ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for s in range(3):
        u = Tokens(layer, [1] * B, lens, seed=83 + s)
        for a, b in ((t.q, u.q), (t.k, u.k), (t.v, u.v)):
            a.copy_(b)
        seq.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        t.pos, t.lens = u.pos, u.lens
        cache.want = cache.host()
        cache.k, cache.v = nib.decode(cache.want, geo["D"])
        check(cache, t.q_out, lens, geo["window"], out)
        check_codes(t, cache, S)
        lens = np.minimum(lens + [1, 255, 0], S)
    assert gqa.gqa_device_status(ws) == 0


def test_two_calls_at_once():
    """Calls on two streams with a workspace each, on the same cache."""
    geo = GEO["global"]
    lens = [700, 33, 2000]
    cache = filled(geo, 3, 2000, False, 91)
    qs = [queries(geo, 3, 92 + i) for i in range(2)]
    want = [run(cache, q, lens, 0, out_dtype=torch.float32) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    wss = [gqa.new_workspace(3, 2000, geo["H"], geo["KVH"], geo["D"], 0, stream=s) for s in streams]
    outs = [torch.empty_like(want[0]) for _ in qs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for q, s, ws, o in zip(qs, streams, wss, outs):
            gqa.gqa_decode_nibble(q, cache.kv, i32(lens), 0, out=o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


@contextlib.contextmanager
def mode(flags):
    prev = gqa.gqa_set_test_mode(flags)
    try:
        yield
    finally:
        gqa.gqa_set_test_mode(prev)


FEW, MANY = "few", "many"


def batch(layer, count, lens):
    """`lens`, for MANY padded with short lengths to at least 2 * 152 segments: another form of the call."""
    B = 24 if layer == "sliding" else 80
    return lens + [(37 * i) % 150 for i in range(B - len(lens))] if count == MANY else lens


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("count", [FEW, MANY])
def test_one_piece_per_segment_agrees(layer, paged, count):
    """Split segments and their merge against GQA_TEST_SINGLE_PIECE, which has none: each within the
    tolerance of the reference."""
    geo = GEO[layer]
    lens = batch(layer, count, [1500, 33, 700, 0, 16])
    cache = filled(geo, len(lens), 1500, paged, 103)
    q = queries(geo, len(lens), 104)
    ws = gqa.new_workspace(len(lens), 1504, geo["H"], geo["KVH"], geo["D"], 0)
    segments = len(lens) * geo["KVH"]

    def pieces():
        torch.cuda.synchronize()
        e = ws[256:256 + 16 * segments].view(torch.int32).reshape(segments, 4).cpu().numpy()
        return (e[:, 1] + e[:, 3]).max()

    skip = [b for b in range(len(lens)) if b > 4 and b % 7]
    out = run(cache, q, lens, 0, out_dtype=torch.float32, workspace=ws)
    assert pieces() > 1
    check(cache, q, lens, 0, out, skip)
    with mode(gqa.GQA_TEST_SINGLE_PIECE):
        out = run(cache, q, lens, 0, out_dtype=torch.float32, workspace=ws)
    assert pieces() == 1
    check(cache, q, lens, 0, out, skip)


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("count", [FEW, MANY])
def test_stalled_call_takes_the_timeout_exit(layer, paged, count):
    """GQA_TEST_STALL: a producer waits 1 ms on a barrier that nothing completes.  The call ends, the
    status says so, and the workspace serves the next call."""
    geo = GEO[layer]
    lens = batch(layer, count, [1, 700, 2100, 3000])
    cache = filled(geo, len(lens), 3000, paged, 105)
    q = queries(geo, len(lens), 106)
    ws = gqa.new_workspace(len(lens), 3008, geo["H"], geo["KVH"], geo["D"], 0)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    with mode(gqa.GQA_TEST_STALL):
        run(cache, q, lens, 0, workspace=ws)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.0
    assert gqa.gqa_device_status(ws) & gqa.GQA_DEVICE_WAIT_TIMEOUT
    for _ in range(2):
        out = run(cache, q, lens, 0, out_dtype=torch.float32, workspace=ws)
        check(cache, q, lens, 0, out, [b for b in range(len(lens)) if b > 3 and b % 7])
    assert gqa.gqa_device_status(ws) == 0


def test_neighbours_stay_as_they_were():
    """The 8-bit and bf16 calls beside the new ones, on one workspace in turn."""
    geo = GEO["sliding"]
    lens = [100, 3]
    cache = filled(geo, 2, 100, False, 95)
    case = inputs.contiguous_case(2, 100, geo["H"], geo["KVH"], geo["D"], lens, 96, device="cuda")
    ws = gqa.new_workspace(2, 100, geo["H"], geo["KVH"], geo["D"], 0)
    args = (case["q"], case["k"], case["v"], case["seq_lens"], 0)
    want = gqa.gqa_decode(*args, workspace=ws)
    mine = run(cache, case["q"], lens, 0, workspace=ws)
    for _ in range(3):
        assert torch.equal(gqa.gqa_decode(*args, workspace=ws), want)
        assert torch.equal(run(cache, case["q"], lens, 0, workspace=ws), mine)
