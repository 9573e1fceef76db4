"""8-bit KV cache calls under the conditions that a serving loop meets and a single warm call
does not: cold caches, many pieces per CTA, test modes (a segment in one piece; a stalled
producer that takes the timeout exit), streams given by argument, captured graphs of whole
steps, and several calls at once.
"""
import contextlib
import time

import numpy as np
import pytest
import torch

import decode_attention_gb300 as gqa
from tests import quant_reference as ref
from tests.test_gpu_quant import (GEO, Cache, check_decode, filled, i32, producer_inputs, queries,
                                  rows, run_decode)

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@contextlib.contextmanager
def mode(flags):
    prev = gqa.gqa_set_test_mode(flags)
    try:
        yield
    finally:
        gqa.gqa_set_test_mode(prev)


# batches below and above the number of segments at which the decode call changes its units
FEW, MANY = "few", "many"


def batch(layer, count, lens):
    """`lens`, padded with short lengths to at least 2 * 152 segments for MANY."""
    if count == FEW:
        return lens
    B = 24 if layer == "sliding" else 80
    return lens + [(37 * i) % 150 for i in range(B - len(lens))]


def new_workspace(geo, B, S):
    return gqa.new_workspace(B, S, geo["H"], geo["KVH"], geo["D"], 0)


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
def test_cold_repeated_calls(layer, paged):
    """Calls after a write larger than L2, over a batch of very uneven lengths (many pieces per
    CTA, dynamic chunks, merges): all equal bit for bit, the first checked."""
    geo = GEO[layer]
    lens = [3, 2914, 130, 17, 1371, 40, 9000, 1, 640, 77, 16, 500]
    lens += [33 + 7 * i for i in range(40 if layer == "sliding" else 10)]
    cache = filled(geo, len(lens), max(lens), paged, seed=101)
    q = queries(geo, len(lens), 102)
    flush = torch.zeros(256 << 20, dtype=torch.uint8, device="cuda")
    for window in (0, 1024):
        outs = []
        for _ in range(8):
            flush.add_(1)
            outs.append(run_decode(cache, q, lens, window, out_dtype=torch.float32))
        torch.cuda.synchronize()
        check_decode(cache, q, lens, window, outs[0], skip=[b for b in range(len(lens)) if b > 8 and b % 5])
        assert all(torch.equal(o, outs[0]) for o in outs[1:])
    assert gqa.gqa_device_status() == 0


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("count", [FEW, MANY])
def test_one_piece_per_segment_agrees(layer, paged, count):
    """GQA_TEST_SINGLE_PIECE: one unit computes every segment whole.  Both sides carry weights to
    at least 2^-16 and fp32 sums in another order: each lies within attend_tolerance of the
    reference, which check_decode holds both to."""
    geo = GEO[layer]
    lens = batch(layer, count, [1500, 33, 700, 0, 16])
    cache = filled(geo, len(lens), 1500, paged, seed=103)
    q = queries(geo, len(lens), 104)
    ws = new_workspace(geo, len(lens), 1504)
    segments = len(lens) * geo["KVH"]

    def pieces():
        e = ws[256:256 + 16 * segments].view(torch.int32).reshape(segments, 4).cpu().numpy()
        return e[:, 1] + e[:, 3]

    out = run_decode(cache, q, lens, 0, out_dtype=torch.float32, workspace=ws)
    torch.cuda.synchronize()
    assert pieces().max() > 1
    check_decode(cache, q, lens, 0, out)
    with mode(gqa.GQA_TEST_SINGLE_PIECE):
        out = run_decode(cache, q, lens, 0, out_dtype=torch.float32, workspace=ws)
    torch.cuda.synchronize()
    assert pieces().max() == 1
    check_decode(cache, q, lens, 0, out)


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("count", [FEW, MANY])
def test_stalled_call_takes_the_timeout_exit(layer, paged, count):
    """GQA_TEST_STALL: a producer waits 1 ms on a barrier that nothing completes.  The call
    ends, the status says so, and the workspace serves the next call."""
    geo = GEO[layer]
    lens = batch(layer, count, [1, 700, 2100, 3000])
    cache = filled(geo, len(lens), 3000, paged, seed=105)
    q = queries(geo, len(lens), 106)
    ws = new_workspace(geo, len(lens), 3008)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    with mode(gqa.GQA_TEST_STALL):
        run_decode(cache, q, lens, 0, workspace=ws)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.0
    assert gqa.gqa_device_status(ws) & gqa.GQA_DEVICE_WAIT_TIMEOUT
    for _ in range(2):
        out = run_decode(cache, q, lens, 0, out_dtype=torch.float32, workspace=ws)
        torch.cuda.synchronize()
        check_decode(cache, q, lens, 0, out)
    assert gqa.gqa_device_status(ws) == 0


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_captured_step(layer):
    """Append, producer, attention and read-back captured as one graph and replayed over changed
    inputs: each replay equals the same calls made one by one on a cache in the same state."""
    geo, S, B = GEO[layer], 64, 3
    H, KVH, D = geo["H"], geo["KVH"], geo["D"]
    gen = torch.Generator(device="cuda").manual_seed(107)
    lens = [20, 7, 41]
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    k_new, v_new = rows(gen, (off[-1], KVH, D)), rows(gen, (off[-1], KVH, D))
    raw = producer_inputs(geo, B, 108)
    args = (raw["q_raw"], raw["k_raw"], raw["v_raw"], raw["w_q"], raw["w_k"])
    seq, seq1, offs = i32(lens), i32([L + 1 for L in lens]), i32(off)
    ws = new_workspace(geo, B, S)

    def state():
        c = Cache(geo, B, S, False)
        return c, torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda"), \
            torch.zeros(B, H, D, device="cuda"), \
            [torch.zeros(B, S, KVH, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]

    def step(c, q_out, out, outs):
        gqa.gqa_append_quant(k_new, v_new, offs, seq, *c.args)
        gqa.gqa_prepare_decode_quant(*args, seq1, q_out, *c.args)
        gqa.gqa_decode_quant(q_out, *c.args, seq1, 0, out=out, workspace=ws)
        gqa.gqa_read_quant(*c.args, seq1, 0, *outs)

    live = state()
    step(*live)                       # (also: first use of each kernel ahead of the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*live)
    for i in range(3):
        for x in (k_new, v_new, raw["q_raw"], raw["k_raw"], raw["v_raw"]):
            x.copy_(rows(gen, x.shape))
        graph.replay()
        torch.cuda.synchronize()
        plain = state()
        step(*plain)
        torch.cuda.synchronize()
        assert torch.equal(live[1], plain[1]) and torch.equal(live[2], plain[2])
        for t in range(2):
            assert torch.equal(live[3][t], plain[3][t])
            for b, L in enumerate(lens):
                assert torch.equal(live[0].codes[t].view(torch.uint8)[b, :L + 1],
                                   plain[0].codes[t].view(torch.uint8)[b, :L + 1])
    assert gqa.gqa_device_status(ws) == 0


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_streams_given_by_argument(layer):
    """Two whole steps at once on two streams passed as arguments, caches and workspaces of their
    own, while the current stream is another."""
    geo, S, B = GEO[layer], 320, 2
    KVH, D = geo["KVH"], geo["D"]
    gen = torch.Generator(device="cuda").manual_seed(109)
    lens = [300, 123]
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    streams = [torch.cuda.Stream() for _ in range(2)]
    todo = []
    for i in range(2):
        c = Cache(geo, B, S, i == 1, seed=i)
        todo.append((c, rows(gen, (off[-1], KVH, D)), rows(gen, (off[-1], KVH, D)),
                     queries(geo, B, 110 + i), new_workspace(geo, B, S),
                     torch.zeros(B, geo["H"], D, device="cuda")))
    offs, seq = i32(off), i32(lens)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (c, kn, vn, q, ws, out) in zip(streams, todo):
            if c.paged:
                gqa.gqa_append_quant_paged(kn, vn, offs, c.table, seq, *c.args, stream=s)
                gqa.gqa_decode_quant_paged(q, *c.args, c.table, seq, 0, out=out, workspace=ws, stream=s)
            else:
                gqa.gqa_append_quant(kn, vn, offs, seq, *c.args, stream=s)
                gqa.gqa_decode_quant(q, *c.args, seq, 0, out=out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c, kn, vn, q, ws, out in todo:
        for t, x in enumerate((kn, vn)):
            x = x.double().cpu().numpy()
            for b in range(B):
                for h in range(KVH):
                    c.ref[t][b][h].append(x[off[b]:off[b + 1], h], 0)
        check_decode(c, q, lens, 0, out)
        assert gqa.gqa_device_status(ws) == 0


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_many_segments_repeated(layer):
    """A batch of many segments, some of them long: equal calls, all sequences checked."""
    geo = GEO[layer]
    B = 40 if layer == "sliding" else 90
    lens = [(61 * i) % 700 for i in range(B - 2)] + [3300, 5000]
    cache = filled(geo, B, 5000, True, seed=115)
    q = queries(geo, B, 116)
    outs = [run_decode(cache, q, lens, 0, out_dtype=torch.float32) for _ in range(6)]
    torch.cuda.synchronize()
    check_decode(cache, q, lens, 0, outs[0])
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


def test_one_tensor_as_keys_and_values():
    """Keys and values may be the same cache (both are only read)."""
    geo, lens = GEO["global"], [200, 31]
    cache = filled(geo, 2, 200, False, seed=111)
    q = queries(geo, 2, 112)
    k, ks = cache.codes[0], cache.scales[0]
    out = gqa.gqa_decode_quant(q, k, k, ks, ks, i32(lens), 0, out_dtype=torch.float32)
    cache.ref[1] = cache.ref[0]
    check_decode(cache, q, lens, 0, out)


def test_positions_beyond_32_bit_offsets():
    """A cache of more than 2^32 codes: the last sequence and position are written, read and
    attended."""
    geo, S = GEO["sliding"], 16384
    B = 66                                            # 66 * 16384 * 4096 > 2^32
    k = torch.zeros((B, S, 16, 256), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.zeros((B, S, 16, 256), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ks, vs = (torch.zeros(B, S // 16, 16, device="cuda") for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(113)
    n = 100
    kn, vn = rows(gen, (n, 16, 256)), rows(gen, (n, 16, 256))
    lens = [0] * (B - 1) + [S]
    off = [0] * B + [n]
    gqa.gqa_append_quant(kn, vn, i32(off), i32(lens), k, v, ks, vs)
    q = queries(geo, B, 114)
    out = gqa.gqa_decode_quant(q, k, v, ks, vs, i32(lens), n, out_dtype=torch.float32)
    torch.cuda.synchronize()
    host_q = q[B - 1].double().cpu().numpy()
    for h in range(16):
        seqs = []
        for x in (kn, vn):
            s = ref.Sequence(112, 256)
            s.v[:] = 0.0
            s.e[:] = -64                              # zero scales
            s.append(x[:, h].double().cpu().numpy(), 12)   # 16384 - 100 = 12 modulo 16
            seqs.append(s.stored(12, 112))
        want = ref.attend(host_q[2 * h:2 * h + 2], *seqs)
        tol = ref.attend_tolerance(host_q[2 * h:2 * h + 2], *seqs)
        got = out[B - 1, 2 * h:2 * h + 2].double().cpu().numpy()
        assert np.max(np.abs(got - want)) <= tol
    assert torch.all(k.view(torch.uint8)[:B - 1] == 0)
    assert torch.all(k.view(torch.uint8)[B - 1, :S - n] == 0)


@pytest.mark.parametrize("layer,count", [("sliding", 9), ("sliding", 10), ("global", 4), ("global", 5)])
def test_partials_of_few_and_more_segments(layer, count):
    """Batches on both sides of the step between the forms of the combine kernel, with pieces
    in numbers from none (an empty sequence) to dozens."""
    geo = GEO[layer]
    lens = [6000 if layer == "global" else 2500, 0, 16, 1100, 333, 1, 1500, 1023, 97, 700][:count]
    cache = filled(geo, count, max(lens), True, seed=121)
    q = queries(geo, count, 122)
    out = run_decode(cache, q, lens, 0, out_dtype=torch.float32)
    check_decode(cache, q, lens, 0, out)
    assert torch.all(out[1] == 0)
    assert torch.equal(out, run_decode(cache, q, lens, 0, out_dtype=torch.float32))
    bad = cache.table.clone()
    bad[0, 60] = -1                                    # one piece of many is NaN
    got = run_decode(cache, q, lens, 0, table=bad, out_dtype=torch.float32)
    assert torch.all(torch.isnan(got[0])) and torch.equal(got[1:], out[1:])
    assert gqa.gqa_device_status() == gqa.GQA_DEVICE_BAD_PAGE
