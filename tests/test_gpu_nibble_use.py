"""GPU tests of the 4-bit cache's calls as a serving loop makes them: first calls inside a capture, graphs
that share a workspace, batches padded behind their last sequence, and every choice of units."""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import decode_attention_gb300 as gqa
from decode_attention_gb300 import inputs

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from tests.test_gpu_nibble import FILL, GEO, Cache, Tokens, f64, i32, near, rows  # noqa: E402
from tests.test_gpu_nibble_decode import check, filled, queries, run  # noqa: E402

# Nothing of the library has run in this process but the workspace's making.
FIRST_CALLS = """
import torch
import decode_attention_gb300 as gqa
KVH, D, planes = {KVH}, {D}, {KVH} * {D} // 256
make = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
off, lens, table = i32([0, 3, 8]), i32([3, 40]), i32([[4, 1, 0], [2, 5, 3]])
q, k, v, wq, wk = make(8, 32, D), make(8, KVH, D), make(8, KVH, D), make(D), make(D)
kv = torch.zeros((6, planes, 16, 272), dtype=torch.uint8, device="cuda")
kb, vb = (torch.zeros((6, 16, KVH, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
q_out, last = torch.zeros_like(q), torch.zeros((2, 32, D), dtype=torch.bfloat16, device="cuda")
out = torch.zeros((2, 32, D), device="cuda")
ko, vo = (torch.zeros((2, 48, KVH, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
ws = gqa.new_workspace(2, 48, 32, KVH, D, 0)

def step():
    gqa.gqa_append_nibble_paged(k, v, off, table, lens, kv)
    gqa.gqa_prepare_tokens_paged(q, k, v, wq, wk, off, table, lens, q_out, kb, vb)
    gqa.gqa_prepare_tokens_nibble_paged(q, k, v, wq, wk, off, table, lens, q_out, kv)
    gqa.gqa_decode_nibble_paged(q_out[2::5].contiguous(), kv, table, lens, 7, out=out, workspace=ws)
    gqa.gqa_read_nibble_paged(kv, table, lens, 7, ko, vo)

results = (kv, kb, vb, q_out, out, ko, vo)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
captured = [x.clone() for x in results]
for x in results:
    x.zero_()
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, results))
assert out.abs().max() > 0 and gqa.gqa_device_status(ws) == 0
print("agree")
"""


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_first_calls_inside_a_capture(layer):
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(KVH=GEO[layer]["KVH"], D=GEO[layer]["D"])],
                       cwd=Path(__file__).parents[1], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("agree"), r.stderr[-2000:]


def graph_of(call):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


def test_graphs_that_share_a_workspace():
    """A captured decode over the 4-bit cache and one over a bf16 cache, replayed by turns on one stream."""
    geo = GEO["global"]
    lens = [3000, 17, 1200]
    cache = filled(geo, 3, 3000, True, 61)
    case = inputs.contiguous_case(3, 3000, geo["H"], geo["KVH"], geo["D"], lens, 62, device="cuda")
    ws = gqa.new_workspace(3, 3008, geo["H"], geo["KVH"], geo["D"], 0)
    mine, other = (torch.empty((3, 32, geo["D"]), device="cuda") for _ in range(2))
    seq = i32(lens)
    graphs = (graph_of(lambda: gqa.gqa_decode_nibble_paged(case["q"], cache.kv, cache.table, seq, 0, out=mine, workspace=ws)),
              graph_of(lambda: gqa.gqa_decode(case["q"], case["k"], case["v"], case["seq_lens"], 0, out=other, workspace=ws)))
    want = run(cache, case["q"], lens, 0, out_dtype=torch.float32)
    beside = gqa.gqa_decode(case["q"], case["k"], case["v"], case["seq_lens"], 0, out_dtype=torch.float32)
    check(cache, case["q"], lens, 0, want)
    for turn in range(4):
        mine.fill_(3.0)
        other.fill_(3.0)
        for g in graphs if turn % 2 else graphs[::-1]:
            g.replay()
        assert torch.equal(mine, want) and torch.equal(other, beside)
    assert gqa.gqa_device_status(ws) == 0


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("call", ["append", "tokens", "step"])
def test_rows_behind_the_last_sequence(layer, call):
    """A packed batch padded to a fixed number of tokens, and a batch padded with empty sequences."""
    t = Tokens(layer, [4, 0, 2, 7], [4, 9, 30, 18], seed=63)
    off = i32([0, 4, 4, 6, 6])                      # the last seven tokens are padding
    lens = i32([4, 9, 30, 0])
    geo = GEO[layer]
    q, k, v = t.exact()
    if call == "tokens":
        kb, vb = (torch.full((4, 32, t.KVH, t.D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        gqa.gqa_prepare_tokens(t.q, t.k, t.v, t.wq, t.wk, off, lens, t.q_out, kb, vb)
        for c, want in ((kb, k), (vb, v)):
            near(c[0, :4], want[:4])
            near(c[2, 28:30], want[4:6])
            assert torch.all(c[0, 4:] == 3.0) and torch.all(c[2, :28] == 3.0) and torch.all(c[2, 30:] == 3.0)
            assert torch.all(c[1] == 3.0) and torch.all(c[3] == 3.0)
    else:
        cache = Cache(geo, 4, 32, True, seed=2)
        if call == "append":
            gqa.gqa_append_nibble_paged(t.k, t.v, off, cache.table, lens, cache.kv)
            cache.note(f64(t.k), f64(t.v), [0, 4, 4, 6, 6], [4, 9, 30, 0])
            cache.check()
        else:
            gqa.gqa_prepare_tokens_nibble_paged(t.q, t.k, t.v, t.wq, t.wk, off, cache.table, lens, t.q_out, cache.kv)
            got = cache.host()
            assert np.all(got[[1, 3]] == FILL) and np.all(got[0, 4:] == FILL)
            assert np.all(got[2, :28] == FILL) and np.all(got[2, 30:] == FILL)
            assert not np.any(np.all(got[0, :4] == FILL, axis=-1)) and not np.any(np.all(got[2, 28:30] == FILL, axis=-1))
    if call != "append":
        near(t.q_out[:6], q[:6])
        assert torch.all(t.q_out[6:] == 3.0)


# positions of a sequence, batch: few positions in long segments take one or two units of a CTA's three
@pytest.mark.parametrize("layer,B,L", [("sliding", 1, 400), ("sliding", 1, 1500), ("sliding", 3, 1500), ("sliding", 5, 1024),
                                       ("sliding", 8, 1040), ("sliding", 16, 100), ("global", 1, 2048), ("global", 1, 8192),
                                       ("global", 1, 16384), ("global", 2, 5001), ("global", 1, 32768), ("global", 16, 100)])
@pytest.mark.parametrize("paged", [False, True])
def test_every_choice_of_units(layer, B, L, paged):
    geo = GEO[layer]
    cache = filled(geo, B, L, paged, 64)
    lens = [L - 3 * b for b in range(B)]
    q = queries(geo, B, 65)
    out = run(cache, q, lens, geo["window"], out_dtype=torch.float32)
    check(cache, q, lens, geo["window"], out)
    assert torch.equal(run(cache, q, lens, geo["window"], out_dtype=torch.float32), out)


def test_one_token_at_the_largest_batch():
    """256 sequences of one new token each, the first of them at position 0, into pages and behind them."""
    t = Tokens("global", [1] * 256, [1 + 5 * b % 97 for b in range(256)], seed=66)
    cache = Cache(GEO["global"], 256, 96, True, seed=3)
    gqa.gqa_prepare_tokens_nibble_paged(*t.args, cache.table, i32(t.lens), t.q_out, cache.kv)
    near(t.q_out, t.exact()[0])
    cache.note(*(np.zeros((256, t.KVH, t.D)) for _ in "kv"), t.off, t.lens, 96)
    untouched = np.all(cache.want == FILL, axis=-1)
    assert np.all(np.all(cache.host() == FILL, axis=-1) == untouched)   # (length 97 does not fit)


def test_two_producers_at_once():
    """Two streams write two caches from the same raw tokens."""
    t = Tokens("sliding", [70, 9], [80, 9], seed=67)
    caches = [Cache(GEO["sliding"], 2, 80, False) for _ in range(2)]
    outs = [torch.empty_like(t.q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    off, lens = i32(t.off), i32(t.lens)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, c, o in zip(streams, caches, outs):
            gqa.gqa_prepare_tokens_nibble(t.q, t.k, t.v, t.wq, t.wk, off, lens, o, c.kv, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(caches[0].kv, caches[1].kv)
    near(outs[0], t.exact()[0])


def test_append_of_what_was_read():
    """Values of a cache, appended to another, are coded as any others."""
    g = torch.Generator(device="cuda").manual_seed(68)
    geo, n = GEO["sliding"], 50
    k, v = rows(g, n, geo, 6), rows(g, n, geo, 6)
    caches = [Cache(geo, 1, n, False) for _ in range(2)]
    off, lens = i32([0, n]), i32([n])
    gqa.gqa_append_nibble(k, v, off, lens, caches[0].kv)
    k1, v1 = gqa.gqa_read_nibble(caches[0].kv, lens, 0)
    gqa.gqa_append_nibble(k1[0].contiguous(), v1[0].contiguous(), off, lens, caches[1].kv)
    caches[1].note(f64(k1[0]), f64(v1[0]), [0, n], [n])
    caches[1].check()
