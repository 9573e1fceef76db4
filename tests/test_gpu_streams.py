"""Outputs that a call on a given stream makes itself, while the current stream is busy: nothing
the current stream still has to do may reach them."""
import pytest
import torch

import decode_attention_gb300 as gqa
from decode_attention_gb300 import inputs
from tests.test_gpu_quant import GEO, filled, i32, queries, run_decode

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


class Busy:
    """Some tens of milliseconds of matrix products on the current stream."""

    def __init__(self):
        self.a = torch.full((4096, 4096), 1e-3, device="cuda")
        self.b = self.a @ self.a
        self.done = torch.cuda.Event()

    def start(self):
        for _ in range(20):
            torch.mm(self.a, self.a, out=self.b)
        self.done.record()

    def late_fill(self, shapes, dtype):
        """Values written by the current stream after all that, into memory given back at once."""
        for s in shapes:
            torch.full(s, 7.0, dtype=dtype, device="cuda")


@pytest.mark.parametrize("paged", [False, True])
def test_outputs_made_on_a_given_stream(paged):
    geo, lens, S = GEO["sliding"], [40, 333], 333
    cache = filled(geo, 2, S, paged, seed=201, nan_rows=False)
    for t in range(2):                                 # (NaN codes compare unequal)
        c = cache.codes[t].view(torch.uint8)
        c[(c & 0x7f) == 0x7f] = 0x35
    q, seq = queries(geo, 2, 202), i32(lens)
    read = gqa.gqa_read_quant_paged if paged else gqa.gqa_read_quant
    cache_args = (*cache.args, cache.table) if paged else cache.args
    want_kv = read(*cache_args, seq, 0)
    want = run_decode(cache, q, lens, 0, out_dtype=torch.float32)
    stream, busy = torch.cuda.Stream(), Busy()
    torch.cuda.synchronize()
    for _ in range(3):
        busy.start()
        busy.late_fill([want_kv[0].shape] * 2, torch.bfloat16)
        busy.late_fill([want.shape], torch.float32)
        got_kv = read(*cache_args, seq, 0, stream=stream)
        if paged:
            got = gqa.gqa_decode_quant_paged(q, *cache.args, cache.table, seq, 0,
                                             out_dtype=torch.float32, stream=stream)
        else:
            got = gqa.gqa_decode_quant(q, *cache.args, seq, 0, out_dtype=torch.float32, stream=stream)
        stream.synchronize()
        assert not busy.done.query(), "the current stream was to be busy throughout"
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert all(torch.equal(a, b) for a, b in zip(got_kv, want_kv))


@pytest.mark.parametrize("layer", ["sliding", "global"])
def test_bf16_outputs_made_on_a_given_stream(layer):
    geo = GEO[layer]
    H, KVH, D = geo["H"], geo["KVH"], geo["D"]
    case = inputs.contiguous_case(2, 333, H, KVH, D, [40, 333], 203, device="cuda")
    args = (case["q"], case["k"], case["v"], case["seq_lens"], geo["window"])
    mq = (torch.stack([case["q"], case["q"]], 1).contiguous(), *args[1:])
    want, want_mq = gqa.gqa_decode(*args), gqa.gqa_decode_mq(*mq)
    stream, busy = torch.cuda.Stream(), Busy()
    torch.cuda.synchronize()
    for _ in range(3):
        busy.start()
        busy.late_fill([want.shape], want.dtype)
        busy.late_fill([want_mq.shape], want.dtype)
        ws = gqa.new_workspace(2, 333, H, KVH, D, geo["window"], stream=stream)
        got = gqa.gqa_decode(*args, workspace=ws, stream=stream)
        got_mq = gqa.gqa_decode_mq(*mq, stream=stream)
        stream.synchronize()
        assert not busy.done.query(), "the current stream was to be busy throughout"
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_mq, want_mq)
