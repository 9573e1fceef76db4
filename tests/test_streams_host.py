"""Tensors that a call allocates belong to the stream the call runs on.  The caching allocator
hands out memory in the order of the stream that is current when it is asked, so an output made
on another stream may still be in use there, and a fill enqueued there is not ordered with the
kernel.  Host side: tensors that say they are on a GPU, allocations recorded with the stream that
is current at that moment, and no launch."""
import contextlib

import pytest
import torch

import decode_attention_gb300 as gqa
from decode_attention_gb300 import _native

BF16, E4M3, I32, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.float32


class OnGpu(torch.Tensor):
    """A CPU tensor that answers as one on CUDA device 0."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def get_device(self):
        return 0


def tensor(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class FakeStream:
    cuda_stream = 0x1234


@pytest.fixture
def made(monkeypatch):
    """The (function, current stream) of every allocation."""
    log, current = [], [None]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def recorded(name):
        plain = getattr(torch, name)

        def make(*args, **kw):
            log.append((name, current[-1]))
            kw.pop("device", None)
            return plain(*args, **kw).as_subclass(OnGpu)
        return make

    class NoLaunch:
        def __getattr__(self, name):
            return lambda *args: gqa.GQA_OK

    for name in ("empty", "zeros", "zeros_like", "empty_like"):
        monkeypatch.setattr(torch, name, recorded(name))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(_native, "_call_on", lambda *args: None)
    monkeypatch.setattr(_native, "_lib_on", lambda device: NoLaunch())
    monkeypatch.setattr(_native, "_stream_handle", lambda stream, device: 0)
    return log


def quant_cache(paged):
    if paged:
        return [tensor((9, 16, 16, 256), E4M3) for _ in "kv"] + [tensor((9, 16), F32) for _ in "kv"]
    return [tensor((2, 40, 16, 256), E4M3) for _ in "kv"] + [tensor((2, 3, 16), F32) for _ in "kv"]


def read(paged, **kw):
    cache, lens = quant_cache(paged), tensor((2,), I32)
    if paged:
        return gqa.gqa_read_quant_paged(*cache, tensor((2, 3), I32), lens, 0, **kw)
    return gqa.gqa_read_quant(*cache, lens, 0, **kw)


def decode(paged, **kw):
    cache, lens, q = quant_cache(paged), tensor((2,), I32), tensor((2, 32, 256), BF16)
    if paged:
        return gqa.gqa_decode_quant_paged(q, *cache, tensor((2, 3), I32), lens, 0, **kw)
    return gqa.gqa_decode_quant(q, *cache, lens, 0, **kw)


@pytest.mark.parametrize("call", [read, decode])
@pytest.mark.parametrize("paged", [False, True])
def test_outputs_of_the_8_bit_calls(made, call, paged):
    stream = FakeStream()
    call(paged, stream=stream)           # (its inputs are made with no stream current)
    outputs = 2 if call is read else 1
    assert [s for _, s in made if s is not None] == [stream] * outputs
    made.clear()
    call(paged)
    assert all(s is None for _, s in made), "the current stream when none is given"


def bf16_call(name, **kw):
    """One of the calls over a bf16 cache, at the smallest shapes it takes."""
    KVH, D = (4, 512) if "keqv" in name else (16, 256)
    q = tensor((2, 2, 32, D) if "mq" in name else (2, 32, D), BF16)
    paged = name.endswith("paged")
    cache = [tensor((5, 16, KVH, D) if paged else (2, 40, KVH, D), BF16) for _ in "kv"]
    if "keqv" in name:
        cache = [cache[0], tensor((D,), BF16)]
    args = [q, *cache] + ([tensor((2, 3), I32)] if paged else []) + [tensor((2,), I32)]
    return getattr(gqa, name)(*args, *([] if "keqv" in name else [8]), **kw)


@pytest.mark.parametrize("name", ["gqa_decode", "gqa_decode_paged", "gqa_decode_ring", "gqa_decode_keqv",
                                  "gqa_decode_keqv_paged", "gqa_decode_mq", "gqa_decode_mq_paged"])
def test_outputs_of_the_bf16_calls(made, name):
    stream = FakeStream()
    bf16_call(name, stream=stream)
    assert [s for _, s in made if s is not None] == [stream]
    made.clear()
    bf16_call(name)
    assert all(s is None for _, s in made)


def test_new_workspace(made):
    """The workspace's zeros are written on the stream that it is made for."""
    stream = FakeStream()
    lib = type("Lib", (), {"gqa_workspace_init": lambda *args: gqa.GQA_OK})()
    size = gqa.gqa_workspace_size(2, 40, 32, 16, 256, 0)
    with pytest.MonkeyPatch.context() as patch:
        patch.setattr(_native, "gqa_workspace_size", lambda *args: size)
        patch.setattr(_native, "load_library", lambda: lib)
        ws = gqa.new_workspace(2, 40, 32, 16, 256, 0, stream=stream)
        assert made == [("empty", stream)] and ws.numel() == size
        gqa.new_workspace(2, 40, 32, 16, 256, 0)
    assert made[1:] == [("empty", None)]
