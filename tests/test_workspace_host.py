"""The size of a workspace that a call passes on is never more than the tensor's memory: the
elements of an expanded tensor are one in memory, and the library would write past it."""
import pytest
import torch

import decode_attention_gb300 as gqa
from decode_attention_gb300 import _native
from tests.test_streams_host import BF16, I32, OnGpu, bf16_call, quant_cache, tensor


def ws(t):
    return t.as_subclass(OnGpu)


@pytest.mark.parametrize("workspace,size", [
    (torch.zeros(4096, dtype=torch.uint8), 4096),
    (torch.zeros(1024, dtype=torch.int32)[512:], 2048),
    (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), 1),
    (torch.zeros(64, dtype=torch.uint8)[32:33].expand(4096), 32),
    (torch.zeros(4096, dtype=torch.uint8)[::2], 2048),
])
def test_bytes_passed_on(monkeypatch, workspace, size):
    seen = []

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                seen.append(args)
                return gqa.GQA_OK
            return call

    monkeypatch.setattr(_native, "_call_on", lambda dev, stream, name, *args: seen.append(args))
    monkeypatch.setattr(_native, "_lib_on", lambda device: Lib())
    monkeypatch.setattr(_native, "load_library", lambda: Lib())
    monkeypatch.setattr(_native, "_stream_handle", lambda stream, device: 0)
    w = ws(workspace)
    gqa.gqa_decode_quant(tensor((2, 32, 256), BF16), *quant_cache(False), tensor((2,), I32), 0,
                         out=tensor((2, 32, 256), BF16), workspace=w)
    assert seen[-1][-1] == size
    outs = {"gqa_decode": (2, 32, 256), "gqa_decode_keqv": (2, 32, 512), "gqa_decode_mq": (2, 2, 32, 256)}
    for name in ("gqa_decode", "gqa_decode_paged", "gqa_decode_ring", "gqa_decode_keqv",
                 "gqa_decode_keqv_paged", "gqa_decode_mq", "gqa_decode_mq_paged"):
        shape = outs.get(name.removesuffix("_paged").removesuffix("_ring"))
        bf16_call(name, out=tensor(shape, BF16), workspace=w)
        assert seen[-1][-2] == size, name
    gqa.gqa_workspace_init(w)
    assert seen[-1][1] == size
