"""GPU test of gqa_decode_nibble called again and again: every call gives the same bits.

A slot of the ring that is copied into while a warp still reads it changes single codes of a row, now and
then: without the fence between a warp's loads and the arrival that frees the slot one call in a thousand
was wrong, over contiguous caches whose rows do not begin on whole lines of memory, in batches of a hundred
sequences and more.  So: thousands of calls of such batches, back to back.
"""
import numpy as np
import pytest
import torch

import decode_attention_gb300 as gqa
from decode_attention_gb300 import inputs

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

CALLS, TOGETHER = 3000, 6   # calls, of which six run behind one another before their outputs are looked at


@pytest.mark.parametrize("layer,B,top,window", [("sliding", 256, 4095, 0), ("sliding", 200, 973, 0), ("sliding", 152, 6748, 1024),
                                                ("sliding", 100, 9793, 1024), ("sliding", 8, 4001, 0),
                                                ("global", 100, 4001, 0)])
@pytest.mark.parametrize("paged", [False, True])
def test_thousands_of_calls_agree(layer, B, top, window, paged):
    geo = inputs.SLIDING if layer == "sliding" else inputs.GLOBAL
    planes = geo["KVH"] * geo["D"] // 256
    lens = (top ** np.random.default_rng(7).random(B)).astype(np.int32)    # spread over the logarithm
    lens[B // 2] = top
    g = torch.Generator(device="cuda").manual_seed(8)
    blocks = (top + 15) // 16
    shape = (B * blocks, planes, 16, 272) if paged else (B, planes, top, 272)
    kv = torch.randint(0x11, 0x100, shape, dtype=torch.uint8, generator=g, device="cuda")
    kv[..., 256:] = torch.randint(96, 112, (*shape[:3], 16), dtype=torch.uint8, generator=g, device="cuda")
    table = (torch.randperm(B * blocks, generator=g, device="cuda").view(B, blocks).int(),) if paged else ()
    q = (0.05 * torch.randn((B, geo["H"], geo["D"]), generator=g, device="cuda")).to(torch.bfloat16)
    seq = torch.tensor(lens, device="cuda")
    ws = gqa.new_workspace(B, blocks * 16, geo["H"], geo["KVH"], geo["D"], window)
    fn = gqa.gqa_decode_nibble_paged if paged else gqa.gqa_decode_nibble
    want = fn(q, kv, *table, seq, window, out_dtype=torch.float32, workspace=ws)
    outs = torch.empty((TOGETHER, *want.shape), device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(CALLS // TOGETHER):
        for out in outs:
            fn(q, kv, *table, seq, window, out=out, workspace=ws)
        differ += (outs != want).flatten(1).any(dim=1).sum()
    assert differ.item() == 0, f"{differ.item()} of {CALLS} calls differ from the first"
    assert gqa.gqa_device_status(ws) == 0 and not torch.isnan(want).any()
