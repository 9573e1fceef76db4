"""GPU test of the decode calls over 8-bit and bf16 caches made again and again: every call gives the same
bits.  (Shared memory that is copied into while a warp still reads it would change a value now and then.)
Many sequences of very unlike lengths, so that pieces begin and end all the time, six calls behind one
another before their outputs are looked at.
"""
import numpy as np
import pytest
import torch

import decode_attention_gb300 as gqa
from decode_attention_gb300 import inputs

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

CALLS, TOGETHER = 1200, 6


def random_cache(kind, shape, scales, g):
    """The caches: K and V, and the scales of 8-bit ones."""
    if kind == "bf16":
        return [torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in "kv"]
    codes = [torch.randint(0, 0x7f, shape, dtype=torch.uint8, generator=g, device="cuda") for _ in "kv"]
    signs = [torch.randint(0, 2, shape, dtype=torch.uint8, generator=g, device="cuda") << 7 for _ in "kv"]
    return ([(c | s).view(torch.float8_e4m3fn) for c, s in zip(codes, signs)]
            + [torch.exp2(torch.randint(-8, -5, scales, generator=g, device="cuda").float()) for _ in "kv"])


@pytest.mark.parametrize("kind", ["8-bit", "bf16"])
@pytest.mark.parametrize("layer,B,top,window", [("sliding", 200, 973, 0), ("sliding", 100, 4001, 1024), ("global", 100, 2001, 0)])
@pytest.mark.parametrize("paged", [False, True])
def test_thousands_of_calls_agree(kind, layer, B, top, window, paged):
    geo = inputs.SLIDING if layer == "sliding" else inputs.GLOBAL
    lens = (top ** np.random.default_rng(7).random(B)).astype(np.int32)    # spread over the logarithm
    lens[B // 2] = top
    g = torch.Generator(device="cuda").manual_seed(8)
    blocks = (top + 15) // 16
    row = (geo["KVH"], geo["D"])
    if paged:
        cache = random_cache(kind, (B * blocks, 16, *row), (B * blocks, geo["KVH"]), g)
        cache.append(torch.randperm(B * blocks, generator=g, device="cuda").view(B, blocks).int())
    else:
        cache = random_cache(kind, (B, top, *row), (B, blocks, geo["KVH"]), g)
    q = (0.05 * torch.randn((B, geo["H"], geo["D"]), generator=g, device="cuda")).to(torch.bfloat16)
    seq = torch.tensor(lens, device="cuda")
    ws = gqa.new_workspace(B, blocks * 16, geo["H"], geo["KVH"], geo["D"], window)
    fn = getattr(gqa, {"bf16": "gqa_decode", "8-bit": "gqa_decode_quant"}[kind] + ("_paged" if paged else ""))
    want = fn(q, *cache, seq, window, out_dtype=torch.float32, workspace=ws)
    outs = torch.empty((TOGETHER, *want.shape), device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(CALLS // TOGETHER):
        for out in outs:
            fn(q, *cache, seq, window, out=out, workspace=ws)
        differ += (outs != want).flatten(1).any(dim=1).sum()
    assert differ.item() == 0, f"{differ.item()} of {CALLS} calls differ from the first"
    assert gqa.gqa_device_status(ws) == 0 and not torch.isnan(want).any()
