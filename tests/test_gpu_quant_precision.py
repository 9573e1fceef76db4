"""8-bit decode attention held to the precision it states, on scores of a few units (many
positions carry weight): quant_precision's bound, which weights of 16 bits or a lost position
break (test_quant_precision_host)."""
import numpy as np
import pytest
import torch

from tests.quant_precision import attend_and_bound
from tests.test_gpu_quant import GEO, filled, run_decode

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("layer", ["sliding", "global"])
@pytest.mark.parametrize("paged,many", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("exact_scores", [True, False])
def test_weights_and_sums(layer, paged, many, exact_scores):
    """Lengths in one piece and in several; `many`: enough segments for the smaller units.  With
    one channel in q, a power of two, the scores are exact."""
    geo = GEO[layer]
    H, KVH, D = geo["H"], geo["KVH"], geo["D"]
    lens = [2, 3, 16, 17, 33, 100]
    if many:
        B = 24 if layer == "sliding" else 80
        lens += [1 + (37 * i) % 150 for i in range(B - len(lens))]
    else:
        lens += [1, 700, 2049]
    B = len(lens)
    cache = filled(geo, B, max(lens), paged, seed=401, spread=1)
    q = torch.zeros((B, H, D), dtype=torch.bfloat16, device="cuda")
    if exact_scores:
        q[..., 7] = torch.tensor([2.0, -2.0, 1.0, -1.0, 4.0, -4.0, 2.0, 0.5] * (H // 8)).cuda().bfloat16()
    else:
        g = torch.Generator(device="cuda").manual_seed(402)
        q = (torch.randn((B, H, D), generator=g, device="cuda") * 1.5 / D ** 0.5).bfloat16()
    for window in (0, 64):
        out = run_decode(cache, q, lens, window, out_dtype=torch.float32).double().cpu().numpy()
        G, qd = H // KVH, q.double().cpu().numpy()
        for b, L in enumerate(lens):
            lo = max(0, L - window) if window else 0
            for h in range(KVH):
                k, v = (cache.ref[t][b][h].stored(lo, L) for t in range(2))
                o, bound = attend_and_bound(qd[b, h * G:(h + 1) * G], k, v, exact_scores)
                worst = float(np.max(np.abs(out[b, h * G:(h + 1) * G] - o) - bound))
                assert worst <= 0, (b, h, L, window)
