"""8-bit KV cache, host side: the argument checks of the gqa_*_quant calls return before
anything touches a device, and the 64-bit reference used by the GPU tests agrees with the
format's definition."""
import numpy as np
import pytest
import torch

import decode_attention_gb300 as gqa
from tests import quant_reference as ref

F = 0x10000   # aligned address, never dereferenced
SLIDING, GLOBAL = (32, 16, 256), (32, 4, 512)
BAD, UNSUPPORTED, OK = gqa.GQA_ERR_INVALID_ARGUMENT, gqa.GQA_ERR_UNSUPPORTED, gqa.GQA_OK


@pytest.fixture(scope="module")
def lib():
    return gqa.load_library()


def append(lib, B=2, N=5, S=64, geo=SLIDING, kn=F, vn=F, off=F, lens=F, k=F, v=F, ks=F, vs=F):
    return lib.gqa_append_quant(kn, vn, off, lens, B, N, S, geo[1], geo[2], k, v, ks, vs, None)


def append_paged(lib, B=2, N=5, P=8, mp=4, ps=16, geo=GLOBAL, bt=F, k=F, v=F):
    return lib.gqa_append_quant_paged(F, F, F, bt, F, B, N, P, mp, ps, geo[1], geo[2], k, v, F, F, None)


def read(lib, B=2, S=64, geo=SLIDING, window=0, ko=F, vo=F, rows=64, dtype=0, k=F, ks=F, lens=F):
    return lib.gqa_read_quant(k, F, ks, F, lens, B, S, geo[1], geo[2], window, ko, vo, rows, dtype, None)


def read_paged(lib, B=2, P=8, mp=4, ps=16, geo=GLOBAL, bt=F, rows=64):
    return lib.gqa_read_quant_paged(F, F, F, F, bt, F, B, P, mp, ps, geo[1], geo[2], 0, F, F, rows, 0, None)


def prepare(lib, B=2, geo=SLIDING, q=F, v=F, wq=F, out=F, k=F, ks=F, rows=64):
    return lib.gqa_prepare_decode_quant(q, F, v, wq, F, F, B, *geo, out, k, F, ks, F, rows, None)


def prepare_paged(lib, B=2, P=8, mp=4, ps=16, geo=GLOBAL, bt=F):
    return lib.gqa_prepare_decode_quant_paged(F, F, F, F, F, bt, F, B, P, mp, ps, *geo, F, F, F, F, F, None)


def decode(lib, B=2, S=64, geo=SLIDING, window=0, q=F, k=F, ks=F, vs=F, lens=F, out=F, dtype=0):
    return lib.gqa_decode_quant(q, k, F, ks, vs, lens, B, S, *geo, window, out, dtype, None, 0, None)


def decode_paged(lib, B=2, P=8, mp=4, ps=16, geo=GLOBAL, bt=F, ks=F):
    return lib.gqa_decode_quant_paged(F, F, F, ks, F, bt, F, B, P, mp, ps, *geo, 0, F, 0, None, 0, None)


@pytest.mark.parametrize("call", [append, append_paged, read, read_paged, prepare, prepare_paged,
                                  decode, decode_paged])
def test_geometry_and_batch(lib, call):
    for geo in [(32, 8, 256), (32, 16, 512), (32, 4, 256)]:
        assert call(lib, geo=geo) == UNSUPPORTED
    assert call(lib, B=-1) == BAD
    assert call(lib, B=257) == BAD
    assert call(lib, B=0) == OK


@pytest.mark.parametrize("call", [append_paged, read_paged, prepare_paged, decode_paged])
def test_page_arguments(lib, call):
    for kw in (dict(ps=32), dict(P=0), dict(mp=0), dict(mp=16385), dict(bt=None), dict(bt=F + 2)):
        assert call(lib, **kw) == BAD, kw


def test_heads_of_the_producer_and_decode(lib):
    assert prepare(lib, geo=(16, 16, 256)) == UNSUPPORTED
    assert decode(lib, geo=(16, 16, 256)) == UNSUPPORTED


def test_append_arguments(lib):
    for name in ("kn", "vn", "off", "lens", "k", "v", "ks", "vs"):
        assert append(lib, **{name: None}) == BAD, name
    for kw in (dict(kn=F + 8), dict(k=F + 8), dict(ks=F + 2), dict(off=F + 2), dict(S=0),
               dict(S=262145), dict(N=-1), dict(N=256 * 262144 + 1)):
        assert append(lib, **kw) == BAD, kw
    assert append(lib, N=0, kn=None, k=None) == OK


def test_read_arguments(lib):
    for kw in (dict(ko=None), dict(vo=None), dict(k=None), dict(ks=None), dict(lens=None), dict(ko=F + 8),
               dict(rows=0), dict(rows=262145), dict(window=-1), dict(dtype=5), dict(S=0)):
        assert read(lib, **kw) == BAD, kw


def test_prepare_arguments(lib):
    for kw in (dict(q=None), dict(v=None), dict(wq=None), dict(out=None), dict(k=None), dict(ks=None),
               dict(q=F + 8), dict(wq=F + 2), dict(rows=0), dict(rows=262145)):
        assert prepare(lib, **kw) == BAD, kw


def test_decode_arguments(lib):
    for kw in (dict(q=None), dict(k=None), dict(ks=None), dict(vs=None), dict(lens=None), dict(out=None),
               dict(q=F + 8), dict(k=F + 8), dict(ks=F + 2), dict(window=-1), dict(S=0),
               dict(S=262145), dict(dtype=9)):
        assert decode(lib, **kw) == BAD, kw
    assert decode_paged(lib, ks=None) == BAD


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 32, 256, dtype=torch.bfloat16)
    k = torch.zeros(1, 16, 16, 256, dtype=torch.float8_e4m3fn)
    s = torch.zeros(1, 1, 16)
    lens = torch.zeros(1, dtype=torch.int32)
    off = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        gqa.gqa_decode_quant(q, k, k, s, s, lens, 0)
    with pytest.raises(ValueError):
        gqa.gqa_append_quant(q[:, :16], q[:, :16], off, lens, k, k, s, s)
    with pytest.raises(ValueError):
        gqa.gqa_read_quant(k, k, s, s, lens, 0)
    with pytest.raises(ValueError):
        gqa.gqa_prepare_decode_quant(q, q[:, :16], q[:, :16], q[0, 0], q[0, 0], lens, q, k, k, s, s)


def test_reference_rounds_like_the_format():
    # every code stands for itself; midpoints go to the even code; torch's e4m3 agrees
    v = ref.VALUES[~np.isnan(ref.VALUES)]
    assert np.array_equal(ref.e4m3(v), v)
    pos = np.sort(v[v >= 0])
    mid = (pos[1:] + pos[:-1]) / 2
    x = np.concatenate([mid, -mid, mid * (1 + 1e-12), mid * (1 - 1e-12)])
    t = torch.tensor(x, dtype=torch.float64).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(x[:2 * len(mid)]), t[:2 * len(mid)])
    assert np.all(ref.e4m3(mid * (1 + 1e-12)) == pos[1:])
    assert np.all(ref.e4m3(mid * (1 - 1e-12)) == pos[:-1])
    assert np.all(np.abs(ref.e4m3(x) - x) <= ref.half_step(x))


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (224.0, -1), (0.0, -64), (1e-30, -64),
                                    (448.0 * 2.0 ** 64, 64), (1e38, 64)])
def test_reference_exponent(amax, e):
    assert ref.exponent(amax) == e
