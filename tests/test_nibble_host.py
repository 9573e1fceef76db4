"""4-bit KV cache and the producer for many tokens, host side: argument checks return before
anything touches a device, the binding's refusals, what it passes on, and the 64-bit reference of
the GPU tests against the format's definition."""
import numpy as np
import pytest
import torch

import decode_attention_gb300 as gqa
from decode_attention_gb300 import _native
from tests import nibble_reference as ref
from tests.test_streams_host import BF16, FakeStream, I32, made, tensor  # noqa: F401

F = 0x10000   # aligned address, never dereferenced
SLIDING, GLOBAL = (32, 16, 256), (32, 4, 512)
BAD, UNSUPPORTED, OK = gqa.GQA_ERR_INVALID_ARGUMENT, gqa.GQA_ERR_UNSUPPORTED, gqa.GQA_OK
U8 = torch.uint8


@pytest.fixture(scope="module")
def lib():
    return gqa.load_library()


def append(lib, B=2, N=5, S=64, geo=SLIDING, kn=F, vn=F, off=F, lens=F, kv=F):
    return lib.gqa_append_nibble(kn, vn, off, lens, B, N, S, geo[1], geo[2], kv, None)


def append_paged(lib, B=2, N=5, P=8, mp=4, ps=16, geo=GLOBAL, bt=F, kv=F):
    return lib.gqa_append_nibble_paged(F, F, F, bt, F, B, N, P, mp, ps, geo[1], geo[2], kv, None)


def read(lib, B=2, S=64, geo=SLIDING, window=0, ko=F, vo=F, rows=64, dtype=0, kv=F, lens=F):
    return lib.gqa_read_nibble(kv, lens, B, S, geo[1], geo[2], window, ko, vo, rows, dtype, None)


def read_paged(lib, B=2, P=8, mp=4, ps=16, geo=GLOBAL, bt=F, rows=64):
    return lib.gqa_read_nibble_paged(F, bt, F, B, P, mp, ps, geo[1], geo[2], 0, F, F, rows, 0, None)


def tokens(lib, B=2, N=5, geo=SLIDING, q=F, k=F, v=F, wq=F, wk=F, off=F, lens=F, out=F, kc=F, vc=F, rows=64,
           ring=0):
    return lib.gqa_prepare_tokens(q, k, v, wq, wk, off, lens, B, N, *geo, out, kc, vc, rows, ring, None)


def tokens_paged(lib, B=2, N=5, P=8, mp=4, ps=16, geo=GLOBAL, bt=F, v=F, kc=F, vc=F):
    return lib.gqa_prepare_tokens_paged(F, F, v, F, F, F, bt, F, B, N, P, mp, ps, *geo, F, kc, vc, None)


def step(lib, B=2, N=5, geo=SLIDING, q=F, k=F, v=F, wq=F, wk=F, off=F, lens=F, out=F, kv=F, S=64):
    return lib.gqa_prepare_tokens_nibble(q, k, v, wq, wk, off, lens, B, N, *geo, out, kv, S, None)


def step_paged(lib, B=2, N=5, P=8, mp=4, ps=16, geo=GLOBAL, bt=F, v=F, kv=F):
    return lib.gqa_prepare_tokens_nibble_paged(F, F, v, F, F, F, bt, F, B, N, P, mp, ps, *geo, F, kv, None)


def decode(lib, B=2, S=64, geo=SLIDING, window=0, q=F, kv=F, lens=F, out=F, dtype=0):
    return lib.gqa_decode_nibble(q, kv, lens, B, S, *geo, window, out, dtype, None, 0, None)


def decode_paged(lib, B=2, P=8, mp=4, ps=16, geo=GLOBAL, bt=F, kv=F):
    return lib.gqa_decode_nibble_paged(F, kv, bt, F, B, P, mp, ps, *geo, 0, F, 0, None, 0, None)


ALL = [append, append_paged, read, read_paged, tokens, tokens_paged, step, step_paged, decode, decode_paged]


@pytest.mark.parametrize("call", ALL)
def test_geometry_and_batch(lib, call):
    for geo in [(32, 8, 256), (32, 16, 512), (32, 4, 256)]:
        assert call(lib, geo=geo) == UNSUPPORTED
    assert call(lib, B=-1) == BAD
    assert call(lib, B=257) == BAD
    assert call(lib, B=0) == OK


@pytest.mark.parametrize("call", [append_paged, read_paged, tokens_paged, step_paged, decode_paged])
def test_page_arguments(lib, call):
    for kw in (dict(ps=32), dict(P=0), dict(mp=0), dict(mp=16385), dict(bt=None), dict(bt=F + 2)):
        assert call(lib, **kw) == BAD, kw


@pytest.mark.parametrize("call", [tokens, step, decode])
def test_query_heads(lib, call):
    assert call(lib, geo=(16, 16, 256)) == UNSUPPORTED


@pytest.mark.parametrize("call", [append, append_paged, tokens, tokens_paged, step, step_paged])
def test_token_counts(lib, call):
    assert call(lib, N=-1) == BAD
    assert call(lib, N=256 * 262144 + 1) == BAD
    assert call(lib, N=0) == OK


def test_append_arguments(lib):
    for name in ("kn", "vn", "off", "lens", "kv"):
        assert append(lib, **{name: None}) == BAD, name
    for kw in (dict(kn=F + 8), dict(vn=F + 8), dict(kv=F + 8), dict(off=F + 2), dict(lens=F + 2), dict(S=0),
               dict(S=262145)):
        assert append(lib, **kw) == BAD, kw
    assert append_paged(lib, kv=None) == BAD and append_paged(lib, kv=F + 8) == BAD


def test_read_arguments(lib):
    for kw in (dict(ko=None), dict(vo=None), dict(kv=None), dict(lens=None), dict(ko=F + 8), dict(kv=F + 8),
               dict(rows=0), dict(rows=262145), dict(window=-1), dict(dtype=5), dict(S=0), dict(S=262145)):
        assert read(lib, **kw) == BAD, kw


@pytest.mark.parametrize("call,cache", [(tokens, "vc"), (tokens, "kc"), (step, "kv")])
def test_producer_arguments(lib, call, cache):
    size = "rows" if call is tokens else "S"
    for name in ("q", "k", "wq", "wk", "off", "lens", "out", cache):
        assert call(lib, **{name: None}) == BAD, name
    for kw in (dict(q=F + 8), dict(k=F + 8), dict(v=F + 8), dict(out=F + 8), dict(wq=F + 2), dict(wk=F + 2),
               dict(off=F + 2), dict(lens=F + 2), {cache: F + 8}, {size: 0}, {size: 262145}):
        assert call(lib, **kw) == BAD, kw


def test_values_equal_to_keys(lib):
    assert tokens(lib, v=None) == UNSUPPORTED                     # sliding layers project values
    assert tokens(lib, geo=GLOBAL, v=None, vc=None) == BAD
    assert step(lib, v=None) == BAD and step(lib, geo=GLOBAL, v=None) == BAD
    assert tokens(lib, ring=2) == BAD
    assert tokens_paged(lib, v=None, vc=None) == BAD and tokens_paged(lib, kc=None) == BAD


def test_decode_arguments(lib):
    for kw in (dict(q=None), dict(kv=None), dict(lens=None), dict(out=None), dict(q=F + 8), dict(kv=F + 8),
               dict(lens=F + 2), dict(out=F + 8), dict(window=-1), dict(S=0), dict(S=262145), dict(dtype=9)):
        assert decode(lib, **kw) == BAD, kw
    assert decode_paged(lib, kv=None) == BAD


def test_row_constants_match_the_header():
    import re
    from tests.test_abi_host import HEADER
    defines = dict(re.findall(r"#define (GQA_NIBBLE_[A-Z]+) (\d+)", open(HEADER).read()))
    assert defines == {"GQA_NIBBLE_PLANE": str(gqa.GQA_NIBBLE_PLANE), "GQA_NIBBLE_ROW": str(gqa.GQA_NIBBLE_ROW)}


# ---------------------------------------------------------------------------- binding

def inputs_of(name, paged, geo=SLIDING, **change):
    """Arguments of a call at its smallest shapes; `change` replaces one by name."""
    H, KVH, D = geo
    planes = KVH * D // 256
    t = dict(q=tensor((2, H, D), BF16), q_raw=tensor((5, H, D), BF16), k_raw=tensor((5, KVH, D), BF16),
             v_raw=tensor((5, KVH, D), BF16), w_q=tensor((D,), BF16), w_k=tensor((D,), BF16),
             token_offsets=tensor((3,), I32), q_out=tensor((5, H, D), BF16),
             block_table=tensor((2, 3), I32), seq_lens=tensor((2,), I32),
             kv=tensor((9, planes, 16, 272) if paged else (2, planes, 40, 272), U8),
             k_cache=tensor((9, 16, KVH, D) if paged else (2, 40, KVH, D), BF16),
             v_cache=tensor((9, 16, KVH, D) if paged else (2, 40, KVH, D), BF16))
    t.update(change)
    order = {"gqa_append_nibble": "k_raw v_raw token_offsets block_table seq_lens kv",
             "gqa_read_nibble": "kv block_table seq_lens",
             "gqa_prepare_tokens": "q_raw k_raw v_raw w_q w_k token_offsets block_table seq_lens q_out k_cache v_cache",
             "gqa_prepare_tokens_nibble": "q_raw k_raw v_raw w_q w_k token_offsets block_table seq_lens q_out kv",
             "gqa_decode_nibble": "q kv block_table seq_lens"}[name].split()
    args = [t[n] for n in order if paged or n != "block_table"]
    return args + ([0] if name in ("gqa_read_nibble", "gqa_decode_nibble") else [])


CALLS = ["gqa_append_nibble", "gqa_read_nibble", "gqa_prepare_tokens", "gqa_prepare_tokens_nibble",
         "gqa_decode_nibble"]


def call(name, paged, geo=SLIDING, kw=None, **change):
    return getattr(gqa, name + ("_paged" if paged else ""))(*inputs_of(name, paged, geo, **change), **(kw or {}))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("geo", [SLIDING, GLOBAL])
def test_calls_that_fit_pass_every_argument(monkeypatch, name, paged, geo):
    seen = []
    monkeypatch.setattr(_native, "_call_on", lambda dev, stream, fn, *args: seen.append((fn, args)))
    kw = {}
    if name == "gqa_decode_nibble":
        kw = dict(out=tensor((2, 32, geo[2]), BF16))
    if name == "gqa_read_nibble":
        kw = {n: tensor((2, 7, geo[1], geo[2]), BF16) for n in ("k_out", "v_out")}
    call(name, paged, geo, kw)
    fn, args = seen[0]
    assert fn == name + ("_paged" if paged else "")
    # every argument but the stream, in number as the C signature takes them
    assert len(args) == len(getattr(gqa.load_library(), fn).argtypes) - 1
    assert set(geo[1:]) <= set(args)


def wrong(name, geo=SLIDING):
    H, KVH, D = geo
    yield dict(seq_lens=tensor((3,), I32))
    yield dict(seq_lens=tensor((2,), torch.int64))
    yield dict(seq_lens=tensor((2, 1), I32))
    if name != "gqa_prepare_tokens":
        yield dict(kv=tensor((2, 16, 40, 270), U8))
        yield dict(kv=tensor((2, 4, 40, 272), U8))
        yield dict(kv=tensor((2, 8, 40, 272), U8)) if name != "gqa_read_nibble" else dict(kv=tensor((2, 40, 272), U8))
        yield dict(kv=tensor((2, 16, 40, 272), torch.int8))
        yield dict(kv=tensor((2, 16, 272, 40), U8).transpose(2, 3))
        yield dict(kv=None)
    if name not in ("gqa_read_nibble", "gqa_decode_nibble"):
        yield dict(token_offsets=tensor((2,), I32))
        yield dict(k_raw=tensor((5, KVH, D + 1), BF16))
        yield dict(v_raw=tensor((4, KVH, D), BF16))
        yield dict(k_raw=torch.ones((5, KVH, D), dtype=BF16))   # on the CPU
    if name.startswith("gqa_prepare"):
        yield dict(q_out=tensor((4, H, D), BF16))
        yield dict(w_k=tensor((D - 1,), BF16))
        yield dict(q_raw=tensor((5, H, D), torch.float16))
        yield dict(q_raw=tensor((5, H * D), BF16))
    if name == "gqa_prepare_tokens":
        yield dict(v_cache=tensor((2, 40, KVH, 2 * D), BF16))
        yield dict(k_cache=tensor((2, 41, KVH, D), BF16))
        yield dict(v_cache=None)
    if name == "gqa_prepare_tokens_nibble":
        yield dict(v_raw=None)
    if name == "gqa_decode_nibble":
        yield dict(q=tensor((2, 32, 512), BF16))
        yield dict(q=torch.ones((2, 32, 256), dtype=BF16))


@pytest.mark.parametrize("name", CALLS)
def test_binding_refuses(monkeypatch, made, name):  # noqa: F811
    changes = list(wrong(name))
    monkeypatch.setattr(_native, "_call_on", lambda *args: pytest.fail("the call went through"))
    for change in changes:
        with pytest.raises(ValueError):
            call(name, False, **change)
    if name != "gqa_prepare_tokens":
        with pytest.raises(ValueError):
            call(name, True, block_table=tensor((3, 3), I32))
    with pytest.raises(ValueError):
        call(name, True, block_table=None)
    with pytest.raises(ValueError):
        call(name, True, block_table=tensor((2,), I32))


@pytest.mark.parametrize("name,outputs", [("gqa_read_nibble", 2), ("gqa_decode_nibble", 1)])
@pytest.mark.parametrize("paged", [False, True])
def test_outputs_belong_to_the_stream_of_the_call(made, name, outputs, paged):  # noqa: F811
    stream = FakeStream()
    call(name, paged, kw=dict(stream=stream))
    assert [s for _, s in made if s is not None] == [stream] * outputs
    made.clear()
    call(name, paged)
    assert all(s is None for _, s in made)


def test_workspace_bytes(monkeypatch):
    seen = []
    monkeypatch.setattr(_native, "_call_on", lambda dev, stream, fn, *args: seen.append(args))
    w = tensor((1,), U8).expand(1 << 20)
    call("gqa_decode_nibble", False, kw=dict(out=tensor((2, 32, 256), BF16), workspace=w))
    assert seen[0][-1] == 1


# ---------------------------------------------------------------------------- reference

def test_scales_are_f16_numbers():
    bits = (np.arange(ref.TOP + 1, dtype=np.uint16) << 7).view(np.float16)
    assert np.array_equal(ref.SCALES, bits.astype(np.float64))
    assert ref.SCALES[-1] == 60 and np.isnan((np.array([0xFF], dtype=np.uint16) << 7).view(np.float16)[0])


def test_reference_rounds_as_the_format_says():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((2048, 32)) * np.exp2(rng.uniform(-20, 8, (2048, 1)))
    x = ref.bf16(x)
    byte, u = ref.code_group(x)
    s = ref.SCALES[byte]
    amax = np.abs(x).max(1)
    inside = amax <= 450
    assert np.all(amax[inside] <= 7.5 * s[inside])
    assert np.all((byte == 0) | (amax > 7.5 * ref.SCALES[np.maximum(byte - 1, 0)]))
    assert u.min() >= 1 and u.max() <= 15
    y = (u - 8) * s[:, None]
    assert np.all(np.abs(y - x)[inside] <= s[inside][:, None] / 2)
    # no other code is nearer, and of two as near the one further from zero is taken
    for d in (-1, 1):
        v = np.clip(u + d, 1, 15)
        other = np.abs((v - 8) * s[:, None] - x)
        mine = np.abs(y - x)
        assert np.all(mine <= other)
        tie = (mine == other) & (v != u)
        assert np.all(np.abs(u - 8)[tie] > np.abs(v - 8)[tie])
    # the bytes of a row stand for the same
    k = x.reshape(-1, 16, 256)
    back = ref.decode(ref.encode(k, -k), 256)
    assert np.array_equal(back[0], y.reshape(k.shape)) and np.array_equal(back[1], -back[0])


def test_reference_ends():
    one = np.zeros((6, 32))
    one[1, 3] = 450.0
    one[2, 3] = 1e6
    one[3, 3] = 2.0 ** -18
    one[4, 3] = np.nan
    one[5, 3] = -np.inf
    byte, u = ref.code_group(one)
    assert byte.tolist() == [0, ref.TOP, ref.TOP, 1, ref.NAN, ref.NAN]
    assert u[:, 3].tolist() == [8, 15, 15, 9, 8, 8]


def test_normal_values_are_held_to_a_tenth():
    """The error of four bits on normally distributed values, 32 to a scale: the rms of a uniform
    error of one step is s / sqrt(12), and s is on average 2.35 / 7.2 of the values' rms."""
    x = ref.bf16(np.random.default_rng(6).standard_normal((4000, 32)))
    byte, u = ref.code_group(x)
    err = (u - 8) * ref.SCALES[byte][:, None] - x
    assert 0.08 < np.sqrt(np.mean(err ** 2)) < 0.105
