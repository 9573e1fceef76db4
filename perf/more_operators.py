"""Cases and plain forms of the 4-bit KV cache operators and of the many-token producer.

One cache format: K and V of 256 channels of a KV head (a plane) stand in a row of 272 bytes per
position: 128 bytes of K codes, 128 of V codes, 8 scales of K, 8 of V.  A code u stands for
(u - 8) * s; s, one for 32 channels, is an f16 number with 3 mantissa bits, held as its bits 14 to 7.
Contiguous caches are [B, planes, S, 272], page pools [P, planes, 16, 272].

* ``decode``  attention of one new token per sequence over the cache
* ``append``  K/V rows of a ragged batch of prompts or chunks, quantised as they are written, and
              the rows back as the prefill's attention takes them
* ``read``    cached rows back as bf16 or fp32
* ``step``    the ragged producer (norms, rotary positions; any number of new tokens per sequence)
              writing the 4-bit cache, and the new rows back
* ``tokens``  the same producer writing a bf16 cache

``run`` computes them in elementary torch operations, or, with ``own`` set, through the package's
entry points.
"""
import math

import torch

own = False

DEVICE = "cuda"
PAGE = 16                  # positions per page
PLANE = 256                # channels of a plane
ROW = 272                  # bytes of a plane's row
GROUP = 32                 # channels that share a scale
TOP_SCALE = 0xA7           # byte of the largest scale (60)
NAN_SCALE = 0xFF
RMS_EPS = 1e-6
# the package's two layer geometries: heads, head size, window, rotated pairs and their base
GEOMETRY = {
    "sliding": dict(H=32, KVH=16, D=256, window=1024, pairs=128, theta=1.0e4),
    "global": dict(H=32, KVH=4, D=512, window=0, pairs=64, theta=1.0e6),
}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one request on a sliding layer: a full window, the latency of a single call
        dict(name="decode_sliding_b1", op="decode", layer="sliding", B=1, lo=2048, hi=2048,
             before=0, paged=False, f32=False),
        # a few chat requests of mixed length on a global layer, pages
        dict(name="decode_global_b8_paged", op="decode", layer="global", B=8, lo=1, hi=8192,
             before=0, paged=True, f32=False),
        # a full batch on a sliding layer, windows that start inside a page, fp32 for a caller that sums on
        dict(name="decode_sliding_b64_paged", op="decode", layer="sliding", B=64, lo=1, hi=8192,
             before=0, paged=True, f32=True),
        # long contexts on a global layer: the largest call
        dict(name="decode_global_b16_long", op="decode", layer="global", B=16, lo=65536,
             hi=131072, before=0, paged=False, f32=False),
        # one short chunk of a chat turn behind an odd number of cached positions
        dict(name="append_chunk_b1", op="append", layer="sliding", B=1, lo=37, hi=37, before=1003,
             paged=True, f32=False),
        # prompts of a serving batch, fresh caches
        dict(name="append_prompts_b16", op="append", layer="sliding", B=16, lo=100, hi=8192,
             before=0, paged=False, f32=False),
        # one sliding window back for a prefill kernel
        dict(name="read_sliding_b2", op="read", layer="sliding", B=2, lo=1500, hi=2047, before=0,
             paged=False, f32=False),
        # cached prompts of a batch back
        dict(name="read_global_b16_paged", op="read", layer="global", B=16, lo=1, hi=32768,
             before=0, paged=True, f32=False),
        # the producer of one request's next token
        dict(name="step_sliding_b1", op="step", layer="sliding", B=1, lo=1, hi=1, before=2042,
             paged=False, f32=False),
        # prompts of a serving batch on a global layer, pages, behind a shared system prompt's length
        dict(name="step_prompts_b16_paged", op="step", layer="global", B=16, lo=100, hi=4096,
             before=517, paged=True, f32=False),
        # the verify step of speculative decoding: eight draft tokens of each of 64 requests
        dict(name="tokens_verify_b64", op="tokens", layer="sliding", B=64, lo=8, hi=8, before=2001,
             paged=False, f32=False),
        # chunks of long prompts on a global layer, pages
        dict(name="tokens_chunks_b8_paged", op="tokens", layer="global", B=8, lo=511, hi=2050,
             before=4099, paged=True, f32=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One case of the listed ranges: any operator, geometry, cache form, batch and lengths."""
    op = rng.choice(["decode", "decode", "append", "read", "step", "tokens"])
    case = dict(op=op, layer=rng.choice(["sliding", "global"]), paged=rng.random() < 0.5,
                f32=op in ("decode", "read") and rng.random() < 0.3, before=0)
    # bound on the positions of the whole batch
    if op == "decode":
        case["B"] = _log_int(rng, 1, 256)
        top = min(131072, (1 << 20) // case["B"])
    elif op == "read":
        case["B"] = _log_int(rng, 1, 64)
        top = min(32768, (1 << 18) // case["B"])
    else:
        case["B"] = _log_int(rng, 1, 256)
        top = min(8192, 65536 // case["B"])
        if rng.random() < 0.7:
            case["before"] = _log_int(rng, 1, min(5000, (1 << 17) // case["B"]))
    case["hi"] = _log_int(rng, 1, top)
    case["lo"] = _log_int(rng, 1, case["hi"])
    return case


def lengths(case):
    """The batch's lengths (new tokens where the operator writes): spread over [lo, hi] by the
    golden ratio, both ends first."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    got = [hi, lo] + [lo + int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(1, B)]
    return got[:B]


def _writes(case):
    return case["op"] in ("append", "step", "tokens")


def _window(case):
    """Positions that a decode or a read back reaches from the end; 0: all."""
    if case["op"] in ("append", "step"):
        return case["hi"]
    return GEOMETRY[case["layer"]]["window"]


def _attended(case, end):
    w = _window(case)
    return min(end, w) if w else end


def work(case):
    """Bytes each input read once and each output written once; operations of the products."""
    g = GEOMETRY[case["layer"]]
    H, KVH, D, B = g["H"], g["KVH"], g["D"], case["B"]
    row, cached = KVH * D, KVH * D // PLANE * ROW
    lens = lengths(case)
    n = sum(lens)
    if case["op"] == "decode":
        n = sum(_attended(case, L) for L in lens)
        out = B * H * D * (4 if case["f32"] else 2)
        return {"bytes": n * cached + 2 * B * H * D + out + 4 * B, "flops": 4 * n * H * D}
    if case["op"] == "read":
        n = sum(_attended(case, L) for L in lens)
        return {"bytes": n * (cached + 2 * row * (4 if case["f32"] else 2)), "flops": 4 * n * row}
    if case["op"] == "append":
        back = sum(_attended(case, L + case["before"]) for L in lens)
        return {"bytes": n * (4 * row + cached) + back * 4 * row, "flops": 8 * n * row}
    vec = (H + 2 * KVH) * D
    moved = n * (2 * vec + 2 * H * D)
    if case["op"] == "tokens":
        return {"bytes": moved + 4 * n * row, "flops": 8 * n * vec}
    back = sum(_attended(case, L + case["before"]) for L in lens)
    return {"bytes": moved + n * cached + back * 4 * row, "flops": 8 * n * vec}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rms_rows(gen, shape, weight=None):
    """bf16 rows of unit root mean square, times a channel weight: what the norms ahead of the
    cache give."""
    x = torch.randn(shape, generator=gen, device=DEVICE)
    x *= torch.rsqrt(x.square().mean(-1, keepdim=True) + RMS_EPS)
    if weight is not None:
        x *= weight
    return x.to(torch.bfloat16)


def _channel_weight(gen, D):
    """A norm weight around 1 with a few large channels, as key caches have them."""
    w = 1.0 + 0.25 * torch.randn(D, generator=gen, device=DEVICE)
    w[torch.randint(D, (4,), generator=gen, device=DEVICE)] *= 4.0
    return w


def _scale_values(dtype=torch.float32):
    """The scales of the bytes 0 .. TOP_SCALE: f16 numbers given by their bits 14 to 7."""
    c = torch.arange(TOP_SCALE + 1, device=DEVICE, dtype=torch.int16)
    return (c << 7).view(torch.float16).to(dtype)


def _coded(x):
    """Codes [..., C / 2] and scale bytes [..., C / 32] of bf16 rows [..., C]."""
    shape = x.shape
    x = x.to(torch.float32).reshape(*shape[:-1], shape[-1] // GROUP, GROUP)
    amax = x.abs().amax(-1)
    table = _scale_values()
    # the smallest scale with amax <= 7.5 s (the products are exact)
    byte = torch.searchsorted(7.5 * table, amax).clamp_(max=TOP_SCALE)
    s = table[byte][..., None]
    # to the nearest, ties away from zero: a bf16 number over a scale of four bits is a tie or far
    # from one, and an fp32 division keeps both apart
    step = torch.floor(x.abs() / s + 0.5).clamp_(max=7.0)
    u = (torch.where(s > 0, torch.copysign(step, x), torch.zeros_like(x)) + 8.0).nan_to_num_(8.0)
    lost = ~torch.isfinite(amax)
    u = u.masked_fill_(lost[..., None], 8.0).to(torch.uint8).reshape(shape)
    byte = byte.masked_fill_(lost, NAN_SCALE).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4), byte


def _records(k, v):
    """Rows [n, planes, 272] of bf16 K and V [n, KVH, D]."""
    n = k.shape[0]
    (kc, ks), (vc, vs) = (_coded(t.reshape(n, -1, PLANE)) for t in (k, v))
    return torch.cat([kc, vc, ks, vs], -1)


def _page_table(case, ends, seed):
    """Pages in a random order with a few spare ones: (block table, pages)."""
    need = [-(-L // PAGE) for L in ends]
    gen = torch.Generator(device="cpu").manual_seed(seed)
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=gen, dtype=torch.int64).to(torch.int32)
    table = torch.full((case["B"], max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table.to(DEVICE), pages


def _filled(gen, outer, rows, KVH, D, w_k):
    """A 4-bit cache [outer, planes, rows, 272] written earlier, in pieces that bound the memory in
    flight."""
    planes = KVH * D // PLANE
    kv = torch.empty((outer, planes, rows, ROW), dtype=torch.uint8, device=DEVICE)
    step = max(1, (1 << 26) // (KVH * D * rows))
    cut = max(1, (1 << 26) // (KVH * D))
    for o in range(0, outer, step):
        m = min(step, outer - o)
        for r in range(0, rows, cut):
            n = min(cut, rows - r)
            k, v = (_rms_rows(gen, (m * n, KVH, D), w) for w in (w_k, None))
            kv[o:o + m, :, r:r + n] = _records(k, v).view(m, n, planes, ROW).transpose(1, 2)
    return kv


def prepare(case, seed):
    g = GEOMETRY[case["layer"]]
    H, KVH, D, B = g["H"], g["KVH"], g["D"], case["B"]
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    lens = lengths(case)
    ends = [n + case["before"] for n in lens] if _writes(case) else lens
    wide = max(ends)
    w_k = _channel_weight(gen, D)
    table, pages = _page_table(case, ends, seed) if case["paged"] else (None, 0)
    outer, rows = (pages, PAGE) if case["paged"] else (B, wide)
    st = dict(case=case, g=g, table=table, rows=rows, window=_window(case),
              most=max(_attended(case, L) for L in ends),
              seq_lens=torch.tensor(ends, dtype=torch.int32, device=DEVICE))
    if case["op"] == "tokens":
        for name in ("k", "v"):
            st[name] = torch.empty((outer, rows, KVH, D), dtype=torch.bfloat16, device=DEVICE)
            st[name].normal_(generator=gen)
    else:
        st["kv"] = _filled(gen, outer, rows, KVH, D, w_k)
    if case["op"] == "decode":
        # query weight 1/4: scores of a few units, so that many positions carry weight
        st["q"] = _rms_rows(gen, (B, H, D), torch.tensor(0.25, device=DEVICE))
        st["out"] = torch.empty((B, H, D), dtype=torch.float32 if case["f32"] else torch.bfloat16,
                                device=DEVICE)
        return st
    if case["op"] != "tokens":
        dtype = torch.float32 if case["f32"] else torch.bfloat16
        st["k_out"] = torch.zeros((B, wide, KVH, D), dtype=dtype, device=DEVICE)
        st["v_out"] = torch.zeros((B, wide, KVH, D), dtype=dtype, device=DEVICE)
    if case["op"] == "read":
        return st
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    N = off[-1]
    st["offsets"] = torch.tensor(off, dtype=torch.int32, device=DEVICE)
    if case["op"] == "append":
        st["k_new"] = _rms_rows(gen, (N, KVH, D), w_k)
        st["v_new"] = _rms_rows(gen, (N, KVH, D))
        return st
    for name, heads, size in (("q_raw", H, 2.0), ("k_raw", KVH, 3.0), ("v_raw", KVH, 1.5)):
        st[name] = torch.empty((N, heads, D), dtype=torch.bfloat16, device=DEVICE)
        st[name].normal_(0.0, size, generator=gen)
    st["w_q"] = (0.25 * _channel_weight(gen, D)).to(torch.bfloat16)
    st["w_k"] = w_k.to(torch.bfloat16)
    st["q_out"] = torch.empty((N, H, D), dtype=torch.bfloat16, device=DEVICE)
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _slots(st, b, pos):
    """(outer, row) of positions pos of sequences b (tensors of one shape)."""
    if st["table"] is None:
        return b, pos
    return st["table"].long()[b, pos // PAGE], pos % PAGE


def _values(codes, scales):
    """fp32 values [..., 256] of codes [..., 128] and scale bytes [..., 8]."""
    u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    s = (scales.to(torch.int16) << 7).view(torch.float16).to(torch.float32)
    s = s.masked_fill_(scales == NAN_SCALE, math.nan)
    x = u.to(torch.float32).sub_(8.0).view(*s.shape, GROUP)
    return x.mul_(s[..., None]).flatten(-2)


def _cached(st, outer, row):
    """fp32 K and V [..., KVH, D] of cache rows."""
    g = st["g"]
    r = st["kv"][outer, :, row]                      # [..., planes, 272]
    shape = (*r.shape[:-2], g["KVH"], g["D"])
    return (_values(r[..., :128], r[..., 256:264]).view(shape),
            _values(r[..., 128:256], r[..., 264:]).view(shape))


def _window_rows(st):
    """(positions, outer, row, there) of the last `most` positions of every sequence, [B, most]."""
    L = st["seq_lens"].long()[:, None]
    w = st["window"]
    first = (L - w).clamp(min=0) if w else torch.zeros_like(L)
    pos = first + torch.arange(st["most"], device=L.device)
    there = pos < L
    pos = torch.where(there, pos, first)
    b = torch.arange(L.shape[0], device=L.device)[:, None].expand_as(pos)
    return (pos, *_slots(st, b, pos), there)


def _plain_decode(st):
    g, q = st["g"], st["q"].to(torch.float32)
    H, KVH, D, B = g["H"], g["KVH"], g["D"], q.shape[0]
    _, outer, row, there = _window_rows(st)
    k, v = _cached(st, outer, row)
    score = torch.einsum("bkgd,bskd->bkgs", q.view(B, KVH, H // KVH, D), k)
    score = score.masked_fill_(~there[:, None, None, :], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    o = torch.einsum("bkgs,bskd->bkgd", p, v).reshape(B, H, D)
    return o if st["case"]["f32"] else o.to(torch.bfloat16)


def _plain_read(st):
    pos, outer, row, there = _window_rows(st)
    b = torch.arange(pos.shape[0], device=pos.device)[:, None].expand_as(pos)
    # (a place past a sequence's end takes its first row once more)
    for name, x in zip(("k_out", "v_out"), _cached(st, outer, row)):
        st[name][b, pos] = x.to(st[name].dtype)


def _new_rows(st):
    """(sequence, position) of each packed token."""
    off, L = st["offsets"].long(), st["seq_lens"].long()
    i = torch.arange(int(st["k_new" if "k_new" in st else "k_raw"].shape[0]), device=L.device)
    b = torch.searchsorted(off[1:], i, right=True)
    return b, L[b] - off[b + 1] + i


def _plain_append(st, k_new, v_new):
    outer, row = _slots(st, *_new_rows(st))
    st["kv"][outer, :, row] = _records(k_new, v_new)


def _norm_rope(x, weight, pos, g, rope=True):
    """rope(x / rms(x) * weight) at positions pos, in x's type (angles in 64 bits)."""
    D, n = g["D"], g["pairs"]
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + RMS_EPS)
    if weight is not None:
        y = y * weight.to(x.dtype)
    if not rope:
        return y
    i = torch.arange(n, device=x.device, dtype=torch.float64)
    angle = pos.double()[:, None, None] * g["theta"] ** (-2.0 * i / D)
    c, s = torch.cos(angle).to(x.dtype), torch.sin(angle).to(x.dtype)
    lo, hi = y[..., :n], y[..., D // 2:D // 2 + n]
    return torch.cat([lo * c - hi * s, y[..., n:D // 2], hi * c + lo * s, y[..., D // 2 + n:]], -1)


def _plain_producer(st, wide):
    """q into q_out; K and V rows in bf16, computed in `wide` (64 bits ahead of the 4-bit codes: a
    value on the other side of a border between codes is a whole step off)."""
    g = st["g"]
    b, pos = _new_rows(st)
    st["q_out"].copy_(_norm_rope(st["q_raw"].to(torch.float32), st["w_q"], pos, g))
    k = _norm_rope(st["k_raw"].to(wide), st["w_k"], pos, g).to(torch.bfloat16)
    v = _norm_rope(st["v_raw"].to(wide), None, pos, g, rope=False).to(torch.bfloat16)
    return b, pos, k, v


def _plain_tokens(st):
    b, pos, k, v = _plain_producer(st, torch.float32)
    outer, row = _slots(st, b, pos)
    st["k"][outer, row] = k
    st["v"][outer, row] = v


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _run_own(st):
    import decode_attention_gb300 as gqa
    op, table, lens, window = st["case"]["op"], st["table"], st["seq_lens"], st["window"]
    pages = () if table is None else (table,)
    call = (lambda name: getattr(gqa, name)) if table is None else \
           (lambda name: getattr(gqa, name + "_paged"))
    if op == "decode":
        return call("gqa_decode_nibble")(st["q"], st["kv"], *pages, lens, window, out=st["out"])
    if op == "append":
        call("gqa_append_nibble")(st["k_new"], st["v_new"], st["offsets"], *pages, lens, st["kv"])
    elif op == "step":
        call("gqa_prepare_tokens_nibble")(st["q_raw"], st["k_raw"], st["v_raw"], st["w_q"],
                                          st["w_k"], st["offsets"], *pages, lens, st["q_out"],
                                          st["kv"])
    elif op == "tokens":
        call("gqa_prepare_tokens")(st["q_raw"], st["k_raw"], st["v_raw"], st["w_q"], st["w_k"],
                                   st["offsets"], *pages, lens, st["q_out"], st["k"], st["v"])
    if op != "tokens":
        call("gqa_read_nibble")(st["kv"], *pages, lens, window, st["k_out"], st["v_out"])
    return _outputs(st)


def _outputs(st):
    """The written cache as the values it stands for."""
    op = st["case"]["op"]
    if op == "tokens":
        return {"q": st["q_out"], "k": st["k"], "v": st["v"]}
    got = {"k": st["k_out"], "v": st["v_out"]}
    if op == "step":
        got["q"] = st["q_out"]
    return got


def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    if op == "decode":
        return _plain_decode(st)
    if op == "tokens":
        _plain_tokens(st)
        return _outputs(st)
    if op == "append":
        _plain_append(st, st["k_new"], st["v_new"])
    elif op == "step":
        _, _, k, v = _plain_producer(st, torch.float64)
        _plain_append(st, k, v)
    _plain_read(st)
    return _outputs(st)


# ---------------------------------------------------------------------------
# The definition in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------

def _row_of(st, b, pos):
    """Index arrays of the positions `pos` of sequence b."""
    if st["table"] is None:
        return torch.full_like(pos, b), pos
    return st["table"][b].long()[torch.div(pos, PAGE, rounding_mode="floor")], pos.remainder(PAGE)


def _meaning(bytes_, scales):
    """64-bit values of code bytes [n, planes, 128] with scale bytes [n, planes, 8]."""
    n, planes, _ = bytes_.shape
    x = torch.empty((n, planes, PLANE), dtype=torch.float64, device=DEVICE)
    x[..., 0::2] = bytes_.remainder(16).double() - 8
    x[..., 1::2] = torch.div(bytes_, 16, rounding_mode="floor").double() - 8
    c = scales.long()
    e, m = c // 8, (c % 8).double()
    s = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 18), m * 2.0 ** -17)
    s = torch.where(c > TOP_SCALE, torch.full_like(s, math.nan), s)
    return x * s.repeat_interleave(GROUP, -1)


def _coarse(x):
    """What finite bf16 rows [n, C] are held as, in 64 bits: for 32 channels the step is the
    smallest of the scales that reaches the largest of them with 7.5 steps."""
    y = x.double().view(-1, GROUP)
    amax = y.abs().amax(1, keepdim=True)
    # amax / 7.5 rounded up to 4 significant bits, or to a multiple of 2^-17 below 2^-14
    want = amax / 7.5
    _, e = torch.frexp(want)
    unit = torch.exp2((e - 4).clamp(min=-17).double())
    step = torch.ceil(want / unit) * unit
    step = torch.where((step - unit) * 7.5 >= amax, step - unit, step)   # (a rounded quotient)
    step = step.clamp(min=0.0, max=60.0)
    ratio = torch.where(step > 0, y / step.clamp(min=2.0 ** -30), torch.zeros_like(y))
    whole = torch.trunc(ratio)
    whole = whole + torch.sign(ratio) * ((ratio - whole).abs() >= 0.5)
    return (whole.clamp(-7, 7) * step).view(x.shape)


def _normed(x, weight=None):
    x = x.double()
    y = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + RMS_EPS).sqrt()
    return y if weight is None else y * weight.double()


def _turned(y, pos, g):
    """Pairs (i, i + D / 2), i < pairs, as complex numbers turned by pos * theta^(-2 i / D)."""
    half, n = g["D"] // 2, g["pairs"]
    rate = torch.exp(torch.arange(n, device=DEVICE).double() * (-2.0 / g["D"] * math.log(g["theta"])))
    z = torch.complex(y[..., :half], y[..., half:])
    z[..., :n] *= torch.exp(1j * pos.double()[:, None] * rate)[:, None, :]
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    st = prepare(case, seed)
    g, lens = st["g"], st["seq_lens"].tolist()
    H, KVH, D, B = g["H"], g["KVH"], g["D"], case["B"]
    first = [L - _attended(case, L) for L in lens]
    if _writes(case) and sum(lengths(case)) > 80000:
        return None

    def stored(b, lo, hi):
        outer, row = _row_of(st, b, torch.arange(lo, hi, device=DEVICE))
        r = st["kv"][outer, :, row]
        return [_meaning(c, s).view(hi - lo, KVH, D)
                for c, s in ((r[..., :128], r[..., 256:264]), (r[..., 128:256], r[..., 264:272]))]

    if case["op"] == "decode":
        out = torch.empty((B, H, D), dtype=torch.float64, device=DEVICE)
        for b in range(B):
            k, v = stored(b, first[b], lens[b])
            q = st["q"][b].double().view(KVH, H // KVH, D)
            score = torch.matmul(q, k.permute(1, 2, 0))
            out[b] = torch.matmul(torch.softmax(score, -1), v.permute(1, 0, 2)).reshape(H, D)
        return out
    got = {}
    off = st["offsets"].tolist() if _writes(case) else None
    new = {}
    if case["op"] == "append":
        new = {"k": st["k_new"], "v": st["v_new"]}
    elif case["op"] in ("step", "tokens"):
        pos = torch.cat([torch.arange(lens[b] - off[b + 1] + off[b], lens[b], device=DEVICE)
                         for b in range(B)])
        got["q"] = _turned(_normed(st["q_raw"], st["w_q"]), pos, g)
        new = {"k": _turned(_normed(st["k_raw"], st["w_k"]), pos, g), "v": _normed(st["v_raw"])}
    if case["op"] == "tokens":
        for name in ("k", "v"):
            full = st[name].double()
            for b in range(B):
                outer, row = _row_of(st, b, torch.arange(lens[b] - off[b + 1] + off[b], lens[b],
                                                         device=DEVICE))
                full[outer, row] = new[name][off[b]:off[b + 1]]
            got[name] = full
        return got
    for name in ("k", "v"):
        got[name] = torch.zeros(st[name + "_out"].shape, dtype=torch.float64, device=DEVICE)
    for b in range(B):
        for name, x in zip(("k", "v"), stored(b, first[b], lens[b])):
            got[name][b, first[b]:lens[b]] = x
            if off is not None:
                rows = new[name][off[b]:off[b + 1]].to(torch.bfloat16)
                got[name][b, lens[b] - len(rows):lens[b]] = _coarse(rows.reshape(-1, D)).view(rows.shape)
    return got
