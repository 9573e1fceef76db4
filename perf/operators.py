"""Cases and plain forms of the 8-bit KV cache operators.

Four operators over one cache format: e4m3 codes with a power-of-two scale for each
block of 16 positions and KV head, contiguous or in 16-position pages.

* ``append``   K/V rows of a ragged batch of prompts or chunks, quantised as they are written
* ``read``     cached rows back as bf16
* ``prepare``  the single-token producer (norms, rotary positions) writing the cache
* ``decode``   attention of one new token per sequence over the cache

``run`` computes them in elementary torch operations (32-bit, rotary angles in 64),
or, with ``own`` set, through the package's entry points.
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 16                 # positions that share a scale; positions per page
E4M3_MAX = 448.0           # largest e4m3 value
E_MIN, E_MAX = -64, 64     # range of the scales' exponents
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
             paged=False, f32=False),
        # a few chat requests of mixed length on a global layer
        dict(name="decode_global_b8", op="decode", layer="global", B=8, lo=1, hi=8192,
             paged=False, f32=False),
        # a full batch on a sliding layer, pages, windows that start inside a page
        dict(name="decode_sliding_b64_paged", op="decode", layer="sliding", B=64, lo=1, hi=8192,
             paged=True, f32=False),
        # serving batch on a global layer, pages, fp32 result for a caller that sums on
        dict(name="decode_global_b64_paged", op="decode", layer="global", B=64, lo=700, hi=16384,
             paged=True, f32=True),
        # long contexts on a global layer: the largest call
        dict(name="decode_global_b16_long", op="decode", layer="global", B=16, lo=65536,
             hi=131072, paged=False, f32=False),
        # one short chunk of a chat turn behind an odd number of cached positions
        dict(name="append_chunk_b1", op="append", layer="sliding", B=1, lo=37, hi=37, before=1003,
             paged=True),
        # prompts of a serving batch, fresh caches
        dict(name="append_prompts_b16", op="append", layer="sliding", B=16, lo=100, hi=8192,
             before=0, paged=False),
        # chunks of long prompts on a global layer, pages, behind cached positions
        dict(name="append_chunks_b32_paged", op="append", layer="global", B=32, lo=511, hi=2050,
             before=4099, paged=True),
        # one sliding window back for a prefill kernel
        dict(name="read_sliding_b2", op="read", layer="sliding", B=2, lo=1500, hi=2047, paged=False),
        # cached prompts of a batch back
        dict(name="read_global_b16_paged", op="read", layer="global", B=16, lo=1, hi=32768,
             paged=True),
        # the producer of one request
        dict(name="prepare_sliding_b1", op="prepare", layer="sliding", B=1, lo=2043, hi=2043,
             paged=False),
        # the producer of the largest batch
        dict(name="prepare_sliding_b256_paged", op="prepare", layer="sliding", B=256, lo=1, hi=1024,
             paged=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One case of the listed ranges: any operator, geometry, cache form, batch and lengths."""
    op = rng.choice(["decode", "decode", "append", "read", "prepare"])
    case = dict(op=op, layer=rng.choice(["sliding", "global"]), paged=rng.random() < 0.5)
    # bound on the positions of the whole batch (the listed long call has 16 x 131072)
    if op == "decode":
        case["B"] = _log_int(rng, 1, 256)
        top = min(131072, (1 << 20) // case["B"])
        case["f32"] = rng.random() < 0.25
    elif op == "append":
        case["B"] = _log_int(rng, 1, 256)
        top = min(8192, 65536 // case["B"])
        case["before"] = rng.choice([0, rng.randrange(1, 5000)])
    elif op == "read":
        case["B"] = _log_int(rng, 1, 64)
        top = min(32768, (1 << 18) // case["B"])
    else:
        case["B"] = _log_int(rng, 1, 256)
        top = min(8192, (1 << 18) // case["B"])
    case["hi"] = _log_int(rng, 1, top)
    case["lo"] = _log_int(rng, 1, case["hi"])
    return case


def lengths(case):
    """The batch's lengths (new tokens for append): spread over [lo, hi] by the golden ratio,
    both ends first."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    got = [hi, lo] + [lo + int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(1, B)]
    return got[:B]


def _attended(case, n):
    w = GEOMETRY[case["layer"]]["window"]
    return min(n, w) if w else n


def work(case):
    """Bytes each input read once and each output written once; operations of the products."""
    g = GEOMETRY[case["layer"]]
    H, KVH, D, B = g["H"], g["KVH"], g["D"], case["B"]
    row = KVH * D
    lens = lengths(case)
    if case["op"] == "decode":
        n = sum(_attended(case, L) for L in lens)
        blocks = sum((L - 1) // BLOCK - (L - _attended(case, L)) // BLOCK + 1 for L in lens)
        out = B * H * D * (4 if case["f32"] else 2)
        return {"bytes": 2 * n * row + 8 * blocks * KVH + 2 * B * H * D + out + 4 * B,
                "flops": 4 * n * H * D}
    if case["op"] == "append":
        n = sum(lens)
        return {"bytes": 2 * n * row * 3 + 8 * (n // BLOCK + B) * KVH, "flops": 4 * n * row}
    if case["op"] == "read":
        n = sum(_attended(case, L) for L in lens)
        return {"bytes": 2 * n * row * 3 + 8 * (n // BLOCK + B) * KVH, "flops": 2 * n * row}
    vec = (H + 2 * KVH) * D
    return {"bytes": B * (2 * vec + 2 * H * D + 2 * row + 16 * KVH), "flops": 8 * B * vec}


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


def _scale_exponent(amax):
    """The smallest e with amax <= 448 2^e, in [E_MIN, E_MAX]."""
    m, k = torch.frexp(amax)                       # amax = m 2^k, m in [0.5, 1)
    e = torch.where(m <= 0.875, k - 9, k - 8)      # 448 = 0.875 * 2^9
    e = torch.where(amax == 0, torch.full_like(e, E_MIN), e)
    return e.clamp(E_MIN, E_MAX)


def _power(e, dtype=torch.float32):
    """2^e of whole e, by its bits."""
    if dtype == torch.float64:
        return ((e.long() + 1023) << 52).view(dtype)
    return ((e.int() + 127) << 23).view(dtype)


def _filled(gen, rows, KVH, D, weight):
    """Codes [rows, KVH, D] and scales [rows / 16, KVH] of a cache written earlier, in pieces
    that bound the memory in flight."""
    codes = torch.empty((rows, KVH, D), dtype=torch.float8_e4m3fn, device=DEVICE)
    scales = torch.empty((rows // BLOCK, KVH), dtype=torch.float32, device=DEVICE)
    step = max(BLOCK, (1 << 28) // (KVH * D) // BLOCK * BLOCK)
    for r in range(0, rows, step):
        x = _rms_rows(gen, (min(step, rows - r), KVH, D), weight).float().view(-1, BLOCK, KVH, D)
        s = _power(_scale_exponent(x.abs().amax((1, 3))))
        scales[r // BLOCK:r // BLOCK + x.shape[0]] = s
        codes[r:r + x.shape[0] * BLOCK] = (x / s[:, None, :, None]).view(-1, KVH, D).to(codes.dtype)
    return codes, scales


def _layout(case, ends, seed):
    """Cache rows: contiguous [B, S] (S a whole number of blocks), or pages in a random order
    with a few spare ones. Returns (S or None, block table or None, rows)."""
    need = [-(-L // BLOCK) for L in ends]
    most = max(need)
    if not case["paged"]:
        return most * BLOCK, None, case["B"] * most * BLOCK
    gen = torch.Generator(device="cpu").manual_seed(seed)
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=gen, dtype=torch.int64).to(torch.int32)
    table = torch.full((case["B"], most), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return None, table.to(DEVICE), pages * BLOCK


def prepare(case, seed):
    g = GEOMETRY[case["layer"]]
    H, KVH, D, B = g["H"], g["KVH"], g["D"], case["B"]
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    lens = lengths(case)
    ends = [n + case["before"] for n in lens] if case["op"] == "append" else lens
    S, table, rows = _layout(case, ends, seed)
    w_k = _channel_weight(gen, D)
    st = dict(case=case, g=g, S=S, table=table,
              seq_lens=torch.tensor(ends, dtype=torch.int32, device=DEVICE))
    st["k"], st["ks"] = _filled(gen, rows, KVH, D, w_k)
    st["v"], st["vs"] = _filled(gen, rows, KVH, D, None)
    if case["op"] == "decode":
        # query weight 1/4: scores of a few units, so that many positions carry weight
        st["q"] = _rms_rows(gen, (B, H, D), torch.tensor(0.25, device=DEVICE))
        st["out"] = torch.empty((B, H, D), dtype=torch.float32 if case["f32"] else torch.bfloat16,
                                device=DEVICE)
        st["most"] = max(_attended(case, L) for L in lens)
    elif case["op"] == "append":
        off = [0]
        for n in lens:
            off.append(off[-1] + n)
        st["offsets"] = torch.tensor(off, dtype=torch.int32, device=DEVICE)
        st["k_new"] = _rms_rows(gen, (off[-1], KVH, D), w_k)
        st["v_new"] = _rms_rows(gen, (off[-1], KVH, D))
    elif case["op"] == "read":
        wide = max(lens)
        st["k_out"] = torch.zeros((B, wide, KVH, D), dtype=torch.bfloat16, device=DEVICE)
        st["v_out"] = torch.zeros((B, wide, KVH, D), dtype=torch.bfloat16, device=DEVICE)
        st["most"] = max(_attended(case, L) for L in lens)
    else:
        st["q_raw"] = (2.0 * torch.randn((B, H, D), generator=gen, device=DEVICE)).to(torch.bfloat16)
        st["k_raw"] = (3.0 * torch.randn((B, KVH, D), generator=gen, device=DEVICE)).to(torch.bfloat16)
        st["v_raw"] = (1.5 * torch.randn((B, KVH, D), generator=gen, device=DEVICE)).to(torch.bfloat16)
        st["w_q"] = (0.25 * _channel_weight(gen, D)).to(torch.bfloat16)
        st["w_k"] = w_k.to(torch.bfloat16)
        st["q_out"] = torch.empty((B, H, D), dtype=torch.bfloat16, device=DEVICE)
        st["offsets"] = torch.arange(B + 1, dtype=torch.int32, device=DEVICE)
    # the cache in the shape its user holds it
    if table is None:
        shape, sshape = (B, S, KVH, D), (B, S // BLOCK, KVH)
    else:
        shape, sshape = (rows // BLOCK, BLOCK, KVH, D), (rows // BLOCK, KVH)
    for name in ("k", "v"):
        st[name] = st[name].view(shape)
        st[name + "s"] = st[name + "s"].view(sshape)
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _rows_of(st, b, pos):
    """Cache rows of positions pos of sequences b (tensors of one shape)."""
    if st["table"] is None:
        return b * st["S"] + pos
    return st["table"].long()[b, pos // BLOCK] * BLOCK + pos % BLOCK


def _values(st, name, rows):
    """fp32 values of cache rows: code times scale."""
    KVH, D = st["g"]["KVH"], st["g"]["D"]
    codes = st[name].view(torch.uint8).view(-1, KVH * D)[rows].view(torch.float8_e4m3fn)
    scale = st[name + "s"].view(-1, KVH)[rows // BLOCK]
    return codes.to(torch.float32).view(*rows.shape, KVH, D).mul_(scale[..., None])


def _window_rows(st):
    """(positions, rows, attended) of the last `most` positions of every sequence, [B, most]."""
    L = st["seq_lens"].long()[:, None]
    w = st["g"]["window"]
    first = (L - w).clamp(min=0) if w else torch.zeros_like(L)
    pos = first + torch.arange(st["most"], device=L.device)
    there = pos < L
    b = torch.arange(L.shape[0], device=L.device)[:, None].expand_as(pos)
    return pos, _rows_of(st, b, torch.where(there, pos, first)), there


def _plain_decode(st):
    g, q = st["g"], st["q"].to(torch.float32)
    H, KVH, D, B = g["H"], g["KVH"], g["D"], q.shape[0]
    _, rows, there = _window_rows(st)
    score = torch.einsum("bkgd,bskd->bkgs", q.view(B, KVH, H // KVH, D), _values(st, "k", rows))
    score = score.masked_fill_(~there[:, None, None, :], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    o = torch.einsum("bkgs,bskd->bkgd", p, _values(st, "v", rows)).reshape(B, H, D)
    return o if st["case"]["f32"] else o.to(torch.bfloat16)


def _plain_append(st, k_new, v_new):
    """Quantises the new rows (fp32 [N, KVH, D]) into the cache, re-coding the earlier rows of a
    block whose scale grows."""
    KVH, D = st["g"]["KVH"], st["g"]["D"]
    off, L = st["offsets"].long(), st["seq_lens"].long()
    i = torch.arange(k_new.shape[0], device=L.device)
    b = torch.searchsorted(off[1:], i, right=True)
    start = L - (off[1:] - off[:-1])                    # first new position of each sequence
    pos = start[b] + i - off[b]
    rows = _rows_of(st, b, pos)
    blk = rows // BLOCK
    first = _rows_of(st, torch.arange(L.shape[0], device=L.device), start)
    slot = start % BLOCK                                 # earlier rows in each first block
    j = torch.arange(BLOCK - 1, device=L.device)
    old = torch.where(j < slot[:, None], (first - slot)[:, None] + j, first[:, None])
    for name, x in (("k", k_new), ("v", v_new)):
        codes = st[name].view(torch.uint8).view(-1, KVH, D)
        scales = st[name + "s"].view(-1, KVH)
        amax = torch.zeros_like(scales)
        amax.scatter_reduce_(0, blk[:, None].expand(-1, KVH), x.abs().amax(-1), "amax")
        need = _power(_scale_exponent(amax))
        kept = torch.zeros_like(scales)                  # scales of blocks with earlier rows
        kept[first // BLOCK] = scales[first // BLOCK] * (slot > 0)[:, None]
        fit = torch.maximum(need, kept)
        recoded = _values(st, name, old) / fit[old // BLOCK][..., None]
        codes[old] = recoded.to(torch.float8_e4m3fn).view(torch.uint8)
        codes[rows] = (x / fit[blk][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[blk] = fit[blk]


def _plain_read(st):
    pos, rows, there = _window_rows(st)
    wide = st["k_out"].shape[1]
    b = torch.arange(pos.shape[0], device=pos.device)[:, None].expand_as(pos)
    to = torch.where(there, b * wide + pos, b * wide + pos[:, :1])
    rows = torch.where(there, rows, rows[:, :1])
    for name in ("k", "v"):
        out = st[name + "_out"]
        out.view(-1, *out.shape[2:])[to] = _values(st, name, rows).to(torch.bfloat16)


def _norm_rope(x, weight, seq_lens, g, rope=True):
    """rope(x / rms(x) * weight) at position L - 1, in x's type (angles in 64 bits)."""
    D, n = g["D"], g["pairs"]
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + RMS_EPS)
    if weight is not None:
        y = y * weight.to(x.dtype)
    if not rope:
        return y
    i = torch.arange(n, device=x.device, dtype=torch.float64)
    angle = (seq_lens - 1).double()[:, None, None] * g["theta"] ** (-2.0 * i / D)
    c, s = torch.cos(angle).to(x.dtype), torch.sin(angle).to(x.dtype)
    lo, hi = y[..., :n], y[..., D // 2:D // 2 + n]
    return torch.cat([lo * c - hi * s, y[..., n:D // 2], hi * c + lo * s, y[..., D // 2 + n:]], -1)


def _plain_prepare(st):
    g, L = st["g"], st["seq_lens"]
    st["q_out"].copy_(_norm_rope(st["q_raw"].to(torch.float32), st["w_q"], L, g))
    _plain_append(st, _norm_rope(st["k_raw"].to(torch.float32), st["w_k"], L, g),
                  _norm_rope(st["v_raw"].to(torch.float32), None, L, g, rope=False))


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _run_own(st):
    import decode_attention_gb300 as gqa
    op, table, window = st["case"]["op"], st["table"], st["g"]["window"]
    cache = (st["k"], st["v"], st["ks"], st["vs"])
    if op == "decode":
        if table is None:
            return gqa.gqa_decode_quant(st["q"], *cache, st["seq_lens"], window, out=st["out"])
        return gqa.gqa_decode_quant_paged(st["q"], *cache, table, st["seq_lens"], window,
                                       out=st["out"])
    if op == "append":
        if table is None:
            gqa.gqa_append_quant(st["k_new"], st["v_new"], st["offsets"], st["seq_lens"], *cache)
        else:
            gqa.gqa_append_quant_paged(st["k_new"], st["v_new"], st["offsets"], table,
                                    st["seq_lens"], *cache)
    elif op == "read":
        if table is None:
            gqa.gqa_read_quant(*cache, st["seq_lens"], window, st["k_out"], st["v_out"])
        else:
            gqa.gqa_read_quant_paged(*cache, table, st["seq_lens"], window, st["k_out"], st["v_out"])
    elif table is None:
        gqa.gqa_prepare_decode_quant(st["q_raw"], st["k_raw"], st["v_raw"], st["w_q"], st["w_k"],
                                  st["seq_lens"], st["q_out"], *cache)
    else:
        gqa.gqa_prepare_decode_quant_paged(st["q_raw"], st["k_raw"], st["v_raw"], st["w_q"],
                                        st["w_k"], table, st["seq_lens"], st["q_out"], *cache)
    return _outputs(st)


def _outputs(st):
    if st["case"]["op"] == "read":
        return {"k": st["k_out"], "v": st["v_out"]}
    got = {"k": st["k"], "v": st["v"], "k_scales": st["ks"], "v_scales": st["vs"]}
    if st["case"]["op"] == "prepare":
        got["q"] = st["q_out"]
    return got


def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    if op == "decode":
        return _plain_decode(st)
    if op == "append":
        _plain_append(st, st["k_new"].to(torch.float32), st["v_new"].to(torch.float32))
    elif op == "read":
        _plain_read(st)
    else:
        _plain_prepare(st)
    return _outputs(st)


# ---------------------------------------------------------------------------
# The definition in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------

def _seq_rows(st, b, lo, hi):
    pos = torch.arange(lo, hi, device=DEVICE)
    if st["table"] is None:
        return b * st["S"] + pos
    pages = st["table"][b].long()
    return pages[torch.div(pos, BLOCK, rounding_mode="floor")] * BLOCK + pos.remainder(BLOCK)


def _flat(st, name):
    KVH, D = st["g"]["KVH"], st["g"]["D"]
    return st[name].reshape(-1, KVH, D), st[name + "s"].reshape(-1, KVH)


def _stored(codes, scales, rows):
    part = codes.view(torch.uint8)[rows].view(torch.float8_e4m3fn).double()
    return part * scales[rows // BLOCK].double()[..., None]


def _round_e4m3(x):
    """Nearest e4m3 value, ties to even, of 64-bit values of magnitude <= 448."""
    _, k = torch.frexp(x)
    step = _power((k - 1).clamp(min=-6) - 3, torch.float64)   # spacing of x's binade
    return torch.round(x / step) * step


def _exact_write(values, scale, new, pos0):
    """Writes rows `new` (64-bit [n, KVH, D]) at position pos0 of one sequence whose cache is
    `values` (code values [S, KVH, D]) and `scale` ([S / 16, KVH]), block by block."""
    n = new.shape[0]
    at = pos0
    while at < pos0 + n:
        blk, j0 = at // BLOCK, at % BLOCK
        end = min(pos0 + n, (blk + 1) * BLOCK)
        part = new[at - pos0:end - pos0]
        amax = part.abs().amax((0, 2))
        # the logarithm is within one of the exponent; the comparisons settle it
        e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / E4M3_MAX)).clamp(E_MIN, E_MAX)
        s = _power(e, torch.float64)
        s = torch.where((amax > E4M3_MAX * s) & (e < E_MAX), 2 * s, s)
        s = torch.where((amax <= E4M3_MAX * s / 2) & (e > E_MIN), s / 2, s)
        if j0:
            s = torch.maximum(s, scale[blk])
            kept = values[blk * BLOCK:at] * (scale[blk] / s)[None, :, None]
            values[blk * BLOCK:at] = _round_e4m3(kept)
        values[at:end] = _round_e4m3(part / s[None, :, None])
        scale[blk] = s
        at = end


def exact(case, seed):
    st = prepare(case, seed)
    g, lens = st["g"], st["seq_lens"].tolist()
    H, KVH, D, B = g["H"], g["KVH"], g["D"], case["B"]
    (kc, ks), (vc, vs) = _flat(st, "k"), _flat(st, "v")
    first = [max(0, L - g["window"]) if g["window"] else 0 for L in lens]
    if case["op"] == "decode":
        out = torch.empty((B, H, D), dtype=torch.float64, device=DEVICE)
        for b in range(B):
            rows = _seq_rows(st, b, first[b], lens[b])
            q = st["q"][b].double().view(KVH, H // KVH, D)
            score = torch.matmul(q, _stored(kc, ks, rows).permute(1, 2, 0))
            o = torch.matmul(torch.softmax(score, -1), _stored(vc, vs, rows).permute(1, 0, 2))
            out[b] = o.reshape(H, D)
        return out
    if case["op"] == "read":
        got = {}
        for name, codes, scales in (("k", kc, ks), ("v", vc, vs)):
            out = torch.zeros(st[name + "_out"].shape, dtype=torch.float64, device=DEVICE)
            for b in range(B):
                out[b, first[b]:lens[b]] = _stored(codes, scales, _seq_rows(st, b, first[b], lens[b]))
            got[name] = out
        return got
    off = st["offsets"].tolist()
    if off[-1] > 80000:
        return None
    if case["op"] == "append":
        new = {"k": st["k_new"].double(), "v": st["v_new"].double()}
        got = {}
    else:
        L = st["seq_lens"]
        new = {"k": _norm_rope(st["k_raw"].double(), st["w_k"], L, g),
               "v": _norm_rope(st["v_raw"].double(), None, L, g, rope=False)}
        got = {"q": _norm_rope(st["q_raw"].double(), st["w_q"], L, g)}
    for name, codes, scales in (("k", kc, ks), ("v", vc, vs)):
        full, full_s = codes.double(), scales.double()
        for b in range(B):
            n = off[b + 1] - off[b]
            lo = (lens[b] - n) // BLOCK * BLOCK
            hi = -(-lens[b] // BLOCK) * BLOCK
            rows = _seq_rows(st, b, lo, hi)
            values, scale = full[rows], full_s[rows[::BLOCK] // BLOCK]
            _exact_write(values, scale, new[name][off[b]:off[b + 1]], lens[b] - n - lo)
            full[rows], full_s[rows[::BLOCK] // BLOCK] = values, scale
        got[name] = full.view(st[name].shape)
        got[name + "_scales"] = full_s.view(st[name + "s"].shape)
    return got
