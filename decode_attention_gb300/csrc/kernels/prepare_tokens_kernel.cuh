// The producer (prepare_kernel.cuh: norms, rotary positions) for any number of new tokens per
// sequence, packed as the appends take them, writing a bf16 cache or the 4-bit one
// (nibble_cache.cuh).
//
// A CTA takes a token at a time: its first n_rot threads make the angles of the token's position,
// once for all its heads, and its warps take the token's H + 2 KVH head vectors (q heads, then k,
// then v), the next one's load in flight behind each.  Few tokens are shared by several CTAs
// (blockIdx.y).
//
// For the 4-bit cache a k or v vector is rounded to fp32 and to bf16, as a row that an append gets,
// and coded from there.  An fp32 error moves a value over a border between two bf16 numbers once
// in some 10^4, and one in forty of those goes over a border between codes, a whole step.  Norm,
// weight and rotation of k and v are therefore taken to some 2^-30 there (twofold.cuh).
#pragma once

#include "nibble_cache.cuh"
#include "prepare_quant_kernel.cuh"   // head_norm_rope, head_norm_rope_twofold

namespace gqa {

constexpr int kTokensThreads = 256;

struct PrepareTokensParams {
    const __nv_bfloat16* q_raw;     // [N, H, D]
    const __nv_bfloat16* k_raw;     // [N, KVH, D]
    const __nv_bfloat16* v_raw;     // [N, KVH, D], or null (bf16 only): values = keys
    const __nv_bfloat16* w_q;       // [D]
    const __nv_bfloat16* w_k;       // [D]
    const int32_t* token_offsets;   // [B + 1]
    const int32_t* seq_lens;        // [B], lengths after the append
    __nv_bfloat16* q_out;           // [N, H, D]
    __nv_bfloat16* k_cache;         // bf16 cache: [B, rows, KVH, D] or [P, 16, KVH, D]; null if values = keys
    __nv_bfloat16* v_cache;
    NibbleCache cache;              // the 4-bit cache; of the bf16 one rows, block_table, max_pages, num_pages
    int ring;                       // bf16, contiguous: 1 = position s at row s mod rows
    int B, N, H, KVH;
    int n_rot;                      // rotated pairs
    uint64_t turn[kPrepareMaxRot];  // turns per position of pair i, a 64-bit fraction
};

template <int D, bool kNibble>
__global__ void __launch_bounds__(kTokensThreads)
    gqa_prepare_tokens_kernel(const PrepareTokensParams p) {
    constexpr int kHalf = D / 2;
    constexpr int kPer = kHalf / 32;              // elements per lane in each half: 4 or 8
    constexpr int kWarps = kTokensThreads / 32;
    constexpr int kShare = kNibbleGroup / kPer;   // lanes that share a scale
    __shared__ TokenIndex idx;
    __shared__ float2 cs[2][kPrepareMaxRot];      // (cos, sin), of this token and the one before
    __shared__ float2 cs_l[kNibble ? 2 : 1][kPrepareMaxRot];   // their low parts

    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    idx.load(p.token_offsets, p.seq_lens, p.B);

    const NibbleCache& c = p.cache;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_vec = p.H + 2 * p.KVH;
    const int first = blockIdx.y * kWarps + warp, step = gridDim.y * kWarps;
    const bool keqv = p.v_raw == nullptr;
    const size_t stride = kNibble ? c.plane_stride() : 0;

    // this lane's elements [kPer l, kPer l + kPer) of each half of a vector
    auto load = [&](int i, int vec, uint2 (&raw)[2][kPer / 4]) {
        const bool is_q = vec < p.H, is_k = !is_q && vec < p.H + p.KVH;
        const int kvh = is_k ? vec - p.H : vec - p.H - p.KVH;
        const __nv_bfloat16* src =
            is_q ? p.q_raw + (static_cast<size_t>(i) * p.H + vec) * D
                 : (is_k || keqv ? p.k_raw : p.v_raw) + (static_cast<size_t>(i) * p.KVH + kvh) * D;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < kPer; e += 4)
                raw[h][e / 4] = __ldcs(reinterpret_cast<const uint2*>(src + h * kHalf + kPer * lane + e));
    };

    int turn = 0;
    for (int i = blockIdx.x; i < p.N; i += gridDim.x) {
        int b, pos;
        if (!idx.find(p.B, p.N, i, &b, &pos)) continue;   // (the whole CTA alike)
        uint2 next[2][kPer / 4];
        if (first < n_vec) load(i, first, next);
        float2* cst = cs[turn & 1];
        float2* cst_l = cs_l[kNibble ? turn & 1 : 0];
        ++turn;
        if (tid < p.n_rot) {
            Twofold co, si;
            cos_sin_of_turn(static_cast<uint64_t>(pos) * p.turn[tid], &co, &si);
            cst[tid] = make_float2(co.h, si.h);
            if (kNibble) cst_l[tid] = make_float2(co.l, si.l);
        }
        // the token's place: null when it is not written
        uint8_t* row = nullptr;
        if (kNibble) {
            if (pos < c.capacity()) row = c.row(b, pos);
        }
        bool have_slot = false;
        size_t slot = 0;   // bf16 cache: its row
        if (!kNibble) {
            if (c.block_table) {
                const int page = pos < c.capacity()
                                     ? c.block_table[static_cast<size_t>(b) * c.max_pages + pos / kNibblePage] : -1;
                have_slot = page >= 0 && page < c.num_pages;
                slot = static_cast<size_t>(page) * kNibblePage + pos % kNibblePage;
            } else {
                // (a ring keeps the last `rows` positions)
                have_slot = p.ring ? pos >= idx.len[b] - c.rows : pos < c.rows;
                slot = static_cast<size_t>(b) * c.rows + (p.ring ? pos % c.rows : pos);
            }
        }
        __syncthreads();

        for (int vec = first; vec < n_vec; vec += step) {
            float x[2][kPer];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < kPer; e += 4) {
                    const uint2 t = next[h][e / 4];
                    x[h][e] = __uint_as_float(t.x << 16);
                    x[h][e + 1] = __uint_as_float(t.x & 0xffff0000u);
                    x[h][e + 2] = __uint_as_float(t.y << 16);
                    x[h][e + 3] = __uint_as_float(t.y & 0xffff0000u);
                }
            if (vec + step < n_vec) load(i, vec + step, next);
            const bool is_q = vec < p.H, is_k = !is_q && vec < p.H + p.KVH;
            const int kvh = is_k ? vec - p.H : vec - p.H - p.KVH;
            if (!is_q && (kNibble ? row == nullptr : !have_slot || (is_k && keqv))) continue;
            const __nv_bfloat16* w = is_q ? p.w_q : is_k ? p.w_k : nullptr;
            if (!kNibble || is_q)
                head_norm_rope<D>(x, w, cst, p.n_rot, lane);
            else
                head_norm_rope_twofold<D>(x, w, cst, cst_l, p.n_rot, lane,
                                          [](Twofold a) { return fast_sum(a.h, a.l).h; });

            uint32_t y[2][kPer / 2];   // in bf16
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < kPer; e += 2) {
                    const __nv_bfloat162 t = __floats2bfloat162_rn(x[h][e], x[h][e + 1]);
                    y[h][e / 2] = *reinterpret_cast<const uint32_t*>(&t);
                }
            if (!kNibble || is_q) {
                __nv_bfloat16* dst =
                    is_q ? p.q_out + (static_cast<size_t>(i) * p.H + vec) * D
                         : (is_k ? p.k_cache : p.v_cache) + (slot * p.KVH + kvh) * D;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < kPer / 2; e += 2)
                        *reinterpret_cast<uint2*>(dst + h * kHalf + kPer * lane + 2 * e) =
                            make_uint2(y[h][e], y[h][e + 1]);
                continue;
            }
            if constexpr (kNibble) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t m = 0;
#pragma unroll
                    for (int e = 0; e < kPer / 2; ++e) m = __vmaxu2(m, y[h][e] & 0x7fff7fffu);
                    m = max(m & 0xffffu, m >> 16);
#pragma unroll
                    for (int off = 1; off < kShare; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
                    uint32_t scale = kNibbleNanScale, codes = 0x88888888u;
                    if (m < 0x7f80u) {
                        scale = nibble_scale_byte(__uint_as_float(m << 16));
                        const float inv = nibble_inverse(nibble_scale(scale));
                        codes = 0;
#pragma unroll
                        for (int e = 0; e < kPer / 2; ++e) {
                            codes |= nibble_code(__uint_as_float(y[h][e] << 16), inv) << (8 * e);
                            codes |= nibble_code(__uint_as_float(y[h][e] & 0xffff0000u), inv) << (8 * e + 4);
                        }
                    }
                    // D = 256: both halves in the head's plane; D = 512: one each
                    uint8_t* r = row + (D == 256 ? kvh : 2 * kvh + h) * stride + (is_k ? 0 : kNibblePlane / 2);
                    if constexpr (kPer == 4)
                        *reinterpret_cast<uint16_t*>(r + h * 64 + 2 * lane) = static_cast<uint16_t>(codes);
                    else
                        *reinterpret_cast<uint32_t*>(r + 4 * lane) = codes;
                    if (lane % kShare == 0) {
                        uint8_t* scales = r + (is_k ? kNibbleScales : kNibbleScales + 8 - kNibblePlane / 2);
                        scales[(D == 256 ? 4 * h : 0) + lane / kShare] = static_cast<uint8_t>(scale);
                    }
                }
            }
        }
    }
}

}  // namespace gqa
