// Quantising K/V rows into the 8-bit cache (quant_cache.cuh) as they are written.
//
// The new rows of sequence b are the packed tokens [off_b, off_{b+1}); they go to the
// positions [L_b - n_b, L_b).  One item is a block of 16 positions of one KV head of K or V:
// its new rows are loaded once into registers (16 bytes of a row per lane), the largest
// magnitude is taken, and the codes and the scale are written.  D / 256 warps share an
// item, 16 / (D / 256) rows each, so that a lane holds 64 registers of data at both head
// sizes and 16 warps fit an SM (one warp per item at D = 512 needs 171 registers and left 8
// warps: append_chunks_b32_paged 97.6 us).  In a block that holds earlier rows of the
// sequence the scale never shrinks; when it grows the earlier rows are re-coded.  Rows
// behind the last new one are left as they are.
#pragma once

#include "quant_cache.cuh"

namespace gqa {

constexpr int kAppendThreads = 256;

struct AppendQuantParams {
    const __nv_bfloat16* k_new;     // [N, KVH, D]
    const __nv_bfloat16* v_new;     // [N, KVH, D]
    const int32_t* token_offsets;   // [B + 1]
    const int32_t* seq_lens;        // [B], lengths after the append
    QuantCache cache;
    int B, N;
};

template <int D>
__global__ void __launch_bounds__(kAppendThreads, 2)
    gqa_append_quant_kernel(const AppendQuantParams p) {
    constexpr int kWarps = kAppendThreads / 32;
    constexpr int kShare = D / 256;               // warps per item
    constexpr int kRows = kQuantBlock / kShare;   // block rows per warp
    constexpr int kItems = kWarps / kShare;       // items a CTA works on at a time
    __shared__ BlockIndex idx;
    __shared__ uint32_t top[2][kWarps];           // [turn parity]: largest magnitude of each warp

    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    const QuantCache& c = p.cache;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sub = warp % kShare, slot = warp / kShare;
    const int capacity = c.capacity();
    // blocks of positions that sequence b writes; 0 when its offsets or length do not fit
    idx.build(p.B, [&](int b) {
        const int o0 = p.token_offsets[b], o1 = p.token_offsets[b + 1], L = p.seq_lens[b];
        if (o0 < 0 || o1 <= o0 || o1 > p.N || L < o1 - o0 || L > capacity) return 0;
        return (L - 1) / kQuantBlock - (L - (o1 - o0)) / kQuantBlock + 1;
    });
    const uint32_t per_block = 2u * c.KVH;   // K heads, then V heads
    const uint64_t total = static_cast<uint64_t>(idx.pref[p.B]) * per_block;
    uint32_t turn = 0;
    // the largest of the sharing warps' values (the other parity is written next, after this
    // exchange's barrier)
    auto share_max = [&](uint32_t m) {
        m = __reduce_max_sync(0xffffffffu, m);
        if constexpr (kShare > 1) {
            uint32_t* t = top[turn & 1u];
            ++turn;
            if (lane == 0) t[warp] = m;
            ptx::named_barrier_sync(1 + slot, 32 * kShare);
#pragma unroll
            for (int i = 0; i < kShare; ++i) m = max(m, t[slot * kShare + i]);
        }
        return m;
    };

    for (uint64_t it = static_cast<uint64_t>(blockIdx.x) * kItems + slot; it < total;
         it += static_cast<uint64_t>(gridDim.x) * kItems) {
        const uint32_t x = static_cast<uint32_t>(it / per_block);
        const int th = static_cast<int>(it - static_cast<uint64_t>(x) * per_block);
        const bool is_v = th >= c.KVH;
        const int kvh = is_v ? th - c.KVH : th;
        const int b = idx.seq_of(p.B, x);
        const int o0 = p.token_offsets[b], n = p.token_offsets[b + 1] - o0;
        const int start = p.seq_lens[b] - n;               // first new position
        const int blk = start / kQuantBlock + static_cast<int>(x - idx.pref[b]);
        const int base = blk * kQuantBlock;
        const int j0 = start > base ? start - base : 0;    // new rows [j0, j1) of the block
        const int j1 = min(start + n - base, kQuantBlock);
        size_t row, scale_row;
        if (!c.locate(b, blk, &row, &scale_row)) continue;

        // this warp's rows: sub, sub + kShare, ... of the block
        const size_t stride = static_cast<size_t>(c.KVH) * D;
        const __nv_bfloat16* src = (is_v ? p.v_new : p.k_new) +
                                   (static_cast<int64_t>(o0) + base - start) * static_cast<int64_t>(stride) +
                                   static_cast<size_t>(kvh) * D + lane * 8;
        uint8_t* dst = (is_v ? c.v : c.k) + (row * c.KVH + kvh) * D + lane * 8;
        float* scale = (is_v ? c.v_scales : c.k_scales) + scale_row * c.KVH + kvh;

        uint4 w[kRows][kShare];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int q = 0; q < kShare; ++q) {
                const int j = i * kShare + sub;
                w[i][q] = make_uint4(0, 0, 0, 0);
                if (j >= j0 && j < j1)
                    w[i][q] = __ldcs(reinterpret_cast<const uint4*>(src + j * stride + q * 256));
            }
        const float old = j0 > 0 ? *scale : 0.0f;
        // largest magnitude: the bits of |bf16| order like the values, NaN above infinity
        uint32_t m2 = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int q = 0; q < kShare; ++q) {
                m2 = __vmaxu2(m2, w[i][q].x & 0x7fff7fffu);
                m2 = __vmaxu2(m2, w[i][q].y & 0x7fff7fffu);
                m2 = __vmaxu2(m2, w[i][q].z & 0x7fff7fffu);
                m2 = __vmaxu2(m2, w[i][q].w & 0x7fff7fffu);
            }
        uint32_t m = share_max(max(m2 & 0xffffu, m2 >> 16));
        const bool non_finite = m >= 0x7f80u;
        if (non_finite) {   // the largest finite one instead
            m = 0;
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
                for (int q = 0; q < kShare; ++q) {
                    const uint32_t u[4] = {w[i][q].x, w[i][q].y, w[i][q].z, w[i][q].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = u[e] & 0x7fffu, hi = (u[e] >> 16) & 0x7fffu;
                        m = max(m, lo < 0x7f80u ? lo : 0u);
                        m = max(m, hi < 0x7f80u ? hi : 0u);
                    }
                }
            m = share_max(m);
        }
        int e = quant_exponent(__uint_as_float(m << 16));
        if (j0 > 0) {
            const int eo = scale_exponent(old);
            if (e > eo) {
                const float f = pow2f(max(eo - e, -126));
                for (int j = sub; j < j0; j += kShare)
#pragma unroll
                    for (int q = 0; q < kShare; ++q) {
                        uint2* r = reinterpret_cast<uint2*>(dst + j * stride + q * 256);
                        const uint2 t = *r;
                        *r = make_uint2(recode4(t.x, f), recode4(t.y, f));
                    }
            } else {
                e = eo;
            }
        }
        const float inv = pow2f(-e);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int j = i * kShare + sub;
            if (j < j0 || j >= j1) continue;
#pragma unroll
            for (int q = 0; q < kShare; ++q) {
                const uint32_t u[4] = {w[i][q].x, w[i][q].y, w[i][q].z, w[i][q].w};
                uint16_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float lo = __uint_as_float(u[k] << 16) * inv;
                    float hi = __uint_as_float(u[k] & 0xffff0000u) * inv;
                    if (non_finite) {
                        lo = inf_to_nan(lo);
                        hi = inf_to_nan(hi);
                    }
                    o[k] = ptx::float2_to_e4m3x2(lo, hi);
                }
                __stcs(reinterpret_cast<uint2*>(dst + j * stride + q * 256),
                       make_uint2(o[0] | (static_cast<uint32_t>(o[1]) << 16),
                                  o[2] | (static_cast<uint32_t>(o[3]) << 16)));
            }
        }
        // (the sharing warps have all read the old scale: each did before the exchange)
        if (sub == 0 && lane == 0) *scale = pow2f(e);
    }
}

}  // namespace gqa
