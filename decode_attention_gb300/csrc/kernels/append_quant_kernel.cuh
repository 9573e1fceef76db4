// Quantising K/V rows into the 8-bit cache (quant_cache.cuh) as they are written.
//
// The new rows of sequence b are the packed tokens [off_b, off_{b+1}); they go to the
// positions [L_b - n_b, L_b).  A warp takes one block of 16 positions of one KV head of K
// or V: it loads the block's new rows once (each lane 16 bytes of a row at a time), takes
// the largest magnitude, and writes the codes and the scale.  In a block that holds
// earlier rows of the sequence the scale never shrinks; when it grows the earlier rows
// are re-coded.  Rows behind the last new one are left as they are.
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
__global__ void __launch_bounds__(kAppendThreads)
    gqa_append_quant_kernel(const AppendQuantParams p) {
    constexpr int kVec = D / 256;   // 16-byte loads per lane and row
    __shared__ BlockIndex idx;

    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    const QuantCache& c = p.cache;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int capacity = c.capacity();
    // blocks of positions that sequence b writes; 0 when its offsets or length do not fit
    idx.build(p.B, [&](int b) {
        const int o0 = p.token_offsets[b], o1 = p.token_offsets[b + 1], L = p.seq_lens[b];
        if (o0 < 0 || o1 <= o0 || o1 > p.N || L < o1 - o0 || L > capacity) return 0;
        return (L - 1) / kQuantBlock - (L - (o1 - o0)) / kQuantBlock + 1;
    });
    const uint32_t per_block = 2u * c.KVH;   // K heads, then V heads
    const uint32_t items = idx.pref[p.B];
    const uint64_t total = static_cast<uint64_t>(items) * per_block;

    for (uint64_t it = static_cast<uint64_t>(blockIdx.x) * (kAppendThreads / 32) + warp; it < total;
         it += static_cast<uint64_t>(gridDim.x) * (kAppendThreads / 32)) {
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

        const __nv_bfloat16* src =
            (is_v ? p.v_new : p.k_new) +
            (static_cast<size_t>(o0 + base - start + j0) * c.KVH + kvh) * D + lane * 8;
        uint8_t* dst = (is_v ? c.v : c.k) + (row * c.KVH + kvh) * D + lane * 8;
        float* scale = (is_v ? c.v_scales : c.k_scales) + scale_row * c.KVH + kvh;
        const size_t stride = static_cast<size_t>(c.KVH) * D;

        uint4 w[kQuantBlock][kVec];
#pragma unroll
        for (int j = 0; j < kQuantBlock; ++j)
#pragma unroll
            for (int q = 0; q < kVec; ++q) {
                w[j][q] = make_uint4(0, 0, 0, 0);
                if (j < j1 - j0)
                    w[j][q] = __ldcs(reinterpret_cast<const uint4*>(src + j * stride + q * 256));
            }
        const float old = j0 > 0 ? *scale : 0.0f;
        // largest magnitude: the bits of |bf16| order like the values, NaN above infinity
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < kQuantBlock; ++j)
#pragma unroll
            for (int q = 0; q < kVec; ++q) {
                m = __vmaxu2(m, w[j][q].x & 0x7fff7fffu);
                m = __vmaxu2(m, w[j][q].y & 0x7fff7fffu);
                m = __vmaxu2(m, w[j][q].z & 0x7fff7fffu);
                m = __vmaxu2(m, w[j][q].w & 0x7fff7fffu);
            }
        m = max(m & 0xffffu, m >> 16);
        m = __reduce_max_sync(0xffffffffu, m);
        const bool non_finite = m >= 0x7f80u;
        if (non_finite) {   // the largest finite one instead
            m = 0;
#pragma unroll
            for (int j = 0; j < kQuantBlock; ++j)
#pragma unroll
                for (int q = 0; q < kVec; ++q) {
                    const uint32_t u[4] = {w[j][q].x, w[j][q].y, w[j][q].z, w[j][q].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t lo = u[i] & 0x7fffu, hi = (u[i] >> 16) & 0x7fffu;
                        m = max(m, lo < 0x7f80u ? lo : 0u);
                        m = max(m, hi < 0x7f80u ? hi : 0u);
                    }
                }
            m = __reduce_max_sync(0xffffffffu, m);
        }
        int e = quant_exponent(__uint_as_float(m << 16));
        if (j0 > 0) {
            const int eo = scale_exponent(old);
            if (e > eo) {
                const float f = pow2f(max(eo - e, -126));
                for (int j = 0; j < j0; ++j)
#pragma unroll
                    for (int q = 0; q < kVec; ++q) {
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
        for (int j = 0; j < kQuantBlock; ++j) {
            if (j >= j1 - j0) break;
#pragma unroll
            for (int q = 0; q < kVec; ++q) {
                const uint32_t u[4] = {w[j][q].x, w[j][q].y, w[j][q].z, w[j][q].w};
                uint16_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo = __uint_as_float(u[i] << 16) * inv;
                    float hi = __uint_as_float(u[i] & 0xffff0000u) * inv;
                    if (non_finite) {
                        lo = inf_to_nan(lo);
                        hi = inf_to_nan(hi);
                    }
                    o[i] = ptx::float2_to_e4m3x2(lo, hi);
                }
                *reinterpret_cast<uint2*>(dst + (j0 + j) * stride + q * 256) =
                    make_uint2(o[0] | (static_cast<uint32_t>(o[1]) << 16),
                               o[2] | (static_cast<uint32_t>(o[3]) << 16));
            }
        }
        if (lane == 0) *scale = pow2f(e);
    }
}

}  // namespace gqa
