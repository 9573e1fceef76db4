// Reading the 8-bit cache (quant_cache.cuh) back: out[b, s] = scale * code for the
// positions s in [lo_b, min(L_b, out_rows)), in bf16 (exact: 4 significant bits, exponents
// within range) or fp32.  Other rows of the output are left as they are.
//
// A CTA takes one block of 16 positions of K or V (16 * KVH * D contiguous codes), or a
// quarter of one when whole blocks would leave SMs idle (kParts); a thread keeps the loads of
// 8 x 8 codes in flight.  Bound by the memory's read and write rate: bf16 491 us for 3.18 GB
// (read_global_b16_paged, the copy rate's 470), fp32 1095 us for 5.30 GB (782), two stores for
// every load.
#pragma once

#include "quant_cache.cuh"

namespace gqa {

constexpr int kReadThreads = 256;

struct ReadQuantParams {
    QuantCache cache;
    const int32_t* seq_lens;   // [B]
    void* k_out;               // [B, out_rows, KVH, D]
    void* v_out;
    int B, window, out_rows;
};

template <int KVH, int D, bool kF32, int kParts>
__global__ void __launch_bounds__(kReadThreads)
    gqa_read_quant_kernel(const ReadQuantParams p) {
    constexpr int kRow = KVH * D;                                 // codes per position
    constexpr int kSteps = kQuantBlock * kRow / (8 * kReadThreads) / kParts;
    constexpr int kBatch = kSteps < 8 ? kSteps : 8;               // loads in flight per thread
    __shared__ BlockIndex idx;

    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    const QuantCache& c = p.cache;
    const int capacity = c.capacity();
    auto range = [&](int b, int* lo) {   // positions [*lo, returned)
        const int L = min(max(p.seq_lens[b], 0), capacity);
        *lo = p.window > 0 && L > p.window ? L - p.window : 0;
        return min(L, p.out_rows);
    };
    idx.build(p.B, [&](int b) {
        int lo;
        const int hi = range(b, &lo);
        return hi > lo ? (hi - 1) / kQuantBlock - lo / kQuantBlock + 1 : 0;
    });
    const uint32_t total = 2u * kParts * idx.pref[p.B];   // <= 2 * 4 * 256 * 2^14

    for (uint32_t it = blockIdx.x; it < total; it += gridDim.x) {
        const uint32_t x = it / (2u * kParts), sub = it % (2u * kParts);
        const bool is_v = sub >= kParts;
        const int at0 = static_cast<int>(sub % kParts) * (kQuantBlock * kRow / kParts) +
                        static_cast<int>(threadIdx.x) * 8;
        const int b = idx.seq_of(p.B, x);
        int lo;
        const int hi = range(b, &lo);
        const int blk = lo / kQuantBlock + static_cast<int>(x - idx.pref[b]);
        const int base = blk * kQuantBlock;
        size_t row, scale_row;
        if (!c.locate(b, blk, &row, &scale_row)) continue;
        const uint8_t* src = (is_v ? c.v : c.k) + row * kRow;
        const float* scale = (is_v ? c.v_scales : c.k_scales) + scale_row * KVH;
        const size_t out0 = (static_cast<size_t>(b) * p.out_rows + base) * kRow;
#pragma unroll 1
        for (int s0 = 0; s0 < kSteps; s0 += kBatch) {
            uint2 codes[kBatch];
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                const int at = at0 + (s0 + s) * kReadThreads * 8, pos = base + at / kRow;
                codes[s] = make_uint2(0, 0);
                if (pos >= lo && pos < hi) codes[s] = __ldcs(reinterpret_cast<const uint2*>(src + at));
            }
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                const int at = at0 + (s0 + s) * kReadThreads * 8, pos = base + at / kRow;
                if (pos < lo || pos >= hi) continue;
                const uint2 w = codes[s];
                const float f = pow2f(scale_exponent(__ldg(scale + (at % kRow) / D)));
                float2 v[4] = {ptx::e4m3x2_to_float2(static_cast<uint16_t>(w.x)),
                               ptx::e4m3x2_to_float2(static_cast<uint16_t>(w.x >> 16)),
                               ptx::e4m3x2_to_float2(static_cast<uint16_t>(w.y)),
                               ptx::e4m3x2_to_float2(static_cast<uint16_t>(w.y >> 16))};
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = make_float2(v[i].x * f, v[i].y * f);
                if (kF32) {
                    float4* o = reinterpret_cast<float4*>(static_cast<float*>(is_v ? p.v_out : p.k_out) + out0 + at);
                    __stcs(o, make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
                    __stcs(o + 1, make_float4(v[2].x, v[2].y, v[3].x, v[3].y));
                } else {
                    uint4 o;
                    uint32_t* ow = &o.x;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 t = __floats2bfloat162_rn(v[i].x, v[i].y);
                        ow[i] = *reinterpret_cast<const uint32_t*>(&t);
                    }
                    __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? p.v_out : p.k_out) + out0 + at), o);
                }
            }
        }
    }
}

}  // namespace gqa
