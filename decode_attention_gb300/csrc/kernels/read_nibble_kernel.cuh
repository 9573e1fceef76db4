// Reading the 4-bit cache (nibble_cache.cuh) back: out[b, s] = (u - 8) s for the positions s in
// [lo_b, min(L_b, out_rows)), in bf16 (exact) or fp32.  Other rows of the output are left as they
// are.
//
// One item is kPlanes planes of a position, taken by a warp: lane l reads the word of channels
// 8l .. 8l + 7 of K and of V.  In bf16 it writes them, 16 bytes; in fp32 it takes half a word of another
// lane, twice, so that a store fills whole lines.
//
// Bound by the memory's rate, four fifths of it writes: 16 decodeGQA sequences of up to 32768 positions, paged,
// 448 to 454 us in bf16, 0.87 of a copy's rate; of up to 16384 in fp32 378 us, 0.93 (570 with a lane's own
// channels, whose two stores each filled half of their sectors).
#pragma once

#include "nibble_cache.cuh"
#include "quant_cache.cuh"   // BlockIndex

namespace gqa {

constexpr int kReadNibbleThreads = 256;

struct ReadNibbleParams {
    NibbleCache cache;
    const int32_t* seq_lens;   // [B]
    void* k_out;               // [B, out_rows, KVH, D]
    void* v_out;
    int B, window, out_rows;
};

// n channels of a word (from its lowest bits on) as floats, in channel order.
template <int n>
__device__ __forceinline__ void nibble_values(uint32_t w, uint32_t scale, float (&x)[n]) {
    const float s = scale > kNibbleTopScale ? __uint_as_float(0x7fc00000u) : nibble_scale(scale);
#pragma unroll
    for (int i = 0; i < n; ++i)   // 2^23 + u less 2^23 + 8
        x[i] = (__uint_as_float(0x4b000000u | ((w >> (4 * i)) & 15u)) - (0x1p23f + 8.0f)) * s;
}

template <int kPlanes, bool kF32>
__global__ void __launch_bounds__(kReadNibbleThreads, kF32 ? 6 : 8)
    gqa_read_nibble_kernel(const ReadNibbleParams p) {
    __shared__ BlockIndex idx;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    const NibbleCache& c = p.cache;
    const int lane = threadIdx.x & 31;
    const int capacity = c.capacity();
    auto range = [&](int b, int* lo) {   // positions [*lo, returned)
        const int L = min(max(p.seq_lens[b], 0), capacity);
        *lo = p.window > 0 && L > p.window ? L - p.window : 0;
        return min(L, p.out_rows);
    };
    idx.build(p.B, [&](int b) {   // in positions
        int lo;
        const int hi = range(b, &lo);
        return max(hi - lo, 0);
    });
    const uint32_t per_pos = static_cast<uint32_t>(c.planes / kPlanes);
    const uint32_t total = idx.pref[p.B] * per_pos;   // (at most 2^26 positions, 16 planes)
    const size_t stride = c.plane_stride();
    constexpr int kWarps = kReadNibbleThreads / 32;
    for (uint32_t it = blockIdx.x * kWarps + (threadIdx.x >> 5); it < total; it += gridDim.x * kWarps) {
        const uint32_t x = it / per_pos;
        const int plane = static_cast<int>(it % per_pos) * kPlanes;
        const int b = idx.seq_of(p.B, x);
        int lo;
        range(b, &lo);
        const int pos = lo + static_cast<int>(x - idx.pref[b]);
        const uint8_t* row = c.row(b, pos);
        if (!row) continue;
        row += plane * stride;
        uint32_t kw[kPlanes], vw[kPlanes], ks[kPlanes], vs[kPlanes];
#pragma unroll
        for (int j = 0; j < kPlanes; ++j) {
            const uint8_t* r = row + j * stride;
            kw[j] = __ldg(reinterpret_cast<const uint32_t*>(r) + lane);
            vw[j] = __ldg(reinterpret_cast<const uint32_t*>(r + kNibblePlane / 2) + lane);
            ks[j] = __ldg(r + kNibbleScales + lane / 4);
            vs[j] = __ldg(r + kNibbleScales + 8 + lane / 4);
        }
        const size_t at = ((static_cast<size_t>(b) * p.out_rows + pos) * c.planes + plane) * kNibblePlane;
#pragma unroll
        for (int j = 0; j < kPlanes; ++j)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t w = t ? vw[j] : kw[j], sc = t ? vs[j] : ks[j];
                if (kF32) {
                    float* out = static_cast<float*>(t ? p.v_out : p.k_out) + at + j * kNibblePlane + 4 * lane;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // channels 128 h + 4 lane .. + 3
                        const int from = 16 * h + (lane >> 1);
                        const uint32_t half = __shfl_sync(0xffffffffu, w, from) >> (16 * (lane & 1));
                        float y[4];
                        nibble_values(half, __shfl_sync(0xffffffffu, sc, from), y);
                        __stcs(reinterpret_cast<float4*>(out + 128 * h), make_float4(y[0], y[1], y[2], y[3]));
                    }
                } else {
                    float y[8];
                    nibble_values(w, sc, y);
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(t ? p.v_out : p.k_out) + at + j * kNibblePlane;
                    __stcs(reinterpret_cast<uint4*>(out + 8 * lane),
                           make_uint4(bf16x2_bits(y[0], y[1]), bf16x2_bits(y[2], y[3]),
                                      bf16x2_bits(y[4], y[5]), bf16x2_bits(y[6], y[7])));
                }
            }
    }
}

}  // namespace gqa
