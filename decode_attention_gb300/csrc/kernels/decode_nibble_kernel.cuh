// Decode attention over the 4-bit cache (nibble_cache.cuh): attn.core of the gemma-4-31B Model
// Spec for one new token per sequence.
//
// One CTA per sequence and KV head.  Each of its warps takes every eighth position: lane l holds
// channels 8l .. 8l + 7 of each plane, makes their products with the G query heads, and keeps the
// running maximum, sum and output of its positions; the warps' states are merged at the end.
#pragma once

#include "decode_kernel.cuh"
#include "nibble_cache.cuh"
#include "read_nibble_kernel.cuh"   // nibble_values

namespace gqa {

constexpr int kDecodeNibbleWarps = 8;

struct DecodeNibbleParams {
    DecodeParams d;
    NibbleCache cache;
};

template <int G, int D>
__global__ void __launch_bounds__(kDecodeNibbleWarps * 32)
    gqa_decode_nibble_kernel(const DecodeNibbleParams np) {
    constexpr int kPlanes = D / kNibblePlane;
    const DecodeParams& p = np.d;
    const NibbleCache& c = np.cache;
    __shared__ float sm_m[kDecodeNibbleWarps], sm_l[kDecodeNibbleWarps];
    __shared__ float sm_acc[kDecodeNibbleWarps][D];

    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / p.KVH, kvh = blockIdx.x % p.KVH;
    int L = p.seq_lens[b];
    if (L < 0 || L > p.capacity) {
        if (threadIdx.x == 0) atomicOr(p.ws_flags, kFlagBadLength);
        L = L < 0 ? 0 : p.capacity;
    }
    const int lo = p.window > 0 && L > p.window ? L - p.window : 0;
    const size_t out = (static_cast<size_t>(b) * p.H + kvh * G) * D;

    uint32_t q[G][kPlanes][4];
    float m[G], l[G], acc[G][kPlanes][8];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.0f;
#pragma unroll
        for (int j = 0; j < kPlanes; ++j) {
            const uint4 t = *reinterpret_cast<const uint4*>(p.q + out + g * D + j * kNibblePlane + lane * 8);
            q[g][j][0] = t.x;
            q[g][j][1] = t.y;
            q[g][j][2] = t.z;
            q[g][j][3] = t.w;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[g][j][e] = 0.0f;
        }
    }
    for (int pos = lo + warp; pos < L; pos += kDecodeNibbleWarps) {
        const uint8_t* row = c.row(b, pos);
        const bool bad = row == nullptr;
        if (bad && lane == 0) atomicOr(p.ws_flags, kFlagBadPage);
        float k[kPlanes][8], v[kPlanes][8];
#pragma unroll
        for (int j = 0; j < kPlanes; ++j) {
            const uint8_t* r = bad ? c.kv : row + (kvh * kPlanes + j) * c.plane_stride();
            nibble_values(reinterpret_cast<const uint32_t*>(r)[lane], r[kNibbleScales + lane / 4], k[j]);
            nibble_values(reinterpret_cast<const uint32_t*>(r + kNibblePlane / 2)[lane],
                          r[kNibbleScales + 8 + lane / 4], v[j]);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < kPlanes; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s = fmaf(e % 2 ? bf16hi(q[g][j][e / 2]) : bf16lo(q[g][j][e / 2]), k[j][e], s);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            s = bad ? __uint_as_float(0x7fc00000u) : s * kLog2e;
            const float top = fmaxf(m[g], s);
            const float a = m[g] == -INFINITY ? 0.0f : ptx::ex2(m[g] - top);
            const float w = ptx::ex2(s - top);
            m[g] = top;
            l[g] = l[g] * a + w;
#pragma unroll
            for (int j = 0; j < kPlanes; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[g][j][e] = fmaf(w, v[j][e], acc[g][j][e] * a);
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
        __syncthreads();
        if (lane == 0) {
            sm_m[warp] = m[g];
            sm_l[warp] = l[g];
        }
#pragma unroll
        for (int j = 0; j < kPlanes; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) sm_acc[warp][j * kNibblePlane + lane * 8 + e] = acc[g][j][e];
        __syncthreads();
        float top = -INFINITY, den = 0.0f, f[kDecodeNibbleWarps];
        for (int w = 0; w < kDecodeNibbleWarps; ++w) top = fmaxf(top, sm_m[w]);
        for (int w = 0; w < kDecodeNibbleWarps; ++w) {
            f[w] = sm_l[w] == 0.0f ? 0.0f : ptx::ex2(sm_m[w] - top);
            den += f[w] * sm_l[w];
        }
        for (int d = threadIdx.x; d < D; d += blockDim.x) {
            float x = 0.0f;
            for (int w = 0; w < kDecodeNibbleWarps; ++w) x += f[w] * sm_acc[w][d];
            store_out(p, out + g * D + d, den == 0.0f ? 0.0f : x / den);
        }
    }
}

}  // namespace gqa
