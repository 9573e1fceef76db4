// Decode attention over the 8-bit cache (quant_cache.cuh): attn.core of the gemma-4-31B
// Model Spec for one new token per sequence, over k = s_k code_k and v = s_v code_v.
//
// One CTA per (KV head, sequence).  It walks the attended positions in blocks of 16 that
// share their scales, widens the codes through shared memory and keeps an online softmax
// in fp32.
#pragma once

#include "decode_kernel.cuh"
#include "quant_cache.cuh"

namespace gqa {

constexpr int kDecodeQuantThreads = 256;

struct DecodeQuantParams {
    DecodeParams d;
    QuantCache cache;
};

template <int G, int D>
__global__ void __launch_bounds__(kDecodeQuantThreads)
    gqa_decode_quant_kernel(const DecodeQuantParams p) {
    constexpr int kPer = D / kDecodeQuantThreads;   // output dims per thread
    __shared__ __nv_bfloat16 qs[G][D];
    __shared__ float kv[kQuantBlock][D];
    __shared__ float sc[G][kQuantBlock];

    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    const QuantCache& c = p.cache;
    const int kvh = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int capacity = c.capacity();
    int L = p.d.seq_lens[b];
    if (L < 0 || L > capacity) {
        if (kvh == 0 && tid == 0) atomicOr(p.d.ws_flags, kFlagBadLength);
        L = L < 0 ? 0 : capacity;
    }
    const int lo = p.d.window > 0 && L > p.d.window ? L - p.d.window : 0;
    const size_t out0 = (static_cast<size_t>(b) * p.d.H + kvh * G) * D;
    for (int i = tid; i < G * D; i += kDecodeQuantThreads)
        qs[i / D][i % D] = p.d.q[out0 + i];

    float acc[G][kPer], m[G], l[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[h][i] = 0.0f;
    }
    bool bad = false;
    const size_t stride = static_cast<size_t>(c.KVH) * D;
    for (int blk = lo / kQuantBlock; blk * kQuantBlock < L; ++blk) {
        const int j0 = max(lo - blk * kQuantBlock, 0);
        const int j1 = min(L - blk * kQuantBlock, kQuantBlock);
        size_t row, scale_row;
        if (!c.locate(b, blk, &row, &scale_row)) {
            bad = true;
            continue;
        }
        const size_t base = (row * c.KVH + kvh) * D;
        const float fk = pow2f(scale_exponent(c.k_scales[scale_row * c.KVH + kvh]));
        const float fv = pow2f(scale_exponent(c.v_scales[scale_row * c.KVH + kvh]));
        auto widen = [&](const uint8_t* codes, float f) {
            __syncthreads();
            for (int i = tid * 2; i < kQuantBlock * D; i += 2 * kDecodeQuantThreads) {
                const int j = i / D, d = i % D;
                float2 v = make_float2(0.0f, 0.0f);
                if (j >= j0 && j < j1)
                    v = ptx::e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(codes + base + j * stride + d));
                kv[j][d] = v.x * f;
                kv[j][d + 1] = v.y * f;
            }
            __syncthreads();
        };
        widen(c.k, fk);
        for (int t = warp; t < G * kQuantBlock; t += kDecodeQuantThreads / 32) {
            const int h = t / kQuantBlock, j = t % kQuantBlock;
            float s = 0.0f;
            for (int d = lane; d < D; d += 32) s = fmaf(__bfloat162float(qs[h][d]), kv[j][d], s);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            if (lane == 0) sc[h][j] = j >= j0 && j < j1 ? s * kLog2e : -INFINITY;
        }
        widen(c.v, fv);
#pragma unroll
        for (int h = 0; h < G; ++h) {
            float mn = m[h];
#pragma unroll
            for (int j = 0; j < kQuantBlock; ++j) mn = fmaxf(mn, sc[h][j]);
            const float mm = mn == -INFINITY ? 0.0f : mn;   // no finite score so far
            const float alpha = exp2f(m[h] - mm);
            l[h] *= alpha;
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[h][i] *= alpha;
            for (int j = 0; j < kQuantBlock; ++j) {
                const float w = exp2f(sc[h][j] - mm);
                l[h] += w;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    acc[h][i] = fmaf(w, kv[j][tid + i * kDecodeQuantThreads], acc[h][i]);
            }
            m[h] = mn;
        }
    }
    if (bad && tid == 0) atomicOr(p.d.ws_flags, kFlagBadPage);
    const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int h = 0; h < G; ++h)
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            store_out(p.d, out0 + h * D + tid + i * kDecodeQuantThreads,
                      bad ? nan : (l[h] == 0.0f ? 0.0f : acc[h][i] / l[h]));
}

}  // namespace gqa
