// The 8-bit KV cache format: e4m3 codes with one power-of-two scale for each block of
// 16 positions and KV head.
//
//   x ~ s * code,   s = 2^e,   e = the smallest integer with amax <= 448 * 2^e,
//   clamped to [-64, 64];   amax = the largest finite magnitude written to the block.
//
// A power of two costs nothing against amax / 448 (e4m3 is a floating format: its
// relative step does not depend on the scale) and makes x / s, code * s and the
// re-coding of a block whose scale grows exact, apart from values that fall among the
// subnormal codes.  So every value is rounded once (to nearest even), and the codes do
// not depend on the order in which a machine sums or compares.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace gqa {

constexpr int kQuantBlock = 16;        // positions that share a scale (= positions per page)
constexpr int kQuantMinExp = -64;
constexpr int kQuantMaxExp = 64;
constexpr uint32_t kQuantNanCode = 0x7f;

// 2^e, e in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// Exponent of the scale of values of magnitude up to amax (finite, >= 0): 448 = 1.75 * 2^8.
__device__ __forceinline__ int quant_exponent(float amax) {
    const int bits = __float_as_int(amax);
    const int e = (bits >> 23) - (127 + 8) + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
    return min(max(e, kQuantMinExp), kQuantMaxExp);
}

// Exponent that a stored scale stands for: its exponent field, clamped (a scale that is no
// power of two in range was not written by this library).
__device__ __forceinline__ int scale_exponent(float s) {
    const int e = ((__float_as_int(s) >> 23) & 0xff) - 127;
    return min(max(e, kQuantMinExp), kQuantMaxExp);
}

// A value as it is coded: infinities take the NaN code.
__device__ __forceinline__ float inf_to_nan(float x) {
    return fabsf(x) == INFINITY ? __uint_as_float(0x7fc00000u) : x;
}

// Four codes (a 32-bit word, low byte first) times f, rounded to codes again.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float f) {
    const float2 a = ptx::e4m3x2_to_float2(static_cast<uint16_t>(w));
    const float2 b = ptx::e4m3x2_to_float2(static_cast<uint16_t>(w >> 16));
    return ptx::float2_to_e4m3x2(a.x * f, a.y * f) |
           (static_cast<uint32_t>(ptx::float2_to_e4m3x2(b.x * f, b.y * f)) << 16);
}

// Where the cache holds a block of positions: contiguous [B, rows, KVH, D] with scales
// [B, ceil(rows / 16), KVH], or page pools [P, 16, KVH, D] with scales [P, KVH].
struct QuantCache {
    uint8_t* k;
    uint8_t* v;
    float* k_scales;
    float* v_scales;
    const int32_t* block_table;   // [B, max_pages]; null: contiguous
    int rows;                     // contiguous: positions per sequence
    int max_pages, num_pages;     // paged
    int KVH;

    __host__ __device__ int capacity() const {
        return block_table ? max_pages * kQuantBlock : rows;
    }
    // First row (in units of KVH * D codes) and scale row (in units of KVH scales) of block
    // `blk` of sequence b; false when its page id is out of range.
    __device__ __forceinline__ bool locate(int b, int blk, size_t* row, size_t* scale_row) const {
        if (block_table) {
            const int page = block_table[static_cast<size_t>(b) * max_pages + blk];
            if (page < 0 || page >= num_pages) return false;
            *row = static_cast<size_t>(page) * kQuantBlock;
            *scale_row = static_cast<size_t>(page);
        } else {
            const int nblk = (rows + kQuantBlock - 1) / kQuantBlock;
            *row = static_cast<size_t>(b) * rows + static_cast<size_t>(blk) * kQuantBlock;
            *scale_row = static_cast<size_t>(b) * nblk + blk;
        }
        return true;
    }
};

// Sequences of a ragged call laid end to end in blocks: sequence b owns the items
// [pref[b], pref[b + 1]).  Built by the whole CTA (blockDim.x >= 256); count(b) is called
// once for every b < B.
struct BlockIndex {
    uint32_t pref[257];
    uint32_t warp_sum[8];

    template <class Count>
    __device__ __forceinline__ void build(int B, Count count) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        uint32_t own = 0, incl = 0;
        if (tid < 256) {
            own = tid < B ? static_cast<uint32_t>(count(tid)) : 0u;
            incl = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t t = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += t;
            }
            if (lane == 31) warp_sum[warp] = incl;
        }
        __syncthreads();
        if (tid < 256) {
            uint32_t base = 0;
            for (int w = 0; w < warp; ++w) base += warp_sum[w];
            pref[tid + 1] = base + incl;
            if (tid == 0) pref[0] = 0;
        }
        __syncthreads();
    }
    // The sequence that owns item x (x < pref[B]).
    __device__ __forceinline__ int seq_of(int B, uint32_t x) const {
        int lo = 0, hi = B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pref[mid] <= x)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    }
};

}  // namespace gqa
