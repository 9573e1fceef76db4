// The 4-bit KV cache format.  256 channels of one KV head are a plane (one per head at
// D = 256, two at D = 512); a position's K and V of a plane are one row of 272 bytes:
//
//   [0, 128)    codes of K: channel 2i in the low half of byte i, 2i + 1 in the high half
//   [128, 256)  codes of V
//   [256, 264)  scales of K, one byte for 32 channels
//   [264, 272)  scales of V
//
//   x ~ (u - 8) s,   u in 1 .. 15,   s = the f16 number with bits (byte << 7)
//
// A scale is an f16 number of three mantissa bits, bytes 0 .. 0xa7 (60).  s is the smallest
// with amax <= 7.5 s, so that no value is further than half a step from its code; u - 8 is
// x / s to the nearest whole number, ties away from zero, at most 7.  Channels of which one is
// not finite have the scale byte 0xff (an f16 NaN) and codes 8.
//
// Why this form.  (u - 8) s has at most seven significant bits, so it is exact in f16 and in
// bf16, and one f16x2 fma makes it of two codes.  (e2m1 codes, of four bits too, are 6 to 9%
// further off for normally distributed values, by how their scale is rounded: rms 0.102 to 0.105
// of the values' against 0.096, 32 to a scale.)  A
// row stands by itself: a new token touches no other row.  K, V and scales of 16 positions are
// one run of memory, 4352 bytes, which one bulk copy moves, and rows of 17 16-byte units are
// read without bank conflicts.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx_more.cuh"

namespace gqa {

constexpr int kNibblePlane = 256;     // channels of a plane
constexpr int kNibbleRow = 272;       // bytes of a plane's row
constexpr int kNibbleGroup = 32;      // channels that share a scale
constexpr int kNibbleScales = 256;    // offset of the scales in a row
constexpr int kNibblePage = 16;       // positions per page
constexpr uint32_t kNibbleTopScale = 0xa7, kNibbleNanScale = 0xff;

// Two floats as packed bf16 (lo in the low half).
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}

// The scale that a byte stands for.
__device__ __forceinline__ float nibble_scale(uint32_t byte) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// The byte of the smallest scale s with amax <= 7.5 s (amax finite, >= 0; the largest where none is).
__device__ __forceinline__ uint32_t nibble_scale_byte(float amax) {
    // a guess within one of it, settled by exact products
    const float want = fminf(amax * (1.0f / 7.5f), 60.0f);
    int c = (__half_as_ushort(__float2half_ru(want)) + 0x7f) >> 7;
    if (amax > 7.5f * nibble_scale(static_cast<uint32_t>(c))) ++c;
    if (c > 0 && amax <= 7.5f * nibble_scale(static_cast<uint32_t>(c - 1))) --c;
    return min(static_cast<uint32_t>(c), kNibbleTopScale);
}

// Codes (one word) and the scale byte of a lane's eight channels, packed bf16 in channel order; four
// neighbouring lanes hold a group.  Some 60 operations.
//
// The byte.  amax has the bits (e << 7 | f): it is A 2^n, A = 128 + f.  In the octave above 120 the scales'
// bounds 7.5 s are 120, 135, 150, ... times 2^n, one byte apart, so the byte is that of 120, 8 e - 920, and
// ceil((A - 120) / 15) more.  (Below byte 8 the scales are subnormal and spaced evenly.)
// The codes.  x is a bf16 number and s has four bits, so x / s is a tie between two codes or at least
// 2^-8 of itself away from one: the reciprocal taken 2^-16 too large turns ties away from zero and
// changes nothing else.  x is kept below 7.5 s (a bf16 number), rounded by one fma to 1.5 2^23 + 8 + x / s,
// and the words' low bits are added up by place, less what the rest of the words adds up to.
__device__ __forceinline__ uint32_t nibble_codes(const uint32_t (&u)[4], uint32_t* scale) {
    // largest magnitude: the bits of |bf16| order like the values, infinity and NaN above
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, u[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    uint32_t c = ((m >> 4) & 0xff8u) - 920u + ((((m & 0x7fu) + 22u) * 137u) >> 11), byte = c;
    float up = 1.0f + 0x1p-16f;
    if (c - 8u > kNibbleTopScale - 8u) {   // (seldom) subnormal scales, zeros, beyond the largest, not finite
        const bool finite = m < 0x7f80u;
        byte = finite ? nibble_scale_byte(__uint_as_float(m << 16)) : kNibbleNanScale;
        c = finite && byte > 0 ? byte : 8u;
        if (!finite) up = 0.0f;            // codes 8
    }
    *scale = byte;
    const float s = nibble_scale(c);
    const float inv = ptx::rcp(s) * up;
    const uint32_t top = __byte_perm(__float_as_uint(7.5f * s), 0u, 0x3232) - 0x00010001u, low = top | 0x80008000u;
    constexpr uint32_t kOne = 0x4b400000u;   // of 1.5 2^23
    uint32_t r = 0u - kOne * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = ptx::bf16x2_max(ptx::bf16x2_min(u[i], top), low);
        r += __float_as_uint(fmaf(__uint_as_float(x << 16), inv, 0x1.8p23f + 8.0f)) << (8 * i);
        r += __float_as_uint(fmaf(__uint_as_float(x & 0xffff0000u), inv, 0x1.8p23f + 8.0f)) << (8 * i + 4);
    }
    return r;
}

// Where the cache holds a row: contiguous [B, planes, rows, 272] or pools [P, planes, 16, 272].
struct NibbleCache {
    uint8_t* kv;
    const int32_t* block_table;   // [B, max_pages]; null: contiguous
    int rows;                     // contiguous: positions per sequence
    int max_pages, num_pages;     // paged
    int planes;                   // KVH * D / 256

    __host__ __device__ int capacity() const { return block_table ? max_pages * kNibblePage : rows; }
    // Bytes from a plane's row to the next plane's.
    __device__ __forceinline__ size_t plane_stride() const {
        return static_cast<size_t>(block_table ? kNibblePage : rows) * kNibbleRow;
    }
    // Plane 0's row of position pos (below the capacity) of sequence b; null when its page id is
    // out of range.
    __device__ __forceinline__ uint8_t* row(int b, int pos) const {
        if (block_table) {
            const int page = block_table[static_cast<size_t>(b) * max_pages + pos / kNibblePage];
            if (page < 0 || page >= num_pages) return nullptr;
            return kv + (static_cast<size_t>(page) * planes * kNibblePage + pos % kNibblePage) * kNibbleRow;
        }
        return kv + (static_cast<size_t>(b) * planes * rows + pos) * kNibbleRow;
    }
};

// The tokens of a ragged call: those of sequence b are rows [off_b, off_{b+1}) of the packed
// arrays, at the positions [L_b - n_b, L_b).
struct TokenIndex {
    int off[257];
    int len[256];

    // By the whole CTA, ending with a barrier.
    __device__ __forceinline__ void load(const int32_t* token_offsets, const int32_t* seq_lens, int B) {
        for (int i = threadIdx.x; i <= B; i += blockDim.x) {
            off[i] = token_offsets[i];
            if (i < B) len[i] = seq_lens[i];
        }
        __syncthreads();
    }
    // Sequence and position of packed token i < N; false when it belongs to no sequence, or to one
    // whose offsets lie outside [0, N] or whose length is below its number of new tokens.  (Offsets
    // that do not ascend are found or not, but never give a token a place outside its sequence.)
    __device__ __forceinline__ bool find(int B, int N, int i, int* b, int* pos) const {
        int lo = 0, hi = B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (off[mid] <= i)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int o0 = off[lo], o1 = off[lo + 1], L = len[lo];
        *b = lo;
        *pos = L - o1 + i;
        return o0 >= 0 && o0 <= i && i < o1 && o1 <= N && L >= o1 - o0;
    }
};

}  // namespace gqa
