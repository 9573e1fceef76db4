// The decode-step producer (prepare_kernel.cuh: norms, rotary positions) writing the new
// token of each sequence into the 8-bit cache (quant_cache.cuh).
//
// The same grid: a warp per head vector.  A k or v warp codes its row; at the first position
// of a block the scale starts anew, later in the block it never shrinks, and when it grows
// the warp re-codes the block's earlier rows of its head.
//
// An fp32 error of 2^-22 moves a value over a border between two codes once in some 10^5
// values, a whole step each time.  Norm, weight and rotation of k and v are therefore taken to
// some 2^-30 (twofold.cuh): codes and scales are those of the formulas but for one value in
// 10^7.  In a graph that costs 2.9 us in place of 2.6 for one sequence and 9.8 in place of 7.7
// for 256; a loop of calls is bound by the host either way (11 and 12.4 us).
#pragma once

#include "prepare_kernel.cuh"
#include "quant_cache.cuh"
#include "twofold.cuh"

namespace gqa {

struct PrepareQuantParams {
    const __nv_bfloat16* q_raw;   // [B, H, D]
    const __nv_bfloat16* k_raw;   // [B, KVH, D]
    const __nv_bfloat16* v_raw;   // [B, KVH, D]
    const __nv_bfloat16* w_q;     // [D]
    const __nv_bfloat16* w_k;     // [D]
    const int32_t* seq_lens;      // [B], lengths after the append
    __nv_bfloat16* q_out;         // [B, H, D]
    QuantCache cache;
    int B, H;
    int n_rot;                    // rotated pairs
    uint64_t turn[kPrepareMaxRot];   // turns per position of pair i, a 64-bit fraction
};

// The angle of position pos is pos turns of `turn`: the product wraps at whole turns, so it is
// reduced exactly in integers.  turn is off by at most 2^-52 of itself (a double's steps), a
// position below 2^18 by 2^-36 turns.  (In fp64, at 2 operations a clock, the angles of the eight
// CTAs of a sequence would cost more than its data.)

// One k or v head vector over a warp, as head_norm_rope: x becomes floats that round to a code
// as the values do.
template <int D>
__device__ __forceinline__ void head_norm_rope_to_odd(float (&x)[2][D / 64], const __nv_bfloat16* w,
                                                      const float2* cs, const float2* cs_l, int n_rot,
                                                      int lane) {
    constexpr int kHalf = D / 2;
    constexpr int kPer = kHalf / 32;
    float ss = 0.0f, ss_l = 0.0f;   // (the square of a bf16 value is exact)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const Twofold t = exact_sum(ss, __fmul_rn(x[h][e], x[h][e]));
            ss = t.h;
            ss_l += t.l;
        }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const Twofold t = exact_sum(ss, __shfl_xor_sync(0xffffffffu, ss, off));
        ss = t.h;
        ss_l = __fadd_rn(ss_l, __shfl_xor_sync(0xffffffffu, ss_l, off)) + t.l;
    }
    if (!(ss < INFINITY)) ss_l = 0.0f;   // NaN, or beyond fp32
    constexpr float kInvD = 1.0f / static_cast<float>(D);
    const Twofold inv = reciprocal_sqrt(add(Twofold{ss * kInvD, ss_l * kInvD}, twofold(1e-6)));
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int i = kPer * lane + e;
        Twofold a = mul(inv, x[0][e]), b = mul(inv, x[1][e]);
        if (w) {
            a = mul(a, __bfloat162float(w[i]));
            b = mul(b, __bfloat162float(w[kHalf + i]));
            if (i < n_rot) {
                const Twofold c{cs[i].x, cs_l[i].x}, s{cs[i].y, cs_l[i].y};
                const Twofold a0 = a;
                a = add(mul(a, c), neg(mul(b, s)));
                b = add(mul(b, c), mul(a0, s));
            }
        }
        x[0][e] = to_odd(a);
        x[1][e] = to_odd(b);
    }
}

template <int D>
__global__ void __launch_bounds__(kPrepareThreads)
    gqa_prepare_quant_kernel(const PrepareQuantParams p) {
    constexpr int kHalf = D / 2;
    constexpr int kPer = kHalf / 32;   // elements per lane in each half: 4 or 8
    constexpr int kWords = kPer / 4;   // code words per lane in each half
    __shared__ float2 cs[kPrepareMaxRot], cs_l[kPrepareMaxRot];   // (cos, sin): both floats of each

    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    const QuantCache& c = p.cache;
    const int b = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int vec = blockIdx.y * (kPrepareThreads / 32) + warp;   // q heads, k heads, v heads
    const int L = p.seq_lens[b];
    const bool is_q = vec < p.H;
    const bool is_k = !is_q && vec < p.H + c.KVH;
    const int kvh = is_q ? 0 : (is_k ? vec - p.H : vec - p.H - c.KVH);
    // the raw vector first: its load does not wait for the length, page and scale
    float x[2][kPer];
    if (vec < p.H + 2 * c.KVH) {
        const __nv_bfloat16* src =
            is_q ? p.q_raw + (static_cast<size_t>(b) * p.H + vec) * D
                 : (is_k ? p.k_raw : p.v_raw) + (static_cast<size_t>(b) * c.KVH + kvh) * D;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < kPer; e += 4) {
                const uint2 t = *reinterpret_cast<const uint2*>(src + h * kHalf + kPer * lane + e);
                x[h][e] = __uint_as_float(t.x << 16);
                x[h][e + 1] = __uint_as_float(t.x & 0xffff0000u);
                x[h][e + 2] = __uint_as_float(t.y << 16);
                x[h][e + 3] = __uint_as_float(t.y & 0xffff0000u);
            }
    }
    const int pos = L - 1;
    if (pos < 0) return;   // no new token
    size_t row = 0, scale_row = 0;
    const bool active =
        vec < p.H + 2 * c.KVH &&
        (is_q || (pos < c.capacity() && c.locate(b, pos / kQuantBlock, &row, &scale_row)));
    const int slot = pos % kQuantBlock;
    const size_t stride = static_cast<size_t>(c.KVH) * D;
    uint8_t* codes = nullptr;   // this head's first row of the block
    float* scale = nullptr;
    float old = 0.0f;
    if (active && !is_q) {
        codes = (is_k ? c.k : c.v) + (row * c.KVH + kvh) * D;
        scale = (is_k ? c.k_scales : c.v_scales) + scale_row * c.KVH + kvh;
        if (slot > 0) old = *scale;
    }
    if (tid < p.n_rot && blockIdx.y * (kPrepareThreads / 32) < p.H + c.KVH) {   // (v is not rotated)
        Twofold co, si;
        cos_sin_of_turn(static_cast<uint64_t>(pos) * p.turn[tid], &co, &si);
        cs[tid] = make_float2(co.h, si.h);
        cs_l[tid] = make_float2(co.l, si.l);
    }
    __syncthreads();
    if (!active) return;

    if (is_q) {
        head_norm_rope<D>(x, p.w_q, cs, p.n_rot, lane);
        __nv_bfloat16* dst = p.q_out + (static_cast<size_t>(b) * p.H + vec) * D;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < kPer; e += 2)
                *reinterpret_cast<__nv_bfloat162*>(dst + h * kHalf + kPer * lane + e) =
                    __floats2bfloat162_rn(x[h][e], x[h][e + 1]);
        return;
    }

    head_norm_rope_to_odd<D>(x, is_k ? p.w_k : nullptr, cs, cs_l, p.n_rot, lane);
    float amax = 0.0f;   // largest finite magnitude
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            x[h][e] = inf_to_nan(x[h][e]);
            amax = fmaxf(amax, fabsf(x[h][e]));   // a NaN is passed over
        }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    int e = quant_exponent(amax);
    if (slot > 0) {
        const int eo = scale_exponent(old);
        if (e > eo) {
            const float f = pow2f(max(eo - e, -126));
            for (int j = 0; j < slot; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t* r = reinterpret_cast<uint32_t*>(codes + j * stride + h * kHalf + kPer * lane);
#pragma unroll
                    for (int w = 0; w < kWords; ++w) r[w] = recode4(r[w], f);
                }
        } else {
            e = eo;
        }
    }
    const float inv = pow2f(-e);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t* r = reinterpret_cast<uint32_t*>(codes + slot * stride + h * kHalf + kPer * lane);
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const float* y = &x[h][4 * w];
            r[w] = ptx::float2_to_e4m3x2(y[0] * inv, y[1] * inv) |
                   (static_cast<uint32_t>(ptx::float2_to_e4m3x2(y[2] * inv, y[3] * inv)) << 16);
        }
    }
    if (lane == 0) *scale = pow2f(e);
}

}  // namespace gqa
