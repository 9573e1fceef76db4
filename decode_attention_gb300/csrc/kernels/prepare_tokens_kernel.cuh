// The producer (prepare_kernel.cuh: norms, rotary positions) for any number of new tokens per
// sequence, packed as the appends take them, writing a bf16 cache or the 4-bit one
// (nibble_cache.cuh).
//
// A CTA takes a token at a time.  Its threads make the angles of the token's position, once for all its
// heads, and its warps take the token's heads (q, then k, then v) by turns, 512 channels at a
// time: one head vector at D = 512, two at D = 256, where each takes half of the lanes.  So a lane
// holds 8 channels of each half of a vector (a word of codes each, four lanes to a scale).  Each warp
// keeps copies of its next three units in flight, in a ring of its own in shared memory; the angles of
// the next two tokens are made while the warps work on two, with one barrier per two.  Few tokens are
// shared by several CTAs (blockIdx.y).
//
// Bound by the memory's rate into a bf16 cache, by instructions into the 4-bit one: some 18 for an
// element, where the memory's rate leaves time for 20 (D = 512).
//
// For the 4-bit cache a k or v vector is rounded to fp32 and to bf16, as a row that an append gets,
// and coded from there.  An fp32 error moves a value over a border between two bf16 numbers once
// in some 10^4, and one in forty of those goes over a border between codes, a whole step.  So k and v
// are looked at: a vector with a value within its error bound of such a border, one in ten, is taken
// again with norm, weight and rotation to some 2^-30 (twofold.cuh).
#pragma once

#include "nibble_cache.cuh"
#include "prepare_quant_kernel.cuh"   // head_norm_rope_twofold

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

constexpr int kTokensUnit = 512;   // channels that a warp takes together

constexpr int kTokensRing = 4;     // units of a warp in shared memory: one in work, the others on their way

template <bool kNibble>
struct TokensSmem {
    uint4 raw[kTokensThreads / 32][kTokensRing][kTokensUnit / 8];
    // (cos, sin) of two tokens, and of the next two: pair 8 l + e at [e][l] (a lane's eight on distinct banks
    // from its neighbours'); and in order, with their low parts, for what is taken again
    float2 cs[2][2][8][kPrepareMaxRot / 8];
    float2 cs_h[kNibble ? 2 : 1][kNibble ? 2 : 1][kPrepareMaxRot], cs_l[kNibble ? 2 : 1][kNibble ? 2 : 1][kPrepareMaxRot];
    int2 place[2][2];                                  // sequence (-1: none) and position
    TokenIndex idx;
};

enum class HeadKind { kQuery, kKey, kValue };

// Norm, weight and rotation of a head vector over D / 16 lanes in fp32, rounded to bf16; raw, y: this
// lane's elements [8 l, 8 l + 8) of each half, packed.  `turns`: they are rotated by co, si.  kDoubt:
// returns whether an error of fp32 may have changed a bf16 number of this lane.
template <int D, HeadKind kKind, bool kDoubt>
__device__ __forceinline__ bool head_to_bf16(const uint32_t (&raw)[2][4], const float (&w)[2][8],
                                             const float (&co)[8], const float (&si)[8], bool turns,
                                             uint32_t (&y)[2][4]) {
    constexpr int kPer = 8, kWords = 4;
    float x[2][kPer];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
            x[h][2 * e] = __uint_as_float(raw[h][e] << 16);
            x[h][2 * e + 1] = __uint_as_float(raw[h][e] & 0xffff0000u);
        }
    // 1 / sqrt(mean(x^2) + 1e-6); the squares are exact and are added up in pairs
    float sq[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) sq[e] = fmaf(x[0][e], x[0][e], __fmul_rn(x[1][e], x[1][e]));
#pragma unroll
    for (int n = kPer / 2; n > 0; n >>= 1)
#pragma unroll
        for (int e = 0; e < n; ++e) sq[e] += sq[e + n];
    float ss = sq[0];
#pragma unroll
    for (int off = D / 32; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float inv = ptx::rsqrt(fmaf(ss, 1.0f / static_cast<float>(D), 1e-6f));
    // The fp32 error of a value y, in units of 2^-24: of |y| what all of the vector share, the sum's 9
    // levels at most, halved by the root, its scaling 1/4 and the reciprocal root 2.2, then the product
    // with x, the weight or a rotation's sum 1/2 each, and 1 for the sums below: 8.95 (a rotation: 8.45).
    // Of |a| + |d|, which a rotated y is made of, the products with x, the weight, cosine or sine and
    // its product 1/2 each.
    constexpr float kError = 9.0f * 0x1p-24f, kTurnError = 2.0f * 0x1p-24f;
    const bool rotated = kKind != HeadKind::kValue && (D == 256 || turns);
    float err[kPer];   // of a rotated pair
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            x[h][e] *= inv;
            if (kKind != HeadKind::kValue) x[h][e] *= w[h][e];
        }
    if (rotated) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const float a = x[0][e], d = x[1][e];
            x[0][e] = fmaf(a, co[e], -__fmul_rn(d, si[e]));
            x[1][e] = fmaf(d, co[e], __fmul_rn(a, si[e]));
            if (kDoubt) err[e] = (fabsf(a) + fabsf(d)) * kTurnError;
        }
    }
    uint32_t differ = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
            const float v0 = x[h][2 * e], v1 = x[h][2 * e + 1];
            if (kDoubt) {   // (where both ends round alike, so does v)
                const float e0 = fmaf(fabsf(v0), kError, rotated ? err[2 * e] : 0.0f);
                const float e1 = fmaf(fabsf(v1), kError, rotated ? err[2 * e + 1] : 0.0f);
                y[h][e] = bf16x2_bits(v0 + e0, v1 + e1);
                differ |= y[h][e] ^ bf16x2_bits(v0 - e0, v1 - e1);
            } else {
                y[h][e] = bf16x2_bits(v0, v1);
            }
        }
    return differ != 0;
}

template <int D, bool kNibble>
__global__ void __launch_bounds__(kTokensThreads, kNibble ? 2 : 3)
    gqa_prepare_tokens_kernel(const PrepareTokensParams p) {
    constexpr int kHalf = D / 2, kLanes = D / 16, kHeads = kTokensUnit / D;   // lanes of a vector, vectors of a unit
    constexpr int kWarps = kTokensThreads / 32;
    __shared__ TokensSmem<kNibble> sm;

    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    const NibbleCache& c = p.cache;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int l = lane % kLanes, head = lane / kLanes;   // place in a vector, and which of a unit's it is
    const int q_units = p.H / kHeads, kv_units = p.KVH / kHeads, n_units = q_units + 2 * kv_units;
    const int first = blockIdx.y * kWarps + warp, step = gridDim.y * kWarps;
    const bool keqv = p.v_raw == nullptr;
    const size_t stride = kNibble ? c.plane_stride() : 0;
    // this lane's place in the ring, by slot, and the next unit to copy
    const uint32_t ring = ptx::smem_addr(sm.raw[warp][0]) + lane * 16;
    int next_i = blockIdx.x, next_u = first;
    uint32_t fetched = 0, taken = 0;
    auto fetch = [&] {   // (a group of copies for each unit, empty ones behind the last)
        if (next_i < p.N) {
            const bool is_q = next_u < q_units, is_k = !is_q && next_u < q_units + kv_units;
            const __nv_bfloat16* src =
                (is_q ? p.q_raw + (static_cast<size_t>(next_i) * q_units + next_u) * kTokensUnit
                      : (is_k || keqv ? p.k_raw : p.v_raw) +
                            (static_cast<size_t>(next_i) * kv_units + next_u - q_units - (is_k ? 0 : kv_units)) *
                                kTokensUnit) + lane * 8;
            const uint32_t dst = ring + (fetched % kTokensRing) * (kTokensUnit * 2);
            ptx::cp_async16(dst, src);
            ptx::cp_async16(dst + 512, src + 256);
            next_u += step;
            if (next_u >= n_units) {
                next_u = first;
                next_i += gridDim.x;
            }
        }
        ++fetched;
        ptx::cp_async_commit();
    };
    // places and angles of token i and the CTA's next to stage s
    auto angles = [&](int i, int s) {
        const int sub = tid / p.n_rot, pair = tid % p.n_rot;
        i += sub * gridDim.x;
        if (sub > 1 || i >= p.N) return;
        int b, pos;
        const bool found = sm.idx.find(p.B, p.N, i, &b, &pos);
        if (pair == 0) sm.place[s][sub] = make_int2(found ? b : -1, pos);
        if (!found) return;
        Twofold co, si;
        cos_sin_of_turn(static_cast<uint64_t>(pos) * p.turn[pair], &co, &si);
        sm.cs[s][sub][pair % 8][pair / 8] = make_float2(co.h, si.h);
        if constexpr (kNibble) {
            sm.cs_h[s][sub][pair] = make_float2(co.h, si.h);
            sm.cs_l[s][sub][pair] = make_float2(co.l, si.l);
        }
    };

    for (int n = 0; n + 1 < kTokensRing; ++n) fetch();
    // weights of this lane's elements [8 l, 8 l + 8) of each half
    float wq[2][8], wk[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const uint32_t a = __ldg(reinterpret_cast<const uint32_t*>(p.w_q + h * kHalf + 8 * l + e));
            const uint32_t b = __ldg(reinterpret_cast<const uint32_t*>(p.w_k + h * kHalf + 8 * l + e));
            wq[h][e] = __uint_as_float(a << 16);
            wq[h][e + 1] = __uint_as_float(a & 0xffff0000u);
            wk[h][e] = __uint_as_float(b << 16);
            wk[h][e + 1] = __uint_as_float(b & 0xffff0000u);
        }
    sm.idx.load(p.token_offsets, p.seq_lens, p.B);
    angles(blockIdx.x, 0);
    __syncthreads();

    const bool turns = 8 * l < p.n_rot;   // (n_rot is a multiple of 8)
    int s = 0;   // stage of the angles
    for (int i = blockIdx.x, sub = 0; i < p.N; i += gridDim.x) {
        if (sub == 0) angles(i + 2 * gridDim.x, s ^ 1);
        const int b = sm.place[s][sub].x, pos = sm.place[s][sub].y;
        // the token's place: null (no slot) when it is not written
        uint8_t* row = nullptr;
        bool have_slot = false;
        size_t slot = 0;   // bf16 cache: its row
        if (b >= 0 && kNibble) {
            if (pos < c.capacity()) row = c.row(b, pos);
        } else if (b >= 0 && c.block_table) {
            const int page = pos < c.capacity()
                                 ? c.block_table[static_cast<size_t>(b) * c.max_pages + pos / kNibblePage] : -1;
            have_slot = page >= 0 && page < c.num_pages;
            slot = static_cast<size_t>(page) * kNibblePage + pos % kNibblePage;
        } else if (b >= 0) {
            // (a ring keeps the last `rows` positions)
            have_slot = p.ring ? pos >= sm.idx.len[b] - c.rows : pos < c.rows;
            slot = static_cast<size_t>(b) * c.rows + (p.ring ? pos % c.rows : pos);
        }
        float co[8], si[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 x = sm.cs[s][sub][e][turns ? l : 0];
            co[e] = x.x;
            si[e] = x.y;
        }
        for (int u = first; u < n_units; u += step) {
            fetch();
            ptx::cp_async_wait<kTokensRing - 1>();
            __syncwarp();   // (a warp's copies are its lanes')
            const uint4* from = sm.raw[warp][taken++ % kTokensRing] + head * (D / 8) + l;
            const uint4 r0 = from[0], r1 = from[D / 16];
            __syncwarp();   // (the slot is filled again)
            const bool is_q = u < q_units, is_k = !is_q && u < q_units + kv_units;
            if (b < 0 || (!is_q && (kNibble ? row == nullptr : !have_slot || (is_k && keqv)))) continue;
            // this lane's head of q, k or v
            const int mine = (is_q ? u : is_k ? u - q_units : u - q_units - kv_units) * kHeads + head;
            const uint32_t raw[2][4] = {{r0.x, r0.y, r0.z, r0.w}, {r1.x, r1.y, r1.z, r1.w}};
            uint32_t y[2][4];
            bool doubt = false;
            if (is_q)
                head_to_bf16<D, HeadKind::kQuery, false>(raw, wq, co, si, turns, y);
            else if (is_k)
                doubt = head_to_bf16<D, HeadKind::kKey, kNibble>(raw, wk, co, si, turns, y);
            else
                doubt = head_to_bf16<D, HeadKind::kValue, kNibble>(raw, wk, co, si, turns, y);
            if (!kNibble || is_q) {
                __nv_bfloat16* dst = is_q ? p.q_out + (static_cast<size_t>(i) * p.H + mine) * D
                                          : (is_k ? p.k_cache : p.v_cache) + (slot * p.KVH + mine) * D;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<uint4*>(dst + h * kHalf + 8 * l) =
                        make_uint4(y[h][0], y[h][1], y[h][2], y[h][3]);
                continue;
            }
            if constexpr (kNibble) {
                if (__any_sync(0xffffffffu, doubt)) {
                    float x[2][8];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[h][2 * e] = __uint_as_float(raw[h][e] << 16);
                            x[h][2 * e + 1] = __uint_as_float(raw[h][e] & 0xffff0000u);
                        }
                    head_norm_rope_twofold<D, kLanes>(x, is_k ? p.w_k : nullptr, sm.cs_h[s][sub], sm.cs_l[s][sub],
                                                      p.n_rot, l, [](Twofold a) { return fast_sum(a.h, a.l).h; });
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[h][e] = bf16x2_bits(x[h][2 * e], x[h][2 * e + 1]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t scale;
                    const uint32_t codes = nibble_codes(y[h], &scale);
                    // D = 256: both halves in the head's plane; D = 512: one each
                    uint8_t* r = row + (D == 256 ? mine : 2 * mine + h) * stride;
                    const int at = D == 256 ? h * 16 + l : l;   // the word's place in the plane
                    *reinterpret_cast<uint32_t*>(r + (is_k ? 0 : kNibblePlane / 2) + 4 * at) = codes;
                    if (l % 4 == 0)
                        r[kNibbleScales + (is_k ? 0 : 8) + at / 4] = static_cast<uint8_t>(scale);
                }
            }
        }
        if (++sub == 2) {   // the next two tokens' angles are there, and these may go
            __syncthreads();
            sub = 0;
            s ^= 1;
        }
    }
    ptx::cp_async_wait<0>();
}

}  // namespace gqa
