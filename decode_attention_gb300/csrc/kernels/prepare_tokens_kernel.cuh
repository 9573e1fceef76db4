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
// Bound by the memory's rate into a bf16 cache, 10200 tokens at D = 512 in 128 us, 0.96 of a copy's rate (at
// D = 256 0.96), and at D = 512 into the 4-bit one, 33000 tokens in 402 us, 0.92; by instructions into the
// 4-bit one at D = 256, where half of the channels are coded, 17000 tokens in 234 us, 0.57.  Two CTAs an SM:
// three, at 80 registers, spilled (148 us for 127) or, with the weights in shared memory or packed, took 15
// to 25% more instructions (525 to 555 us for 475 then).  Pairs of channels go through packed fp32
// operations (516 to 475, 303 to 278; into bf16 140 to 127 with the registers), the ends are coded once where
// they agree and leave codes' seldom cases to one branch (to 451 and 251), and what a warp branches on is
// seen to be the warp's (to 400 and 229; the error's bound, wider since, costs 2 and 5).
//
// For the 4-bit cache a k or v vector is rounded to fp32 and to bf16, as a row that an append gets,
// and coded from there.  An fp32 error moves a value over a border between two bf16 numbers once
// in some 10^4, and one in forty of those goes over a border between codes, a whole step.  So k and v
// are looked at: where a value is within its error bound of a border between bf16 numbers (two in five of
// 512 rotated channels, one in eight of others), both ends are coded, and where the codes differ (one in a
// hundred) the vectors are taken again with norm, weight and rotation to some 2^-30 (twofold.cuh).
#pragma once

#include "nibble_cache.cuh"
#include "prepare_quant_kernel.cuh"   // head_norm_rope_twofold

namespace gqa {

constexpr int kTokensThreads = 256;
constexpr int kTokensPerSm = 2;   // CTAs

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
    // cosines and sines of two tokens, and of the next two: those of the pairs 8 l + 2 e and 8 l + 2 e + 1 at [e][l]
    // (lanes on distinct banks); and (cos, sin) in order, with their low parts, for what is taken again
    float4 cs[2][2][4][kPrepareMaxRot / 8];
    float2 cs_h[kNibble ? 2 : 1][kNibble ? 2 : 1][kPrepareMaxRot], cs_l[kNibble ? 2 : 1][kNibble ? 2 : 1][kPrepareMaxRot];
    int2 place[2][2];                                  // sequence (-1: none) and position
    TokenIndex idx;
};

enum class HeadKind { kQuery, kKey, kValue };

// Norm, weight and rotation of a head vector over D / 16 lanes in fp32, rounded to bf16; raw, y: this
// lane's elements [8 l, 8 l + 8) of each half, packed.  `turns`: they are rotated by co, si.  kDoubt: y and
// below are what the ends of fp32's error round to; returns whether they differ in this lane.
template <int D, HeadKind kKind, bool kDoubt>
__device__ __forceinline__ bool head_to_bf16(const uint32_t (&raw)[2][4], const uint64_t (&w)[2][4],
                                             const uint64_t (&co)[4], const uint64_t (&si)[4], bool turns,
                                             uint32_t (&y)[2][4], uint32_t (&below)[2][4]) {
    constexpr int kWords = 4;   // pairs of neighbouring channels
    uint64_t x[2][kWords];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kWords; ++e) x[h][e] = ptx::f2_from_bf16x2(raw[h][e]);
    // 1 / sqrt(mean(x^2) + 1e-6); the squares are exact and are added up in pairs
    uint64_t sq[kWords];
#pragma unroll
    for (int e = 0; e < kWords; ++e) sq[e] = ptx::f2_fma(x[0][e], x[0][e], ptx::f2_mul(x[1][e], x[1][e]));
    const float2 s2 = ptx::f2_unpack(ptx::f2_add(ptx::f2_add(sq[0], sq[2]), ptx::f2_add(sq[1], sq[3])));
    float ss = s2.x + s2.y;
#pragma unroll
    for (int off = D / 32; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float inv = ptx::rsqrt(fmaf(ss, 1.0f / static_cast<float>(D), 1e-6f));
    // The fp32 error of a value y, in units of 2^-24, of which a rounding takes one at most.  Of |y|: what all
    // of the vector share, the sum's 9 levels and its scaling, halved by the root, and the reciprocal root 2.2;
    // then the product with x and the weight, or a rotation's sum; and 1 for the sums below: 10.2 (a value:
    // 9.2, a rotation: 9.2).  Of |a| + |d|, which a rotated y is made of, the products with x and the weight,
    // cosine or sine (the nearest float of what is good to 2^-30) and its product: 4.
    constexpr float kError = 10.5f * 0x1p-24f, kValueError = 10.0f * 0x1p-24f, kTurnError = 4.01f * 0x1p-24f;
    const bool rotated = kKind != HeadKind::kValue && (D == 256 || turns);
    const uint64_t inv2 = ptx::f2_pack(inv, inv);
    float2 err[kWords];   // of rotated pairs
#pragma unroll
    for (int e = 0; e < kWords; ++e) err[e] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
            x[h][e] = ptx::f2_mul(x[h][e], inv2);
            if (kKind != HeadKind::kValue) x[h][e] = ptx::f2_mul(x[h][e], w[h][e]);
        }
    if (rotated) {
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
            const uint64_t a = x[0][e], d = x[1][e];
            x[0][e] = ptx::f2_sub(ptx::f2_mul(a, co[e]), ptx::f2_mul(d, si[e]));
            x[1][e] = ptx::f2_fma(d, co[e], ptx::f2_mul(a, si[e]));
            if (kDoubt) {
                const float2 a2 = ptx::f2_unpack(a), d2 = ptx::f2_unpack(d);
                err[e] = ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(fabsf(a2.x) + fabsf(d2.x), fabsf(a2.y) + fabsf(d2.y)),
                                                    ptx::f2_pack(kTurnError, kTurnError)));
            }
        }
    }
    uint32_t differ = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
            const float2 v = ptx::f2_unpack(x[h][e]);
            if (kDoubt) {   // (where both ends round alike, so does v)
                float2 up, down;
                if (kKind == HeadKind::kValue) {   // (by magnitude; both factors are fp32 numbers)
                    up = ptx::f2_unpack(ptx::f2_mul(x[h][e], ptx::f2_pack(1.0f + kValueError, 1.0f + kValueError)));
                    down = ptx::f2_unpack(ptx::f2_mul(x[h][e], ptx::f2_pack(1.0f - kValueError, 1.0f - kValueError)));
                } else {
                    const uint64_t r = ptx::f2_pack(fmaf(fabsf(v.x), kError, err[e].x), fmaf(fabsf(v.y), kError, err[e].y));
                    up = ptx::f2_unpack(ptx::f2_add(x[h][e], r));
                    down = ptx::f2_unpack(ptx::f2_sub(x[h][e], r));
                }
                y[h][e] = bf16x2_bits(up.x, up.y);
                below[h][e] = bf16x2_bits(down.x, down.y);
                differ |= y[h][e] ^ below[h][e];
            } else {
                y[h][e] = bf16x2_bits(v.x, v.y);
            }
        }
    return differ != 0;
}

template <int D, bool kNibble>
__global__ void __launch_bounds__(kTokensThreads, kTokensPerSm)
    gqa_prepare_tokens_kernel(const PrepareTokensParams p) {
    constexpr int kHalf = D / 2, kLanes = D / 16, kHeads = kTokensUnit / D;   // lanes of a vector, vectors of a unit
    constexpr int kWarps = kTokensThreads / 32;
    __shared__ TokensSmem<kNibble> sm;

    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    const NibbleCache& c = p.cache;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (so that branches on it are seen to be a warp's)
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
        cos_sin_nearest(static_cast<uint64_t>(pos) * p.turn[pair], &co, &si);
        float* at = &sm.cs[s][sub][pair % 8 / 2][pair / 8].x + pair % 2;
        at[0] = co.h;
        at[2] = si.h;
        if constexpr (kNibble) {
            sm.cs_h[s][sub][pair] = make_float2(co.h, si.h);
            sm.cs_l[s][sub][pair] = make_float2(co.l, si.l);
        }
    };

    for (int n = 0; n + 1 < kTokensRing; ++n) fetch();
    // weights of this lane's elements [8 l, 8 l + 8) of each half
    uint64_t wq[2][4], wk[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            wq[h][e] = ptx::f2_from_bf16x2(__ldg(reinterpret_cast<const uint32_t*>(p.w_q + h * kHalf + 8 * l) + e));
            wk[h][e] = ptx::f2_from_bf16x2(__ldg(reinterpret_cast<const uint32_t*>(p.w_k + h * kHalf + 8 * l) + e));
        }
    sm.idx.load(p.token_offsets, p.seq_lens, p.B);
    angles(blockIdx.x, 0);
    __syncthreads();

    const bool turns = 8 * l < p.n_rot;   // (n_rot is a multiple of 8)
    int s = 0;   // stage of the angles
    for (int i = blockIdx.x, sub = 0; i < p.N; i += gridDim.x) {
        if (sub == 0) angles(i + 2 * gridDim.x, s ^ 1);
        const int2 at = sm.place[s][sub];
        const int b = at.x, pos = at.y;
        const bool found = __any_sync(0xffffffffu, b >= 0);   // (one answer for the warp)
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
        const bool kept = __any_sync(0xffffffffu, kNibble ? row != nullptr : have_slot);
        uint64_t co[4], si[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 x = sm.cs[s][sub][e][turns ? l : 0];
            co[e] = ptx::f2_pack(x.x, x.y);
            si[e] = ptx::f2_pack(x.z, x.w);
        }
        for (int u = first; u < n_units; u += step) {
            fetch();
            ptx::cp_async_wait<kTokensRing - 1>();
            __syncwarp();   // (a warp's copies are its lanes')
            const uint4* from = sm.raw[warp][taken++ % kTokensRing] + head * (D / 8) + l;
            const uint4 r0 = from[0], r1 = from[D / 16];
            __syncwarp();   // (the slot is filled again)
            const bool is_q = u < q_units, is_k = !is_q && u < q_units + kv_units;
            if (!found || (!is_q && (!kept || (!kNibble && is_k && keqv)))) continue;
            // this lane's head of q, k or v
            const int mine = (is_q ? u : is_k ? u - q_units : u - q_units - kv_units) * kHeads + head;
            const uint32_t raw[2][4] = {{r0.x, r0.y, r0.z, r0.w}, {r1.x, r1.y, r1.z, r1.w}};
            uint32_t y[2][4], below[2][4];
            bool doubt = false;
            if (is_q)
                head_to_bf16<D, HeadKind::kQuery, false>(raw, wq, co, si, turns, y, below);
            else if (is_k)
                doubt = head_to_bf16<D, HeadKind::kKey, kNibble>(raw, wk, co, si, turns, y, below);
            else
                doubt = head_to_bf16<D, HeadKind::kValue, kNibble>(raw, wk, co, si, turns, y, below);
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
                // The ends by magnitude, y the larger (a value's are so already).  Codes and scale grow with it, so
                // where both ends' agree, all between do (ends of two signs are not compared).
                const bool twice = __any_sync(0xffffffffu, doubt);
                bool open = false;
                if (twice && is_k) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t up = y[h][e], down = below[h][e];
                            const uint32_t minus = ((up >> 15) & 0x00010001u) * 0xffffu;
                            open |= ((up ^ down) & 0x80008000u) != 0;
                            y[h][e] = (down & minus) | (up & ~minus);
                            below[h][e] = (up & minus) | (down & ~minus);
                        }
                }
                uint32_t codes[2], scale[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) codes[h] = nibble_codes(y[h], &scale[h]);
                if (twice) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t other;
                        open |= nibble_codes(below[h], &other) != codes[h] || other != scale[h];
                    }
                }
                if (twice && __any_sync(0xffffffffu, open)) {
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
#pragma unroll
                    for (int h = 0; h < 2; ++h) codes[h] = nibble_codes(y[h], &scale[h]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // D = 256: both halves in the head's plane; D = 512: one each
                    uint8_t* r = row + (D == 256 ? mine : 2 * mine + h) * stride;
                    const int at = D == 256 ? h * 16 + l : l;   // the word's place in the plane
                    *reinterpret_cast<uint32_t*>(r + (is_k ? 0 : kNibblePlane / 2) + 4 * at) = codes[h];
                    if (l % 4 == 0)
                        r[kNibbleScales + (is_k ? 0 : 8) + at / 4] = static_cast<uint8_t>(scale[h]);
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
