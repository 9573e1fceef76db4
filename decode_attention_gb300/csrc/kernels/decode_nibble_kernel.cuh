// Decode attention over the 4-bit cache (nibble_cache.cuh): attn.core of the gemma-4-31B Model
// Spec for one new token per sequence.
//
// Mathematics.  With x_s = log2(e) <q, k_s> the weights are 2^(x_s - M + 12), M a whole number at
// most 3 below the running maximum and never above what it was; o = sum of weights times v_s over the
// sum of weights.  The accumulators are rescaled by powers of two, and seldom; weights lie in (0, 2^15],
// where f16 hi + lo parts hold them to 22 bits.  The 12 stands apart from M, so that scores of 2^24
// and more, where floats have a spacing above 1, need no sum of the two.
//
// Both contractions run as warp-level f16 mma (m16n8k16, fp32 accumulate) with the cache as the A
// operand, so that the g <= 8 query heads of a KV head fill the 8 columns of B.  A value
// (u - 8) s is exact in f16 and takes one fma of two codes: the codes j and j + 4 of a word (or code j
// of two positions) lie in the low four bits of its halves, and 0x6400 | u is the f16 number
// 1024 + u, so the value is (1024 + u) s - 1032 s; codes one place up are 1024 + 16 u, times
// s / 16, less 72 s; a shift by 8 brings the rest.  (With bf16 in place of f16, whose 7 bits of
// mantissa leave no room for a second place, it takes three shifts for a word and not one.)  The
// constants are exact as well: 1032 s has 11 bits and is at most 61920.  q is scaled by a power of
// two per head (at g = 8 per half of D), which makes its bf16 numbers exact in f16 down to 2^-31 of the
// largest, and within 2^-39 of it below.
//   scores  S[pos, h] = K[pos, :] . q[h, :] for the 16 positions of a block.  Lane (g, t) reads the
//           chunks (16 bytes, 32 channels, one scale) t and t + 4 of the rows of its A fragments; what
//           order the channels take in k does not matter, q's B fragments take the same
//   P.V     O^T[c, h] += V^T[c, pos] P[pos, h]: lane (g, t) reads the chunk of its g from the rows of
//           its four positions, a byte permute pairs positions, and code 2m (2m + 1) of every chunk is
//           the row g (g + 8) of the m-th tile.  movmatrix turns the weights from the scores'
//           layout into B fragments.  At g = 2 the hi and lo parts of P are columns of one mma; at
//           g = 8 they are two mma.
// A row of the scores' fragment g (g + 8) stands for position perm(g) (8 + perm(g)), perm(g) =
// g / 2 + 4 (g % 2): with rows of 17 16-byte units this is what keeps the 8 lanes of a shared-memory
// phase on distinct banks in both contractions.
// An mma truncates its sum, so long chains of them drift: a block's products start from zero and
// are added to the accumulators by ordinary additions.
//
// Work split and timeouts are those of decode_quant_kernel.cuh: a persistent CTA per SM, a plan built
// from seq_lens on the device, pieces of whole blocks, several units per CTA with a schedule each, NC
// warps of a unit (at g = 8 pairs, a plane each) on a block each with a ring of slots of their
// own, states merged through shared memory at a piece's end, split segments by the combine kernel.  A
// slot is one block of K, V and scales: one bulk copy per plane of exactly the attended rows.
#pragma once

#include "decode_kernel.cuh"
#include "nibble_cache.cuh"
#include "piece_walk.cuh"

namespace gqa {

struct DecodeNibbleParams {
    DecodeParams d;
    const uint8_t* kv;       // [B, planes, rows, 272] or [P, planes, 16, 272]
    int rows;                // contiguous: positions per sequence
};

struct NibblePlanTuning {
    static constexpr int kAlign = kNibblePage, kExtra = 12;
    static constexpr int kMinShare = 1024, kChunksPerCta = 4;
};

template <int kG, int kGroups, int kBlocksAtOnce, int kRing>
struct NibblePolicy {
    static constexpr int G = kG;
    static constexpr int SPLIT = kG == 2 ? 1 : 2;        // warps per block, a plane each
    static constexpr int D = kNibblePlane * SPLIT;
    static constexpr int GROUPS = kGroups;               // units of the plan per CTA
    static constexpr int NC = kBlocksAtOnce;             // blocks a unit works on at a time
    static constexpr int RING = kRing;                   // slots per block in work
    static constexpr int GW = NC * SPLIT;                // consumer warps per unit
    static constexpr int kConsumers = GROUPS * GW;
    static constexpr int kFeeds = NC / 2;                // producers per unit, two rings each
    static constexpr int kWarps = kConsumers + kFeeds * GROUPS;
    static constexpr int kThreads = kWarps * 32;
    static constexpr bool kSplitCols = G == 2;           // hi and lo parts of P in one mma
    static constexpr int kMergeCols = kSplitCols ? 2 * G : G;
    static constexpr int kMergeDims = 128 / SPLIT;       // channels of a warp merged per round
    static constexpr int kMergeTiles = kMergeDims / 16;  // tiles of a round: 2 channels of each chunk
    static constexpr int kMergePitch = 2 * kMergeTiles + 2;   // floats per chunk
    static_assert((G == 2 || G == 8) && (NC == 2 || NC == 4), "shape");
    static_assert(kThreads >= kPlanWarps * 32, "the plan takes eight warps");
};

template <class Pol>
struct alignas(128) NibbleSmem {
    static constexpr int kTileBytes = kNibblePage * kNibbleRow;
    struct Unit {
        alignas(8) uint64_t full[Pol::NC * Pol::RING];
        alignas(8) uint64_t empty[Pol::NC * Pol::RING];
        alignas(8) uint64_t piece_full, piece_empty;
        int bad[Pol::NC * Pol::RING];            // the block's page id is out of range
        BlockPiece piece;
        float wm[Pol::NC][8], wl[Pol::NC][8];    // M and l per column of each warp (pair)
        alignas(16) float wacc[Pol::SPLIT][Pol::NC][Pol::kMergeCols][8 * Pol::kMergePitch];   // being merged
    };
    uint8_t kv[Pol::GROUPS][Pol::NC * Pol::RING][Pol::SPLIT][kTileBytes];   // [slot][plane][16 rows][272 B]
    Unit unit[Pol::GROUPS];
    alignas(8) uint64_t stall_bar;               // kTestStall: a barrier nothing completes
    PlanSmem plan;
    int len[kMaxBatch];                          // clamped lengths
    int abort_flag;
};

// Two codes (in the low four bits, or one place up, of the halves of w) as f16 values.
struct NibbleScale {
    uint32_t s, less, s16, less16;   // s, -1032 s, s / 16, -72 s

    // bits: the scale bytes of the two halves, each shifted to bits 7 .. 14 of its own
    __device__ __forceinline__ explicit NibbleScale(uint32_t bits)
        : s(bits), less(ptx::f16x2_mul(bits, 0xe408e408u)), s16(ptx::f16x2_mul(bits, 0x2c002c00u)),
          less16(ptx::f16x2_mul(bits, 0xd480d480u)) {}
    __device__ __forceinline__ uint32_t low(uint32_t w) const {
        return ptx::f16x2_fma((w & 0x000f000fu) | 0x64006400u, s, less);
    }
    __device__ __forceinline__ uint32_t high(uint32_t w) const {
        return ptx::f16x2_fma((w & 0x00f000f0u) | 0x64006400u, s16, less16);
    }
};

template <class Pol>
struct NibbleConsumer {
    static constexpr int G = Pol::G, D = Pol::D;
    static constexpr int kTiles = kNibblePlane / 16;
    static constexpr float kBase = 12.0f;   // exponent of the weight of a score equal to M
    static constexpr float kTop = 15.0f;    // largest exponent of a weight (f16 ends at 2^16)
    static constexpr float kLowest = -3.402823466e38f;   // M of no score yet

    uint32_t qb[kTiles][2];      // B fragments of q (column g = head g % G) for this warp's plane
    float q_undo[2];             // undo their scaling for columns 2t and 2t + 1, times log2(e)
    float acc[kTiles][4];        // tile m: channels 2m (0, 1) and 2m + 1 (2, 3) of chunk(g); columns 2t, 2t + 1
    float ms[2];                 // M of columns 2t, 2t + 1
    float l[2];                  // this lane's share of their normalisers

    __device__ static __forceinline__ int perm(int g) { return (g >> 1) + 4 * (g & 1); }

    // q_heads: [G][D] bf16 in global memory; `half`: which plane of the head is this warp's.
    __device__ __forceinline__ void begin(const __nv_bfloat16* q_heads, int half, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const __nv_bfloat16* row = q_heads + (g % G) * D + half * kNibblePlane + 32 * t;
        uint32_t top = 0;   // largest |q|: the bits of |bf16| order like the values
        uint4 raw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // channels 8 (i % 4) .. + 7 of chunk t + 4 (i / 4)
            raw[i] = __ldg(reinterpret_cast<const uint4*>(row + (i >> 2) * 128 + (i & 3) * 8));
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu),
                                         __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu)));
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(static_cast<int>(top >> 7) - 127, -88);   // |q| < 2^(e + 1)
        const float f = __int_as_float((14 - e + 127) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // pairs of channels (0, 4), (1, 5), (2, 6), (3, 7)
            qb[2 * i][0] = ptx::f16x2_pack(bf16lo(raw[i].x) * f, bf16lo(raw[i].z) * f);
            qb[2 * i][1] = ptx::f16x2_pack(bf16hi(raw[i].x) * f, bf16hi(raw[i].z) * f);
            qb[2 * i + 1][0] = ptx::f16x2_pack(bf16lo(raw[i].y) * f, bf16lo(raw[i].w) * f);
            qb[2 * i + 1][1] = ptx::f16x2_pack(bf16hi(raw[i].y) * f, bf16hi(raw[i].w) * f);
        }
        const float undo = __int_as_float((e - 14 + 127) << 23) * kLog2e;
        q_undo[0] = __shfl_sync(0xffffffffu, undo, 8 * t);
        q_undo[1] = __shfl_sync(0xffffffffu, undo, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
        ms[0] = ms[1] = kLowest;
        l[0] = l[1] = 0.0f;
    }

    // This plane's share of a block's scores in units of log2: rows g (0, 1) and g + 8 (2, 3),
    // columns 2t, 2t + 1.
    __device__ __forceinline__ void scores(uint32_t tile, float (&z)[4], int lane) {
        const int g = lane >> 2, t = lane & 3;
        const uint32_t row = tile + perm(g) * kNibbleRow;
        constexpr uint32_t k8 = 8 * kNibbleRow;
        float c[4][4];   // four independent chains
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i][j] = 0.0f;
        const uint2 sa = ptx::lds64(row + kNibbleScales), sb = ptx::lds64(row + k8 + kNibbleScales);
        const uint32_t sel = 0x0404u | (t << 4) | (t << 12);   // byte t to the upper bytes of both halves
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 a = ptx::lds128(row + 16 * t + 64 * i), b = ptx::lds128(row + k8 + 16 * t + 64 * i);
            const NibbleScale fa(__byte_perm(i ? sa.y : sa.x, 0u, sel) >> 1);
            const NibbleScale fb(__byte_perm(i ? sb.y : sb.x, 0u, sel) >> 1);
            const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int u = 8 * i + 2 * w;
                ptx::mma_f16_16816(c[w], fa.low(wa[w]), fb.low(wb[w]), fa.high(wa[w]), fb.high(wb[w]),
                                   qb[u][0], qb[u][1]);
                const uint32_t ha = wa[w] >> 8, hb = wb[w] >> 8;
                ptx::mma_f16_16816(c[w], fa.low(ha), fb.low(hb), fa.high(ha), fb.high(hb),
                                   qb[u + 1][0], qb[u + 1][1]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            z[i] = ((c[0][i] + c[1][i]) + (c[2][i] + c[3][i])) * q_undo[i & 1];
    }

    // The rest of a block, from its scores: weights, M, l, and P.V for this warp's plane.  Rows
    // [first, last) are attended; bad: their page does not exist, and their weights are NaN.
    __device__ __forceinline__ void weigh(const float (&z)[4], uint32_t tile, int first, int last, bool bad,
                                          int lane) {
        const int g = lane >> 2, t = lane & 3, pos = perm(g);
        const bool row_ok[2] = {pos >= first && pos < last, pos + 8 >= first && pos + 8 < last};
        float x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // rows outside the range weigh 2^-inf
            x[i] = row_ok[i >> 1] ? (bad ? __uint_as_float(0x7fc00000u) : z[i]) : -INFINITY;
            y[i] = x[i] - ms[i & 1] + kBase;
        }
        // M moves only when a weight would pass 2^kTop (and on the first block)
        const float ym = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
        if (__any_sync(0xffffffffu, ym > kTop)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float top = fmaxf(x[j], x[j + 2]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = ceilf(fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)));
                const float m = fmaxf(ms[j], top);   // (never of a NaN)
                const float alpha = ptx::ex2(ms[j] - m);
                ms[j] = m;
                l[j] *= alpha;
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    acc[i][j] *= alpha;
                    acc[i][j + 2] *= alpha;
                }
                y[j] = x[j] - m + kBase;
                y[j + 2] = x[j + 2] - m + kBase;
            }
        }
        uint32_t hi[2], lo[2];   // B fragments: column g, positions perm(2t), perm(2t + 1) of each half
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float p0 = ptx::ex2(y[2 * i]), p1 = ptx::ex2(y[2 * i + 1]);
            l[0] += p0;
            l[1] += p1;
            hi[i] = ptx::f16x2_pack(p0, p1);
            const float2 h = ptx::f16x2_unpack(hi[i]);
            lo[i] = ptx::f16x2_pack(p0 - h.x, p1 - h.y);
            if (Pol::kSplitCols) {   // columns 2t, 2t + 1: the hi parts at even t, the lo parts at odd
                hi[i] = ptx::movmatrix_trans((t & 1) ? lo[i] : hi[i]);
            } else {
                hi[i] = ptx::movmatrix_trans(hi[i]);
                lo[i] = ptx::movmatrix_trans(lo[i]);
            }
        }
        // the chunk of this g in positions t, t + 4, t + 8, t + 12; rows outside the range hold
        // anything, and 0 * NaN is NaN: their scale is taken as 0
        const int chunk = perm(g);
        const uint32_t row = tile + t * kNibbleRow;
        uint32_t sc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sc[j] = ptx::lds8(row + 4 * j * kNibbleRow + kNibbleScales + 8 + chunk);
            if (t + 4 * j < first || t + 4 * j >= last) sc[j] = 0;
        }
        const NibbleScale f0(__byte_perm(sc[0], sc[1], 0x5410) << 7), f1(__byte_perm(sc[2], sc[3], 0x5410) << 7);
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = ptx::lds128(row + 4 * j * kNibbleRow + kNibblePlane / 2 + 16 * chunk);
        const uint32_t w[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w},
                                  {v[2].x, v[2].y, v[2].z, v[2].w}, {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {   // codes 2k, 2k + 1 of word i
                uint32_t a = __byte_perm(w[0][i], w[1][i], k < 2 ? 0x5410 : 0x7632);
                uint32_t b = __byte_perm(w[2][i], w[3][i], k < 2 ? 0x5410 : 0x7632);
                if (k & 1) {
                    a >>= 8;
                    b >>= 8;
                }
                float d[4];
                const uint32_t a0 = f0.low(a), a1 = f0.high(a), a2 = f1.low(b), a3 = f1.high(b);
                if (Pol::kSplitCols) {
                    ptx::mma_f16_16816_zero(d, a0, a1, a2, a3, hi[0], hi[1]);
                } else {
                    ptx::mma_f16_16816_zero(d, a0, a1, a2, a3, lo[0], lo[1]);
                    ptx::mma_f16_16816(d, a0, a1, a2, a3, hi[0], hi[1]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[4 * i + k][j] += d[j];
            }
    }

    // The end of this warp's share of a piece: M and l of its columns to wm and wl (the planes of a
    // head hold the same), with M itself as the exponent of the weights.
    __device__ __forceinline__ void finish(typename NibbleSmem<Pol>::Unit& sm, int own, int half,
                                           int lane) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float ls = l[j];
            ls += __shfl_xor_sync(0xffffffffu, ls, 4);
            ls += __shfl_xor_sync(0xffffffffu, ls, 8);
            ls += __shfl_xor_sync(0xffffffffu, ls, 16);
            if (half == 0 && lane < 4) {
                sm.wm[own][2 * lane + j] = ms[j];
                sm.wl[own][2 * lane + j] = ls * 0x1p-12f;
            }
        }
    }

    // Merge of the warps' states: the output (slot < 0; the piece is the whole segment) or
    // the partial (acc, m, l) at workspace slot `slot`.  The M are whole numbers, so the
    // factors 2^(M_w - M) are exact.  Called by all consumer warps, after finish() and a barrier.
    __device__ __forceinline__ void merge(typename NibbleSmem<Pol>::Unit& sm, const DecodeParams& p,
                                          size_t out_base, int slot, int bar, int own, int half,
                                          int lane) {
        const int g = lane >> 2, t = lane & 3, tid = own * 32 + lane;
        constexpr int kThreads = Pol::NC * 32;          // of each plane
        constexpr int W = Pol::kMergeDims, kPer = Pol::kMergeTiles, kPitch = Pol::kMergePitch;
        // a round merges G heads x W channels; a thread takes two channels of every kHeadStep-th head
        constexpr int kHeadStep = kThreads / (W / 2);
        static_assert(kHeadStep * (W / 2) == kThreads && G % kHeadStep == 0, "two channels per thread");
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < Pol::NC; ++w) top = fmaxf(top, sm.wm[w][2 * t + j]);
            // (a warp without a score weighs 0 beside one with; its NaN stay)
            const float f = ptx::ex2(ms[j] - top) * 0x1p-12f;
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                acc[i][j] *= f;
                acc[i][j + 2] *= f;
            }
        }
        float top[G / kHeadStep], ls[G / kHeadStep], inv[G / kHeadStep];   // of this thread's heads
#pragma unroll
        for (int k = 0; k < G / kHeadStep; ++k) {
            const int h = k * kHeadStep + tid / (W / 2);
            top[k] = -INFINITY;
            ls[k] = 0.0f;
#pragma unroll
            for (int w = 0; w < Pol::NC; ++w) top[k] = fmaxf(top[k], sm.wm[w][h]);
#pragma unroll
            for (int w = 0; w < Pol::NC; ++w) ls[k] += ptx::ex2(sm.wm[w][h] - top[k]) * sm.wl[w][h];
            inv[k] = slot < 0 ? 1.0f / ls[k] : 1.0f;
            if (slot >= 0 && half == 0 && tid % (W / 2) == 0)
                *reinterpret_cast<float2*>(p.ws_ml + (static_cast<size_t>(slot) * G + h) * 2) =
                    make_float2(top[k], ls[k]);
        }
        const bool floats = slot >= 0 || p.out_f32;
        float* to = slot < 0 ? static_cast<float*>(p.out) + out_base
                             : p.ws_acc + static_cast<size_t>(slot) * G * D;
        const int pair = tid % (W / 2), chunk = pair / kPer, within = 2 * (pair % kPer);
#pragma unroll
        for (int r = 0; r < kTiles / kPer; ++r) {
            if (2 * t < Pol::kMergeCols) {   // (at kSplitCols t = 1 holds the lo parts' products)
#pragma unroll
                for (int i = 0; i < kPer; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        *reinterpret_cast<float2*>(&sm.wacc[half][own][2 * t + j][perm(g) * kPitch + 2 * i]) =
                            make_float2(acc[r * kPer + i][j], acc[r * kPer + i][j + 2]);
            }
            ptx::named_barrier_sync(bar, Pol::GW * 32);
#pragma unroll
            for (int k = 0; k < G / kHeadStep; ++k) {
                const int h = k * kHeadStep + tid / (W / 2);
                float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < Pol::NC; ++w)
#pragma unroll
                    for (int c = 0; c < Pol::kMergeCols; c += G) {
                        const float2 x =
                            *reinterpret_cast<const float2*>(&sm.wacc[half][w][c + h][chunk * kPitch + within]);
                        s.x += x.x;
                        s.y += x.y;
                    }
                const size_t at = static_cast<size_t>(h) * D + half * kNibblePlane + 32 * chunk + 2 * kPer * r + within;
                if (floats)
                    *reinterpret_cast<float2*>(to + at) = make_float2(s.x * inv[k], s.y * inv[k]);
                else
                    *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + out_base + at) =
                        __floats2bfloat162_rn(s.x * inv[k], s.y * inv[k]);
            }
            // (wacc is filled again: in the next round, or after the barrier that ends the next piece)
            if (r + 1 < kTiles / kPer) ptx::named_barrier_sync(bar, Pol::GW * 32);
        }
    }
};

template <class Pol, bool kPaged>
__global__ void __launch_bounds__(Pol::kThreads, 1) gqa_decode_nibble_kernel(const DecodeNibbleParams np) {
    constexpr int G = Pol::G, D = Pol::D, RING = Pol::RING, GROUPS = Pol::GROUPS, SPLIT = Pol::SPLIT;
    constexpr int NC = Pol::NC, kBlock = kNibblePage;
    constexpr std::integral_constant<int, NibblePlanTuning::kExtra> kExtra{};
    constexpr uint32_t kTileBytes = NibbleSmem<Pol>::kTileBytes;
    const DecodeParams& p = np.d;

    extern __shared__ uint8_t smem_raw[];
    NibbleSmem<Pol>& sm = *reinterpret_cast<NibbleSmem<Pol>*>(
        smem_raw + ((128u - (ptx::smem_addr(smem_raw) & 127u)) & 127u));

    const int tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    const int B = p.B, KVH = p.KVH, H = p.H;
    const int cta = blockIdx.x, ctas = static_cast<int>(gridDim.x);
    PlanSmem& pl = sm.plan;

    if (tid < GROUPS) {
        typename NibbleSmem<Pol>::Unit& un = sm.unit[tid];
        for (int s = 0; s < NC * RING; ++s) {
            ptx::mbar_init(ptx::smem_addr(&un.full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&un.empty[s]), SPLIT);
        }
        ptx::mbar_init(ptx::smem_addr(&un.piece_full), 1);
        ptx::mbar_init(ptx::smem_addr(&un.piece_empty), Pol::GW + Pol::kFeeds - 1);   // who reads it
        if (tid == 0) {
            ptx::mbar_init(ptx::smem_addr(&sm.stall_bar), 1);
            sm.abort_flag = 0;
        }
        ptx::fence_mbar_init();
    }
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    // (the plan's barriers make the lengths visible)
    for (int b = tid; b < B; b += blockDim.x)
        sm.len[b] = min(max(__ldg(p.seq_lens + b), 0), p.capacity);
    build_plan<NibblePlanTuning>(pl, p, ctas * GROUPS, warp, lane, cta, kBlock,
                                 reinterpret_cast<uint32_t*>(&sm.kv[0][0][0][0]));

    // zeros for empty sequences and the segments' partial lists, as in decode_kernel.cuh.  (Unit
    // cta + ctas * i is this CTA's i-th: few units still spread over all CTAs.)
    const bool has_work = cta < pl.g_eff;
    if (!has_work || warp < Pol::kConsumers) {
        const int nt = has_work ? Pol::kConsumers * 32 : static_cast<int>(blockDim.x);
        for (int b = cta; b < B; b += ctas) {
            if (pl.n[b] != 0) continue;
            const size_t base = static_cast<size_t>(b) * H * D;
            for (int i = tid; i < H * D; i += nt) store_out(p, base + i, 0.0f);
        }
        const int U = B * KVH;
        const int u_end = (cta + 1) * U / ctas;
        for (int u = cta * U / ctas + tid; u < u_end; u += nt) {
            const int b = u / KVH, kvh = u - b * KVH;
            int4 e = make_int4(0, 0, 0, 0);
            if (pl.n[b] != 0 && pl.g_eff > 0) {
                const SegmentParts sp(pl, b, kvh, p.dyn_slot_base, kExtra);
                e = make_int4(sp.first_s, sp.ns_parts, sp.dk0, sp.nd_parts);
            }
            p.ws_segs[u] = e;
        }
    }
    if (!has_work) return;

    // this warp's unit (a group without a unit has nothing to do)
    const int group = warp < Pol::kConsumers ? warp / Pol::GW : (warp - Pol::kConsumers) / Pol::kFeeds;
    const int unit = cta + ctas * group;
    if (unit >= pl.g_eff) return;
    typename NibbleSmem<Pol>::Unit& un = sm.unit[group];
    const uint32_t kv_base = ptx::smem_addr(&sm.kv[group][0][0][0]);
    const uint32_t piece_full = ptx::smem_addr(&un.piece_full), piece_empty = ptx::smem_addr(&un.piece_empty);

    if (warp >= Pol::kConsumers) {
        // ======== producers: a thread per two rings of the unit ========
        // The unit's first walks the schedule and publishes each piece; each fills the slots of
        // its rings.
        const uint32_t edge = static_cast<uint32_t>(static_unit_begin(pl, unit + (lane & 1)));
        StaticWalk<NibblePlanTuning> walk(pl, B, __shfl_sync(0xffffffffu, edge, 0),
                                          __shfl_sync(0xffffffffu, edge, 1));
        if (lane != 0) return;
        constexpr int kFeeds = Pol::kFeeds, kLoads = 2;   // rings of a producer
        const int me = (warp - Pol::kConsumers) % kFeeds;
        const uint64_t policy = ptx::policy_evict_first();
        ptx::fence_proxy_async_smem();   // the plan used the slots
        const bool dynamic = pl.n_dyn > 0;
        const size_t plane = static_cast<size_t>(kPaged ? kBlock : np.rows) * kNibbleRow;   // bytes of a plane
        uint32_t filled[kLoads];   // blocks sent to rings me, me + kFeeds
#pragma unroll
        for (int k = 0; k < kLoads; ++k) filled[k] = 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            int b, kvh, blk0, blk1, lo, hi;
            if (me == 0) {
                // the description is free once the others have read the one before
                ok = wait_bounded(piece_empty, (n & 1u) ^ 1u, &sm.abort_flag, p.ws_flags);
                if (!ok) break;
                Piece w;
                bool whole = false;   // the piece is its segment
                if (walk.next(pl, KVH, unit, w)) {
                    whole = w.p1 - w.p0 == pl.n[w.b];
                } else {
                    int claimed = -1;
                    if (!dynamic || !claim_piece(pl, p, claimed, w)) {
                        un.piece.done = 1;
                        ptx::mbar_arrive(piece_full);
                        break;
                    }
                }
                const int L = sm.len[w.b];
                un.piece.b = b = w.b;
                un.piece.kvh = kvh = w.kvh;
                un.piece.p0 = w.p0;
                un.piece.p1 = w.p1;
                un.piece.lo = lo = p.window > 0 && L > p.window ? L - p.window : 0;
                un.piece.hi = hi = L;
                un.piece.slot = whole ? -1 : w.slot;
                un.piece.done = 0;
                blk0 = w.p0 / kBlock;
                blk1 = w.p1 / kBlock;
                ptx::mbar_arrive(piece_full);
            } else {
                ok = wait_bounded(piece_full, n & 1u, &sm.abort_flag, p.ws_flags);
                if (!ok || un.piece.done) break;
                b = un.piece.b;
                kvh = un.piece.kvh;
                blk0 = un.piece.p0 / kBlock;
                blk1 = un.piece.p1 / kBlock;
                lo = un.piece.lo;
                hi = un.piece.hi;
                ptx::mbar_arrive(piece_empty);
            }
            const int32_t* bt_row =
                kPaged ? p.block_table + static_cast<size_t>(b) * p.max_pages : nullptr;
            // the head's planes of sequence b, or of page 0
            const uint8_t* head =
                np.kv + (static_cast<size_t>(kPaged ? 0 : b) * KVH + kvh) * SPLIT * plane;
            int page[kLoads];   // page ids of the next round, loaded one round ahead
            if (kPaged) {
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const int blk = blk0 + me + kFeeds * k;
                    page[k] = blk < blk1 ? __ldg(bt_row + blk) : 0;
                }
            }
            for (int round = blk0; ok && round < blk1; round += NC) {
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const int ring = me + kFeeds * k, blk = round + ring;
                    if (blk >= blk1) break;
                    const int s = ring * RING + static_cast<int>(filled[k] % RING);
                    ok = wait_bounded(ptx::smem_addr(&un.empty[s]), ((filled[k] / RING) & 1u) ^ 1u,
                                      &sm.abort_flag, p.ws_flags);
                    if (!ok) break;
                    const uint32_t full_bar = ptx::smem_addr(&un.full[s]);
                    // the attended rows of the block (at least one), no others
                    const int r0 = max(lo - blk * kBlock, 0), r1 = min(hi - blk * kBlock, kBlock);
                    const uint32_t bytes = static_cast<uint32_t>(r1 - r0) * kNibbleRow;
                    const uint8_t* src;
                    bool bad = false;
                    if (kPaged) {
                        bad = page[k] < 0 || page[k] >= p.num_pages;
                        src = head + (static_cast<size_t>(page[k]) * KVH * SPLIT * kBlock + r0) * kNibbleRow;
                        un.bad[s] = bad;
                        if (blk + NC < blk1) page[k] = __ldg(bt_row + blk + NC);
                    } else {
                        src = head + (static_cast<size_t>(blk) * kBlock + r0) * kNibbleRow;
                    }
                    if (bad) {   // nothing to load: the consumer's weights are NaN
                        atomicOr(p.ws_flags, kFlagBadPage);
                        ptx::mbar_arrive(full_bar);
                    } else {
                        ptx::mbar_arrive_expect_tx(full_bar, SPLIT * bytes);
#pragma unroll
                        for (int h = 0; h < SPLIT; ++h)
                            ptx::bulk_copy_g2s(kv_base + (s * SPLIT + h) * kTileBytes + r0 * kNibbleRow,
                                               src + h * plane, bytes, full_bar, policy);
                    }
                    ++filled[k];
                    if ((p.test_flags & kTestStall) && group == 0 && me == 0 && k == 0 && filled[0] == 1)
                        ok = wait_bounded(ptx::smem_addr(&sm.stall_bar), 0u, &sm.abort_flag,
                                          p.ws_flags, kTestStallNs);
                    if (!ok) break;
                }
            }
        }
        // every copy issued lands before the CTA can exit (its consumer may have given up)
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
            for (uint32_t f = filled[k] > RING ? filled[k] - RING : 0u; f < filled[k]; ++f)
                wait_drain(ptx::smem_addr(&un.full[(me + kFeeds * k) * RING + f % RING]), (f / RING) & 1u);
        return;
    }

    // ===================== consumers =====================
    // Every warp of a unit passes the same barriers for every piece, whatever its waits return:
    // one that gave up (or saw the end) makes all of them leave at the piece's last barrier.
    const int gwarp = warp - group * Pol::GW, own = gwarp / SPLIT, half = gwarp % SPLIT;
    const int bar = 1 + group, pair_bar = 1 + GROUPS + group * NC + own;
    NibbleConsumer<Pol> c;
    uint32_t taken = 0;   // blocks this warp has processed (its ring's fills, in order)
    for (uint32_t n = 0;; ++n) {
        const bool there = __all_sync(0xffffffffu, wait_bounded(piece_full, n & 1u, &sm.abort_flag, p.ws_flags));
        BlockPiece pc{};
        pc.done = 1;
        if (there) pc = un.piece;
        bool gone = pc.done != 0;
        if (SPLIT > 1) gone = ptx::named_barrier_or(pair_bar, 2 * 32, gone);
        __syncwarp();
        const size_t out_base = (static_cast<size_t>(pc.b) * H + pc.kvh * G) * D;
        if (!gone) {
            if (lane == 0) ptx::mbar_arrive(piece_empty);   // every lane has read it
            c.begin(p.q + out_base, half, lane);
            // (block i of a piece is warp i % NC's, whatever came before: the order of the sums
            // does not depend on the schedule)
            for (int pos = pc.p0 + own * kBlock; pos < pc.p1; pos += NC * kBlock) {
                const int s = own * RING + static_cast<int>(taken % RING);
                gone = !__all_sync(0xffffffffu, wait_bounded(ptx::smem_addr(&un.full[s]), (taken / RING) & 1u,
                                                             &sm.abort_flag, p.ws_flags));
                const uint32_t tile = kv_base + (s * SPLIT + half) * kTileBytes;
                float z[4];
                if (SPLIT == 1) {
                    if (gone) break;
                    c.scores(tile, z, lane);
                } else {
                    // the planes' scores cross over through the K codes of this warp's tile, which
                    // it has read: lane l's at row l / 2
                    const uint32_t at = (lane >> 1) * kNibbleRow + (lane & 1) * 16;
                    const uint32_t other = kv_base + (s * SPLIT + 1 - half) * kTileBytes;
                    if (!gone) {
                        c.scores(tile, z, lane);
                        __syncwarp();
                        ptx::sts128(tile + at, __float_as_uint(z[0]), __float_as_uint(z[1]),
                                    __float_as_uint(z[2]), __float_as_uint(z[3]));
                    }
                    gone = ptx::named_barrier_or(pair_bar, 2 * 32, gone);
                    if (gone) break;
                    const uint4 o = ptx::lds128(other + at);
                    z[0] += __uint_as_float(o.x);
                    z[1] += __uint_as_float(o.y);
                    z[2] += __uint_as_float(o.z);
                    z[3] += __uint_as_float(o.w);
                }
                const bool bad = kPaged && un.bad[s] != 0;
                c.weigh(z, tile, pc.lo - pos, pc.hi - pos, bad, lane);
                if (SPLIT > 1) ptx::fence_proxy_async_smem();   // (the scores, before the next copy)
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&un.empty[s]));
                ++taken;
            }
            c.finish(un, own, half, lane);
        }
        if (ptx::named_barrier_or(bar, Pol::GW * 32, gone)) break;
        c.merge(un, p, out_base, pc.slot, bar, own, half, lane);
    }
}

// slidingDecodeGQA and decodeGQA, for few and for many segments
using NibbleSliding = NibblePolicy<2, 2, 4, 4>;
using NibbleSlidingMany = NibblePolicy<2, 4, 2, 4>;
using NibbleGlobal = NibblePolicy<8, 1, 4, 4>;
using NibbleGlobalMany = NibblePolicy<8, 2, 2, 4>;

}  // namespace gqa
