// Decode attention over the 8-bit cache (quant_cache.cuh): attn.core of the gemma-4-31B
// Model Spec for one new token per sequence, on the values k = 2^ek ck and v = 2^ev cv
// (c: e4m3 codes; ek, ev: exponents of the block scales).
//
// Mathematics.  With x_s = log2(e) <q, k_s> + ev_s the weights of the value CODES are
// 2^(x_s - M), and the normaliser is l = sum 2^(x_s - ev_s - M), for any M; o = sum
// 2^(x_s - M) cv_s / l.  So the scales never touch the codes: ek multiplies a finished
// score, ev moves an exponent.  M is a whole number, at least the running maximum of x
// less 15: differences of exponents are then exact, the accumulators are rescaled by
// powers of two (and seldom), and the weights lie in (0, 2^15], where f16 hi + lo parts
// hold them to 22 bits.  M is held in two parts, the ceiling of the score that set it and the
// ev beside it less 12, and x - M is formed part by part: from 2^24 on, where floats have a spacing
// above 1, a sum of the two would lose ev and could pass 2^15.  Equal scores weigh the same
// whatever their blocks' scales.
//
// Both contractions run as warp-level f16 mma (m16n8k16, fp32 accumulate) with the cache
// as the A operand, so that the g <= 8 query heads of a KV head fill the 8 columns of B
// and no row is idle.  e4m3 widens to f16 exactly, two codes per instruction.  q is scaled
// by a power of two per head, which makes its bf16 values exact in f16 down to 2^-31 of
// the largest (at g = 8 of the largest in each half of D).
//   scores  S[pos, h] = K[pos, :] . q[h, :] for the 16 positions of a block; the k index
//           pairs of an A fragment are the bytes (4t, 4t+1) and (4t+2, 4t+3) of a 16-byte
//           unit, q's B fragment in the same order
//   P.V     O^T[d, h] += V^T[d, pos] P[pos, h]; 16-bit ldmatrix.trans delivers dims (2g, 2g+1)
//           of two positions, one byte permute makes them rows g and g+8 of A.  movmatrix
//           turns the weights from the scores' layout into B fragments.  At g = 2 the hi
//           and lo parts of P are columns of one mma; at g = 8 they are two mma.
// An mma truncates its sum, so long chains of them drift: a block's products start from
// zero and are added to the accumulators by ordinary additions.
//
// Work split and timeouts are those of decode_kernel.cuh: a persistent CTA per SM, a plan
// built from seq_lens on the device; split segments are merged by the combine kernel.  Pieces
// start and end on blocks.  A CTA holds several units of the plan, each with a schedule of
// its own, so that one computes while another begins or ends a piece.  In a unit, NC warps (at
// g = 8, where the accumulators would take 128 registers and leave one warp per scheduler, NC
// pairs, half of D each, which add their halves of the scores) work on a block each: block i of
// a piece goes to warp i % NC, into that warp's own ring of slots, and the warp keeps M, l and
// the D x 8 accumulators until the piece ends, when the NC states are merged through shared
// memory.  (A ring shared by the warps would let a warp wait on a slot's barrier two fills
// ahead of its last completion, which a parity cannot tell apart.)  Producer threads walk the
// schedules and issue the TMA copies, one slot per block.
//
// NC = 4 or 2 (kernels_quant.cu has the rule and what both measure): larger units leave fewer
// partials to merge and read longer runs, smaller ones overlap more ends of pieces, which
// cost 2-3 us each.  A piece of one block takes a warp 3.2 us: 0.7 for q, 1.3 for the block, 1.0
// for the merge.  Much of that is fetching instructions (each warp is somewhere else in some 20 KB
// of code), so code that is kept short, with one form for all cases, is faster here.
//
// Measured on the way (decode_sliding_b64_paged / decode_global_b64_paged, now 83-86 / 334-344 us):
// the 8 warps sharing each tile, with a score tile between the contractions, 171 / 386 us
// (every warp repeats the softmax of all positions); blocks dealt to the warps in turn and one
// producer thread, 153 / 447 us (its ~700 cycles per 16 KB are the time HBM takes for them);
// units of one warp or pair, 92 / 353 us.
#pragma once

#include "decode_kernel.cuh"
#include "quant_cache.cuh"

namespace gqa {

struct DecodeQuantParams {
    DecodeParams d;
    const float* k_scales;   // [B, blocks, KVH] or [P, KVH]
    const float* v_scales;
    int blocks;              // blocks per sequence (contiguous)
};

// The plan's constants for this kernel: a piece costs a unit about as much as kExtra blocks,
// and dynamic chunks are fewer and begin at more work than for bf16 rows, which stream half as
// fast.  Measured with 4 extra blocks, 256 positions and 8 chunks, and with these:
// decode_global_b8 37.3 and 31.7 us, decode_sliding_b64_paged 89.4 and 84.6,
// decode_global_b64_paged 350 and 341.
struct QuantPlanTuning {
    static constexpr int kAlign = kQuantBlock, kExtra = 12;
    static constexpr int kMinShare = 1024, kChunksPerCta = 4;
};

template <int kG, int kD, int kGroups, int kBlocksAtOnce, int kSplitD, int kRing>
struct QuantPolicy {
    static constexpr int G = kG, D = kD;
    static constexpr int GROUPS = kGroups;               // units of the plan per CTA
    static constexpr int NC = kBlocksAtOnce;             // blocks a unit works on at a time
    static constexpr int SPLIT = kSplitD;                // warps per block, D / SPLIT dims each
    static constexpr int RING = kRing;                   // slots per block in work: one block of K and V each
    static constexpr int GW = NC * SPLIT;                // consumer warps per unit
    static constexpr int kConsumers = GROUPS * GW;
    static constexpr int kFeeds = NC / 2;                // producers per unit, two rings each
    static constexpr int kWarps = kConsumers + kFeeds * GROUPS;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kOwnUnits = D / 16 / SPLIT;     // 16-dim steps of one warp
    static constexpr bool kSplitCols = G == 2;           // hi and lo parts of P in one mma
    static constexpr int kMergeDims = 128 / SPLIT;       // dims of a warp merged per round
    static constexpr int kMergeStride = kMergeDims + 4;  // conflict-free float2 stores
    static constexpr int kMergeCols = kSplitCols ? 2 * G : G;
    static_assert((G == 2 || G == 8) && (SPLIT == 1 || SPLIT == 2) && (NC == 2 || NC == 4), "shape");
    static_assert(kOwnUnits % 8 == 0 && (D / SPLIT) % kMergeDims == 0, "shape");
    static_assert(kThreads >= kPlanWarps * 32, "the plan takes eight warps");
};

// One piece of work.
struct QuantPiece {
    int b, kvh;
    int p0, p1;     // positions, whole blocks
    int lo, hi;     // attended positions of the sequence
    int slot;       // workspace slot of the partial; -1: the piece is the whole segment
    int done;       // no more pieces
};

// The static pieces of one unit of the plan in order: a search and a division for the first (on
// every call's way to its first copy), steps from there.  Each segment's tiles begin with kExtra
// that hold no positions.
struct StaticWalk {
    static constexpr int kExtra = QuantPlanTuning::kExtra;
    uint32_t x, stop;   // the unit's tiles
    int b, kvh, k;      // the segment that holds tile x, and x's place in it

    __device__ __forceinline__ static int tiles(const PlanSmem& pl, int b) {
        return kExtra + pl.sn[b] / kQuantBlock;   // (sn is whole blocks)
    }
    __device__ __forceinline__ StaticWalk(const PlanSmem& pl, int B, uint32_t first, uint32_t end)
        : x(first), stop(end), b(0), kvh(0), k(0) {
        if (x >= stop) return;
        b = upper_seq(pl.spref, B, x);
        const uint32_t st = static_cast<uint32_t>(tiles(pl, b)), rel = x - pl.spref[b];
        kvh = static_cast<int>(rel / st);
        k = static_cast<int>(rel - static_cast<uint32_t>(kvh) * st);
    }
    __device__ __forceinline__ bool next(const PlanSmem& pl, int KVH, int unit, Piece& w) {
        while (x < stop) {
            const int st = tiles(pl, b), k0 = k;
            const int take = min(static_cast<int>(min(stop - x, 0x7fffffffu)), st - k0);
            w.b = b;
            w.kvh = kvh;
            w.p0 = pl.lo[b] + max(k0 - kExtra, 0) * kQuantBlock;
            w.p1 = pl.lo[b] + (k0 + take - kExtra) * kQuantBlock;
            w.slot = unit + b * KVH + kvh;
            x += static_cast<uint32_t>(take);
            k += take;
            if (k == st) {
                k = 0;
                if (++kvh == KVH) {
                    kvh = 0;
                    if (x < stop)
                        do ++b;
                        while (pl.sn[b] == 0);   // (ends: tile x is in a later sequence)
                }
            }
            if (k0 + take > kExtra) return true;   // else only tiles without positions
        }
        return false;
    }
};

template <class Pol>
struct alignas(1024) QuantSmem {
    static constexpr int kTileBytes = kQuantBlock * Pol::D;
    struct Unit {
        alignas(8) uint64_t full[Pol::NC * Pol::RING];
        alignas(8) uint64_t empty[Pol::NC * Pol::RING];
        alignas(8) uint64_t piece_full, piece_empty;
        float scales[Pol::NC * Pol::RING][2];
        int bad[Pol::NC * Pol::RING];            // the block's page id is out of range
        QuantPiece piece;
        float wm[Pol::NC][8], wl[Pol::NC][8];    // M and l per column of each warp (pair)
        alignas(16) float wacc[Pol::SPLIT][Pol::NC][Pol::kMergeCols][Pol::kMergeStride];   // dims being merged
    };
    uint8_t kv[Pol::GROUPS][Pol::NC * Pol::RING][2][kTileBytes];   // [slot][K, V][chunk][16 rows][128 B]
    Unit unit[Pol::GROUPS];
    alignas(8) uint64_t stall_bar;               // kTestStall: a barrier nothing completes
    PlanSmem plan;
    int len[kMaxBatch];                          // clamped lengths
    int abort_flag;
};

template <class Pol>
struct QuantConsumer {
    static constexpr int G = Pol::G, D = Pol::D, kOwnUnits = Pol::kOwnUnits;
    static constexpr float kTop = 15.0f;    // largest exponent of a weight (f16 ends at 2^16)
    static constexpr float kRoom = 3.0f;    // binades left above the maximum when M is set
    static constexpr float kLowest = -3.402823466e38f;   // ms of no score yet (differences are numbers)
    // Scores wait for the keys' scale as 2^-kPark of themselves: a product <q, code> may be up to
    // 2^147, and with a scale down to 2^-64 the score is a float all the same.  At the other end
    // what is lost to fp32's smallest numbers is below 2^-60 of a unit after any key scale.
    static constexpr int kPark = 24;
    // Weights of codes below 2^-126 are flushed.  l is at least 2^(11 - 64), so at value scales
    // from 2^kLowExp up the flushed shares are below 2^-41 of it; below, they are taken apart.
    static constexpr int kLowExp = -32;

    uint2 qb[kOwnUnits];         // B fragments of q (column g = head g % G) for this warp's dims
    float q_undo[2];             // undo their scaling for columns 2t and 2t + 1, times 2^-kPark
    float acc[kOwnUnits][4];     // rows: dims 2g (0, 1) and 2g + 1 (2, 3); columns 2t, 2t + 1
    float ms[2], me[2];          // M = ms + me of columns 2t, 2t + 1: of the scores, of the scales
    float l[2];                  // this lane's share of their normalisers

    // Byte address of 16-byte unit `unit` of row r of a block.
    __device__ static __forceinline__ uint32_t unit_addr(uint32_t block, int r, int unit) {
        return block + (unit >> 3) * 2048 + r * 128 + (((unit & 7) ^ (r & 7)) << 4);
    }

    // q_heads: [G][D] bf16 in global memory; `half`: which part of D is this warp's.
    __device__ __forceinline__ void begin(const __nv_bfloat16* q_heads, int half, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const __nv_bfloat16* row = q_heads + (g % G) * D + half * (kOwnUnits * 16) + 4 * t;
        uint32_t top = 0;   // largest |q|: the bits of |bf16| order like the values
#pragma unroll
        for (int u = 0; u < kOwnUnits; ++u) {
            qb[u] = __ldg(reinterpret_cast<const uint2*>(row + u * 16));
            top = __vmaxu2(top, __vmaxu2(qb[u].x & 0x7fff7fffu, qb[u].y & 0x7fff7fffu));
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(static_cast<int>(top >> 7) - 127, -88);   // |q| < 2^(e + 1)
        const float f = pow2f(14 - e);
#pragma unroll
        for (int u = 0; u < kOwnUnits; ++u)
            qb[u] = make_uint2(ptx::f16x2_pack(bf16lo(qb[u].x) * f, bf16hi(qb[u].x) * f),
                               ptx::f16x2_pack(bf16lo(qb[u].y) * f, bf16hi(qb[u].y) * f));
        const float undo = pow2f(e - 14 - kPark);
        q_undo[0] = __shfl_sync(0xffffffffu, undo, 8 * t);
        q_undo[1] = __shfl_sync(0xffffffffu, undo, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < kOwnUnits; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
        ms[0] = ms[1] = kLowest;
        me[0] = me[1] = 0.0f;
        l[0] = l[1] = 0.0f;
    }

    // This warp's share of a block's products 2^-kPark <q, code>: rows g (0, 1) and g + 8 (2, 3),
    // columns 2t, 2t + 1.
    __device__ __forceinline__ void scores(uint32_t k_blk, int half, float (&z)[4], int lane) {
        const int mat = lane >> 3, r = (mat & 1) * 8 + (lane & 7);
        float c[4][4];   // four independent chains
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i][j] = 0.0f;
        // (8 units fill one of unit_addr's chunks)
        const uint32_t k_half = k_blk + half * (kOwnUnits / 8) * 2048;
#pragma unroll
        for (int u = 0; u < kOwnUnits; u += 2) {
            uint32_t a[4];   // rows g, g + 8 of unit u, then of unit u + 1
            ptx::ldmatrix_x4(unit_addr(k_half, r, u + (mat >> 1)), a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t a0, a1, a2, a3;
                ptx::e4m3x4_to_f16x2(a[2 * i], a0, a2);
                ptx::e4m3x4_to_f16x2(a[2 * i + 1], a1, a3);
                ptx::mma_f16_16816(c[(u + i) & 3], a0, a1, a2, a3, qb[u + i].x, qb[u + i].y);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            z[i] = ((c[0][i] + c[1][i]) + (c[2][i] + c[3][i])) * q_undo[i & 1];
    }

    // Zeroes this warp's dims of the V rows outside [first, last): they hold anything, and 0 * NaN
    // is NaN.  (As masks on every unit in weigh() it cost 1% of decode_global_b64_paged; a masked
    // and a whole form of weigh() took 0.2 us more everywhere, by the size of their code.)
    __device__ static __forceinline__ void clear_rows(uint32_t v_blk, int first, int last, int half, int lane) {
        const uint32_t v_half = v_blk + half * (kOwnUnits / 8) * 2048;
        const int r = lane & 15;
        if (r < first || r >= last) {
#pragma unroll
            for (int i = 0; i < kOwnUnits; i += 2)
                ptx::sts128(unit_addr(v_half, r, i + (lane >> 4)), 0u, 0u, 0u, 0u);
        }
        __syncwarp();
    }

    // The rest of a block, from its products z: weights, M, l, and P.V for this warp's dims.  Rows
    // [first, last) are attended; bad: their page does not exist, and their weights are NaN.
    __device__ __forceinline__ void weigh(const float (&z)[4], uint32_t v_blk, float k_scale,
                                          float v_scale, int first, int last, bool bad, int half,
                                          int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int mat = lane >> 3, r = (mat & 1) * 8 + (lane & 7);
        // x = log2(e) score, rows g (0, 1) and g + 8 (2, 3), and the weights' exponents y = x + ev - M;
        // rows outside the range weigh 2^-inf
        const float f = pow2f(scale_exponent(k_scale) + kPark) * kLog2e;
        const int ev = scale_exponent(v_scale);
        const float evf = bad ? __uint_as_float(0x7fc00000u) : static_cast<float>(ev);
        const bool row_ok[2] = {g >= first && g < last, g + 8 >= first && g + 8 < last};
        float x[4], y[4];
        // (the rounding of x is left out of y while it is below 1; from 2^23 on M bounds rounded x
        // only.  With rounded x throughout the outputs' error was a tenth larger, 1.8e-7 in place
        // of 1.6e-7 for 1 to 40 positions, and the time up to 1% less on some short sliding calls.)
        auto level = [&](int i) {
            const float d = fabsf(x[i]) < 0x1p23f ? fmaf(z[i], f, -ms[i & 1]) : x[i] - ms[i & 1];
            return d + (evf - me[i & 1]);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = row_ok[i >> 1] ? __fmul_rn(z[i], f) : -INFINITY;
            y[i] = level(i);
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
                const float up = (top - ms[j]) + (evf - (kTop - kRoom) - me[j]);
                if (up > 0.0f) {   // (never of a NaN)
                    ms[j] = top;
                    me[j] = evf - (kTop - kRoom);
                }
                // (in two steps for l, which may be near 2^100 when the values so far were tiny)
                const float dm = up > 0.0f ? fmaxf(-up, -252.0f) : 0.0f;
                const float a1 = ptx::ex2(floorf(0.5f * dm)), a2 = ptx::ex2(dm - floorf(0.5f * dm));
                const float alpha = a1 * a2;
                l[j] = l[j] * a1 * a2;
#pragma unroll
                for (int i = 0; i < kOwnUnits; ++i) {
                    acc[i][j] *= alpha;
                    acc[i][j + 2] *= alpha;
                }
                y[j] = level(j);
                y[j + 2] = level(j + 2);
            }
        }
        uint32_t hi[2], lo[2];   // B fragments: column g, positions (2t, 2t + 1) of each half
        const float unscale = pow2f(-ev);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float p0 = ptx::ex2(y[2 * i]), p1 = ptx::ex2(y[2 * i + 1]);
            if (ev >= kLowExp) {
                l[0] = fmaf(p0, unscale, l[0]);
                l[1] = fmaf(p1, unscale, l[1]);
            } else {
                l[0] += ptx::ex2(y[2 * i] - evf);
                l[1] += ptx::ex2(y[2 * i + 1] - evf);
            }
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
        const uint32_t v_half = v_blk + half * (kOwnUnits / 8) * 2048;
#pragma unroll
        for (int u = 0; u < kOwnUnits; u += 2) {
            uint32_t w[4];   // positions 0-7, 8-15 of unit u, then of unit u + 1
            ptx::ldmatrix_x4_trans(unit_addr(v_half, r, u + (mat >> 1)), w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t a0, a1, a2, a3;
                ptx::e4m3x4_to_f16x2(__byte_perm(w[2 * i], 0u, 0x3120), a0, a1);
                ptx::e4m3x4_to_f16x2(__byte_perm(w[2 * i + 1], 0u, 0x3120), a2, a3);
                float d[4];
                if (Pol::kSplitCols) {
                    ptx::mma_f16_16816_zero(d, a0, a1, a2, a3, hi[0], hi[1]);
                } else {
                    ptx::mma_f16_16816_zero(d, a0, a1, a2, a3, lo[0], lo[1]);
                    ptx::mma_f16_16816(d, a0, a1, a2, a3, hi[0], hi[1]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[u + i][j] += d[j];
            }
        }
    }

    // The end of this warp's share of a piece: M and l of its columns to wm and wl (the halves
    // of D hold the same).  From here on l is in [1, 2) and M has its exponent: between equal
    // shares of the softmax the M of the weights of codes differ by up to 128, and a merge
    // would flush one of them.  l[j] becomes the factor by which the accumulators lag behind M.
    // M is one float again.  Where that has a spacing above 1 (from 2^24 on) l keeps what M
    // cannot hold, at most 2^19 either way: l 2^M lies within [2^-1, 2^18] times 2^x of the
    // largest x, and that x is a float.  ms[j] becomes M.
    __device__ __forceinline__ void finish(typename QuantSmem<Pol>::Unit& sm, int own, int half,
                                           int lane) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float ls = l[j];
            ls += __shfl_xor_sync(0xffffffffu, ls, 4);
            ls += __shfl_xor_sync(0xffffffffu, ls, 8);
            ls += __shfl_xor_sync(0xffffffffu, ls, 16);
            const int e = ls > 0.0f && ls < INFINITY ? (__float_as_int(ls) >> 23) - 127 : 0;
            const float m = ms[j] + (me[j] + static_cast<float>(e));
            l[j] = pow2f(static_cast<int>(me[j] - (m - ms[j])));
            ms[j] = m;
            if (half == 0 && lane < 4) {
                sm.wm[own][2 * lane + j] = m;
                sm.wl[own][2 * lane + j] = ls * l[j];
            }
        }
    }

    // Merge of the warps' states: the output (slot < 0; the piece is the whole segment) or
    // the partial (acc, m, l) at workspace slot `slot`.  The M are whole numbers, so the
    // factors 2^(M_w - M) are exact.  Called by all consumer warps, after finish() and a barrier.
    __device__ __forceinline__ void merge(typename QuantSmem<Pol>::Unit& sm, const DecodeParams& p,
                                          size_t out_base, int slot, int bar, int own, int half,
                                          int lane) {
        const int g = lane >> 2, t = lane & 3, tid = own * 32 + lane;
        constexpr int kThreads = Pol::NC * 32;          // of each half of D
        constexpr int W = Pol::kMergeDims;
        // a round merges G heads x W dims; a thread takes two dims of every kHeadStep-th head
        constexpr int kHeadStep = kThreads / (W / 2);
        static_assert(kHeadStep * (W / 2) == kThreads && G % kHeadStep == 0, "two dims per thread");
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < Pol::NC; ++w) top = fmaxf(top, sm.wm[w][2 * t + j]);
            // (a warp without a score weighs 0 beside one with; its NaN stay)
            const float f = ptx::ex2(ms[j] - top) * l[j];
#pragma unroll
            for (int i = 0; i < kOwnUnits; ++i) {
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
#pragma unroll
        for (int r = 0; r < D / Pol::SPLIT / W; ++r) {
            if (2 * t < Pol::kMergeCols) {   // (at kSplitCols t = 1 holds the lo parts' products)
#pragma unroll
                for (int i = 0; i < W / 16; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        *reinterpret_cast<float2*>(&sm.wacc[half][own][2 * t + j][i * 16 + 2 * g]) =
                            make_float2(acc[r * (W / 16) + i][j], acc[r * (W / 16) + i][j + 2]);
            }
            ptx::named_barrier_sync(bar, Pol::GW * 32);
#pragma unroll
            for (int k = 0; k < G / kHeadStep; ++k) {
                const int h = k * kHeadStep + tid / (W / 2), d = 2 * (tid % (W / 2));
                float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < Pol::NC; ++w)
#pragma unroll
                    for (int c = 0; c < Pol::kMergeCols; c += G) {
                        const float2 x = *reinterpret_cast<const float2*>(&sm.wacc[half][w][c + h][d]);
                        s.x += x.x;
                        s.y += x.y;
                    }
                const size_t at = static_cast<size_t>(h) * D + half * (D / Pol::SPLIT) + r * W + d;
                if (floats)
                    *reinterpret_cast<float2*>(to + at) = make_float2(s.x * inv[k], s.y * inv[k]);
                else
                    *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + out_base + at) =
                        __floats2bfloat162_rn(s.x * inv[k], s.y * inv[k]);
            }
            // (wacc is filled again: in the next round, or after the barrier that ends the next piece)
            if (r + 1 < D / Pol::SPLIT / W) ptx::named_barrier_sync(bar, Pol::GW * 32);
        }
    }
};

template <class Pol, bool kPaged>
__global__ void __launch_bounds__(Pol::kThreads, 1)
    gqa_decode_quant_kernel(const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const DecodeQuantParams qp) {
    constexpr int G = Pol::G, D = Pol::D, RING = Pol::RING, GROUPS = Pol::GROUPS, SPLIT = Pol::SPLIT;
    constexpr int NC = Pol::NC;
    constexpr std::integral_constant<int, QuantPlanTuning::kExtra> kExtra{};
    constexpr uint32_t kTileBytes = QuantSmem<Pol>::kTileBytes;
    const DecodeParams& p = qp.d;

    extern __shared__ uint8_t smem_raw[];
    QuantSmem<Pol>& sm = *reinterpret_cast<QuantSmem<Pol>*>(
        smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u));

    const int tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    const int B = p.B, KVH = p.KVH, H = p.H;
    const int cta = blockIdx.x, ctas = static_cast<int>(gridDim.x);
    PlanSmem& pl = sm.plan;

    if (tid < GROUPS) {
        typename QuantSmem<Pol>::Unit& un = sm.unit[tid];
        for (int s = 0; s < NC * RING; ++s) {
            ptx::mbar_init(ptx::smem_addr(&un.full[s]), 2);   // the tiles' bytes, the scales
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
    if (warp == Pol::kConsumers && lane == 0) {
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
    }
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    // (the plan's barriers make the lengths visible)
    for (int b = tid; b < B; b += blockDim.x)
        sm.len[b] = min(max(__ldg(p.seq_lens + b), 0), p.capacity);
    build_plan<QuantPlanTuning>(pl, p, ctas * GROUPS, warp, lane, cta, kQuantBlock,
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
    typename QuantSmem<Pol>::Unit& un = sm.unit[group];
    const uint32_t kv_base = ptx::smem_addr(&sm.kv[group][0][0][0]);
    const uint32_t piece_full = ptx::smem_addr(&un.piece_full), piece_empty = ptx::smem_addr(&un.piece_empty);

    if (warp >= Pol::kConsumers) {
        // ======== producers: a thread per two rings of the unit ========
        // The unit's first walks the schedule and publishes each piece; each fills the slots of
        // its rings.  (One thread spends ~700 cycles on 16 KB -- its TMA instructions,
        // the scales, its barriers -- which is the time HBM takes to deliver them.)
        const uint32_t edge = static_cast<uint32_t>(static_unit_begin(pl, unit + (lane & 1)));
        StaticWalk walk(pl, B, __shfl_sync(0xffffffffu, edge, 0), __shfl_sync(0xffffffffu, edge, 1));
        if (lane != 0) return;
        constexpr int kFeeds = Pol::kFeeds, kLoads = 2;   // rings of a producer
        const int me = (warp - Pol::kConsumers) % kFeeds;
        const uint64_t policy = ptx::policy_evict_first();
        ptx::fence_proxy_async_smem();   // the plan used the slots
        const bool dynamic = pl.n_dyn > 0;
        uint32_t filled[kLoads];   // blocks sent to rings me, me + kFeeds
#pragma unroll
        for (int k = 0; k < kLoads; ++k) filled[k] = 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            int b, kvh, blk0, blk1;
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
                un.piece.lo = p.window > 0 && L > p.window ? L - p.window : 0;
                un.piece.hi = L;
                un.piece.slot = whole ? -1 : w.slot;
                un.piece.done = 0;
                blk0 = w.p0 / kQuantBlock;
                blk1 = w.p1 / kQuantBlock;
                ptx::mbar_arrive(piece_full);
            } else {
                ok = wait_bounded(piece_full, n & 1u, &sm.abort_flag, p.ws_flags);
                if (!ok || un.piece.done) break;
                b = un.piece.b;
                kvh = un.piece.kvh;
                blk0 = un.piece.p0 / kQuantBlock;
                blk1 = un.piece.p1 / kQuantBlock;
                ptx::mbar_arrive(piece_empty);
            }
            const int32_t* bt_row =
                kPaged ? p.block_table + static_cast<size_t>(b) * p.max_pages : nullptr;
            const int chunk0 = kvh * (D / 128);
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
                    int outer = b;
                    if (kPaged) {
                        const bool bad = page[k] < 0 || page[k] >= p.num_pages;
                        outer = bad ? 0 : page[k];   // (loaded, and masked by the consumer)
                        un.bad[s] = bad;
                        if (bad) atomicOr(p.ws_flags, kFlagBadPage);
                        if (blk + NC < blk1) page[k] = __ldg(bt_row + blk + NC);
                    }
                    const uint32_t full_bar = ptx::smem_addr(&un.full[s]);
                    ptx::mbar_arrive_expect_tx(full_bar, 2 * kTileBytes);
                    const uint32_t k_dst = kv_base + s * 2 * kTileBytes;
                    const int row = kPaged ? 0 : blk * kQuantBlock;
                    ptx::tma_load_4d(k_dst, &tm_k, full_bar, 0, row, chunk0, outer, policy);
                    ptx::tma_load_4d(k_dst + kTileBytes, &tm_v, full_bar, 0, row, chunk0, outer, policy);
                    const size_t at = (kPaged ? static_cast<size_t>(outer)
                                              : static_cast<size_t>(b) * qp.blocks + blk) * KVH + kvh;
                    const uint32_t sc_dst = ptx::smem_addr(&un.scales[s][0]);
                    ptx::cp_async4(sc_dst, qp.k_scales + at);
                    ptx::cp_async4(sc_dst + 4, qp.v_scales + at);
                    ptx::cp_async_mbar_arrive(full_bar);
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
    QuantConsumer<Pol> c;
    uint32_t taken = 0;   // blocks this warp has processed (its ring's fills, in order)
    for (uint32_t n = 0;; ++n) {
        const bool there = __all_sync(0xffffffffu, wait_bounded(piece_full, n & 1u, &sm.abort_flag, p.ws_flags));
        QuantPiece pc{};
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
            for (int pos = pc.p0 + own * kQuantBlock; pos < pc.p1; pos += NC * kQuantBlock) {
                const int s = own * RING + static_cast<int>(taken % RING);
                gone = !__all_sync(0xffffffffu, wait_bounded(ptx::smem_addr(&un.full[s]), (taken / RING) & 1u,
                                                             &sm.abort_flag, p.ws_flags));
                const uint32_t k_tile = kv_base + s * 2 * kTileBytes;
                float z[4];
                if (SPLIT == 1) {
                    if (gone) break;
                    c.scores(k_tile, 0, z, lane);
                } else {
                    // the halves of the scores cross over through this warp's part of the K
                    // tile, which it has read
                    const uint32_t mine = k_tile + half * (kTileBytes / SPLIT) + lane * 16;
                    const uint32_t other = k_tile + (1 - half) * (kTileBytes / SPLIT) + lane * 16;
                    if (!gone) {
                        c.scores(k_tile, half, z, lane);
                        __syncwarp();
                        ptx::sts128(mine, __float_as_uint(z[0]), __float_as_uint(z[1]),
                                    __float_as_uint(z[2]), __float_as_uint(z[3]));
                    }
                    gone = ptx::named_barrier_or(pair_bar, 2 * 32, gone);
                    if (gone) break;
                    const uint4 o = ptx::lds128(other);
                    z[0] += __uint_as_float(o.x);
                    z[1] += __uint_as_float(o.y);
                    z[2] += __uint_as_float(o.z);
                    z[3] += __uint_as_float(o.w);
                }
                const float ks = un.scales[s][0], vs = un.scales[s][1];
                const bool bad = kPaged && un.bad[s] != 0;
                const int first = pc.lo - pos, last = pc.hi - pos;
                const bool part = first > 0 || last < kQuantBlock || bad;
                if (part) c.clear_rows(k_tile + kTileBytes, first, bad ? 0 : last, half, lane);
                c.weigh(z, k_tile + kTileBytes, ks, vs, first, last, bad, half, lane);
                // (the scores and cleared rows, before the next copy)
                if (SPLIT > 1 || part) ptx::fence_proxy_async_smem();
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
using QuantSliding = QuantPolicy<2, 256, 2, 4, 1, 3>;
using QuantSlidingMany = QuantPolicy<2, 256, 4, 2, 1, 3>;
using QuantGlobal = QuantPolicy<8, 512, 1, 4, 2, 3>;
using QuantGlobalMany = QuantPolicy<8, 512, 2, 2, 2, 3>;

}  // namespace gqa
