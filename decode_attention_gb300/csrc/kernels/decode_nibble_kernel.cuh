// Decode attention over the 4-bit cache (nibble_cache.cuh): attn.core of the gemma-4-31B Model
// Spec for one new token per sequence.
//
// Mathematics.  With x_s = log2(e) <q, k_s> the weights are 2^(x_s - M); o = sum of weights times v_s
// over the sum of weights, for any M.  M is a whole number, set 8 below a maximum (rounded up, so that
// from 2^24 on, where floats have a spacing above 1, it is at most 8 below) and kept until a weight
// would pass 2^15: the accumulators are rescaled by powers of two, and seldom.  Weights lie in
// (0, 2^15], where f16 hi + lo parts hold them to 22 bits, or to 2^-25 of a unit, 2^-32 of the largest.
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
//           chunks (16 bytes, 32 channels, one scale) t and t + 4 of rows g and g + 8; what order the
//           channels take in k does not matter, q's B fragments take the same
//   P.V     O^T[c, h] += V^T[c, pos] P[pos, h]: lane (g, t) reads the chunk g from the rows of its
//           four positions, a byte permute pairs positions, and code 2m (2m + 1) of every chunk is
//           the row g (g + 8) of the m-th tile.  movmatrix turns the weights from the scores'
//           layout into B fragments.  At g = 2 the hi and lo parts of P are columns of one mma; at
//           g = 8 they are two mma.
// An mma truncates its sum, so long chains of them drift: a block's products start from zero and
// are added to the accumulators by ordinary additions.
//
// Work split and timeouts are those of decode_quant_kernel.cuh: a persistent CTA per SM, a plan built
// from seq_lens on the device, pieces of whole blocks, several units per CTA with a schedule each, NC
// warps of a unit (at g = 8 pairs, a plane each) on a block each with a ring of slots of their
// own, states merged through shared memory at a piece's end, split segments by the combine kernel.  A
// slot is one block of K, V and scales: one bulk copy per plane of exactly the attended rows.
// A slot is free when its warps' loads are done: each lane's fence between the proxies stands ahead of the
// arrival, as a copy may overtake loads that are only issued.  (Without it one call in some 1000 over large
// sliding batches found other codes in part of a row; it takes no time, 66.9 / 693 us in the cases below.)
//
// Bound by latency at few warps: no unit is full.  Three consumer warps per scheduler (160 registers each,
// what the producers leave) issue in 0.58 of the cycles, some 640 instructions for a block of a plane (4352
// bytes), of which 128 mask codes, 128 make values, 48 (32) are mma; no pipe is busy more than 0.46, and HBM,
// which could bring a block to each scheduler every 740 cycles, half of the time.  Between two instructions of
// a warp pass 6.3 cycles.  At g = 2 a fifth of them are waits at barriers and for loads from global
// memory, which are the starts and ends of pieces, 1.6 fixed latencies and busy pipes; at g = 8 these are
// 2.1, the others 0.7.  Four warps, at 112 registers, took 70 / 709 us where three took 67 / 698.  What the
// steps took, GPU time of decode_sliding_b64_paged / decode_global_b16_long: 8 consumer warps and the mask and
// the constant of 1024 + u two operations, 85 / 990 us; 12 warps 86 / 860; one operation 80 / 766; producers that fill
// their rings lane by lane and sleep 76 / 785; q's fragments in shared memory (fewer spills) 71 / 755; a
// merge that reads whole states 72 / 718; P.V in two halves (less registers), the pair's exchange apart
// from the tiles 69 / 732; a warp's index that the compiler sees to be one (no spills, plain branches) 67 / 698.
// Tried: codes of K masked into the mma as subnormal numbers u 2^-24, a chunk's products scaled in fp32
// afterwards and the 8 taken off with sums of q, 68 / 711, but sums several times the scores, whose
// rounding is twice the error (1.0e-6 for 4.6e-7 in a plain fp32 evaluation, 3.1e-7 here); P.V of one
// block between another's scores, 81 / 874 (slots are held longer); sums kept in the mma's accumulator
// and flushed every 16 blocks, 75 / 711; four chains of scores in place of two 67 / 711; the first codes of V
// loaded ahead of the weights 67 / 700, and 151 us for 149 over 64 sequences of up to 8192 positions.
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
    // Few positions in long segments are better off with fewer units, whose pieces are longer (in blocks, a
    // piece's cost among them).  One, two and three to a CTA, us: slidingDecodeGQA, one sequence of 400
    // positions 7.7 8.4 8.5, of the whole window 8.5 8.5 9.6, two 9.7 9.6 10.8, five 13.5 12.8 13.6, eight
    // 17.3 15.9 16.1; decodeGQA, one of 2048 9.9 11.8 13.7, of 16384 20.4 19.4 20.6, of 32768 31.9 27.5 27.1.
    // Segments of 100 positions, 16 sequences: 11.3 11.7 10.5 and 11.5 12.0 11.2.  (The segments of empty
    // sequences count: a window beside 15 of them takes three units, and 11.9 with their zeros, alone 8.4.)
    static constexpr int kUnitsPerCta = 3;
    __device__ static uint32_t units(uint32_t ctas, uint32_t tiles, uint32_t segments) {
        if (tiles <= 14 * ctas && tiles >= (kExtra + 16) * segments) return ctas;
        if (tiles <= 48 * ctas && tiles > (kExtra + 32) * segments) return 2 * ctas;
        return kUnitsPerCta * ctas;
    }
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
    static constexpr int kConsumers = GROUPS * GW;       // whole warpgroups; then one of producers
    static constexpr int kThreads = (kConsumers + 4) * 32;
    static constexpr int kLaunchRegs = 128, kConsumerRegs = 160, kProducerRegs = 32;
    static constexpr bool kSplitCols = G == 2;           // hi and lo parts of P in one mma
    static constexpr int kLanes = kSplitCols ? 16 : 32;  // lanes whose accumulators are no copies
    static constexpr int kRound = kSplitCols ? 8 : 4;    // tiles merged at a time
    static_assert((G == 2 || G == 8) && (NC == 2 || NC == 4), "shape");
    static_assert(kThreads >= kPlanWarps * 32, "the plan takes eight warps");
    static_assert(kConsumers % 4 == 0 && GROUPS <= 4, "warpgroups");
    static_assert(GROUPS == NibblePlanTuning::kUnitsPerCta, "units");
    static_assert(kConsumers * kConsumerRegs + 4 * kProducerRegs <= (kConsumers + 4) * kLaunchRegs &&
                      kThreads * kLaunchRegs <= 65536,
                  "no share waits for registers that the block was not launched with");
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
    };
    uint8_t kv[Pol::GROUPS][Pol::NC * Pol::RING][Pol::SPLIT][kTileBytes];   // [slot][plane][16 rows][272 B]
    alignas(16) float4 sum[Pol::GROUPS][Pol::SPLIT][Pol::NC][Pol::kRound][Pol::kLanes];   // accumulators being merged
    uint4 q[Pol::GROUPS][Pol::SPLIT][8][32];   // B fragments of q (NibbleConsumer::begin)
    float4 cross[Pol::GROUPS][Pol::NC][2][Pol::SPLIT][32];   // scores on their way between a pair's warps
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
    // base: 0x64006400 in a register
    __device__ __forceinline__ uint32_t low(uint32_t w, uint32_t base) const {
        return ptx::f16x2_fma(ptx::and_or<0x000f000fu>(w, base), s, less);
    }
    __device__ __forceinline__ uint32_t high(uint32_t w, uint32_t base) const {
        return ptx::f16x2_fma(ptx::and_or<0x00f000f0u>(w, base), s16, less16);
    }
};

// wait_bounded (decode_kernel.cuh) for waits that are long as a rule: the thread is suspended between
// its looks at the barrier.  (Producers that wait for a slot took a fifth of the issue slots.)
__device__ __forceinline__ bool wait_suspended(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                               uint32_t* flags, uint64_t limit_ns = kWaitLimitNs) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t round = 0;; ++round) {
        if (ptx::mbar_try_wait_for(bar, parity, 20000u)) return true;
        if (*abort_flag) return false;
        // time limit, with an iteration cap in case the timer does not advance
        if (ptx::globaltimer_ns() - t0 > limit_ns || round > kWaitMaxRounds) {
            *abort_flag = 1;
            atomicOr(flags, kFlagWaitTimeout);
            return false;
        }
    }
}

template <class Pol>
struct NibbleConsumer {
    static constexpr int G = Pol::G, D = Pol::D;
    static constexpr int kTiles = kNibblePlane / 16;
    static constexpr float kBase = 8.0f;    // exponent of the largest weight when M is set
    static constexpr float kTop = 15.0f;    // largest exponent of a weight (f16 ends at 2^16)
    static constexpr float kLowest = -3.402823466e38f;   // M of no score yet

    // Rows that a lane's B fragments of P.V stand for, less 2t.
    __device__ static constexpr int place(int j) { return j < 2 ? j : 6 + j; }   // 0, 1, 8, 9

    float q_undo[2];             // undo q's scaling for columns 2t and 2t + 1, times log2(e)
    // tile m: channels 2n (0, 1) and 2n + 1 (2, 3) of chunk g, n = m or, where g & 2, m ^ 8; columns 2t, 2t + 1
    float acc[kTiles][4];
    float ms[2];                 // M of columns 2t, 2t + 1
    float l[2];                  // this lane's share of their normalisers
    uint32_t base;               // 0x64006400

    // q_heads: [G][D] bf16 in global memory; `half`: which plane of the head is this warp's; q_at: where
    // the plane's B fragments of q (column g = head g % G) stand in shared memory.  The unit's warps write
    // a part each.
    __device__ __forceinline__ void begin(const __nv_bfloat16* q_heads, uint32_t q_at, int own, int half,
                                          int lane) {
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
        const float f = __int_as_float((14 - e + 127) << 23);   // 2^(14 - e)
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // pairs of channels (0, 4), (1, 5), (2, 6), (3, 7)
            if (i % Pol::NC != own) continue;
            ptx::sts128(q_at + i * 512 + lane * 16,
                        ptx::f16x2_pack(bf16lo(raw[i].x) * f, bf16lo(raw[i].z) * f),
                        ptx::f16x2_pack(bf16hi(raw[i].x) * f, bf16hi(raw[i].z) * f),
                        ptx::f16x2_pack(bf16lo(raw[i].y) * f, bf16lo(raw[i].w) * f),
                        ptx::f16x2_pack(bf16hi(raw[i].y) * f, bf16hi(raw[i].w) * f));
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
        base = ptx::in_register(0x64006400u);
    }

    // This plane's share of a block's scores in units of log2: rows g (0, 1) and g + 8 (2, 3),
    // columns 2t, 2t + 1.
    __device__ __forceinline__ void scores(uint32_t tile, uint32_t q_at, float (&z)[4], int lane) {
        const int g = lane >> 2, t = lane & 3;
        const uint32_t row = tile + g * kNibbleRow;
        constexpr uint32_t k8 = 8 * kNibbleRow;
        float c[2][4];   // two chains
#pragma unroll
        for (int i = 0; i < 2; ++i)
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
                const uint4 q = ptx::lds128(q_at + (4 * i + w) * 512 + lane * 16);
                ptx::mma_f16_16816(c[w & 1], fa.low(wa[w], base), fb.low(wb[w], base), fa.high(wa[w], base),
                                   fb.high(wb[w], base), q.x, q.y);
                const uint32_t ha = wa[w] >> 8, hb = wb[w] >> 8;
                ptx::mma_f16_16816(c[w & 1], fa.low(ha, base), fb.low(hb, base), fa.high(ha, base),
                                   fb.high(hb, base), q.z, q.w);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = (c[0][i] + c[1][i]) * q_undo[i & 1];
    }

    // The accumulators of columns 2t and 2t + 1 times a and b.
    __device__ __forceinline__ void scale_by(float a, float b) {
        const uint64_t f = ptx::f2_pack(a, b);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const float2 x = ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(acc[i][j], acc[i][j + 1]), f));
                acc[i][j] = x.x;
                acc[i][j + 1] = x.y;
            }
        }
    }

    // The rest of a block, from its scores: weights, M, l, and P.V for this warp's plane.  Rows
    // [first, last) are attended; bad: their page does not exist, and their weights are NaN.
    __device__ __forceinline__ void weigh(float (&x)[4], uint32_t tile, int first, int last, bool bad,
                                          int lane) {
        const int g = lane >> 2, t = lane & 3;
        // the scales of chunk g in positions 2t, 2t + 1, 2t + 8, 2t + 9
        const uint32_t row = tile + 2 * t * kNibbleRow;
        uint32_t sc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[j] = ptx::lds8(row + place(j) * kNibbleRow + kNibbleScales + 8 + g);
        if (first > 0 || last < kNibblePage || bad) {
            // rows outside the range weigh 2^-inf, and as they hold anything, and 0 * NaN is NaN, their
            // scales are taken as 0
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pos = g + 8 * (i >> 1);
                x[i] = pos >= first && pos < last ? (bad ? __uint_as_float(0x7fc00000u) : x[i]) : -INFINITY;
                if (2 * t + place(i) < first || 2 * t + place(i) >= last) sc[i] = 0;
            }
        }
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = x[i] - ms[i & 1];
        // M moves only when a weight would pass 2^kTop (and on the first block)
        const float ym = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
        if (__any_sync(0xffffffffu, ym > kTop)) {
            float alpha[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float top = fmaxf(x[j], x[j + 2]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const float m = fmaxf(ms[j], __fadd_ru(ceilf(top), -kBase));   // (never of a NaN)
                alpha[j] = ptx::ex2(ms[j] - m);
                ms[j] = m;
                l[j] *= alpha[j];
                y[j] = x[j] - m;
                y[j + 2] = x[j + 2] - m;
            }
            scale_by(alpha[0], alpha[1]);
        }
        uint32_t hi[2], lo[2];   // B fragments: column g, positions 2t, 2t + 1 of each half
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
        const NibbleScale f0(__byte_perm(sc[0], sc[1], 0x5410) << 7), f1(__byte_perm(sc[2], sc[3], 0x5410) << 7);
        // Half a chunk at a time (whole ones took 16 registers more).  Lanes (g, t) and (g + 2, t - 1) share
        // banks: one of them takes its halves the other way round.
        const uint32_t codes = row + kNibblePlane / 2 + 16 * g, flip = 4 * (g & 2);   // 0 or 8 bytes
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = ptx::lds64(codes + place(j) * kNibbleRow + (half ? 8 - flip : flip));
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {   // codes 2k, 2k + 1 of a word
                    uint32_t a = __byte_perm(i ? v[0].y : v[0].x, i ? v[1].y : v[1].x, k < 2 ? 0x5410 : 0x7632);
                    uint32_t b = __byte_perm(i ? v[2].y : v[2].x, i ? v[3].y : v[3].x, k < 2 ? 0x5410 : 0x7632);
                    if (k & 1) {
                        a >>= 8;
                        b >>= 8;
                    }
                    const uint32_t a0 = f0.low(a, base), a1 = f0.high(a, base);
                    const uint32_t a2 = f1.low(b, base), a3 = f1.high(b, base);
                    float d[4];
                    if (Pol::kSplitCols) {
                        ptx::mma_f16_16816_zero(d, a0, a1, a2, a3, hi[0], hi[1]);
                    } else {
                        ptx::mma_f16_16816_zero(d, a0, a1, a2, a3, lo[0], lo[1]);
                        ptx::mma_f16_16816(d, a0, a1, a2, a3, hi[0], hi[1]);
                    }
                    float (&sum)[4] = acc[8 * half + 4 * i + k];
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        const float2 x = ptx::f2_unpack(
                            ptx::f2_add(ptx::f2_pack(sum[j], sum[j + 1]), ptx::f2_pack(d[j], d[j + 1])));
                        sum[j] = x.x;
                        sum[j + 1] = x.y;
                    }
                }
        }
    }

    // Tiles [r kRound, (r + 1) kRound) of the accumulators to this warp's place in shared memory.  (At
    // kSplitCols the columns 4 .. 7 are copies.)
    __device__ __forceinline__ void put(float4 (*sum)[Pol::kLanes], int r, int lane) {
        if (Pol::kSplitCols && (lane & 2)) return;
        const int at = Pol::kSplitCols ? (lane >> 2) * 2 + (lane & 1) : lane;
#pragma unroll
        for (int i = 0; i < Pol::kRound; ++i) {
            const float (&x)[4] = acc[r * Pol::kRound + i];
            sum[i][at] = make_float4(x[0], x[1], x[2], x[3]);
        }
    }

    // The end of this warp's share of a piece: M and l of its columns to wm and wl (the planes of a
    // head hold the same), and the first round's tiles.
    __device__ __forceinline__ void finish(typename NibbleSmem<Pol>::Unit& un, float4 (*sum)[Pol::kLanes],
                                           int own, int half, int lane) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float ls = l[j];
            ls += __shfl_xor_sync(0xffffffffu, ls, 4);
            ls += __shfl_xor_sync(0xffffffffu, ls, 8);
            ls += __shfl_xor_sync(0xffffffffu, ls, 16);
            if (half == 0 && lane < 4) {
                un.wm[own][2 * lane + j] = ms[j];
                un.wl[own][2 * lane + j] = ls;
            }
        }
        put(sum, 0, lane);
    }

    // Merge of the warps' accumulators (of this plane): the output (slot < 0; the piece is the whole
    // segment) or the partial (acc, m, l) at workspace slot `slot`.  The M are whole numbers, so the factors
    // 2^(M_w - M) are exact.  Called by all consumer warps, after finish() and a barrier.
    __device__ __forceinline__ void merge(const typename NibbleSmem<Pol>::Unit& un,
                                          float4 (*sums)[Pol::kRound][Pol::kLanes], const DecodeParams& p,
                                          size_t out_base, int slot, int bar, int own, int half, int lane) {
        const int h0 = Pol::kSplitCols ? 0 : 2 * (lane & 3);
        float f[2][Pol::NC], scale[2];   // of heads h0 and h0 + 1
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float top = -INFINITY, ls = 0.0f;
#pragma unroll
            for (int w = 0; w < Pol::NC; ++w) top = fmaxf(top, un.wm[w][h0 + j]);
#pragma unroll
            for (int w = 0; w < Pol::NC; ++w) {   // (a warp without a score weighs 0 beside one with)
                f[j][w] = ptx::ex2(un.wm[w][h0 + j] - top);
                ls = fmaf(f[j][w], un.wl[w][h0 + j], ls);
            }
            scale[j] = slot < 0 ? 1.0f / ls : 1.0f;
            if (slot >= 0 && half == 0 && own == 0 && lane < (Pol::kSplitCols ? 1 : 4))
                *reinterpret_cast<float2*>(p.ws_ml + (static_cast<size_t>(slot) * G + h0 + j) * 2) =
                    make_float2(top, ls);
        }
        const bool floats = slot >= 0 || p.out_f32;
        float* to = slot < 0 ? static_cast<float*>(p.out) + out_base
                             : p.ws_acc + static_cast<size_t>(slot) * G * D;
        // a warp reads four tiles together, whose channels fill sectors: of all g (at kSplitCols) or of two
        constexpr int kSteps = Pol::kRound / 4 * (Pol::kSplitCols ? 1 : 4);
#pragma unroll
        for (int r = 0; r < kTiles / Pol::kRound; ++r) {
            if (r > 0) {
                ptx::named_barrier_sync(bar, Pol::GW * 32);
                put(sums[own], r, lane);
                ptx::named_barrier_sync(bar, Pol::GW * 32);
            }
#pragma unroll
            for (int step = own; step < kSteps; step += Pol::NC) {
                const int i = 4 * (Pol::kSplitCols ? step : step >> 2) + (lane >> 3);
                const int g = Pol::kSplitCols ? lane & 7 : 2 * (step & 3) + ((lane >> 2) & 1);
                float2 o[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};   // channels 2m, 2m + 1 of the chunk, of both heads
#pragma unroll
                for (int w = 0; w < Pol::NC; ++w) {
                    float4 x;
                    if (Pol::kSplitCols) {   // columns of the hi parts and of the lo parts
                        const float4 hi = sums[w][i][2 * g], lo = sums[w][i][2 * g + 1];
                        x = make_float4(hi.x + lo.x, hi.y + lo.y, hi.z + lo.z, hi.w + lo.w);
                    } else {
                        x = sums[w][i][4 * g + (lane & 3)];
                    }
                    o[0].x = fmaf(x.x, f[0][w], o[0].x);
                    o[1].x = fmaf(x.y, f[1][w], o[1].x);
                    o[0].y = fmaf(x.z, f[0][w], o[0].y);
                    o[1].y = fmaf(x.w, f[1][w], o[1].y);
                }
                const int m = (r * Pol::kRound + i) ^ (4 * (g & 2));   // (weigh()'s halves)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const size_t at = static_cast<size_t>(h0 + j) * D + half * kNibblePlane + 32 * g + 2 * m;
                    const float2 y = make_float2(o[j].x * scale[j], o[j].y * scale[j]);
                    if (floats)
                        *reinterpret_cast<float2*>(to + at) = y;
                    else
                        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + out_base + at) =
                            __floats2bfloat162_rn(y.x, y.y);
                }
            }
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
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // (branches on it are a warp's)
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
        ptx::mbar_init(ptx::smem_addr(&un.piece_empty), Pol::GW);   // who reads it
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

    if (tid == 0) {
        const int units = static_cast<int>(NibblePlanTuning::units(
            static_cast<uint32_t>(ctas), static_cast<uint32_t>(pl.n_static), static_cast<uint32_t>(B * KVH)));
        if (units < pl.g_eff) pl.g_eff = units;
    }
    __syncthreads();

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
    const int group = warp < Pol::kConsumers ? warp / Pol::GW : warp - Pol::kConsumers;
    const int unit = cta + ctas * group;
    const bool idle = group >= GROUPS || unit >= pl.g_eff;
    typename NibbleSmem<Pol>::Unit& un = sm.unit[idle ? 0 : group];
    const uint32_t kv_base = ptx::smem_addr(&sm.kv[idle ? 0 : group][0][0][0]);
    const uint32_t piece_full = ptx::smem_addr(&un.piece_full), piece_empty = ptx::smem_addr(&un.piece_empty);

    if (warp >= Pol::kConsumers) {
        // ======== producer: a warp per unit ========
        // All lanes walk the schedule; lane 0 publishes each piece, lane k fills ring k.
        ptx::fewer_registers<Pol::kProducerRegs>();
        if (idle) return;
        const uint32_t edge = static_cast<uint32_t>(static_unit_begin(pl, unit + (lane & 1)));
        StaticWalk<NibblePlanTuning> walk(pl, B, __shfl_sync(0xffffffffu, edge, 0),
                                          __shfl_sync(0xffffffffu, edge, 1));
        const uint64_t policy = ptx::policy_evict_first();
        ptx::fence_proxy_async_smem();   // the plan used the slots
        const size_t plane = static_cast<size_t>(kPaged ? kBlock : np.rows) * kNibbleRow;   // bytes of a plane
        const int ring = lane < NC ? lane : 0;
        uint32_t filled = 0;   // blocks sent to this lane's ring
        int turn = 0;          // its next slot, and how often the ring went round
        uint32_t laps = 0;
        bool ok = true;
        for (uint32_t n = 0;; ++n) {
            // the description is free once the consumers have read the one before
            if (ok) ok = wait_suspended(piece_empty, (n & 1u) ^ 1u, &sm.abort_flag, p.ws_flags);
            if (!__all_sync(0xffffffffu, ok)) break;
            Piece w;
            bool whole = false;   // the piece is its segment
            if (walk.next(pl, KVH, unit, w)) {
                whole = w.p1 - w.p0 == pl.n[w.b];
            } else {
                int claimed = pl.n_dyn;
                if (pl.n_dyn > 0) {
                    if (lane == 0) claimed = static_cast<int>(atomicAdd(p.ws_claim, 1u));
                    claimed = __shfl_sync(0xffffffffu, claimed, 0);
                }
                if (!claim_piece(pl, p, claimed, w)) {
                    if (lane == 0) {
                        un.piece.done = 1;
                        ptx::mbar_arrive(piece_full);
                    }
                    break;
                }
            }
            const int hi = sm.len[w.b], lo = p.window > 0 && hi > p.window ? hi - p.window : 0;
            if (lane == 0) {
                un.piece.b = w.b;
                un.piece.kvh = w.kvh;
                un.piece.p0 = w.p0;
                un.piece.p1 = w.p1;
                un.piece.lo = lo;
                un.piece.hi = hi;
                un.piece.slot = whole ? -1 : w.slot;
                un.piece.done = 0;
                ptx::mbar_arrive(piece_full);
            }
            if (lane >= NC) continue;
            int blk = w.p0 / kBlock + lane;
            const int blk1 = w.p1 / kBlock;
            const int32_t* bt_row =
                kPaged ? p.block_table + static_cast<size_t>(w.b) * p.max_pages : nullptr;
            // the head's planes of sequence b, or of page 0
            const uint8_t* head =
                np.kv + (static_cast<size_t>(kPaged ? 0 : w.b) * KVH + w.kvh) * SPLIT * plane;
            int page = kPaged && blk < blk1 ? __ldg(bt_row + blk) : 0;   // (loaded one round ahead)
            for (; blk < blk1; blk += NC) {
                const int s = ring * RING + turn;
                ok = wait_suspended(ptx::smem_addr(&un.empty[s]), (laps & 1u) ^ 1u, &sm.abort_flag, p.ws_flags);
                if (!ok) break;
                const uint32_t full_bar = ptx::smem_addr(&un.full[s]);
                // the attended rows of the block (at least one), no others
                const int r0 = max(lo - blk * kBlock, 0), r1 = min(hi - blk * kBlock, kBlock);
                const uint32_t bytes = static_cast<uint32_t>(r1 - r0) * kNibbleRow;
                const uint8_t* src = head;
                bool bad = false;
                if (kPaged) {
                    bad = page < 0 || page >= p.num_pages;
                    src += (static_cast<size_t>(page) * KVH * SPLIT * kBlock + r0) * kNibbleRow;
                    un.bad[s] = bad;
                    if (blk + NC < blk1) page = __ldg(bt_row + blk + NC);
                } else {
                    src += (static_cast<size_t>(blk) * kBlock + r0) * kNibbleRow;
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
                ++filled;
                if (++turn == RING) {
                    turn = 0;
                    ++laps;
                }
                if ((p.test_flags & kTestStall) && group == 0 && lane == 0 && filled == 1) {
                    ok = wait_suspended(ptx::smem_addr(&sm.stall_bar), 0u, &sm.abort_flag, p.ws_flags, kTestStallNs);
                    if (!ok) break;
                }
            }
        }
        // every copy issued lands before the CTA can exit (its consumer may have given up)
        for (uint32_t f = filled > RING ? filled - RING : 0u; f < filled; ++f)
            wait_drain(ptx::smem_addr(&un.full[ring * RING + f % RING]), (f / RING) & 1u);
        return;
    }

    // ===================== consumers =====================
    ptx::more_registers<Pol::kConsumerRegs>();
    if (idle) return;
    // Every warp of a unit passes the same barriers for every piece, whatever its waits return:
    // one that gave up (or saw the end) makes all of them leave at the piece's last barrier.
    const int gwarp = warp - group * Pol::GW, own = gwarp / SPLIT, half = gwarp % SPLIT;
    const int bar = 1 + group, pair_bar = 1 + GROUPS + group * NC + own;
    const uint32_t q_at = ptx::smem_addr(&sm.q[group][half][0][0]);
    float4 (*sums)[Pol::kRound][Pol::kLanes] = sm.sum[group][half];
    NibbleConsumer<Pol> c;
    int turn = 0;         // the next slot of this warp's ring, and how often the ring went round
    uint32_t laps = 0;
    uint32_t swaps = 0;   // blocks whose scores crossed over
    for (uint32_t n = 0;; ++n) {
        const bool there = __all_sync(0xffffffffu, wait_bounded(piece_full, n & 1u, &sm.abort_flag, p.ws_flags));
        BlockPiece pc{};
        pc.done = 1;
        if (there) pc = un.piece;
        bool gone = pc.done != 0;
        __syncwarp();
        const size_t out_base = (static_cast<size_t>(pc.b) * H + pc.kvh * G) * D;
        if (!gone) {
            if (lane == 0) ptx::mbar_arrive(piece_empty);   // every lane has read it
            c.begin(p.q + out_base, q_at, own, half, lane);
        }
        if (ptx::named_barrier_or(bar, Pol::GW * 32, gone)) break;   // (q is there)
        {
            // (block i of a piece is warp i % NC's, whatever came before: the order of the sums
            // does not depend on the schedule)
            for (int pos = pc.p0 + own * kBlock; pos < pc.p1; pos += NC * kBlock) {
                const int s = own * RING + turn;
                gone = !__all_sync(0xffffffffu, wait_bounded(ptx::smem_addr(&un.full[s]), laps & 1u,
                                                             &sm.abort_flag, p.ws_flags));
                const uint32_t tile = kv_base + (s * SPLIT + half) * kTileBytes;
                float z[4];
                if (SPLIT == 1) {
                    if (gone) break;
                    c.scores(tile, q_at, z, lane);
                } else {
                    // the planes' scores cross over (in two places in turn: a warp may be a block ahead)
                    float4* cross = sm.cross[group][own][swaps++ & 1u][0];
                    if (!gone) {
                        c.scores(tile, q_at, z, lane);
                        cross[half * 32 + lane] = make_float4(z[0], z[1], z[2], z[3]);
                    }
                    gone = ptx::named_barrier_or(pair_bar, 2 * 32, gone);
                    if (gone) break;
                    const float4 o = cross[(1 - half) * 32 + lane];
                    z[0] += o.x;
                    z[1] += o.y;
                    z[2] += o.z;
                    z[3] += o.w;
                }
                c.weigh(z, tile, pc.lo - pos, pc.hi - pos, kPaged && un.bad[s] != 0, lane);
                ptx::fence_proxy_async_smem();   // this lane's loads, before the next copy into the slot
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&un.empty[s]));
                if (++turn == RING) {
                    turn = 0;
                    ++laps;
                }
            }
            c.finish(un, sums[own], own, half, lane);
        }
        if (ptx::named_barrier_or(bar, Pol::GW * 32, gone)) break;
        c.merge(un, sums, p, out_base, pc.slot, bar, own, half, lane);
        // (the sums are written again after the barrier that begins the next piece)
    }
}

// slidingDecodeGQA and decodeGQA
using NibbleSliding = NibblePolicy<2, 3, 4, 3>;
using NibbleGlobal = NibblePolicy<8, 3, 2, 2>;

}  // namespace gqa
