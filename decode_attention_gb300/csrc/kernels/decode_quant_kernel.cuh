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
// hold them to 22 bits.
//
// Both contractions run as warp-level f16 mma (m16n8k16, fp32 accumulate) with the cache
// as the A operand, so that the g <= 8 query heads of a KV head fill the 8 columns of B
// and no row is idle.  e4m3 widens to f16 exactly, two codes per instruction.  q is scaled
// by a power of two per head, which makes its bf16 values exact in f16 down to 2^-30 of
// the largest.
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
// A warp works on whole blocks by itself: its own M, l and D x 8 accumulators, no exchange
// with the other warps until the piece ends, when the 8 states are merged through shared
// memory.  (With the 8 warps sharing each tile, one part of the dims each and a score tile
// between the contractions, every warp repeats the softmax of all positions: 1370
// instructions per warp and 128 positions at g = 2 against ~300 here.)
//
// Work split and timeouts are those of decode_kernel.cuh: a persistent CTA per SM, a plan
// built from seq_lens on the device; split segments are merged by the combine kernel (merged
// by the CTA of the last partial, as bf16 sliding calls are, every batch size was slower:
// sliding windows of 1024, B = 1 11.7 us against 10.9, B = 64 96 against 87).  Pieces start and end on
// blocks.  The consumer warps form groups of NC; each group is a unit of the plan with a
// schedule of its own, so that one group computes while another merges its piece (g = 2:
// two groups of 4).  At g = 8 the D x 8 accumulators of a block would take 128 registers and
// leave one warp per scheduler; there two warps share a block, half of D each, and add their
// halves of the scores (one group of 4 pairs).  A group has two
// producer threads: the first walks its schedule and publishes pieces, both stream K and V
// with TMA, one slot per block.  Block i of a piece goes to warp i % NC of the group, into
// that warp's own ring of slots.  (A ring shared by the warps would let a warp wait on a slot's
// barrier two fills ahead of its last completion, which a parity cannot tell apart.)
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

// The plan's constants for this kernel, whose pieces cost 2-3 us of a group (q, merge,
// barriers) while 8-bit rows stream twice as fast as bf16 ones: a piece counts as kExtra
// blocks, and dynamic chunks are fewer and begin at four times the work.  Measured with 4
// extra blocks, 256 positions and 8 chunks per CTA, and with these: decode_global_b8 37.3 and
// 31.7 us, decode_sliding_b64_paged 89.4 and 84.6 us, decode_global_b64_paged 350 and 341 us.
struct QuantPlanTuning {
    static constexpr int kAlign = kQuantBlock, kExtra = 12;
    static constexpr int kMinShare = 1024, kChunksPerCta = 4;
};

template <int kG, int kD, int kGroups, int kSplitD, int kRing>
struct QuantPolicy {
    static constexpr int G = kG, D = kD, GROUPS = kGroups, RING = kRing;
    static constexpr int NC = 4;                         // blocks a group works on at a time
    static constexpr int SPLIT = kSplitD;                // warps per block, D / SPLIT dims each
    static constexpr int GW = NC * SPLIT;                // consumer warps per group
    static constexpr int SLOTS = NC * RING;              // of a group: one block of K and V each
    static constexpr int kConsumers = GROUPS * GW;
    static constexpr int kWarps = kConsumers + 2 * GROUPS;
    static constexpr int kThreads = (kWarps < kPlanWarps ? kPlanWarps : kWarps) * 32;
    static constexpr int kUnits = D / 16;                // 16-dim steps
    static constexpr int kOwnUnits = kUnits / SPLIT;     // those of one warp
    static constexpr bool kSplitCols = G == 2;           // hi and lo parts of P in one mma
    static constexpr int kMergeDims = 128 / SPLIT;       // dims of a warp merged per round
    static constexpr int kMergeStride = kMergeDims + 4;  // conflict-free float2 stores
    static constexpr int kMergeCols = kSplitCols ? 2 * G : G;
    static constexpr int kQStride = D + 16;              // padded row of q: conflict-free 8-byte loads
    static_assert((G == 2 || G == 8) && kOwnUnits % 4 == 0 && (D / SPLIT) % kMergeDims == 0, "shape");
    static_assert(SPLIT == 1 || SPLIT == 2, "a block is one warp's or two's");
};

// One piece of work, published with its q.
struct QuantPiece {
    int b, kvh;
    int p0, p1;     // positions, whole blocks
    int lo, hi;     // attended positions of the sequence
    int slot;       // workspace slot of the partial
    int parts;      // partials of the segment (1: the piece is the whole segment)
    int done;       // no more pieces
};

template <class Pol>
struct alignas(1024) QuantSmem {
    static constexpr int kTileBytes = kQuantBlock * Pol::D;
    struct Group {
        alignas(8) uint64_t full[Pol::SLOTS];
        alignas(8) uint64_t empty[Pol::SLOTS];
        alignas(8) uint64_t q_full, q_empty;
        float scales[Pol::SLOTS][2];
        int bad[Pol::SLOTS];                     // the block's page id is out of range
        QuantPiece piece;
        // a piece's q fragments are last read before its merge, whose last barrier precedes the
        // next piece's
        union alignas(16) {
            uint2 q_frag[Pol::kUnits][32];                      // B fragments of q (column g = head g % G)
            float wacc[Pol::SPLIT][Pol::NC][Pol::kMergeCols][Pol::kMergeStride];   // dims being merged
        };
        alignas(128) __nv_bfloat16 q[Pol::G][Pol::kQStride];
        float wm[Pol::NC][8], wl[Pol::NC][8];    // M and l per column of each warp (pair)
    };
    uint8_t kv[Pol::GROUPS][Pol::SLOTS][2][kTileBytes];   // [slot][K, V][chunk][16 rows][128 B]
    Group group[Pol::GROUPS];
    alignas(8) uint64_t stall_bar;               // kTestStall: a barrier nothing completes
    PlanSmem plan;
    int len[kMaxBatch];                          // clamped lengths
    int abort_flag;
};

template <class Pol>
struct QuantConsumer {
    static constexpr int G = Pol::G, D = Pol::D, kUnits = Pol::kUnits, kOwnUnits = Pol::kOwnUnits;
    static constexpr float kTop = 15.0f;    // largest exponent of a weight (f16 ends at 2^16)
    static constexpr float kRoom = 3.0f;    // binades left above the maximum when M is set

    float q_factor[2];           // undo q's scaling for columns 2t and 2t + 1, times log2(e)
    float acc[kOwnUnits][4];     // rows: dims 2g (0, 1) and 2g + 1 (2, 3); columns 2t, 2t + 1
    float m[2];                  // M of columns 2t, 2t + 1
    float l[2];                  // this lane's share of their normalisers

    // Byte address of 16-byte unit `unit` of row r of a block.
    __device__ static __forceinline__ uint32_t unit_addr(uint32_t block, int r, int unit) {
        return block + (unit >> 3) * 2048 + r * 128 + (((unit & 7) ^ (r & 7)) << 4);
    }

    // q_heads: [G][kQStride] bf16 in shared memory.  Each warp makes its share of the fragments (a
    // barrier follows).
    __device__ __forceinline__ void begin(const __nv_bfloat16* q_heads, uint2 (*frag)[32], int warp,
                                          int lane) {
        const int g = lane >> 2, t = lane & 3;
        const __nv_bfloat16* row = q_heads + (g % G) * Pol::kQStride + 4 * t;
        uint32_t top = 0;   // largest |q|: the bits of |bf16| order like the values
#pragma unroll 8
        for (int u = 0; u < kUnits; ++u) {
            const uint2 w = *reinterpret_cast<const uint2*>(row + u * 16);
            top = __vmaxu2(top, __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu));
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(static_cast<int>(top >> 7) - 127, -100);   // |q| < 2^(e + 1)
        const float f = pow2f(14 - e);
#pragma unroll
        for (int i = 0; i < kUnits / Pol::GW; ++i) {
            const int u = warp * (kUnits / Pol::GW) + i;
            const uint2 w = *reinterpret_cast<const uint2*>(row + u * 16);
            frag[u][lane] = make_uint2(ptx::f16x2_pack(bf16lo(w.x) * f, bf16hi(w.x) * f),
                                       ptx::f16x2_pack(bf16lo(w.y) * f, bf16hi(w.y) * f));
        }
        const float undo = pow2f(e - 14) * kLog2e;
        q_factor[0] = __shfl_sync(0xffffffffu, undo, 8 * t);
        q_factor[1] = __shfl_sync(0xffffffffu, undo, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < kOwnUnits; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
    }

    // This warp's share (`half` of D) of a block's scores, c[i]: rows g (0, 1) and g + 8 (2, 3),
    // columns 2t, 2t + 1.
    __device__ __forceinline__ void scores(uint32_t k_blk, uint32_t q_frag, int half, float (&z)[4],
                                           int lane) {
        const int mat = lane >> 3, r = (mat & 1) * 8 + (lane & 7);
        float c[4][4];   // four independent chains
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i][j] = 0.0f;
        // (unit_addr's chunks: kOwnUnits is a multiple of 8 units or the whole of D)
        const uint32_t k_half = k_blk + half * (kOwnUnits / 8) * 2048;
        const uint32_t q_half = q_frag + half * kOwnUnits * 256;
#pragma unroll
        for (int u = 0; u < kOwnUnits; u += 2) {
            uint32_t a[4];   // rows g, g + 8 of unit u, then of unit u + 1
            ptx::ldmatrix_x4(unit_addr(k_half, r, u + (mat >> 1)), a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint2 q = ptx::lds64(q_half + (u + i) * 256 + lane * 8);
                uint32_t a0, a1, a2, a3;
                ptx::e4m3x4_to_f16x2(a[2 * i], a0, a2);
                ptx::e4m3x4_to_f16x2(a[2 * i + 1], a1, a3);
                ptx::mma_f16_16816(c[(u + i) & 3], a0, a1, a2, a3, q.x, q.y);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = (c[0][i] + c[1][i]) + (c[2][i] + c[3][i]);
    }

    // The rest of a block, from its scores z: weights, M, l, and P.V for this warp's dims.  whole:
    // every row is attended; else rows [first, last) are, and none of them on a bad page.
    template <bool whole>
    __device__ __forceinline__ void weigh(const float (&z)[4], uint32_t v_blk, float k_scale,
                                          float v_scale, int first, int last, bool bad, int half,
                                          int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int mat = lane >> 3, r = (mat & 1) * 8 + (lane & 7);
        // log2 of the weights: y = log2(e) score + ev - M, rows g (0, 1) and g + 8 (2, 3)
        const float fk = pow2f(scale_exponent(k_scale));
        const int ev = scale_exponent(v_scale);
        const float f[2] = {fk * q_factor[0], fk * q_factor[1]};
        // (rows outside the range: 2^-inf)
        const float evf = static_cast<float>(ev);
        bool row_ok[2] = {true, true};
        if (!whole) {
            row_ok[0] = g >= first && g < last;
            row_ok[1] = g + 8 >= first && g + 8 < last;
        }
        auto level = [&](int i, float shift) {
            const float v = fmaf(z[i], f[i & 1], !whole && bad ? __uint_as_float(0x7fc00000u) : shift);
            return row_ok[i >> 1] ? v : -INFINITY;
        };
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = level(i, evf - m[i & 1]);
        }
        // M moves only when a weight would pass 2^kTop (and on the first block, M = -inf)
        const float ym = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
        if (__any_sync(0xffffffffu, ym > kTop)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float top = fmaxf(level(j, evf), level(j + 2, evf));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const float mn = fmaxf(m[j], ceilf(top) - (kTop - kRoom));
                const float alpha = mn == m[j] ? 1.0f : ptx::ex2(m[j] - mn);
                l[j] *= alpha;
#pragma unroll
                for (int i = 0; i < kOwnUnits; ++i) {
                    acc[i][j] *= alpha;
                    acc[i][j + 2] *= alpha;
                }
                m[j] = mn;
                y[j] = level(j, evf - mn);
                y[j + 2] = level(j + 2, evf - mn);
            }
        }
        uint32_t hi[2], lo[2];   // B fragments: column g, positions (2t, 2t + 1) of each half
        const float unscale = pow2f(-ev);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float p0 = ptx::ex2(y[2 * i]), p1 = ptx::ex2(y[2 * i + 1]);
            l[0] = fmaf(p0, unscale, l[0]);
            l[1] = fmaf(p1, unscale, l[1]);
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
        // rows outside the range hold anything: their codes are zeroed (0 * NaN)
        uint32_t mask[2] = {0xffffffffu, 0xffffffffu};
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int pos = 8 * i + 2 * t;
                mask[i] = ((pos >= first && pos < last) ? 0x0000ffffu : 0u) |
                          ((pos + 1 >= first && pos + 1 < last) ? 0xffff0000u : 0u);
                if (bad) mask[i] = 0u;
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
                const uint32_t w0 = whole ? w[2 * i] : w[2 * i] & mask[0];
                const uint32_t w1 = whole ? w[2 * i + 1] : w[2 * i + 1] & mask[1];
                ptx::e4m3x4_to_f16x2(__byte_perm(w0, 0u, 0x3120), a0, a1);
                ptx::e4m3x4_to_f16x2(__byte_perm(w1, 0u, 0x3120), a2, a3);
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

    // Merge of the warps' states: the output (slot < 0; the piece is the whole segment) or
    // the partial (acc, m, l) at workspace slot `slot`.  The M are whole numbers, so the
    // factors 2^(M_w - M) are exact.  Called by all consumer warps, after a barrier that
    // follows the stores of wm and wl.
    __device__ __forceinline__ void merge(typename QuantSmem<Pol>::Group& sm, const DecodeParams& p,
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
            // (a warp without a finite score weighs 0; its NaN stay)
            const float f = m[j] == -INFINITY ? 0.0f : ptx::ex2(m[j] - top);
#pragma unroll
            for (int i = 0; i < kOwnUnits; ++i) {
                acc[i][j] *= f;
                acc[i][j + 2] *= f;
            }
        }
        float top[G / kHeadStep], ls[G / kHeadStep];   // of this thread's heads
#pragma unroll
        for (int k = 0; k < G / kHeadStep; ++k) {
            const int h = k * kHeadStep + tid / (W / 2);
            top[k] = -INFINITY;
            ls[k] = 0.0f;
#pragma unroll
            for (int w = 0; w < Pol::NC; ++w) top[k] = fmaxf(top[k], sm.wm[w][h]);
#pragma unroll
            for (int w = 0; w < Pol::NC; ++w) {
                const float mw = sm.wm[w][h];
                ls[k] += (mw == -INFINITY ? 0.0f : ptx::ex2(mw - top[k])) * sm.wl[w][h];
            }
        }
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
                if (slot < 0) {
                    const float inv = 1.0f / ls[k];
                    store_out2(p, out_base + at, s.x * inv, s.y * inv);
                } else {
                    *reinterpret_cast<float2*>(p.ws_acc + static_cast<size_t>(slot) * G * D + at) = s;
                    if (half == 0 && r == 0 && d == 0) {
                        float* ml = p.ws_ml + (static_cast<size_t>(slot) * G + h) * 2;
                        ml[0] = top[k];
                        ml[1] = ls[k];
                    }
                }
            }
            ptx::named_barrier_sync(bar, Pol::GW * 32);   // wacc is filled again
        }
    }
};

template <class Pol, bool kPaged>
__global__ void __launch_bounds__(Pol::kThreads, 1)
    gqa_decode_quant_kernel(const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const DecodeQuantParams qp) {
    constexpr int G = Pol::G, D = Pol::D, SLOTS = Pol::SLOTS, NC = Pol::NC, RING = Pol::RING;
    constexpr int GROUPS = Pol::GROUPS;
    constexpr int SPLIT = Pol::SPLIT;
    constexpr int kLoads = NC / 2;             // rings a producer fills
    constexpr int kGroupThreads = Pol::GW * 32;   // consumers of a group
    constexpr std::integral_constant<int, QuantPlanTuning::kExtra> kExtra{};
    constexpr uint32_t kTileBytes = QuantSmem<Pol>::kTileBytes;
    constexpr uint32_t kQBytes = G * D * 2;
    const DecodeParams& p = qp.d;

    extern __shared__ uint8_t smem_raw[];
    QuantSmem<Pol>& sm = *reinterpret_cast<QuantSmem<Pol>*>(
        smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u));

    const int tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    const int B = p.B, KVH = p.KVH, H = p.H;
    const int cta = blockIdx.x;
    const int units = static_cast<int>(gridDim.x) * GROUPS;   // units of the plan
    PlanSmem& pl = sm.plan;

    if (tid == 0) {
        for (int g = 0; g < GROUPS; ++g) {
            for (int s = 0; s < SLOTS; ++s) {
                ptx::mbar_init(ptx::smem_addr(&sm.group[g].full[s]), 2);   // the tiles' bytes, the scales
                ptx::mbar_init(ptx::smem_addr(&sm.group[g].empty[s]), SPLIT);
            }
            ptx::mbar_init(ptx::smem_addr(&sm.group[g].q_full), 1);
            ptx::mbar_init(ptx::smem_addr(&sm.group[g].q_empty), 2);   // consumers, second producer
        }
        ptx::mbar_init(ptx::smem_addr(&sm.stall_bar), 1);
        ptx::fence_mbar_init();
        sm.abort_flag = 0;
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
    build_plan<QuantPlanTuning>(pl, p, units, warp, lane, cta, kQuantBlock,
                            reinterpret_cast<uint32_t*>(&sm.kv[0][0][0][0]));

    // zeros for empty sequences and the segments' partial lists, as in decode_kernel.cuh
    const bool has_work = cta * GROUPS < pl.g_eff;
    if (!has_work || warp < Pol::kConsumers) {
        const int nt = has_work ? Pol::kConsumers * 32 : static_cast<int>(blockDim.x);
        for (int b = cta; b < B; b += gridDim.x) {
            if (pl.n[b] != 0) continue;
            const size_t base = static_cast<size_t>(b) * H * D;
            for (int i = tid; i < H * D; i += nt) store_out(p, base + i, 0.0f);
        }
        const int U = B * KVH;
        const int u_end = (cta + 1) * U / static_cast<int>(gridDim.x);
        for (int u = cta * U / static_cast<int>(gridDim.x) + tid; u < u_end; u += nt) {
            const int b = u / KVH, kvh = u - b * KVH;
            int4 e = make_int4(0, 0, 0, 0);
            if (pl.n[b] != 0 && pl.g_eff > 0) {
                const SegmentParts sp(pl, b, kvh, p.dyn_slot_base, kExtra);
                e = make_int4(sp.first_s, sp.ns_parts, sp.dk0, sp.nd_parts);
            }
            p.ws_segs[u] = e;
        }
    }
    // this warp's group and its unit (a group without a unit has nothing to do)
    const int group = warp < Pol::kConsumers ? warp / Pol::GW : (warp - Pol::kConsumers) / 2;
    if (warp >= Pol::kWarps) return;
    const int unit = cta * GROUPS + group;
    if (unit >= pl.g_eff) return;

    typename QuantSmem<Pol>::Group& gr = sm.group[group];
    const uint32_t kv_base = ptx::smem_addr(&sm.kv[group][0][0][0]);
    const uint32_t q_full = ptx::smem_addr(&gr.q_full), q_empty = ptx::smem_addr(&gr.q_empty);

    if (warp >= Pol::kConsumers) {
        // ================= producers: two threads per group =================
        // The first walks the schedule and publishes each piece with its q; both fill the
        // slots of every second warp.  (One thread spends ~700 cycles on 16 KB -- its TMA
        // instructions, the scales, its barriers -- which is the time HBM takes to deliver
        // them.)
        if (lane != 0) return;
        const int me = (warp - Pol::kConsumers) & 1;
        const uint64_t policy = ptx::policy_evict_first();
        const bool dynamic = pl.n_dyn > 0;
        long long x = static_unit_begin(pl, unit);
        const long long stop = static_unit_begin(pl, unit + 1);
        uint32_t filled[kLoads];   // blocks sent to warps me, me + 2, ...
#pragma unroll
        for (int k = 0; k < kLoads; ++k) filled[k] = 0;
        uint32_t n = 0;            // pieces published
        bool ok = true;
        while (true) {
            QuantPiece pc;
            if (me == 0) {
                // the description and q are free once the consumers began the piece before and
                // the other producer has read it
                ok = wait_bounded(q_empty, (n & 1u) ^ 1u, &sm.abort_flag, p.ws_flags);
                if (!ok) break;
                int claimed = -1;
                Piece w;
                if (!next_piece<QuantPlanTuning::kExtra>(pl, p, unit, kQuantBlock, dynamic, x, stop, claimed, w)) {
                    gr.piece.done = 1;
                    ptx::mbar_arrive(q_full);
                    break;
                }
                const int L = sm.len[w.b];
                pc.b = w.b;
                pc.kvh = w.kvh;
                pc.p0 = w.p0;
                pc.p1 = w.p1;
                pc.lo = p.window > 0 && L > p.window ? L - p.window : 0;
                pc.hi = L;
                pc.slot = w.slot;
                pc.parts = SegmentParts(pl, w.b, w.kvh, p.dyn_slot_base, kExtra).count();
                pc.done = 0;
                gr.piece = pc;
                ptx::mbar_arrive_expect_tx(q_full, kQBytes);
#pragma unroll
                for (int h = 0; h < G; ++h)
                    ptx::bulk_copy_g2s(ptx::smem_addr(&gr.q[h][0]),
                                       p.q + (static_cast<size_t>(pc.b) * H + pc.kvh * G + h) * D,
                                       D * 2, q_full);
            } else {
                ok = wait_bounded(q_full, n & 1u, &sm.abort_flag, p.ws_flags);
                if (!ok) break;
                pc = gr.piece;
                if (pc.done) break;
                ptx::mbar_arrive(q_empty);
            }
            ++n;
            const int32_t* bt_row =
                kPaged ? p.block_table + static_cast<size_t>(pc.b) * p.max_pages : nullptr;
            const int blk1 = pc.p1 / kQuantBlock;
            const int chunk0 = pc.kvh * (D / 128);
            int page[kLoads];   // page ids of the next round, loaded one round ahead
            if (kPaged) {
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const int blk = pc.p0 / kQuantBlock + me + 2 * k;
                    page[k] = blk < blk1 ? __ldg(bt_row + blk) : 0;
                }
            }
            for (int round = pc.p0 / kQuantBlock; ok && round < blk1; round += NC) {
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const int w = me + 2 * k, blk = round + w;
                    if (blk >= blk1) break;
                    const int s = w * RING + static_cast<int>(filled[k] % RING);
                    const uint32_t ph = (filled[k] / RING) & 1u;
                    ok = wait_bounded(ptx::smem_addr(&gr.empty[s]), ph ^ 1u, &sm.abort_flag, p.ws_flags);
                    if (!ok) break;
                    int outer = pc.b;
                    if (kPaged) {
                        const bool bad = page[k] < 0 || page[k] >= p.num_pages;
                        outer = bad ? 0 : page[k];   // (loaded, and masked by the consumer)
                        gr.bad[s] = bad;
                        if (bad) atomicOr(p.ws_flags, kFlagBadPage);
                        if (blk + NC < blk1) page[k] = __ldg(bt_row + blk + NC);
                    }
                    const uint32_t full_bar = ptx::smem_addr(&gr.full[s]);
                    ptx::mbar_arrive_expect_tx(full_bar, 2 * kTileBytes);
                    const uint32_t k_dst = kv_base + s * 2 * kTileBytes;
                    const int row = kPaged ? 0 : blk * kQuantBlock;
                    ptx::tma_load_4d(k_dst, &tm_k, full_bar, 0, row, chunk0, outer, policy);
                    ptx::tma_load_4d(k_dst + kTileBytes, &tm_v, full_bar, 0, row, chunk0, outer, policy);
                    const size_t at = (kPaged ? static_cast<size_t>(outer)
                                              : static_cast<size_t>(pc.b) * qp.blocks + blk) * KVH + pc.kvh;
                    const uint32_t sc_dst = ptx::smem_addr(&gr.scales[s][0]);
                    ptx::cp_async4(sc_dst, qp.k_scales + at);
                    ptx::cp_async4(sc_dst + 4, qp.v_scales + at);
                    ptx::cp_async_mbar_arrive(full_bar);
                    ++filled[k];
                    if ((p.test_flags & kTestStall) && me == 0 && k == 0 && filled[0] == 1)
                        ok = wait_bounded(ptx::smem_addr(&sm.stall_bar), 0u, &sm.abort_flag,
                                          p.ws_flags, kTestStallNs);
                    if (!ok) break;
                }
            }
            if (!ok) break;
        }
        if (!ok) {
            // let every copy already issued land before the CTA exits
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
                for (uint32_t f = filled[k] > RING ? filled[k] - RING : 0u; f < filled[k]; ++f)
                    wait_drain(ptx::smem_addr(&gr.full[(me + 2 * k) * RING + f % RING]), (f / RING) & 1u);
            if (me == 0 && n > 0) wait_drain(q_full, (n - 1u) & 1u);
        }
        return;
    }

    // ===================== consumers =====================
    // Every warp of a group passes the same barriers for every piece, whatever its waits
    // return; a warp whose wait gave up (or which saw the end) makes all of them leave at the
    // next one.
    QuantConsumer<Pol> c;
    const int gwarp = warp - group * Pol::GW, gtid = gwarp * 32 + lane, bar = 1 + group;
    const int own = gwarp % NC, half = gwarp / NC;   // ring, part of D
    const uint32_t q_frag = ptx::smem_addr(&gr.q_frag[0][0]);
    uint32_t taken = 0;   // blocks this warp has processed (its ring's fills, in order)
    for (uint32_t n = 0;; ++n) {
        const bool there = __all_sync(0xffffffffu, wait_bounded(q_full, n & 1u, &sm.abort_flag, p.ws_flags));
        QuantPiece pc;
        pc.done = 1;
        if (there) pc = gr.piece;
        if (!pc.done) c.begin(&gr.q[0][0], gr.q_frag, gwarp, lane);
        if (ptx::named_barrier_or(bar, kGroupThreads, pc.done != 0)) break;
        if (gtid == 0) ptx::mbar_arrive(q_empty);   // every warp has read q and the piece

        bool gone = false;
        // (counted from the piece's first block: which warp takes a block, and so the order of
        // the sums, does not depend on the pieces before)
        for (int pos = pc.p0 + own * kQuantBlock; pos < pc.p1; pos += NC * kQuantBlock) {
            const int s = own * RING + static_cast<int>(taken % RING);
            const uint32_t ph = (taken / RING) & 1u;
            gone = !__all_sync(0xffffffffu, wait_bounded(ptx::smem_addr(&gr.full[s]), ph, &sm.abort_flag, p.ws_flags));
            const uint32_t k_tile = kv_base + s * 2 * kTileBytes;
            float z[4];
            if (SPLIT == 1) {
                if (gone) break;
                c.scores(k_tile, q_frag, 0, z, lane);
            } else {
                // the halves of the scores cross over through this warp's part of the K tile,
                // which it has read
                const uint32_t mine = k_tile + half * (kTileBytes / SPLIT) + lane * 16;
                const uint32_t other = k_tile + (1 - half) * (kTileBytes / SPLIT) + lane * 16;
                if (!gone) {
                    c.scores(k_tile, q_frag, half, z, lane);
                    __syncwarp();
                    ptx::sts128(mine, __float_as_uint(z[0]), __float_as_uint(z[1]),
                                __float_as_uint(z[2]), __float_as_uint(z[3]));
                }
                gone = ptx::named_barrier_or(1 + Pol::GROUPS + group * NC + own, 2 * 32, gone);
                if (gone) break;
                const uint4 o = ptx::lds128(other);
                z[0] += __uint_as_float(o.x);
                z[1] += __uint_as_float(o.y);
                z[2] += __uint_as_float(o.z);
                z[3] += __uint_as_float(o.w);
            }
            const float ks = gr.scales[s][0], vs = gr.scales[s][1];
            const bool bad = kPaged && gr.bad[s] != 0;
            const int first = pc.lo - pos, last = pc.hi - pos;
            if (first <= 0 && last >= kQuantBlock && !bad)
                c.template weigh<true>(z, k_tile + kTileBytes, ks, vs, 0, kQuantBlock, false, half, lane);
            else
                c.template weigh<false>(z, k_tile + kTileBytes, ks, vs, first, last, bad, half, lane);
            if (SPLIT > 1) ptx::fence_proxy_async_smem();   // the scores, before the next copy
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&gr.empty[s]));
            ++taken;
        }

        // normalisers of this warp's columns
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float ls = c.l[j];
            ls += __shfl_xor_sync(0xffffffffu, ls, 4);
            ls += __shfl_xor_sync(0xffffffffu, ls, 8);
            ls += __shfl_xor_sync(0xffffffffu, ls, 16);
            if (half == 0 && lane < 4) {   // (the halves hold the same)
                gr.wm[own][2 * lane + j] = c.m[j];
                gr.wl[own][2 * lane + j] = ls;
            }
        }
        if (ptx::named_barrier_or(bar, kGroupThreads, gone)) break;
        const size_t out_base = (static_cast<size_t>(pc.b) * H + pc.kvh * G) * D;
        c.merge(gr, p, out_base, pc.parts == 1 ? -1 : pc.slot, bar, own, half, lane);
    }
}

using QuantSliding = QuantPolicy<2, 256, 2, 1, 3>;   // slidingDecodeGQA
using QuantGlobal = QuantPolicy<8, 512, 1, 2, 3>;    // decodeGQA

}  // namespace gqa
