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
// by a power of two per head and half of D, which makes its bf16 values exact in f16 down
// to 2^-30 of the largest.
//   scores  S[pos, h] = K[pos, :] . q[h, :], 16 positions (one block) per warp; the k index
//           pairs of an A fragment are the bytes (4t, 4t+1) and (4t+2, 4t+3) of a 16-byte
//           unit, q's B fragment in the same order
//   P.V     O^T[d, h] += V^T[d, pos] P[pos, h] for a D/8-wide slice of d per warp: 16-bit
//           ldmatrix.trans delivers dims (2g, 2g+1) of two positions, one byte permute
//           makes them rows g and g+8 of A.  At g = 2 the hi and lo parts of P are four
//           of the 8 columns of one mma; at g = 8 they are two mma.
//
// Work split, pipeline, timeouts and merging are those of decode_kernel.cuh: a persistent
// CTA per SM, a plan built from seq_lens on the device, one producer thread that streams K
// and V tiles with TMA, 8 consumer warps.  Pieces start and end on blocks.
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

template <int kG, int kD, int kTP, int kStages, bool kMerge>
struct QuantPolicy {
    static constexpr int G = kG, D = kD, TP = kTP, STAGES = kStages, NC = 8;
    static constexpr bool kMergeInKernel = kMerge;
    static constexpr int kBlocks = TP / kQuantBlock;    // blocks (m-tiles of the scores) per tile
    static constexpr int kParts = NC / kBlocks;         // parts of D a block's scores are split in
    static constexpr int kUnits = D / kParts / 16;      // 16-dim steps of a warp's scores
    static constexpr int kDimTiles = D / NC / 16;       // m-tiles of 16 dims of a warp's output
    static constexpr bool kSplitCols = G <= 2;          // hi and lo parts of P in one mma
    static constexpr int kSStride = TP + 8;             // padded row of the score tile
    static_assert(NC % kBlocks == 0 && kUnits % 2 == 0 && kDimTiles % 2 == 0, "tile shape");
};

struct QuantTile {
    int b, kvh;
    int vlo, vhi;   // rows [vlo, vhi) of the tile are attended positions
    int slot;       // workspace slot of the partial
    int bad;        // blocks whose page id is out of range, one bit each
    int flags;
};

template <class Pol>
struct alignas(1024) QuantSmem {
    static constexpr int kTileBytes = Pol::TP * Pol::D;
    uint8_t kv[Pol::STAGES][2][kTileBytes];   // [stage][K, V][block][chunk][16 rows][128 B]
    alignas(8) uint64_t full[Pol::STAGES];
    alignas(8) uint64_t empty[Pol::STAGES];
    alignas(8) uint64_t q_empty[2];
    alignas(8) uint64_t stall_bar;            // kTestStall: a barrier nothing completes
    QuantTile tile[Pol::STAGES];
    float scales[Pol::STAGES][2][Pol::kBlocks];
    PlanSmem plan;
    int len[kMaxBatch];                       // clamped lengths
    alignas(128) __nv_bfloat16 q[2][Pol::G * Pol::D];
    alignas(16) float S[2][Pol::kParts][Pol::G][Pol::kSStride];   // [tile parity][part][head][position]
    int abort_flag;
    int merge_last;
};

template <class Pol>
struct QuantConsumer {
    static constexpr int G = Pol::G, D = Pol::D, TP = Pol::TP;
    static constexpr int kBlocks = Pol::kBlocks, kUnits = Pol::kUnits, kDimTiles = Pol::kDimTiles;

    uint32_t qb[kUnits][2];      // B fragments of q (column g = head) for this warp's part of D
    float q_factor[2];           // undo q's scaling for columns 2t and 2t + 1
    float acc[kDimTiles][4];     // rows: dims 2g (0, 1) and 2g + 1 (2, 3); columns 2t, 2t + 1
    float m;                     // M of head column g
    float l;                     // this lane's share of the normaliser of column g

    // Byte address of 16-byte unit `unit` of row r of block `blk` of a tile.
    __device__ static __forceinline__ uint32_t unit_addr(uint32_t tile, int blk, int r, int unit) {
        return tile + blk * (kQuantBlock * D) + (unit >> 3) * 2048 + r * 128 +
               (((unit & 7) ^ (r & 7)) << 4);
    }

    // q_heads: [G][D] bf16 in shared memory
    __device__ __forceinline__ void begin(const __nv_bfloat16* q_heads, int warp, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const bool real = g < G;
        const __nv_bfloat16* row =
            q_heads + (real ? g : 0) * D + (warp / kBlocks) * (kUnits * 16) + 4 * t;
        uint2 w[kUnits];
        uint32_t top = 0;   // largest |q|: the bits of |bf16| order like the values
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            w[u] = *reinterpret_cast<const uint2*>(row + u * 16);
            top = __vmaxu2(top, __vmaxu2(w[u].x & 0x7fff7fffu, w[u].y & 0x7fff7fffu));
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(static_cast<int>(top >> 7) - 127, -100);   // |q| < 2^(e + 1)
        const float f = real ? pow2f(14 - e) : 0.0f;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            qb[u][0] = ptx::f16x2_pack(bf16lo(w[u].x) * f, bf16hi(w[u].x) * f);
            qb[u][1] = ptx::f16x2_pack(bf16lo(w[u].y) * f, bf16hi(w[u].y) * f);
        }
        const float undo = pow2f(e - 14);
        q_factor[0] = __shfl_sync(0xffffffffu, undo, 8 * t);
        q_factor[1] = __shfl_sync(0xffffffffu, undo, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < kDimTiles; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
        m = -INFINITY;
        l = 0.0f;
    }

    // Scores of this warp's block and part of D -> S[part][head][position].
    __device__ __forceinline__ void scores(uint32_t k_tile, const float* k_scales,
                                           float (*S)[G][Pol::kSStride], int warp, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int blk = warp % kBlocks, part = warp / kBlocks;
        const int mat = lane >> 3, r = (mat & 1) * 8 + (lane & 7);
        float c[2][4];   // two independent accumulation chains
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i][j] = 0.0f;
#pragma unroll
        for (int u = 0; u < kUnits; u += 2) {
            uint32_t a[4];   // rows g, g + 8 of unit u, then of unit u + 1
            ptx::ldmatrix_x4(unit_addr(k_tile, blk, r, part * kUnits + u + (mat >> 1)), a[0], a[1],
                             a[2], a[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t lo = a[2 * i], hi = a[2 * i + 1];
                ptx::mma_f16_16816(c[i], ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(lo)),
                                   ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(hi)),
                                   ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(lo >> 16)),
                                   ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(hi >> 16)),
                                   qb[u + i][0], qb[u + i][1]);
            }
        }
        const float fk = pow2f(scale_exponent(k_scales[blk]));
        const int pos = blk * kQuantBlock + g;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int h = 2 * t + j;
            if (h < G) {
                const float f = fk * q_factor[j];
                S[part][h][pos] = (c[0][j] + c[1][j]) * f;
                S[part][h][pos + 8] = (c[0][j + 2] + c[1][j + 2]) * f;
            }
        }
    }

    // Online softmax over the tile (every warp alike), then P.V for this warp's dims.
    __device__ __forceinline__ void softmax_pv(const float (*S)[G][Pol::kSStride], uint32_t v_tile,
                                               const float* v_scales, const QuantTile& d, int warp,
                                               int lane) {
        const int g = lane >> 2, t = lane & 3;
        // the head of column g; at kSplitCols columns G .. 2 G - 1 carry the lo parts
        const bool real = g < (Pol::kSplitCols ? 2 * G : G);
        const int head = Pol::kSplitCols ? g % G : (real ? g : 0);
        const bool whole = d.vlo == 0 && d.vhi == TP && d.bad == 0;
        float x[kBlocks][4];
        int ev[kBlocks];
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            ev[j] = scale_exponent(v_scales[j]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int pos = j * kQuantBlock + 8 * i + 2 * t;
                float2 s = *reinterpret_cast<const float2*>(&S[0][head][pos]);
#pragma unroll
                for (int q = 1; q < Pol::kParts; ++q) {
                    const float2 y = *reinterpret_cast<const float2*>(&S[q][head][pos]);
                    s.x += y.x;
                    s.y += y.y;
                }
                if (!whole) {
                    const float nan = __uint_as_float(0x7fc00000u);
                    if ((d.bad >> j) & 1) s = make_float2(nan, nan);
                    if (pos < d.vlo || pos >= d.vhi) s.x = -INFINITY;
                    if (pos + 1 < d.vlo || pos + 1 >= d.vhi) s.y = -INFINITY;
                }
                x[j][2 * i] = s.x;
                x[j][2 * i + 1] = s.y;
                top = fmaxf(top, fmaf(fmaxf(s.x, s.y), kLog2e, static_cast<float>(ev[j])));
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m, ceilf(top) - 15.0f);
        // (no finite score yet: any finite M)
        const float mm = mn == -INFINITY ? 0.0f : mn;
        if (__any_sync(0xffffffffu, mn != m)) {
            const float alpha = ptx::ex2(m - mm);
            const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * t);
            const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * t + 4);
            l *= alpha;
#pragma unroll
            for (int i = 0; i < kDimTiles; ++i) {
                acc[i][0] *= a0;
                acc[i][1] *= a1;
                acc[i][2] *= a0;
                acc[i][3] *= a1;
            }
        }
        m = mn;
        uint32_t hi[kBlocks][2], lo[kBlocks][2];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const float shift = static_cast<float>(ev[j]) - mm;
            float block_sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float p0 = ptx::ex2(fmaf(x[j][2 * i], kLog2e, shift));
                float p1 = ptx::ex2(fmaf(x[j][2 * i + 1], kLog2e, shift));
                if (!real) p0 = p1 = 0.0f;
                block_sum += p0 + p1;
                hi[j][i] = ptx::f16x2_pack(p0, p1);
                const float2 h = ptx::f16x2_unpack(hi[j][i]);
                lo[j][i] = ptx::f16x2_pack(p0 - h.x, p1 - h.y);
                if (Pol::kSplitCols && g >= G) hi[j][i] = lo[j][i];
            }
            sum += block_sum * pow2f(-ev[j]);
        }
        l += sum;

        const int mat = lane >> 3, r = (mat & 1) * 8 + (lane & 7);
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            // rows outside the range hold anything: their codes are zeroed (0 * NaN)
            uint32_t mask[2] = {0xffffffffu, 0xffffffffu};
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int pos = j * kQuantBlock + 8 * i + 2 * t;
                    mask[i] = ((pos >= d.vlo && pos < d.vhi) ? 0x0000ffffu : 0u) |
                              ((pos + 1 >= d.vlo && pos + 1 < d.vhi) ? 0xffff0000u : 0u);
                    if ((d.bad >> j) & 1) mask[i] = 0u;
                }
            }
#pragma unroll
            for (int n = 0; n < kDimTiles; n += 2) {
                uint32_t w[4];   // positions 0-7, 8-15 of dim tile n, then of n + 1
                ptx::ldmatrix_x4_trans(unit_addr(v_tile, j, r, warp * kDimTiles + n + (mat >> 1)),
                                       w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t a = __byte_perm(w[2 * q] & mask[0], 0u, 0x3120);
                    const uint32_t b = __byte_perm(w[2 * q + 1] & mask[1], 0u, 0x3120);
                    const uint32_t a0 = ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(a));
                    const uint32_t a1 = ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(a >> 16));
                    const uint32_t a2 = ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(b));
                    const uint32_t a3 = ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(b >> 16));
                    ptx::mma_f16_16816(acc[n + q], a0, a1, a2, a3, hi[j][0], hi[j][1]);
                    if (!Pol::kSplitCols)
                        ptx::mma_f16_16816(acc[n + q], a0, a1, a2, a3, lo[j][0], lo[j][1]);
                }
            }
        }
    }

    // The piece's result: the output (slot < 0; the piece is the whole segment) or the partial
    // (acc, m, l) at workspace slot `slot`.
    __device__ __forceinline__ void store(const DecodeParams& p, size_t out_base, int slot, int warp,
                                          int lane) {
        const int g = lane >> 2, t = lane & 3;
        float ls = l;
        ls += __shfl_xor_sync(0xffffffffu, ls, 1);
        ls += __shfl_xor_sync(0xffffffffu, ls, 2);
        if (Pol::kSplitCols) {
            // columns G .. 2 G - 1 (the next t for G = 2) hold the lo parts' products
            static_assert(!Pol::kSplitCols || G == 2, "lo columns are the next lane's");
#pragma unroll
            for (int i = 0; i < kDimTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += __shfl_xor_sync(0xffffffffu, acc[i][j], 1);
        }
        const float inv = 1.0f / ls;
        const float inv0 = __shfl_sync(0xffffffffu, inv, 8 * t);
        const float inv1 = __shfl_sync(0xffffffffu, inv, 8 * t + 4);
        if (2 * t < G) {
#pragma unroll
            for (int i = 0; i < kDimTiles; ++i) {
                const int dim = (warp * kDimTiles + i) * 16 + 2 * g;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int at = (2 * t + j) * D + dim;
                    if (slot < 0) {
                        const float f = j ? inv1 : inv0;
                        store_out2(p, out_base + at, acc[i][j] * f, acc[i][j + 2] * f);
                    } else {
                        *reinterpret_cast<float2*>(p.ws_acc + static_cast<size_t>(slot) * G * D + at) =
                            make_float2(acc[i][j], acc[i][j + 2]);
                    }
                }
            }
        }
        if (slot >= 0 && warp == 0 && t == 0 && g < G) {
            float* ml = p.ws_ml + (static_cast<size_t>(slot) * G + g) * 2;
            ml[0] = m;
            ml[1] = ls;
        }
    }
};

template <class Pol, bool kPaged>
__global__ void __launch_bounds__((Pol::NC + 1) * 32, 1)
    gqa_decode_quant_kernel(const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const DecodeQuantParams qp) {
    constexpr int G = Pol::G, D = Pol::D, TP = Pol::TP, STAGES = Pol::STAGES, NC = Pol::NC;
    constexpr int kBlocks = Pol::kBlocks;
    constexpr int kConsumerThreads = NC * 32;
    constexpr uint32_t kTileBytes = QuantSmem<Pol>::kTileBytes;
    constexpr uint32_t kBoxBytes = kQuantBlock * D;   // one block of one KV head
    const DecodeParams& p = qp.d;

    extern __shared__ uint8_t smem_raw[];
    QuantSmem<Pol>& sm = *reinterpret_cast<QuantSmem<Pol>*>(
        smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u));

    const int tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    const int B = p.B, KVH = p.KVH, H = p.H;
    const int cta = blockIdx.x;
    PlanSmem& pl = sm.plan;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(ptx::smem_addr(&sm.full[s]), 2);   // the tiles' bytes, the scales
            ptx::mbar_init(ptx::smem_addr(&sm.empty[s]), NC);
        }
        ptx::mbar_init(ptx::smem_addr(&sm.q_empty[0]), NC);
        ptx::mbar_init(ptx::smem_addr(&sm.q_empty[1]), NC);
        ptx::mbar_init(ptx::smem_addr(&sm.stall_bar), 1);
        ptx::fence_mbar_init();
        sm.abort_flag = 0;
    }
    if (warp == NC && lane == 0) {
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
    }
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();

    // (the plan's barriers make the lengths visible)
    for (int b = tid; b < B; b += blockDim.x)
        sm.len[b] = min(max(__ldg(p.seq_lens + b), 0), p.capacity);
    build_plan<kQuantBlock>(pl, p, gridDim.x, warp, lane, cta, TP,
                            reinterpret_cast<uint32_t*>(&sm.kv[0][0][0]));

    // zeros for empty sequences and the segments' partial lists, as in decode_kernel.cuh
    const bool has_work = cta < pl.g_eff;
    if (!has_work || warp < NC) {
        const int nt = has_work ? kConsumerThreads : static_cast<int>(blockDim.x);
        for (int b = cta; b < B; b += gridDim.x) {
            if (pl.n[b] != 0) continue;
            const size_t base = static_cast<size_t>(b) * H * D;
            for (int i = tid; i < H * D; i += nt) store_out(p, base + i, 0.0f);
        }
        if (!Pol::kMergeInKernel) {
            const int U = B * KVH;
            const int u_end = (cta + 1) * U / static_cast<int>(gridDim.x);
            for (int u = cta * U / static_cast<int>(gridDim.x) + tid; u < u_end; u += nt) {
                const int b = u / KVH, kvh = u - b * KVH;
                int4 e = make_int4(0, 0, 0, 0);
                if (pl.n[b] != 0 && pl.g_eff > 0) {
                    const SegmentParts sp(pl, b, kvh, p.dyn_slot_base);
                    e = make_int4(sp.first_s, sp.ns_parts, sp.dk0, sp.nd_parts);
                }
                p.ws_segs[u] = e;
            }
        }
    }
    if (!has_work) return;

    const uint32_t kv_base = ptx::smem_addr(&sm.kv[0][0][0]);

    if (warp == NC) {
        // ================= producer: one thread walks the schedule =================
        if (lane != 0) return;
        const uint64_t policy = ptx::policy_evict_first();
        uint32_t t_idx = 0;
        bool ok = true;
        const bool dynamic = pl.n_dyn > 0;
        int claimed = -1;
        uint32_t q_n = 0;
        constexpr uint32_t kQBytes = G * D * 2;

        auto emit_piece = [&](const Piece& pc) -> bool {
            const uint32_t qb = q_n & 1u;
            if (!wait_bounded(ptx::smem_addr(&sm.q_empty[qb]), ((q_n >> 1) & 1u) ^ 1u,
                              &sm.abort_flag, p.ws_flags))
                return false;
            ++q_n;
            const int b = pc.b, kvh = pc.kvh, L = sm.len[b];
            const int first_pos = p.window > 0 && L > p.window ? L - p.window : 0;
            const int chunk0 = kvh * (D / 128);
            const int32_t* bt_row =
                kPaged ? p.block_table + static_cast<size_t>(b) * p.max_pages : nullptr;
            for (int t = pc.p0; t < pc.p1; t += TP) {
                const bool first = t == pc.p0, last = t + TP >= pc.p1;
                const int nbox = min(pc.p1 - t, TP) / kQuantBlock;
                int page[kBlocks], bad = 0;
                if (kPaged) {
#pragma unroll
                    for (int j = 0; j < kBlocks; ++j)
                        page[j] = j < nbox ? __ldg(bt_row + t / kQuantBlock + j) : 0;
#pragma unroll
                    for (int j = 0; j < kBlocks; ++j)
                        if (page[j] < 0 || page[j] >= p.num_pages) {
                            page[j] = 0;   // (loaded, and masked by the consumers)
                            bad |= 1 << j;
                        }
                }
                if (dynamic && pc.unit_end && last)
                    claimed = static_cast<int>(atomicAdd(p.ws_claim, 1u));
                const int s = t_idx % STAGES;
                const uint32_t ph = (t_idx / STAGES) & 1u;
                if (!wait_bounded(ptx::smem_addr(&sm.empty[s]), ph ^ 1u, &sm.abort_flag, p.ws_flags))
                    return false;
                QuantTile& d = sm.tile[s];
                d.b = b;
                d.kvh = kvh;
                d.vlo = max(first_pos - t, 0);
                d.vhi = min(min(L, pc.p1) - t, TP);
                d.slot = pc.slot;
                d.bad = bad;
                d.flags = (first ? kDescFirst : 0) | (last ? kDescLast : 0);
                if (bad) atomicOr(p.ws_flags, kFlagBadPage);
                const uint32_t full_bar = ptx::smem_addr(&sm.full[s]);
                ptx::mbar_arrive_expect_tx(full_bar, static_cast<uint32_t>(nbox) * 2 * kBoxBytes +
                                                         (first ? kQBytes : 0u));
                if (first)
                    ptx::bulk_copy_g2s(ptx::smem_addr(&sm.q[qb][0]),
                                       p.q + (static_cast<size_t>(b) * H + kvh * G) * D, kQBytes,
                                       full_bar);
                const uint32_t k_dst = kv_base + s * 2 * kTileBytes;
                const uint32_t v_dst = k_dst + kTileBytes;
                const uint32_t sc_dst = ptx::smem_addr(&sm.scales[s][0][0]);
#pragma unroll
                for (int j = 0; j < kBlocks; ++j) {
                    if (j >= nbox) break;
                    const int row = kPaged ? 0 : t + j * kQuantBlock;
                    const int outer = kPaged ? page[j] : b;
                    ptx::tma_load_4d(k_dst + j * kBoxBytes, &tm_k, full_bar, 0, row, chunk0, outer, policy);
                    ptx::tma_load_4d(v_dst + j * kBoxBytes, &tm_v, full_bar, 0, row, chunk0, outer, policy);
                    const size_t at =
                        (kPaged ? static_cast<size_t>(page[j])
                                : static_cast<size_t>(b) * qp.blocks + t / kQuantBlock + j) * KVH + kvh;
                    ptx::cp_async4(sc_dst + j * 4, qp.k_scales + at);
                    ptx::cp_async4(sc_dst + (kBlocks + j) * 4, qp.v_scales + at);
                }
                ptx::cp_async_mbar_arrive(full_bar);
                ++t_idx;
                if ((p.test_flags & kTestStall) && t_idx == 1 &&
                    !wait_bounded(ptx::smem_addr(&sm.stall_bar), 0u, &sm.abort_flag, p.ws_flags,
                                  kTestStallNs))
                    return false;
            }
            return true;
        };

        long long x = static_unit_begin(pl, cta);
        const long long stop = static_unit_begin(pl, cta + 1);
        Piece pc;
        while (ok && next_piece(pl, p, cta, TP, dynamic, x, stop, claimed, pc)) ok = emit_piece(pc);
        if (ok) {
            const int s = t_idx % STAGES;
            const uint32_t ph = (t_idx / STAGES) & 1u;
            if (wait_bounded(ptx::smem_addr(&sm.empty[s]), ph ^ 1u, &sm.abort_flag, p.ws_flags)) {
                sm.tile[s].flags = kDescDone;
                ptx::mbar_arrive(ptx::smem_addr(&sm.full[s]));
                ptx::mbar_arrive(ptx::smem_addr(&sm.full[s]));
            }
        } else {
            // let every copy already issued land before the CTA exits
            const uint32_t first = t_idx > static_cast<uint32_t>(STAGES) ? t_idx - STAGES : 0u;
            for (uint32_t tt = first; tt < t_idx; ++tt)
                wait_drain(ptx::smem_addr(&sm.full[tt % STAGES]), (tt / STAGES) & 1u);
        }
        if (Pol::kMergeInKernel && dynamic) {
            if (ptx::atom_add_acq_rel_gpu(p.ws_done, 1u) == static_cast<uint32_t>(pl.g_eff - 1)) {
                atomicExch(p.ws_claim, 0u);
                atomicExch(p.ws_done, 0u);
            }
        }
        return;
    }

    // ===================== consumers: follow the tiles =====================
    QuantConsumer<Pol> c;
    uint32_t q_n = 0;
    for (uint32_t t_idx = 0;; ++t_idx) {
        const int s = t_idx % STAGES;
        const uint32_t ph = (t_idx / STAGES) & 1u;
        // (one decision per warp: the tile's work is warp-wide)
        const bool ok = __all_sync(0xffffffffu, wait_bounded(ptx::smem_addr(&sm.full[s]), ph,
                                                             &sm.abort_flag, p.ws_flags));
        QuantTile d;
        d.flags = kDescDone;
        if (ok) d = sm.tile[s];
        const uint32_t k_tile = kv_base + s * 2 * kTileBytes;
        float(*S)[G][Pol::kSStride] = sm.S[t_idx & 1];
        if (!(d.flags & kDescDone)) {
            if (d.flags & kDescFirst) {
                // q arrived with this tile; release the buffer once every lane has read it
                const uint32_t qb = q_n & 1u;
                c.begin(&sm.q[qb][0], warp, lane);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&sm.q_empty[qb]));
                ++q_n;
            }
            c.scores(k_tile, sm.scales[s][0], S, warp, lane);
        }
        // the scores of every warp are there; and all take the same exit decision (the end, or
        // a wait that gave up)
        if (ptx::named_barrier_or(1, kConsumerThreads, (d.flags & kDescDone) != 0)) break;
        c.softmax_pv(S, k_tile + kTileBytes, sm.scales[s][1], d, warp, lane);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&sm.empty[s]));
        if (!(d.flags & kDescLast)) continue;

        const SegmentParts sp(pl, d.b, d.kvh, p.dyn_slot_base);
        const int nparts = sp.count();
        const size_t out_base = (static_cast<size_t>(d.b) * H + d.kvh * G) * D;
        c.store(p, out_base, nparts == 1 ? -1 : d.slot, warp, lane);
        if constexpr (Pol::kMergeInKernel)
            if (nparts > 1)
                count_and_merge<G, D, kConsumerThreads>(p, sp, d.b * KVH + d.kvh, out_base, tid,
                                                        &sm.merge_last);
    }
}

using QuantSliding = QuantPolicy<2, 256, 128, 3, true>;    // slidingDecodeGQA
using QuantGlobal = QuantPolicy<8, 512, 64, 3, false>;     // decodeGQA

}  // namespace gqa
