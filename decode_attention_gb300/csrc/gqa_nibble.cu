// The calls that write and read the 4-bit cache (include/gqa_decode.h): gqa_append_nibble,
// gqa_read_nibble, gqa_prepare_tokens_nibble, the producer for many tokens into a bf16 cache,
// gqa_prepare_tokens, and their paged forms.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "gqa_decode.h"
#include "kernels/append_nibble_kernel.cuh"
#include "kernels/prepare_tokens_kernel.cuh"
#include "kernels/read_nibble_kernel.cuh"
#include "launch.h"

namespace {

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool geometry_ok(int KVH, int D) { return (KVH == 16 && D == 256) || (KVH == 4 && D == 512); }

bool batch_ok(int B, int N) {
    return B >= 0 && B <= GQA_MAX_BATCH && N >= 0 && N <= GQA_MAX_BATCH * GQA_MAX_SEQ;
}

bool pages_ok(const int32_t* block_table, int P, int max_pages, int page_size) {
    return page_size == GQA_PAGE_SIZE && P >= 1 && max_pages >= 1 && block_table &&
           aligned_to(block_table, 4) &&
           static_cast<int64_t>(max_pages) * GQA_PAGE_SIZE <= GQA_MAX_SEQ;
}

gqa::NibbleCache contiguous_cache(void* kv, int rows, int KVH, int D) {
    gqa::NibbleCache c;
    std::memset(&c, 0, sizeof c);
    c.kv = static_cast<uint8_t*>(kv);
    c.rows = rows;
    c.planes = KVH * D / gqa::kNibblePlane;
    return c;
}

gqa::NibbleCache paged_cache(void* kv, const int32_t* block_table, int P, int max_pages, int KVH, int D) {
    gqa::NibbleCache c = contiguous_cache(kv, 0, KVH, D);
    c.block_table = block_table;
    c.max_pages = max_pages;
    c.num_pages = P;
    return c;
}

template <class Params>
gqa_status_t launch(void (*kernel)(Params), const Params& p, dim3 grid, int threads,
                    gqa_stream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

unsigned clamp_grid(uint64_t want, int per_sm, int sms) {
    const uint64_t most = static_cast<uint64_t>(per_sm) * static_cast<uint64_t>(sms);
    return static_cast<unsigned>(want < 1 ? 1 : (want < most ? want : most));
}

// ---- append ----------------------------------------------------------------------

gqa_status_t check_append(const void* k_new, const void* v_new, const int32_t* token_offsets,
                          const int32_t* seq_lens, int B, int N, int KVH, int D, const void* kv) {
    if (!batch_ok(B, N)) return GQA_ERR_INVALID_ARGUMENT;
    if (!geometry_ok(KVH, D)) return GQA_ERR_UNSUPPORTED;
    if (B == 0 || N == 0) return GQA_OK;
    if (!k_new || !v_new || !token_offsets || !seq_lens || !kv || !aligned_to(k_new, 16) ||
        !aligned_to(v_new, 16) || !aligned_to(token_offsets, 4) || !aligned_to(seq_lens, 4) ||
        !aligned_to(kv, 16))
        return GQA_ERR_INVALID_ARGUMENT;
    return GQA_OK;
}

gqa_status_t run_append(const void* k_new, const void* v_new, const int32_t* token_offsets,
                        const int32_t* seq_lens, int B, int N, const gqa::NibbleCache& cache,
                        gqa_stream_t stream) {
    const int sms = gqa::device_sms();
    if (sms == 0) return GQA_ERR_CUDA;
    gqa::AppendNibbleParams p;
    std::memset(&p, 0, sizeof p);
    p.k_new = static_cast<const __nv_bfloat16*>(k_new);
    p.v_new = static_cast<const __nv_bfloat16*>(v_new);
    p.token_offsets = token_offsets;
    p.seq_lens = seq_lens;
    p.cache = cache;
    p.B = B;
    p.N = N;
    constexpr int kPlanes = 4;
    const uint64_t items = static_cast<uint64_t>(N) * static_cast<uint64_t>(cache.planes / kPlanes);
    constexpr int kWarps = gqa::kAppendNibbleThreads / 32;
    return launch(gqa::gqa_append_nibble_kernel<kPlanes>, p,
                  dim3(clamp_grid((items + kWarps - 1) / kWarps, 4, sms)),
                  gqa::kAppendNibbleThreads, stream);
}

// ---- read ------------------------------------------------------------------------

gqa_status_t check_read(const void* kv, const int32_t* seq_lens, int B, int KVH, int D, int window,
                        const void* k_out, const void* v_out, int out_rows,
                        gqa_out_dtype_t out_dtype) {
    if (B < 0 || B > GQA_MAX_BATCH || window < 0 || out_rows < 1 || out_rows > GQA_MAX_SEQ)
        return GQA_ERR_INVALID_ARGUMENT;
    if (out_dtype != GQA_OUT_BF16 && out_dtype != GQA_OUT_F32) return GQA_ERR_INVALID_ARGUMENT;
    if (!geometry_ok(KVH, D)) return GQA_ERR_UNSUPPORTED;
    if (B == 0) return GQA_OK;
    if (!kv || !seq_lens || !k_out || !v_out || !aligned_to(kv, 16) || !aligned_to(seq_lens, 4) ||
        !aligned_to(k_out, 16) || !aligned_to(v_out, 16))
        return GQA_ERR_INVALID_ARGUMENT;
    return GQA_OK;
}

gqa_status_t run_read(const gqa::NibbleCache& cache, const int32_t* seq_lens, int B, int window,
                      void* k_out, void* v_out, int out_rows, gqa_out_dtype_t out_dtype,
                      gqa_stream_t stream) {
    const int sms = gqa::device_sms();
    if (sms == 0) return GQA_ERR_CUDA;
    gqa::ReadNibbleParams p;
    std::memset(&p, 0, sizeof p);
    p.cache = cache;
    p.seq_lens = seq_lens;
    p.k_out = k_out;
    p.v_out = v_out;
    p.B = B;
    p.window = window;
    p.out_rows = out_rows;
    int most = cache.capacity() < out_rows ? cache.capacity() : out_rows;
    if (window > 0 && window < most) most = window;
    constexpr int kPlanes = 4, kWarps = gqa::kReadNibbleThreads / 32;
    const uint64_t items = static_cast<uint64_t>(B) * static_cast<uint64_t>(most) *
                           static_cast<uint64_t>(cache.planes / kPlanes);
    const dim3 grid(clamp_grid((items + kWarps - 1) / kWarps, 8, sms));
    return out_dtype == GQA_OUT_F32
               ? launch(gqa::gqa_read_nibble_kernel<kPlanes, true>, p, grid, gqa::kReadNibbleThreads, stream)
               : launch(gqa::gqa_read_nibble_kernel<kPlanes, false>, p, grid, gqa::kReadNibbleThreads, stream);
}

// ---- producer --------------------------------------------------------------------

struct ProducerArgs {
    const void *q_raw, *k_raw, *v_raw, *w_q, *w_k;
    const int32_t *token_offsets, *seq_lens;
    int B, N, H, KVH, D;
    void* q_out;
    void *k_cache, *v_cache;   // bf16 cache (null for the 4-bit one)
    void* kv;                  // 4-bit cache (null for the bf16 one)
    int ring;
};

gqa_status_t check_producer(const ProducerArgs& a, bool nibble) {
    if (!batch_ok(a.B, a.N)) return GQA_ERR_INVALID_ARGUMENT;
    if (a.H != 32 || !geometry_ok(a.KVH, a.D)) return GQA_ERR_UNSUPPORTED;
    if (a.B == 0 || a.N == 0) return GQA_OK;
    const bool keqv = !nibble && a.v_raw == nullptr;
    if (keqv && a.D != 512) return GQA_ERR_UNSUPPORTED;   // values = keys on global layers only
    if (!a.q_raw || !a.k_raw || (nibble && !a.v_raw) || !a.w_q || !a.w_k || !a.token_offsets ||
        !a.seq_lens || !a.q_out || (nibble ? !a.kv : !a.v_cache || (!keqv && !a.k_cache)))
        return GQA_ERR_INVALID_ARGUMENT;
    const void* wide[] = {a.q_raw, a.k_raw, a.v_raw, a.q_out, a.k_cache, a.v_cache, a.kv};
    for (const void* x : wide)
        if (x && !aligned_to(x, 16)) return GQA_ERR_INVALID_ARGUMENT;
    if (!aligned_to(a.w_q, 4) || !aligned_to(a.w_k, 4) || !aligned_to(a.token_offsets, 4) ||
        !aligned_to(a.seq_lens, 4))
        return GQA_ERR_INVALID_ARGUMENT;
    return GQA_OK;
}

// Rotary pairs of each geometry (Model Spec, `attn.rope` rows) and, for pair i, the turn per
// position theta^(-2i/D) / (2 pi) as a 64-bit fraction.  Computed once.
struct RopeTurns {
    int pairs;
    uint64_t turn[gqa::kPrepareMaxRot];

    RopeTurns(int D, int n, double theta) : pairs(n) {
        for (int i = 0; i < gqa::kPrepareMaxRot; ++i) {
            const double t = std::pow(theta, -2.0 * i / static_cast<double>(D)) / 6.283185307179586;
            turn[i] = i < n ? static_cast<uint64_t>(t * 18446744073709551616.0) : 0u;
        }
    }
};

const RopeTurns& rope_turns(int D) {
    static const RopeTurns sliding(256, 128, 1.0e4), global(512, 64, 1.0e6);
    return D == 256 ? sliding : global;
}

template <int D, bool kNibble>
gqa_status_t launch_tokens(const gqa::PrepareTokensParams& p, int sms, gqa_stream_t stream) {
    constexpr int kWarps = gqa::kTokensThreads / 32;
    const int n_units = (p.H + 2 * p.KVH) * D / gqa::kTokensUnit, groups = (n_units + kWarps - 1) / kWarps;
    // Few tokens: their heads are dealt to several CTAs, as many as run together (of 100 single tokens at
    // D = 256 6.2 us; 7.8 with twice as many, whose last ones wait, and 6.6 with two thirds).
    const unsigned slots = static_cast<unsigned>(gqa::kTokensPerSm * sms), n = static_cast<unsigned>(p.N);
    const unsigned most = slots / n < static_cast<unsigned>(groups) ? slots / n : static_cast<unsigned>(groups);
    const dim3 grid(clamp_grid(n, gqa::kTokensPerSm, sms), most < 1 ? 1 : most);
    return launch(gqa::gqa_prepare_tokens_kernel<D, kNibble>, p, grid, gqa::kTokensThreads, stream);
}

gqa_status_t run_producer(const ProducerArgs& a, const gqa::NibbleCache& cache, bool nibble,
                          gqa_stream_t stream) {
    const int sms = gqa::device_sms();
    if (sms == 0) return GQA_ERR_CUDA;
    gqa::PrepareTokensParams p;
    std::memset(&p, 0, sizeof p);
    p.q_raw = static_cast<const __nv_bfloat16*>(a.q_raw);
    p.k_raw = static_cast<const __nv_bfloat16*>(a.k_raw);
    p.v_raw = static_cast<const __nv_bfloat16*>(a.v_raw);
    p.w_q = static_cast<const __nv_bfloat16*>(a.w_q);
    p.w_k = static_cast<const __nv_bfloat16*>(a.w_k);
    p.token_offsets = a.token_offsets;
    p.seq_lens = a.seq_lens;
    p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
    p.k_cache = static_cast<__nv_bfloat16*>(a.k_cache);
    p.v_cache = static_cast<__nv_bfloat16*>(a.v_cache);
    p.cache = cache;
    p.ring = a.ring;
    p.B = a.B;
    p.N = a.N;
    p.H = a.H;
    p.KVH = a.KVH;
    const RopeTurns& r = rope_turns(a.D);
    p.n_rot = r.pairs;
    std::memcpy(p.turn, r.turn, sizeof p.turn);
    if (a.D == 256) return nibble ? launch_tokens<256, true>(p, sms, stream) : launch_tokens<256, false>(p, sms, stream);
    return nibble ? launch_tokens<512, true>(p, sms, stream) : launch_tokens<512, false>(p, sms, stream);
}

}  // namespace

extern "C" {

gqa_status_t gqa_append_nibble(const void* k_new, const void* v_new, const int32_t* token_offsets,
                               const int32_t* seq_lens, int B, int N, int S, int KVH, int D,
                               void* kv, gqa_stream_t stream) {
    if (S < 1 || S > GQA_MAX_SEQ) return GQA_ERR_INVALID_ARGUMENT;
    const gqa_status_t st = check_append(k_new, v_new, token_offsets, seq_lens, B, N, KVH, D, kv);
    if (st != GQA_OK || B == 0 || N == 0) return st;
    return run_append(k_new, v_new, token_offsets, seq_lens, B, N, contiguous_cache(kv, S, KVH, D), stream);
}

gqa_status_t gqa_append_nibble_paged(const void* k_new, const void* v_new,
                                     const int32_t* token_offsets, const int32_t* block_table,
                                     const int32_t* seq_lens, int B, int N, int P, int max_pages,
                                     int page_size, int KVH, int D, void* kv_pages,
                                     gqa_stream_t stream) {
    const gqa_status_t st = check_append(k_new, v_new, token_offsets, seq_lens, B, N, KVH, D, kv_pages);
    if (st != GQA_OK || B == 0 || N == 0) return st;
    if (!pages_ok(block_table, P, max_pages, page_size)) return GQA_ERR_INVALID_ARGUMENT;
    return run_append(k_new, v_new, token_offsets, seq_lens, B, N,
                      paged_cache(kv_pages, block_table, P, max_pages, KVH, D), stream);
}

gqa_status_t gqa_read_nibble(const void* kv, const int32_t* seq_lens, int B, int S, int KVH, int D,
                             int window, void* k_out, void* v_out, int out_rows,
                             gqa_out_dtype_t out_dtype, gqa_stream_t stream) {
    if (S < 1 || S > GQA_MAX_SEQ) return GQA_ERR_INVALID_ARGUMENT;
    const gqa_status_t st = check_read(kv, seq_lens, B, KVH, D, window, k_out, v_out, out_rows, out_dtype);
    if (st != GQA_OK || B == 0) return st;
    return run_read(contiguous_cache(const_cast<void*>(kv), S, KVH, D), seq_lens, B, window, k_out,
                    v_out, out_rows, out_dtype, stream);
}

gqa_status_t gqa_read_nibble_paged(const void* kv_pages, const int32_t* block_table,
                                   const int32_t* seq_lens, int B, int P, int max_pages,
                                   int page_size, int KVH, int D, int window, void* k_out,
                                   void* v_out, int out_rows, gqa_out_dtype_t out_dtype,
                                   gqa_stream_t stream) {
    const gqa_status_t st = check_read(kv_pages, seq_lens, B, KVH, D, window, k_out, v_out, out_rows, out_dtype);
    if (st != GQA_OK || B == 0) return st;
    if (!pages_ok(block_table, P, max_pages, page_size)) return GQA_ERR_INVALID_ARGUMENT;
    return run_read(paged_cache(const_cast<void*>(kv_pages), block_table, P, max_pages, KVH, D),
                    seq_lens, B, window, k_out, v_out, out_rows, out_dtype, stream);
}

gqa_status_t gqa_prepare_tokens(const void* q_raw, const void* k_raw, const void* v_raw,
                                const void* w_q, const void* w_k, const int32_t* token_offsets,
                                const int32_t* seq_lens, int B, int N, int H, int KVH, int D,
                                void* q_out, void* k_cache, void* v_cache, int rows, int ring,
                                gqa_stream_t stream) {
    if (rows < 1 || rows > GQA_MAX_SEQ || (ring != 0 && ring != 1)) return GQA_ERR_INVALID_ARGUMENT;
    const ProducerArgs a{q_raw, k_raw, v_raw, w_q, w_k, token_offsets, seq_lens, B, N, H, KVH, D,
                         q_out, k_cache, v_cache, nullptr, ring};
    const gqa_status_t st = check_producer(a, false);
    if (st != GQA_OK || B == 0 || N == 0) return st;
    return run_producer(a, contiguous_cache(nullptr, rows, KVH, D), false, stream);
}

gqa_status_t gqa_prepare_tokens_paged(const void* q_raw, const void* k_raw, const void* v_raw,
                                      const void* w_q, const void* w_k,
                                      const int32_t* token_offsets, const int32_t* block_table,
                                      const int32_t* seq_lens, int B, int N, int P, int max_pages,
                                      int page_size, int H, int KVH, int D, void* q_out,
                                      void* k_pages, void* v_pages, gqa_stream_t stream) {
    const ProducerArgs a{q_raw, k_raw, v_raw, w_q, w_k, token_offsets, seq_lens, B, N, H, KVH, D,
                         q_out, k_pages, v_pages, nullptr, 0};
    const gqa_status_t st = check_producer(a, false);
    if (st != GQA_OK || B == 0 || N == 0) return st;
    if (!pages_ok(block_table, P, max_pages, page_size)) return GQA_ERR_INVALID_ARGUMENT;
    return run_producer(a, paged_cache(nullptr, block_table, P, max_pages, KVH, D), false, stream);
}

gqa_status_t gqa_prepare_tokens_nibble(const void* q_raw, const void* k_raw, const void* v_raw,
                                       const void* w_q, const void* w_k,
                                       const int32_t* token_offsets, const int32_t* seq_lens,
                                       int B, int N, int H, int KVH, int D, void* q_out, void* kv,
                                       int S, gqa_stream_t stream) {
    if (S < 1 || S > GQA_MAX_SEQ) return GQA_ERR_INVALID_ARGUMENT;
    const ProducerArgs a{q_raw, k_raw, v_raw, w_q, w_k, token_offsets, seq_lens, B, N, H, KVH, D,
                         q_out, nullptr, nullptr, kv, 0};
    const gqa_status_t st = check_producer(a, true);
    if (st != GQA_OK || B == 0 || N == 0) return st;
    return run_producer(a, contiguous_cache(kv, S, KVH, D), true, stream);
}

gqa_status_t gqa_prepare_tokens_nibble_paged(const void* q_raw, const void* k_raw,
                                             const void* v_raw, const void* w_q, const void* w_k,
                                             const int32_t* token_offsets,
                                             const int32_t* block_table, const int32_t* seq_lens,
                                             int B, int N, int P, int max_pages, int page_size,
                                             int H, int KVH, int D, void* q_out, void* kv_pages,
                                             gqa_stream_t stream) {
    const ProducerArgs a{q_raw, k_raw, v_raw, w_q, w_k, token_offsets, seq_lens, B, N, H, KVH, D,
                         q_out, nullptr, nullptr, kv_pages, 0};
    const gqa_status_t st = check_producer(a, true);
    if (st != GQA_OK || B == 0 || N == 0) return st;
    if (!pages_ok(block_table, P, max_pages, page_size)) return GQA_ERR_INVALID_ARGUMENT;
    return run_producer(a, paged_cache(kv_pages, block_table, P, max_pages, KVH, D), true, stream);
}

}  // extern "C"
