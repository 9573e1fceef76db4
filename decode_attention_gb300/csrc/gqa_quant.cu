// The calls that write and read the 8-bit cache (include/gqa_decode.h):
// gqa_append_quant, gqa_read_quant, gqa_prepare_decode_quant and their paged forms.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "gqa_decode.h"
#include "kernels/append_quant_kernel.cuh"
#include "kernels/prepare_quant_kernel.cuh"
#include "kernels/read_quant_kernel.cuh"
#include "launch.h"

namespace {

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// 0: slidingDecodeGQA's KV heads, 1: decodeGQA's, -1: neither
int geometry_of(int KVH, int D) {
    if (KVH == 16 && D == 256) return 0;
    if (KVH == 4 && D == 512) return 1;
    return -1;
}

// Codes and scales: not null, and aligned for the vector accesses and the tiled copies.
bool cache_ok(const void* k, const void* v, const void* ks, const void* vs) {
    return k && v && ks && vs && aligned_to(k, 16) && aligned_to(v, 16) && aligned_to(ks, 4) &&
           aligned_to(vs, 4);
}

gqa::QuantCache contiguous_cache(void* k, void* v, float* ks, float* vs, int rows, int KVH) {
    gqa::QuantCache c;
    std::memset(&c, 0, sizeof c);
    c.k = static_cast<uint8_t*>(k);
    c.v = static_cast<uint8_t*>(v);
    c.k_scales = ks;
    c.v_scales = vs;
    c.rows = rows;
    c.KVH = KVH;
    return c;
}

gqa::QuantCache paged_cache(void* k, void* v, float* ks, float* vs, const int32_t* block_table,
                            int P, int max_pages, int KVH) {
    gqa::QuantCache c = contiguous_cache(k, v, ks, vs, 0, KVH);
    c.block_table = block_table;
    c.max_pages = max_pages;
    c.num_pages = P;
    return c;
}

bool pages_ok(const int32_t* block_table, int P, int max_pages, int page_size) {
    return page_size == GQA_PAGE_SIZE && P >= 1 && max_pages >= 1 && block_table &&
           aligned_to(block_table, 4) &&
           static_cast<int64_t>(max_pages) * GQA_PAGE_SIZE <= GQA_MAX_SEQ;
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
                          const int32_t* seq_lens, int B, int N, int KVH, int D, const void* k,
                          const void* v, const float* ks, const float* vs) {
    if (B < 0 || B > GQA_MAX_BATCH || N < 0 || N > GQA_MAX_BATCH * GQA_MAX_SEQ)
        return GQA_ERR_INVALID_ARGUMENT;
    if (geometry_of(KVH, D) < 0) return GQA_ERR_UNSUPPORTED;
    if (B == 0 || N == 0) return GQA_OK;
    if (!k_new || !v_new || !token_offsets || !seq_lens || !aligned_to(k_new, 16) ||
        !aligned_to(v_new, 16) || !aligned_to(token_offsets, 4) || !aligned_to(seq_lens, 4) ||
        !cache_ok(k, v, ks, vs))
        return GQA_ERR_INVALID_ARGUMENT;
    return GQA_OK;
}

gqa_status_t run_append(const void* k_new, const void* v_new, const int32_t* token_offsets,
                        const int32_t* seq_lens, int B, int N, int D, const gqa::QuantCache& cache,
                        gqa_stream_t stream) {
    const int sms = gqa::device_sms();
    if (sms == 0) return GQA_ERR_CUDA;
    gqa::AppendQuantParams p;
    std::memset(&p, 0, sizeof p);
    p.k_new = static_cast<const __nv_bfloat16*>(k_new);
    p.v_new = static_cast<const __nv_bfloat16*>(v_new);
    p.token_offsets = token_offsets;
    p.seq_lens = seq_lens;
    p.cache = cache;
    p.B = B;
    p.N = N;
    // n tokens touch at most (n + 14) / 16 + 1 blocks
    const uint64_t blocks = static_cast<uint64_t>(N) / gqa::kQuantBlock + 2u * static_cast<uint64_t>(B);
    const uint64_t items = blocks * 2 * static_cast<uint64_t>(cache.KVH);
    const uint64_t per_cta = gqa::kAppendThreads / 32 / (D / 256);
    const dim3 grid(clamp_grid((items + per_cta - 1) / per_cta, 2, sms));
    return D == 256 ? launch(gqa::gqa_append_quant_kernel<256>, p, grid, gqa::kAppendThreads, stream)
                    : launch(gqa::gqa_append_quant_kernel<512>, p, grid, gqa::kAppendThreads, stream);
}

// ---- read ------------------------------------------------------------------------

gqa_status_t check_read(const void* k, const void* v, const float* ks, const float* vs,
                        const int32_t* seq_lens, int B, int KVH, int D, int window,
                        const void* k_out, const void* v_out, int out_rows,
                        gqa_out_dtype_t out_dtype) {
    if (B < 0 || B > GQA_MAX_BATCH || window < 0 || out_rows < 1 || out_rows > GQA_MAX_SEQ)
        return GQA_ERR_INVALID_ARGUMENT;
    if (out_dtype != GQA_OUT_BF16 && out_dtype != GQA_OUT_F32) return GQA_ERR_INVALID_ARGUMENT;
    if (geometry_of(KVH, D) < 0) return GQA_ERR_UNSUPPORTED;
    if (B == 0) return GQA_OK;
    if (!seq_lens || !aligned_to(seq_lens, 4) || !k_out || !v_out || !aligned_to(k_out, 16) ||
        !aligned_to(v_out, 16) || !cache_ok(k, v, ks, vs))
        return GQA_ERR_INVALID_ARGUMENT;
    return GQA_OK;
}

gqa_status_t run_read(const gqa::QuantCache& cache, const int32_t* seq_lens, int B, int window,
                      void* k_out, void* v_out, int out_rows, gqa_out_dtype_t out_dtype,
                      gqa_stream_t stream) {
    const int sms = gqa::device_sms();
    if (sms == 0) return GQA_ERR_CUDA;
    gqa::ReadQuantParams p;
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
    const uint64_t blocks = static_cast<uint64_t>(B) * (most / gqa::kQuantBlock + 2) * 2;
    // Few blocks are cut in quarters to reach every SM (260 blocks: 11 us against 22); many are
    // taken whole, which looks up its sequence and page once per block.
    const int parts = blocks < 8u * static_cast<uint64_t>(sms) ? 4 : 1;
    const dim3 grid(clamp_grid(blocks * parts, 8, sms));
    using Kernel = void (*)(gqa::ReadQuantParams);
    static const Kernel kernels[2][2][2] = {   // [decodeGQA][fp32][quarters]
        {{gqa::gqa_read_quant_kernel<16, 256, false, 1>, gqa::gqa_read_quant_kernel<16, 256, false, 4>},
         {gqa::gqa_read_quant_kernel<16, 256, true, 1>, gqa::gqa_read_quant_kernel<16, 256, true, 4>}},
        {{gqa::gqa_read_quant_kernel<4, 512, false, 1>, gqa::gqa_read_quant_kernel<4, 512, false, 4>},
         {gqa::gqa_read_quant_kernel<4, 512, true, 1>, gqa::gqa_read_quant_kernel<4, 512, true, 4>}}};
    return launch(kernels[cache.KVH == 4][out_dtype == GQA_OUT_F32][parts == 4], p, grid,
                  gqa::kReadThreads, stream);
}

// ---- producer --------------------------------------------------------------------

gqa_status_t check_prepare(const void* q_raw, const void* k_raw, const void* v_raw,
                           const void* w_q, const void* w_k, const int32_t* seq_lens, int B, int H,
                           int KVH, int D, const void* q_out, const void* k, const void* v,
                           const float* ks, const float* vs) {
    if (B < 0 || B > GQA_MAX_BATCH) return GQA_ERR_INVALID_ARGUMENT;
    if (H != 32 || geometry_of(KVH, D) < 0) return GQA_ERR_UNSUPPORTED;
    if (B == 0) return GQA_OK;
    if (!q_raw || !k_raw || !v_raw || !w_q || !w_k || !seq_lens || !q_out ||
        !aligned_to(q_raw, 16) || !aligned_to(k_raw, 16) || !aligned_to(v_raw, 16) ||
        !aligned_to(q_out, 16) || !aligned_to(w_q, 4) || !aligned_to(w_k, 4) ||
        !aligned_to(seq_lens, 4) || !cache_ok(k, v, ks, vs))
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

gqa_status_t run_prepare(const void* q_raw, const void* k_raw, const void* v_raw, const void* w_q,
                         const void* w_k, const int32_t* seq_lens, int B, int H, int D,
                         void* q_out, const gqa::QuantCache& cache, gqa_stream_t stream) {
    gqa::PrepareQuantParams p;
    std::memset(&p, 0, sizeof p);
    p.q_raw = static_cast<const __nv_bfloat16*>(q_raw);
    p.k_raw = static_cast<const __nv_bfloat16*>(k_raw);
    p.v_raw = static_cast<const __nv_bfloat16*>(v_raw);
    p.w_q = static_cast<const __nv_bfloat16*>(w_q);
    p.w_k = static_cast<const __nv_bfloat16*>(w_k);
    p.seq_lens = seq_lens;
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.cache = cache;
    p.B = B;
    p.H = H;
    const RopeTurns& r = rope_turns(D);
    p.n_rot = r.pairs;
    std::memcpy(p.turn, r.turn, sizeof p.turn);
    constexpr int kWarps = gqa::kPrepareThreads / 32;
    const dim3 grid(static_cast<unsigned>(B),
                    static_cast<unsigned>((H + 2 * cache.KVH + kWarps - 1) / kWarps));
    return D == 256 ? launch(gqa::gqa_prepare_quant_kernel<256>, p, grid, gqa::kPrepareThreads, stream)
                    : launch(gqa::gqa_prepare_quant_kernel<512>, p, grid, gqa::kPrepareThreads, stream);
}

}  // namespace

extern "C" {

gqa_status_t gqa_append_quant(const void* k_new, const void* v_new, const int32_t* token_offsets,
                              const int32_t* seq_lens, int B, int N, int S, int KVH, int D,
                              void* k, void* v, float* k_scales, float* v_scales,
                              gqa_stream_t stream) {
    if (S < 1 || S > GQA_MAX_SEQ) return GQA_ERR_INVALID_ARGUMENT;
    const gqa_status_t st = check_append(k_new, v_new, token_offsets, seq_lens, B, N, KVH, D, k, v,
                                         k_scales, v_scales);
    if (st != GQA_OK || B == 0 || N == 0) return st;
    return run_append(k_new, v_new, token_offsets, seq_lens, B, N, D,
                      contiguous_cache(k, v, k_scales, v_scales, S, KVH), stream);
}

gqa_status_t gqa_append_quant_paged(const void* k_new, const void* v_new,
                                    const int32_t* token_offsets, const int32_t* block_table,
                                    const int32_t* seq_lens, int B, int N, int P, int max_pages,
                                    int page_size, int KVH, int D, void* k_pages, void* v_pages,
                                    float* k_scales, float* v_scales, gqa_stream_t stream) {
    const gqa_status_t st = check_append(k_new, v_new, token_offsets, seq_lens, B, N, KVH, D,
                                         k_pages, v_pages, k_scales, v_scales);
    if (st != GQA_OK || B == 0 || N == 0) return st;
    if (!pages_ok(block_table, P, max_pages, page_size)) return GQA_ERR_INVALID_ARGUMENT;
    return run_append(k_new, v_new, token_offsets, seq_lens, B, N, D,
                      paged_cache(k_pages, v_pages, k_scales, v_scales, block_table, P, max_pages, KVH),
                      stream);
}

gqa_status_t gqa_read_quant(const void* k, const void* v, const float* k_scales,
                            const float* v_scales, const int32_t* seq_lens, int B, int S, int KVH,
                            int D, int window, void* k_out, void* v_out, int out_rows,
                            gqa_out_dtype_t out_dtype, gqa_stream_t stream) {
    if (S < 1 || S > GQA_MAX_SEQ) return GQA_ERR_INVALID_ARGUMENT;
    const gqa_status_t st = check_read(k, v, k_scales, v_scales, seq_lens, B, KVH, D, window, k_out,
                                       v_out, out_rows, out_dtype);
    if (st != GQA_OK || B == 0) return st;
    return run_read(contiguous_cache(const_cast<void*>(k), const_cast<void*>(v),
                                     const_cast<float*>(k_scales), const_cast<float*>(v_scales), S, KVH),
                    seq_lens, B, window, k_out, v_out, out_rows, out_dtype, stream);
}

gqa_status_t gqa_read_quant_paged(const void* k_pages, const void* v_pages, const float* k_scales,
                                  const float* v_scales, const int32_t* block_table,
                                  const int32_t* seq_lens, int B, int P, int max_pages,
                                  int page_size, int KVH, int D, int window, void* k_out,
                                  void* v_out, int out_rows, gqa_out_dtype_t out_dtype,
                                  gqa_stream_t stream) {
    const gqa_status_t st = check_read(k_pages, v_pages, k_scales, v_scales, seq_lens, B, KVH, D,
                                       window, k_out, v_out, out_rows, out_dtype);
    if (st != GQA_OK || B == 0) return st;
    if (!pages_ok(block_table, P, max_pages, page_size)) return GQA_ERR_INVALID_ARGUMENT;
    return run_read(paged_cache(const_cast<void*>(k_pages), const_cast<void*>(v_pages),
                                const_cast<float*>(k_scales), const_cast<float*>(v_scales),
                                block_table, P, max_pages, KVH),
                    seq_lens, B, window, k_out, v_out, out_rows, out_dtype, stream);
}

gqa_status_t gqa_prepare_decode_quant(const void* q_raw, const void* k_raw, const void* v_raw,
                                      const void* w_q, const void* w_k, const int32_t* seq_lens,
                                      int B, int H, int KVH, int D, void* q_out, void* k, void* v,
                                      float* k_scales, float* v_scales, int rows,
                                      gqa_stream_t stream) {
    if (rows < 1 || rows > GQA_MAX_SEQ) return GQA_ERR_INVALID_ARGUMENT;
    const gqa_status_t st = check_prepare(q_raw, k_raw, v_raw, w_q, w_k, seq_lens, B, H, KVH, D,
                                          q_out, k, v, k_scales, v_scales);
    if (st != GQA_OK || B == 0) return st;
    return run_prepare(q_raw, k_raw, v_raw, w_q, w_k, seq_lens, B, H, D, q_out,
                       contiguous_cache(k, v, k_scales, v_scales, rows, KVH), stream);
}

gqa_status_t gqa_prepare_decode_quant_paged(const void* q_raw, const void* k_raw, const void* v_raw,
                                            const void* w_q, const void* w_k,
                                            const int32_t* block_table, const int32_t* seq_lens,
                                            int B, int P, int max_pages, int page_size, int H,
                                            int KVH, int D, void* q_out, void* k_pages,
                                            void* v_pages, float* k_scales, float* v_scales,
                                            gqa_stream_t stream) {
    const gqa_status_t st = check_prepare(q_raw, k_raw, v_raw, w_q, w_k, seq_lens, B, H, KVH, D,
                                          q_out, k_pages, v_pages, k_scales, v_scales);
    if (st != GQA_OK || B == 0) return st;
    if (!pages_ok(block_table, P, max_pages, page_size)) return GQA_ERR_INVALID_ARGUMENT;
    return run_prepare(q_raw, k_raw, v_raw, w_q, w_k, seq_lens, B, H, D, q_out,
                       paged_cache(k_pages, v_pages, k_scales, v_scales, block_table, P, max_pages, KVH),
                       stream);
}

}  // extern "C"
