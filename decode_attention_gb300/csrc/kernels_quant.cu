// Decode attention kernels over the 8-bit cache, both geometries.
#include "kernels/decode_quant_kernel.cuh"
#include "launch.h"

namespace gqa {

namespace {

template <int G, int D>
cudaError_t launch(const LaunchArgs& a, const DecodeQuantParams& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.p.KVH), static_cast<unsigned>(a.p.B));
    cfg.blockDim = dim3(kDecodeQuantThreads);
    cfg.stream = a.stream;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gqa_decode_quant_kernel<G, D>, p);
}

}  // namespace

cudaError_t launch_quant(const LaunchArgs& a, bool sliding, bool paged) {
    DecodeQuantParams p;
    p.d = a.p;
    p.cache.k = static_cast<uint8_t*>(const_cast<void*>(a.k));
    p.cache.v = static_cast<uint8_t*>(const_cast<void*>(a.v));
    p.cache.k_scales = const_cast<float*>(a.k_scales);
    p.cache.v_scales = const_cast<float*>(a.v_scales);
    p.cache.block_table = paged ? a.p.block_table : nullptr;
    p.cache.rows = static_cast<int>(a.rows);
    p.cache.max_pages = a.p.max_pages;
    p.cache.num_pages = a.p.num_pages;
    p.cache.KVH = a.p.KVH;
    return sliding ? launch<2, 256>(a, p) : launch<8, 512>(a, p);
}

}  // namespace gqa
