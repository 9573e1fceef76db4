// Decode attention kernels over the 4-bit cache, both geometries.
#include "kernels/decode_nibble_kernel.cuh"
#include "launch.h"

namespace gqa {

cudaError_t launch_nibble(const LaunchArgs& a, bool sliding) {
    DecodeNibbleParams p;
    p.d = a.p;
    p.cache.kv = static_cast<uint8_t*>(const_cast<void*>(a.k));
    p.cache.block_table = a.p.block_table;
    p.cache.rows = static_cast<int>(a.rows);
    p.cache.max_pages = a.p.max_pages;
    p.cache.num_pages = a.p.num_pages;
    p.cache.planes = sliding ? 16 : 8;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.p.B * a.p.KVH));
    cfg.blockDim = dim3(kDecodeNibbleWarps * 32);
    cfg.stream = a.stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return sliding ? cudaLaunchKernelEx(&cfg, gqa_decode_nibble_kernel<2, 256>, p)
                   : cudaLaunchKernelEx(&cfg, gqa_decode_nibble_kernel<8, 512>, p);
}

}  // namespace gqa
