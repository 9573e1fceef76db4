// Decode attention kernels over the 8-bit cache, both geometries, contiguous and paged.
#include <mutex>

#include "kernels/combine_kernel.cuh"
#include "kernels/decode_quant_kernel.cuh"
#include "launch.h"

namespace gqa {

namespace {

// Tensor map of K or V codes: 4-D view (128 codes, row, 128-code chunk of the KVH * D row,
// outer), box (128, 16, D / 128, 1) -> shared [D / 128][16 rows][128 B], 16-byte units
// permuted by row so that 8 consecutive rows of one chunk hit distinct banks.
bool encode_codes_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t outer, int KVH,
                      int D) {
    const uint64_t row_bytes = static_cast<uint64_t>(KVH) * D;
    const cuuint64_t dims[4] = {128, rows, row_bytes / 128, outer};
    const cuuint64_t strides[3] = {row_bytes, 128, row_bytes * rows};
    const cuuint32_t box[4] = {128, kQuantBlock, static_cast<cuuint32_t>(D / 128), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims,
                            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Pol, bool kPaged>
cudaError_t launch(const LaunchArgs& a, const DecodeQuantParams& params) {
    constexpr size_t kSmem = sizeof(QuantSmem<Pol>) + 1024;   // + alignment slack
    static_assert(kSmem <= 227 * 1024, "shared memory");
    constexpr int kMaxDevices = 64;
    static std::once_flag once[kMaxDevices];
    static cudaError_t attr_err[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        attr_err[dev] = cudaFuncSetAttribute(gqa_decode_quant_kernel<Pol, kPaged>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kSmem));
    });
    if (attr_err[dev] != cudaSuccess) return attr_err[dev];
    CUtensorMap tm_k, tm_v;
    if (!encode_codes_map(&tm_k, a.k, a.rows, a.outer, a.p.KVH, Pol::D) ||
        !encode_codes_map(&tm_v, a.v, a.rows, a.outer, a.p.KVH, Pol::D))
        return cudaErrorInvalidValue;

    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // The workspace's kMaxCtas + B KVH + kMaxDynUnits partial slots: this kernel's units take
    // the first `units` + B KVH, its dynamic chunks the rest (at least a quarter of theirs).
    constexpr int kMostUnits = kMaxCtas + kMaxDynUnits * 3 / 4;
    const int grid = a.grid < kMostUnits / Pol::GROUPS ? a.grid : kMostUnits / Pol::GROUPS;
    const int units = grid * Pol::GROUPS;
    DecodeQuantParams p = params;
    p.d.dyn_slot_base = units + a.p.B * a.p.KVH;
    p.d.max_dyn = kMaxCtas + kMaxDynUnits - units < kMaxDynUnits ? kMaxCtas + kMaxDynUnits - units
                                                                 : kMaxDynUnits;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(Pol::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = a.stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gqa_decode_quant_kernel<Pol, kPaged>, tm_k, tm_v, p);
    if (e != cudaSuccess) return e;

    const int segments = a.p.B * a.p.KVH;
    // Up to four of its small items per SM the wide form is faster (up to 1024 / 4096 positions,
    // narrow and wide: g = 2, B = 1 9.5 / 9.5 and 8.5 / 8.5 us, B = 8 14.1 / 17.9 and 13.9 /
    // 17.8; g = 8, B = 1 12.4 / 15.1 and 9.6 / 11.2, B = 4 11.7 / 17.1 and 10.6 / 15.0), beyond
    // that its blocks cost more than they hide (B = 12, g = 2 23.2 and 23.8; B = 6, g = 8 19.4 and
    // 19.8; B = 36 67 and 73).
    const bool wide = segments * (Pol::G * Pol::D / 128) <= 4 * grid;
    const int chunk = wide ? 128 : 4 * kCombineThreads;   // outputs per item
    const int items = segments * ((Pol::G * Pol::D + chunk - 1) / chunk);
    const int most = kCombineBlocksPerSm * grid;
    cudaLaunchConfig_t ccfg = cfg;
    ccfg.gridDim = dim3(static_cast<unsigned>(items < most ? items : most));
    ccfg.blockDim = dim3(kCombineThreads);
    ccfg.dynamicSmemBytes = 0;
    if (wide) return cudaLaunchKernelEx(&ccfg, gqa_combine_wide_kernel<Pol::G, Pol::D>, p.d, segments);
    return cudaLaunchKernelEx(&ccfg, gqa_combine_kernel<Pol::G, Pol::D, true>, p.d, segments);
}

}  // namespace

cudaError_t launch_quant(const LaunchArgs& a, bool sliding, bool paged) {
    DecodeQuantParams p;
    p.d = a.p;
    p.k_scales = a.k_scales;
    p.v_scales = a.v_scales;
    p.blocks = static_cast<int>((a.rows + kQuantBlock - 1) / kQuantBlock);
    // Many segments: each CTA meets several pieces, whatever the lengths (which the host does
    // not know), and smaller units overlap more of their ends.  In a graph, large / small units:
    // g = 8 and one segment per CTA (B = 40) at most 16, 256, 1024, 4096 positions 13.7 / 10.4,
    // 18.8 / 18.6, 28.5 / 28.5, 73.3 / 71.6 us; two (B = 72) 15.1 / 11.7, 25.2 / 23.0, 47.3 / 43.0,
    // 116.2 / 116.0; with fewer than one, up to 37% slower.  g = 2 and one (B = 10) 8.3 / 8.0,
    // 11.4 / 11.3, 16.5 / 16.7, 20.6 / 20.8; two (B = 20) 10.9 / 8.3, 14.0 / 13.9, 23.3 / 23.7,
    // 33.5 / 33.4.
    const bool many = a.p.B * a.p.KVH >= (sliding ? 2 : 1) * a.grid;
    if (sliding && many)
        return paged ? launch<QuantSlidingMany, true>(a, p) : launch<QuantSlidingMany, false>(a, p);
    if (sliding) return paged ? launch<QuantSliding, true>(a, p) : launch<QuantSliding, false>(a, p);
    if (many)
        return paged ? launch<QuantGlobalMany, true>(a, p) : launch<QuantGlobalMany, false>(a, p);
    return paged ? launch<QuantGlobal, true>(a, p) : launch<QuantGlobal, false>(a, p);
}

}  // namespace gqa
