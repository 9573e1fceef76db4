// Decode attention kernels over the 4-bit cache, both geometries, contiguous and paged.
#include <mutex>

#include "kernels/combine_kernel.cuh"
#include "kernels/decode_nibble_kernel.cuh"
#include "launch.h"

namespace gqa {

namespace {

template <class Pol, bool kPaged>
cudaError_t launch(const LaunchArgs& a, const DecodeNibbleParams& params) {
    constexpr size_t kSmem = sizeof(NibbleSmem<Pol>) + 128;   // + alignment slack
    static_assert(kSmem <= 227 * 1024, "shared memory");
    constexpr int kMaxDevices = 64;
    static std::once_flag once[kMaxDevices];
    static cudaError_t attr_err[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        attr_err[dev] = cudaFuncSetAttribute(gqa_decode_nibble_kernel<Pol, kPaged>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kSmem));
        // The consumers take the registers that the producers give back of those the block is launched
        // with: fewer at launch would leave them waiting.
        cudaFuncAttributes fa;
        if (attr_err[dev] == cudaSuccess)
            attr_err[dev] = cudaFuncGetAttributes(&fa, gqa_decode_nibble_kernel<Pol, kPaged>);
        if (attr_err[dev] == cudaSuccess && fa.numRegs < Pol::kLaunchRegs)
            attr_err[dev] = cudaErrorInvalidConfiguration;
    });
    if (attr_err[dev] != cudaSuccess) return attr_err[dev];

    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // The workspace's kMaxCtas + B KVH + kMaxDynUnits partial slots: this kernel's units take
    // the first `units` + B KVH, its dynamic chunks the rest (at least a quarter of theirs).
    constexpr int kMostUnits = kMaxCtas + kMaxDynUnits * 3 / 4;
    const int grid = a.grid < kMostUnits / Pol::GROUPS ? a.grid : kMostUnits / Pol::GROUPS;
    const int units = grid * Pol::GROUPS;
    DecodeNibbleParams p = params;
    p.d.dyn_slot_base = units + a.p.B * a.p.KVH;
    p.d.max_dyn = kMaxCtas + kMaxDynUnits - units < kMaxDynUnits ? kMaxCtas + kMaxDynUnits - units
                                                                 : kMaxDynUnits;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(Pol::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = a.stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gqa_decode_nibble_kernel<Pol, kPaged>, p);
    if (e != cudaSuccess) return e;

    // split segments, as over the 8-bit cache (kernels_quant.cu has what both forms measure)
    const int segments = a.p.B * a.p.KVH;
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

cudaError_t launch_nibble(const LaunchArgs& a, bool sliding, bool paged) {
    DecodeNibbleParams p;
    p.d = a.p;
    p.kv = static_cast<const uint8_t*>(a.k);
    p.rows = static_cast<int>(a.rows);
    if (sliding) return paged ? launch<NibbleSliding, true>(a, p) : launch<NibbleSliding, false>(a, p);
    return paged ? launch<NibbleGlobal, true>(a, p) : launch<NibbleGlobal, false>(a, p);
}

}  // namespace gqa
