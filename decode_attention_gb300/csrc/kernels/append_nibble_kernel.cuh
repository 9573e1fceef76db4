// Quantising K/V rows into the 4-bit cache (nibble_cache.cuh).
//
// One item is a token's K and V in kPlanes planes (512 bytes each in bf16), taken by a warp:
// lane l holds channels 8l .. 8l + 7 of each, four lanes share a scale, and a lane's codes are one
// word of the row.  Rows stand by themselves, so there is no order between items and nothing is
// read back.
//
// Bound by the memory's rate: 65500 tokens of slidingDecodeGQA in 220 us, 0.91 of a copy's rate (with codes in
// floating point and by comparisons 307 us, with a branch for each of their seldom cases 228).  Four planes
// an item put eight loads of a lane in flight.  (A row is eight sectors and a half; the shared ones meet in L2.)
#pragma once

#include "nibble_cache.cuh"

namespace gqa {

constexpr int kAppendNibbleThreads = 256;

struct AppendNibbleParams {
    const __nv_bfloat16* k_new;     // [N, KVH, D]
    const __nv_bfloat16* v_new;     // [N, KVH, D]
    const int32_t* token_offsets;   // [B + 1]
    const int32_t* seq_lens;        // [B], lengths after the append
    NibbleCache cache;
    int B, N;
};

template <int kPlanes>
__global__ void __launch_bounds__(kAppendNibbleThreads)
    gqa_append_nibble_kernel(const AppendNibbleParams p) {
    __shared__ TokenIndex idx;
    ptx::grid_dependency_wait();
    ptx::allow_dependent_launch();
    idx.load(p.token_offsets, p.seq_lens, p.B);

    const NibbleCache& c = p.cache;
    const int lane = threadIdx.x & 31;
    const uint32_t per_token = static_cast<uint32_t>(c.planes / kPlanes);
    const int capacity = c.capacity();
    const size_t stride = c.plane_stride();
    const uint32_t total = static_cast<uint32_t>(p.N) * per_token;   // (N <= 2^26, planes <= 16)
    constexpr int kWarps = kAppendNibbleThreads / 32;
    for (uint32_t it = blockIdx.x * kWarps + (threadIdx.x >> 5); it < total; it += gridDim.x * kWarps) {
        const int i = static_cast<int>(it / per_token);
        const int plane = static_cast<int>(it % per_token) * kPlanes;
        const size_t src = (static_cast<size_t>(i) * c.planes + plane) * kNibblePlane + lane * 8;
        uint4 k[kPlanes], v[kPlanes];
#pragma unroll
        for (int j = 0; j < kPlanes; ++j) {
            k[j] = __ldcs(reinterpret_cast<const uint4*>(p.k_new + src + j * kNibblePlane));
            v[j] = __ldcs(reinterpret_cast<const uint4*>(p.v_new + src + j * kNibblePlane));
        }
        int b, pos;
        if (!idx.find(p.B, p.N, i, &b, &pos) || idx.len[b] > capacity) continue;
        uint8_t* row = c.row(b, pos);
        if (!row) continue;
        row += plane * stride;
#pragma unroll
        for (int j = 0; j < kPlanes; ++j) {
            uint32_t ks, vs;
            const uint32_t ku[4] = {k[j].x, k[j].y, k[j].z, k[j].w}, vu[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            const uint32_t kw = nibble_codes(ku, &ks), vw = nibble_codes(vu, &vs);
            uint8_t* r = row + j * stride;
            reinterpret_cast<uint32_t*>(r)[lane] = kw;
            reinterpret_cast<uint32_t*>(r + kNibblePlane / 2)[lane] = vw;
            ks = __shfl_sync(0xffffffffu, ks, (lane & 7) * 4);
            vs = __shfl_sync(0xffffffffu, vs, (lane & 7) * 4);
            if (lane < 16) r[kNibbleScales + lane] = static_cast<uint8_t>(lane < 8 ? ks : vs);
        }
    }
}

}  // namespace gqa
