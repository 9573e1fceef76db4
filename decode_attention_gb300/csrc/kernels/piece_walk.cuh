// The pieces of a unit of the plan (decode_kernel.cuh) in kernels whose pieces start and end on
// blocks of positions (the 8-bit and the 4-bit cache's).
#pragma once

#include "decode_kernel.cuh"

namespace gqa {

// One piece of work.
struct BlockPiece {
    int b, kvh;
    int p0, p1;     // positions, whole blocks
    int lo, hi;     // attended positions of the sequence
    int slot;       // workspace slot of the partial; -1: the piece is the whole segment
    int done;       // no more pieces
};

// The static pieces of one unit of the plan in order: a search and a division for the first (on
// every call's way to its first copy), steps from there.  Each segment's tiles begin with kExtra
// that hold no positions.
template <class Tune>
struct StaticWalk {
    static constexpr int kExtra = Tune::kExtra, kBlock = Tune::kAlign;
    uint32_t x, stop;   // the unit's tiles
    int b, kvh, k;      // the segment that holds tile x, and x's place in it

    __device__ __forceinline__ static int tiles(const PlanSmem& pl, int b) {
        return kExtra + pl.sn[b] / kBlock;   // (sn is whole blocks)
    }
    __device__ __forceinline__ StaticWalk(const PlanSmem& pl, int B, uint32_t first, uint32_t end)
        : x(first), stop(end), b(0), kvh(0), k(0) {
        if (x >= stop) return;
        b = upper_seq(pl.spref, B, x);
        const uint32_t st = static_cast<uint32_t>(tiles(pl, b)), rel = x - pl.spref[b];
        kvh = static_cast<int>(rel / st);
        k = static_cast<int>(rel - static_cast<uint32_t>(kvh) * st);
    }
    __device__ __forceinline__ bool next(const PlanSmem& pl, int KVH, int unit, Piece& w) {
        while (x < stop) {
            const int st = tiles(pl, b), k0 = k;
            const int take = min(static_cast<int>(min(stop - x, 0x7fffffffu)), st - k0);
            w.b = b;
            w.kvh = kvh;
            w.p0 = pl.lo[b] + max(k0 - kExtra, 0) * kBlock;
            w.p1 = pl.lo[b] + (k0 + take - kExtra) * kBlock;
            w.slot = unit + b * KVH + kvh;
            x += static_cast<uint32_t>(take);
            k += take;
            if (k == st) {
                k = 0;
                if (++kvh == KVH) {
                    kvh = 0;
                    if (x < stop)
                        do ++b;
                        while (pl.sn[b] == 0);   // (ends: tile x is in a later sequence)
                }
            }
            if (k0 + take > kExtra) return true;   // else only tiles without positions
        }
        return false;
    }
};

}  // namespace gqa
