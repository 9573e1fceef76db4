// Arithmetic on unevaluated sums of two floats (Knuth's exact sum and Dekker's product, with
// an fma for the product's error), for results good to some 2^-30 and better from fp32
// instructions, of which an SM issues 128 a clock against 2 in fp64.
#pragma once

#include <stdint.h>

namespace gqa {

struct Twofold {
    float h, l;   // value h + l, |l| at most a few ulps of h
};

// The nearest Twofold of a constant.
constexpr __host__ __device__ Twofold twofold(double c) {
    return Twofold{static_cast<float>(c), static_cast<float>(c - static_cast<double>(static_cast<float>(c)))};
}

// a + b, exact.  (The _rn forms are not contracted into other operations.)
__device__ __forceinline__ Twofold fast_sum(float a, float b) {   // |a| >= |b|
    const float h = __fadd_rn(a, b);
    return Twofold{h, __fsub_rn(b, __fsub_rn(h, a))};
}
__device__ __forceinline__ Twofold exact_sum(float a, float b) {
    const float h = __fadd_rn(a, b), t = __fsub_rn(h, a);
    return Twofold{h, __fadd_rn(__fsub_rn(a, __fsub_rn(h, t)), __fsub_rn(b, t))};
}

__device__ __forceinline__ Twofold add(Twofold a, Twofold b) {
    const Twofold s = exact_sum(a.h, b.h);
    return Twofold{s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l))};
}

__device__ __forceinline__ Twofold mul(Twofold a, float b) {
    const float h = __fmul_rn(a.h, b);
    return Twofold{h, __fmaf_rn(a.l, b, __fmaf_rn(a.h, b, -h))};
}

__device__ __forceinline__ Twofold mul(Twofold a, Twofold b) {
    const float h = __fmul_rn(a.h, b.h);
    return Twofold{h, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.h, b.h, -h)))};
}

__device__ __forceinline__ Twofold neg(Twofold a) { return Twofold{-a.h, -a.l}; }

// 1 / sqrt(a), a > 0: one Newton step with its residual 1 - a y^2.  An infinite or NaN a gives
// 1 / sqrtf(a) alone.
__device__ __forceinline__ Twofold reciprocal_sqrt(Twofold a) {
    const float y = 1.0f / sqrtf(a.h);
    if (!(a.h < INFINITY)) return Twofold{y, 0.0f};
    const Twofold p = mul(mul(a, y), y);
    return Twofold{y, __fmul_rn(0.5f * y, __fsub_rn(__fsub_rn(1.0f, p.h), p.l))};
}

// a in one float that rounds as a does to any type of at most 22 bits: cut off at 24 bits, the
// last set when something was.
__device__ __forceinline__ float to_odd(Twofold a) {
    const Twofold t = fast_sum(a.h, a.l);
    const int h = __float_as_int(t.h), cut = h + ((h ^ __float_as_int(t.l)) >> 31);
    return t.l == 0.0f ? t.h : __int_as_float(cut | 1);
}

// (cos, sin) of 2 pi f / 2^64 to 2^-30: whole quarters of a turn are taken off in integers, the
// rest, at most pi / 4, goes through the Taylor series, whose first terms need two floats.
__device__ __forceinline__ void cos_sin_of_turn(uint64_t f, Twofold* c, Twofold* s) {
    const uint64_t quarter = (f + (1ull << 61)) >> 62;
    const int64_t r = static_cast<int64_t>(f - (quarter << 62));   // [-2^61, 2^61)
    // the upper 48 bits, in two floats of 24
    const float r_h = static_cast<float>(static_cast<int32_t>(r >> 38) << 6) * 0x1p-32f;
    const float r_l = static_cast<float>(static_cast<int32_t>((r >> 14) & 0xffffff)) * 0x1p-50f;
    const Twofold a = mul(twofold(6.283185307179586), fast_sum(r_h, r_l));
    const Twofold z = mul(a, a);
    const float zz = z.h;
    // a0 + z (a1 + ...): the constant's and the product's low parts are kept
    auto step = [&](Twofold a0, float hi, float lo) {
        Twofold t = fast_sum(a0.h, hi);
        t.l += lo + a0.l;
        return t;
    };
    Twofold co = step(twofold(1.0 / 24.0),
                      zz * fmaf(fmaf(zz, -1.0f / 3628800.0f, 1.0f / 40320.0f), zz, -1.0f / 720.0f), 0.0f);
    co = mul(z, co);
    co = mul(z, step(twofold(-0.5), co.h, co.l));
    co = step(twofold(1.0), co.h, co.l);
    Twofold si = step(twofold(-1.0 / 6.0),
                      zz * fmaf(fmaf(fmaf(zz, -1.0f / 39916800.0f, 1.0f / 362880.0f), zz, -1.0f / 5040.0f), zz,
                                1.0f / 120.0f), 0.0f);
    si = mul(z, si);
    si = mul(step(twofold(1.0), si.h, si.l), a);
    const bool swap = quarter & 1;
    const Twofold u = swap ? si : co, v = swap ? co : si;
    *c = ((quarter + 1) & 2) ? neg(u) : u;
    *s = (quarter & 2) ? neg(v) : v;
}

// The same with the high parts the nearest floats (above they are off by up to 1.9 x 2^-24, as the low
// parts are).
__device__ __forceinline__ void cos_sin_nearest(uint64_t f, Twofold* c, Twofold* s) {
    cos_sin_of_turn(f, c, s);
    *c = fast_sum(c->h, c->l);
    *s = fast_sum(s->h, s->l);
}

}  // namespace gqa
