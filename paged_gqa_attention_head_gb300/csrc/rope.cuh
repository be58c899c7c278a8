// (cos, sin) of rotary angles in float arithmetic, shared by the decode with rotary embedding
// and the query/key preparation.
#pragma once

#include <cuda_runtime.h>

namespace sinkattn {
namespace {

// 2 pi as three floats for Cody and Waite's reduction: the first has 8 significant bits
// (201 / 32), the second is the float nearest to the rest, the third the float nearest to
// what remains after that.
constexpr float kTwoPi1 = 6.28125f;
constexpr float kTwoPi2 = 1.9353071693331003e-3f;
constexpr float kTwoPi3 = 1.0253376273028358e-11f;
constexpr float kInvTwoPi = 0.15915493667125702f;

// (cos, sin) of the angle p * (hi + lo), both times ms.  p is an integer position below
// 2^24 (exact in float).  The product is split exactly, p * hi = a_hi + a_err (one FMA),
// so the angle is a_hi + a_lo with a_lo = p * lo + a_err; the whole turns k = rint(a / 2 pi)
// come off in three FMAs against the three parts of 2 pi (k * kTwoPi1 is exact, and so is
// the first difference), which keeps the reduced angle within ~1e-6 rad of the exact one,
// where a float product p * theta alone would be off by up to ~1e-2 rad at p = 131072.
__device__ __forceinline__ float2 rope_cs(float p, float hi, float lo, float ms) {
    const float a_hi = p * hi;
    const float a_err = fmaf(p, hi, -a_hi);
    const float a_lo = fmaf(p, lo, a_err);
    const float k = rintf(a_hi * kInvTwoPi);
    float r = fmaf(-k, kTwoPi1, a_hi);
    r = fmaf(-k, kTwoPi2, r);
    r = fmaf(-k, kTwoPi3, r);
    r += a_lo;
    float s, c;
    sincosf(r, &s, &c);
    return make_float2(c * ms, s * ms);
}

}  // namespace
}  // namespace sinkattn
