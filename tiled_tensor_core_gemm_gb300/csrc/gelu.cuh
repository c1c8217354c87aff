// GELU of the operators' epilogues.
#pragma once

#include "ptx_ops.cuh"

namespace tcgemm {

// x * Phi(x), two values at a time.  Phi(-a) = 2^-P(a) for a = |x| >= 0, P a
// polynomial of degree 8 fitted to -log2 Phi(-a) on [0, 5.5] (least squares in
// the Chebyshev basis, reweighted towards the largest error in Phi; 4e-8 in FP32
// arithmetic, where erf's own rounding leaves 6e-8) and above 25 beyond, where
// Phi(-a) no longer counts.  One exponential and eight paired multiply-adds,
// where erff takes about thirty instructions.
__device__ __forceinline__ float2 gelu2(float2 x) {
    const float2 a = make_float2(fabsf(x.x), fabsf(x.y));
    auto both = [](float c) { return make_float2(c, c); };
    float2 r = both(-2.7720716e-06f);                       // -P
    r = __ffma2_rn(r, a, both(3.8620983e-05f));
    r = __ffma2_rn(r, a, both(-1.8254861e-04f));
    r = __ffma2_rn(r, a, both(-1.4586786e-04f));
    r = __ffma2_rn(r, a, both(7.0754690e-03f));
    r = __ffma2_rn(r, a, both(-5.2505028e-02f));
    r = __ffma2_rn(r, a, both(-4.5920491e-01f));
    r = __ffma2_rn(r, a, both(-1.1511058e+00f));
    r = __ffma2_rn(r, a, both(-1.0f));
    const float hx = ptx::exp2_approx(r.x), hy = ptx::exp2_approx(r.y);
    return make_float2(x.x * (x.x > 0.f ? 1.f - hx : hx), x.y * (x.y > 0.f ? 1.f - hy : hy));
}

}  // namespace tcgemm
