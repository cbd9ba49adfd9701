// The activations of the projections' epilogues, in fp32.
#pragma once

#include <math.h>

#include "adafuse.h"

namespace af {

// v / (1 + exp(-w)) by the fast exponential and division: relative to the
// result off by (1.18 |w| + 7) 2^-23 at most.  The exponential is that of -|w|,
// which does not overflow: 1 + exp(-w) for w below -87 would be a divisor that
// the fast division takes to zero, where the result still is a number up to
// 1e-36.  With the exact division a tile's activations took longer than its
// products at d_in below 2000.
__device__ __forceinline__ float gate_by(float v, float w)
{
    const float e = __expf(-fabsf(w));
    return __fdividef(w < 0.f ? v * e : v, 1.f + e);
}

// v times the normal distribution's Q(v) = (1 + erf(v / sqrt 2)) / 2, whose
// plain form cancels for negative v (4 % off at -5, all digits at -6).  For x =
// |v| the tail Q(-x) = exp(-x^2 / 2) erfcx(x / sqrt 2) / 2, and the second factor
// is smooth in t = 1 / (1 + c x) over the whole half axis (the approach of
// Shepherd and Laframboise 1981): t P(t), with P of degree 8 fitted to the
// smallest relative error over x < 14.5, 2.6e-8.  No branch; relative to the
// result it is off by (0.84 v^2 + 10) 2^-23 at most, the first part from the
// exponential.  An epilogue of 2047 x 13824 bf16 takes 45-49 us with it (49-51
// with erff, 64 with erfcf), bound by instructions; silu 32.
__device__ __forceinline__ float gelu(float v)
{
    const float t = __fdividef(1.f, fmaf(0.34375f, fabsf(v), 1.f));
    float p = -0.027582375f;
    p = fmaf(p, t, 0.14280471f);
    p = fmaf(p, t, -0.26968193f);
    p = fmaf(p, t, 0.18874468f);
    p = fmaf(p, t, -0.037908636f);
    p = fmaf(p, t, 0.11210765f);
    p = fmaf(p, t, 0.11686955f);
    p = fmaf(p, t, 0.13752583f);
    p = fmaf(p, t, 0.13712054f);
    p *= t * __expf(-0.5f * v * v);
    return v * (v < 0.f ? p : 1.f - p);
}

__device__ __forceinline__ float activate(float v, uint32_t act)
{
    switch (act) {
        case ADAFUSE_ACT_RELU: return v < 0.f ? 0.f : v;
        case ADAFUSE_ACT_SILU: return gate_by(v, v);
        case ADAFUSE_ACT_GELU: return gelu(v);
        // (1 + tanh u) / 2 = 1 / (1 + exp(-2u)) with u = sqrt(2/pi) (v + 0.044715 v^3)
        case ADAFUSE_ACT_GELU_TANH: return gate_by(v, 1.59576912f * (v + 0.044715f * v * v * v));
        default: return v;
    }
}

// The same for N values, the choice made once.
template <int N>
__device__ __forceinline__ void activate_all(float (&v)[N], uint32_t act)
{
    switch (act) {
        case ADAFUSE_ACT_NONE: return;
        case ADAFUSE_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = activate(v[i], ADAFUSE_ACT_RELU);
            return;
        case ADAFUSE_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = activate(v[i], ADAFUSE_ACT_SILU);
            return;
        case ADAFUSE_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = activate(v[i], ADAFUSE_ACT_GELU);
            return;
        default:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = activate(v[i], ADAFUSE_ACT_GELU_TANH);
            return;
    }
}

}  // namespace af
