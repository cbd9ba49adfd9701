// The activations of the projections' epilogues, in fp32.
#pragma once

#include <math.h>

#include "adafuse.h"

namespace af {

// v / (1 + exp(-w)) by the fast exponential and division (a few fp32 steps
// each; both limits of w give v and 0).  With the exact division a tile's
// activations took longer than its products at d_in below 2000.
__device__ __forceinline__ float gate_by(float v, float w) { return __fdividef(v, 1.f + __expf(-w)); }

__device__ __forceinline__ float activate(float v, uint32_t act)
{
    switch (act) {
        case ADAFUSE_ACT_RELU: return v < 0.f ? 0.f : v;
        case ADAFUSE_ACT_SILU: return gate_by(v, v);
        case ADAFUSE_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678f));
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
