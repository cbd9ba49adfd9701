// The activations of the projections' epilogues, in fp32.
#pragma once

#include <math.h>

#include "adafuse.h"

namespace af {

__device__ __forceinline__ float activate(float v, uint32_t act)
{
    switch (act) {
        case ADAFUSE_ACT_RELU: return v < 0.f ? 0.f : v;
        case ADAFUSE_ACT_SILU: return v / (1.f + expf(-v));
        case ADAFUSE_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678f));
        case ADAFUSE_ACT_GELU_TANH: {
            const float u = 0.79788456f * (v + 0.044715f * v * v * v);
            return 0.5f * v * (1.f + tanhf(u));
        }
        default: return v;
    }
}

}  // namespace af
