// The activations of the matrix product's epilogue and their slopes, in fp32:
// silu(p) = p sigmoid(p), gelu(p) = p (1 + erf(p / sqrt 2)) / 2, relu.
#pragma once

#include "launch.h"

__device__ __forceinline__ float ssd_act(float p, SsdAct act) {
    switch (act) {
        case SsdAct::silu: return ssd_silu(p);
        case SsdAct::gelu: return 0.5f * p * (1.f + erff(p * 0.70710678f));
        case SsdAct::relu: return p < 0.f ? 0.f : p;
        default: return p;
    }
}

__device__ __forceinline__ float ssd_act_slope(float p, SsdAct act) {
    switch (act) {
        case SsdAct::silu: {
            const float sig = __fdividef(1.f, 1.f + __expf(-p));
            return sig * (1.f + p * (1.f - sig));
        }
        case SsdAct::gelu:
            return 0.5f * (1.f + erff(p * 0.70710678f)) +
                   p * 0.39894228f * __expf(-0.5f * p * p);
        case SsdAct::relu: return p > 0.f ? 1.f : 0.f;
        default: return 1.f;
    }
}
