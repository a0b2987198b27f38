// The activations of the matrix product's epilogue and their slopes, in fp32:
// silu(p) = p sigmoid(p), gelu(p) = p (1 + erf(p / sqrt 2)) / 2, relu.
#pragma once

#include "launch.h"
#include "ptx.cuh"

// 1 / (1 + e^-p) by the hardware's exponential and reciprocal, to (1.25 |p| + 8) 2^-24
// of itself (the exponential's argument is one rounded product); below p = -87 it
// runs out of fp32's normal range and is 0.
__device__ __forceinline__ float ssd_sigmoid(float p) {
    return ssdptx::rcp_approx(1.f + ssdptx::ex2_approx(p * -1.44269504f));
}

// The normal distribution's density at p, and its tail beyond |p|: 1 - Phi(|p|) =
// (a1 t + a2 t^2 + a3 t^3 + a4 t^4 + a5 t^5) e^(-p^2/2) / 2, t = 1 / (1 + b |p| / sqrt 2),
// Abramowitz and Stegun's 7.1.26 (error of erf below 1.5e-7).  erff takes three
// times the instructions and bound the activation's backward pass.
struct SsdNormal {
    float density, below;       // below = Phi(p)
    __device__ __forceinline__ explicit SsdNormal(float p) {
        const float t = ssdptx::rcp_approx(1.f + 0.3275911f * 0.70710678f * fabsf(p));
        const float e = ssdptx::ex2_approx(p * p * (-0.5f * 1.44269504f));
        const float q = 0.5f * e * t *
                        (0.254829592f +
                         t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
        density = 0.39894228f * e;
        below = p < 0.f ? q : 1.f - q;
    }
};

__device__ __forceinline__ float ssd_act(float p, SsdAct act) {
    switch (act) {
        case SsdAct::silu: return p * ssd_sigmoid(p);
        case SsdAct::gelu: return p * SsdNormal(p).below;
        case SsdAct::relu: return p < 0.f ? 0.f : p;
        default: return p;
    }
}

__device__ __forceinline__ float ssd_act_slope(float p, SsdAct act) {
    switch (act) {
        case SsdAct::silu: {
            const float sig = ssd_sigmoid(p);
            return sig * (1.f + p * (1.f - sig));
        }
        case SsdAct::gelu: {
            const SsdNormal f(p);
            return f.below + p * f.density;
        }
        case SsdAct::relu: return p > 0.f ? 1.f : 0.f;
        default: return 1.f;
    }
}

// Single elements of the product's output types, and the epilogue of one of its
// values: token m, feature n.
__device__ __forceinline__ float ssd_elt_load(const void *p, long long i, SsdElt t) {
    return t == SSD_ELT_F32 ? static_cast<const float *>(p)[i]
                            : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void ssd_elt_store(void *p, long long i, SsdElt t, float v) {
    if (t == SSD_ELT_F32) static_cast<float *>(p)[i] = v;
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void ssd_finish(const SsdProduct &p, long long m, long long n, float v) {
    if (p.a_scale) v = v * p.a_scale[m] * p.b_scale[n];     // two small scales' product may underflow
    if (p.bias) v += p.bias[n];
    if (p.preact) ssd_elt_store(p.preact, m * p.n + n, p.preact_type, v);
    v = ssd_act(v, p.act);
    if (p.residual) v += ssd_elt_load(p.residual, m * p.residual_row + n, p.out_type);
    ssd_elt_store(p.out, m * p.out_row + n, p.out_type, v);
}
