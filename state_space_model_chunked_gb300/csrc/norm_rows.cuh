// What the norms' kernels share: a row in a CTA's registers, the sums over it, the scale
// of an 8-bit row, and how many threads a row takes.
#pragma once

#include "launch.h"
#include "vec.cuh"

namespace ssdnorm {

constexpr float kE4m3Max = 448.f;
constexpr int kMostWarps = 16;      // a row's CTA: 128 registers a thread

// The CTA's sum, and with kMax its maximum, over its warps (any number of them up to 32).
template <bool kMax>
__device__ __forceinline__ void cta_sum_max(float &sum, float &mx, float (*buf)[32]) {
    sum = ssd_warp_sum(sum);
    if constexpr (kMax) mx = ssd_warp_max(mx);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        buf[0][warp] = sum;
        if constexpr (kMax) buf[1][warp] = mx;
    }
    __syncthreads();
    sum = ssd_warp_sum(lane < warps ? buf[0][lane] : 0.f);
    if constexpr (kMax) mx = ssd_warp_max(lane < warps ? buf[1][lane] : 0.f);
}

// The scale of an 8-bit row and the rounding of one of its values.  Below
// 1e-30 the reciprocal of the scale would leave fp32's range, so those rows
// divide.
struct RowScale {
    float scale, inv;
    bool tiny;
    __device__ __forceinline__ explicit RowScale(float amax) {
        scale = amax / kE4m3Max;
        if (scale == 0.f) scale = 1.f;      // zeros, or values below 3e-43, which are 0 too
        tiny = scale < 1e-30f;
        inv = 1.f / scale;
    }
    __device__ __forceinline__ float apply(float y) const { return tiny ? y / scale : y * inv; }
};

// kC runs of V values of a row: run c of this thread starts at value
// (threadIdx.x + c * blockDim.x) * V; runs past the row read as zero.
template <typename T, int V, int kC>
struct Row {
    SsdRaw<T, V> run[kC];
    __device__ __forceinline__ void load(const T *row, int nvec, bool on) {
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int i = threadIdx.x + c * blockDim.x;
            run[c].zero();
            if (on && i < nvec) run[c].load_cs(row + (size_t)i * V);
        }
    }
};
template <int V, int kC>
__device__ __forceinline__ void load_weight(const float *weight, int nvec, float (&w)[kC][V]) {
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        const int i = threadIdx.x + c * blockDim.x;
        SsdRaw<float, V> r;
        r.zero();
        if (i < nvec) r.load(weight + (size_t)i * V);
#pragma unroll
        for (int k = 0; k < V; ++k) w[c][k] = r.get(k);
    }
}

// Threads and runs a thread for one row: at most `most_runs` runs of V values a
// thread (`want` where the warps allow it), a power of two of warps; 0 warps
// when the row does not fit.
struct RowShape {
    int warps, runs;
};
inline RowShape row_shape(int width, int V, int most_runs, int want) {
    const int nvec = (width + V - 1) / V;
    int w = 1;
    while (w < kMostWarps && (long long)w * 32 * want < nvec) w *= 2;
    const int runs = (nvec + w * 32 - 1) / (w * 32);
    return {runs <= most_runs ? w : 0, runs};
}

// CTAs of a walk over rows: as many as the SMs hold at once.
inline unsigned walkers(long long rows, int sms, int ctas) {
    const long long n = (long long)sms * ctas;
    return (unsigned)(rows < n ? rows : n);
}

inline bool vec8(const void *p, long long stride, int size) {
    return p == nullptr || (((uintptr_t)p & 15u) == 0 && (stride * size) % 16 == 0);
}

}  // namespace ssdnorm
