// Gated linear recurrence, elementwise over the channels of each token:
//
//   f_t = sigmoid(g_t),  h_t = f_t h_{t-1} + (1 - f_t) x_t,  y_t = h_t silu(z_t)
//
// and its gradients: with dh_t = dy_t silu(z_t) (+ dfinal at a sequence's last
// token) and lam_t = dh_t + f_{t+1} lam_{t+1},
//
//   dx_t = (1 - f_t) lam_t,      dg_t = lam_t (h_{t-1} - x_t) f_t (1 - f_t),
//   dz_t = dy_t h_t silu'(z_t),  dinit = f_0 lam_0.
//
// f and 1 - f = sigmoid(-g) each keep their full relative precision; states and gradients are carried in fp32.
#include "launch.h"
#include "vec.cuh"

namespace {

constexpr int kEvery = kSsdCheckpointTokens;

// f = sigmoid(g) and 1 - f = sigmoid(-g).  The smaller of the two is
// e / (1 + e) with e = e^-|g|, to a few 2^-23 of itself; the larger is 1 minus
// it, rounded to nearest: its error has no sign, so it does not add up along a
// memory of thousands of tokens (1 / (1 + e) from the approximate reciprocal
// erred to one side and did).
struct Gate {
    float keep, drop;
    __device__ __forceinline__ explicit Gate(float g) {
        const float e = __expf(-fabsf(g));
        const float small = __fdividef(e, 1.f + e), big = 1.f - small;
        keep = g >= 0.f ? big : small;
        drop = g >= 0.f ? small : big;
    }
};
__device__ __forceinline__ float sigmoidf(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

__device__ __forceinline__ void seq_range(const SsdGated &a, int s, long long &t0, long long &t1) {
    t0 = a.cu ? a.cu[s] : (long long)s * a.length;
    t1 = a.cu ? a.cu[s + 1] : t0 + a.length;
}

template <typename T>
__global__ void __launch_bounds__(128) gated_fwd_kernel(const SsdGatedFwd a) {
    const int c = blockIdx.x * 128 + threadIdx.x, s = blockIdx.y;
    if (c >= a.in.width) return;
    long long t0, t1;
    seq_range(a.in, s, t0, t1);
    float h = a.in.init ? a.in.init[(size_t)s * a.in.width + c] : 0.f;
    for (long long t = t0; t < t1; ++t) {
        if (a.checkpoints && t % kEvery == 0) a.checkpoints[(size_t)(t / kEvery) * a.in.width + c] = h;
        const float x = ssd_ld(static_cast<const T *>(a.in.x) + t * a.in.x_stride + c);
        const Gate f(ssd_ld(static_cast<const T *>(a.in.g) + t * a.in.g_stride + c));
        h = f.keep * h + f.drop * x;
        float y = h;
        if (a.in.z) {
            const float z = ssd_ld(static_cast<const T *>(a.in.z) + t * a.in.z_stride + c);
            y = h * z * sigmoidf(z);
        }
        ssd_st(static_cast<T *>(a.y) + t * a.y_stride + c, y);
    }
    if (a.final_state) a.final_state[(size_t)s * a.in.width + c] = h;
}

template <typename T>
__global__ void __launch_bounds__(128) gated_bwd_kernel(const SsdGatedBwd a) {
    const int c = blockIdx.x * 128 + threadIdx.x, s = blockIdx.y;
    if (c >= a.in.width) return;
    long long t0, t1;
    seq_range(a.in, s, t0, t1);
    const float init = a.in.init ? a.in.init[(size_t)s * a.in.width + c] : 0.f;
    float carry = a.dfinal ? a.dfinal[(size_t)s * a.in.width + c] : 0.f;   // f_{t+1} lam_{t+1}
    float before[kEvery];
    for (long long e = t1; e > t0;) {
        // the block of tokens [b, e) that starts at a kept state or at the sequence's start
        long long b = (e - 1) / kEvery * kEvery;
        float h = b >= t0 ? a.checkpoints[(size_t)(b / kEvery) * a.in.width + c] : init;
        if (b < t0) b = t0;
        for (long long t = b; t < e; ++t) {
            before[t - b] = h;
            const float x = ssd_ld(static_cast<const T *>(a.in.x) + t * a.in.x_stride + c);
            const Gate f(ssd_ld(static_cast<const T *>(a.in.g) + t * a.in.g_stride + c));
            h = f.keep * h + f.drop * x;
        }
        for (long long t = e - 1; t >= b; --t) {
            const float x = ssd_ld(static_cast<const T *>(a.in.x) + t * a.in.x_stride + c);
            const Gate f(ssd_ld(static_cast<const T *>(a.in.g) + t * a.in.g_stride + c));
            const float keep = f.keep, drop = f.drop;
            float dh = ssd_ld(static_cast<const T *>(a.dy) + t * a.dy_stride + c);
            if (a.in.z) {
                const float z = ssd_ld(static_cast<const T *>(a.in.z) + t * a.in.z_stride + c);
                const float sig = sigmoidf(z);
                const float ht = keep * before[t - b] + drop * x;
                ssd_st(static_cast<T *>(a.dz) + t * a.dz_stride + c,
                       dh * ht * sig * (1.f + z * (1.f - sig)));
                dh *= z * sig;
            }
            const float lam = dh + carry;
            ssd_st(static_cast<T *>(a.dx) + t * a.dx_stride + c, drop * lam);
            ssd_st(static_cast<T *>(a.dg) + t * a.dg_stride + c,
                   lam * (before[t - b] - x) * keep * drop);
            carry = keep * lam;
        }
        e = b;
    }
    if (a.dinit) a.dinit[(size_t)s * a.in.width + c] = carry;
}

// One token of every (row, channel): the state is read and written in place.
template <typename T>
__global__ void __launch_bounds__(256) gated_step_kernel(const SsdGatedStep a) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (size_t)a.rows * a.width) return;
    const size_t r = i / a.width, c = i % a.width;
    const Gate f(ssd_ld(static_cast<const T *>(a.g) + r * a.g_stride + c));
    const float x = ssd_ld(static_cast<const T *>(a.x) + r * a.x_stride + c);
    const float h = f.keep * a.state[i] + f.drop * x;
    a.state[i] = h;
    float y = h;
    if (a.z) {
        const float z = ssd_ld(static_cast<const T *>(a.z) + r * a.z_stride + c);
        y = h * z * sigmoidf(z);
    }
    ssd_st(static_cast<T *>(a.y) + i, y);
}

}  // namespace

cudaError_t ssd_launch_gated_fwd(const SsdGatedFwd &a, int, cudaStream_t stream) {
    const dim3 grid((unsigned)((a.in.width + 127) / 128), (unsigned)a.in.nseq);
    if (a.in.bf16) gated_fwd_kernel<__nv_bfloat16><<<grid, 128, 0, stream>>>(a);
    else gated_fwd_kernel<float><<<grid, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t ssd_launch_gated_bwd(const SsdGatedBwd &a, int, cudaStream_t stream) {
    const dim3 grid((unsigned)((a.in.width + 127) / 128), (unsigned)a.in.nseq);
    if (a.in.bf16) gated_bwd_kernel<__nv_bfloat16><<<grid, 128, 0, stream>>>(a);
    else gated_bwd_kernel<float><<<grid, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t ssd_launch_gated_step(const SsdGatedStep &a, cudaStream_t stream) {
    const unsigned grid = (unsigned)(((size_t)a.rows * a.width + 255) / 256);
    if (a.bf16) gated_step_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a);
    else gated_step_kernel<float><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}
