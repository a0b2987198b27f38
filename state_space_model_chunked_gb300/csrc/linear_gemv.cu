// The matrix product for at most four tokens on the fp32 pipe: fp32 inputs, and
// bf16 or E4M3 inputs whose rows do not start on 16-byte boundaries (the others
// go to linear_few.cu).  Every weight is read once and meets kM tokens, so memory
// bounds it, and the multiply-adds run in the shade of the loads.
//
//   out[m][n] = act(sum_k x[m][k] w[n][k] a_scale[m] b_scale[n] + bias[n]) + residual[m][n]
//
// A warp takes kRows features: its lanes read the features' weights in vectors of
// V, kAhead steps of them under way, with the tokens' values of the same k from L1,
// and the lanes' sums are added at the end.  The grid has a warp for every kRows
// features and the hardware hands the CTAs out as SMs free up.
#include <cuda_fp8.h>

#include "act.cuh"
#include "launch.h"
#include "vec.cuh"

namespace {

constexpr int kWarps = 4, kRows = 2, kAhead = 4;

template <typename T, int V>
__device__ __forceinline__ float value(const SsdRaw<T, V> &raw, int i) {
    if constexpr (sizeof(T) == 1) return float(reinterpret_cast<const T *>(raw.w)[i]);
    else return raw.get(i);
}

template <typename T, int kM, int V>
__global__ void __launch_bounds__(32 * kWarps) product_gemv_kernel(const SsdProduct p) {
    const int lane = threadIdx.x & 31;
    const long long n0 = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRows;
    if (n0 >= p.n) return;
    const T *w = static_cast<const T *>(p.b), *x = static_cast<const T *>(p.a);
    float acc[kRows][kM];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int m = 0; m < kM; ++m) acc[r][m] = 0.f;
    constexpr int kStep = 32 * V;
    for (long long k0 = lane * V; k0 < p.k; k0 += kAhead * kStep) {
        SsdRaw<T, V> wr[kAhead][kRows];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                wr[u][r].zero();
                // a row past the end reads the last one; its sums are not used
                if (k0 + u * kStep < p.k)
                    wr[u][r].load_cs(w + min(n0 + r, p.n - 1) * p.b_row + k0 + u * kStep);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (k0 + u * kStep >= p.k) continue;
            float wv[kRows][V];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int i = 0; i < V; ++i) wv[r][i] = value(wr[u][r], i);
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                SsdRaw<T, V> xr;
                xr.load(x + m * p.a_row + k0 + u * kStep);
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        acc[r][m] = fmaf(wv[r][i], value(xr, i), acc[r][m]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            const float v = ssd_warp_sum(acc[r][m]);
            if (lane == r * kM + m && n0 + r < p.n) ssd_finish(p, m, n0 + r, v);
        }
    }
}

template <typename T, int V>
cudaError_t launch(const SsdProduct &p, cudaStream_t stream) {
    const long long per = (long long)kWarps * kRows;
    const dim3 grid((unsigned)((p.n + per - 1) / per)), block(32 * kWarps);
    switch (p.m) {
        case 1: product_gemv_kernel<T, 1, V><<<grid, block, 0, stream>>>(p); break;
        case 2: product_gemv_kernel<T, 2, V><<<grid, block, 0, stream>>>(p); break;
        case 3: product_gemv_kernel<T, 3, V><<<grid, block, 0, stream>>>(p); break;
        default: product_gemv_kernel<T, 4, V><<<grid, block, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace

// K-major operands and at most four tokens.
bool ssd_product_gemv_handles(const SsdProduct &p) {
    return p.m <= 4 && p.a_col == 1 && p.b_col == 1;
}

cudaError_t ssd_launch_product_gemv(const SsdProduct &p, cudaStream_t stream) {
    if (p.in == SSD_ELT_BF16) return launch<__nv_bfloat16, 1>(p, stream);
    if (p.in == SSD_ELT_E4M3) return launch<__nv_fp8_e4m3, 1>(p, stream);
    const auto on_16 = [](const void *q, long long stride) {
        return ((uintptr_t)q & 15u) == 0 && stride % 4 == 0;
    };
    return p.k % 4 == 0 && on_16(p.a, p.a_row) && on_16(p.b, p.b_row) ? launch<float, 4>(p, stream)
                                                                      : launch<float, 1>(p, stream);
}
