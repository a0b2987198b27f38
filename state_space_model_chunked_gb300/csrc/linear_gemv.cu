// The matrix product for a handful of tokens, down to one: every weight is read
// once and meets kM tokens, so memory bounds it, and the multiply-adds run on
// the fp32 pipe in the shade of the loads.
//
//   out[m][n] = act(sum_k x[m][k] w[n][k] a_scale[m] b_scale[n] + bias[n]) + residual[m][n]
//
// A warp takes kRows features: its lanes read the features' weights 16 bytes
// each, kAhead steps of them under way, with the tokens' values of the same k
// from L1, and the lanes' sums are added at the end.  The grid has a warp for
// every kRows features and the hardware hands the CTAs out as SMs free up.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "act.cuh"
#include "launch.h"
#include "vec.cuh"

namespace {

constexpr int kWarps = 4, kRows = 2, kAhead = 4;

// V values of a row as fp32.
template <typename T, int V>
__device__ __forceinline__ void unpack(const SsdRaw<T, V> &raw, float (&v)[V]) {
    if constexpr (sizeof(T) != 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = raw.get(i);
    } else if constexpr (V == 1) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(
            *reinterpret_cast<const __nv_fp8_storage_t *>(raw.w), __NV_E4M3);
        v[0] = __half2float(*reinterpret_cast<const __half *>(&h));
    } else {
        const __nv_fp8x2_storage_t *p = reinterpret_cast<const __nv_fp8x2_storage_t *>(raw.w);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(p[i], __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
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
            for (int r = 0; r < kRows; ++r) unpack(wr[u][r], wv[r]);
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                SsdRaw<T, V> xr;
                xr.load(x + m * p.a_row + k0 + u * kStep);
                float xv[V];
                unpack(xr, xv);
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[r][m] = fmaf(wv[r][i], xv[i], acc[r][m]);
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

template <typename T>
cudaError_t launch_type(const SsdProduct &p, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    const auto on_16 = [](const void *q, long long stride) {
        return ((uintptr_t)q & 15u) == 0 && (stride * sizeof(T)) % 16 == 0;
    };
    if (p.k % V == 0 && on_16(p.a, p.a_row) && on_16(p.b, p.b_row)) return launch<T, V>(p, stream);
    return launch<T, 1>(p, stream);
}

}  // namespace

// K-major operands and at most four tokens.
bool ssd_product_gemv_handles(const SsdProduct &p) {
    return p.m <= 4 && p.a_col == 1 && p.b_col == 1;
}

cudaError_t ssd_launch_product_gemv(const SsdProduct &p, cudaStream_t stream) {
    if (p.in == SSD_ELT_F32) return launch_type<float>(p, stream);
    if (p.in == SSD_ELT_BF16) return launch_type<__nv_bfloat16>(p, stream);
    return launch_type<__nv_fp8_e4m3>(p, stream);
}
