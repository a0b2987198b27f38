// The matrix product in fp32 multiply-adds, for every type, stride and
// alignment: the path of fp32 inputs and of operands whose rows do not start
// on 16-byte boundaries; and the pass in front of the product's gradients.
//
//   out[m][n] = act(sum_k A(m,k) B(n,k) a_scale[m] b_scale[n] + bias[n]) + residual[m][n]
//
// Bound by the fp32 pipe: a CTA's 64 x 64 tile takes 16 values of k a step
// through shared memory, each of 256 threads a 4 x 4 block of sums.
#include <cuda_fp8.h>

#include "act.cuh"
#include "launch.h"
#include "vec.cuh"

namespace {

constexpr int kTile = 64, kStep = 16;

__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ld(const __nv_fp8_e4m3 *p) { return float(*p); }

__device__ __forceinline__ float ld_any(const void *p, long long i, SsdElt t) {
    return t == SSD_ELT_F32 ? static_cast<const float *>(p)[i]
                            : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void st_any(void *p, long long i, SsdElt t, float v) {
    if (t == SSD_ELT_F32) static_cast<float *>(p)[i] = v;
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// kStep x kTile values of one operand, row-major by k in shared memory.  The
// thread order follows the operand's unit stride, so loads are coalesced.
template <typename T>
__device__ __forceinline__ void load_tile(float (*dst)[kTile + 4], const T *p, long long row0,
                                          long long rows, long long k0, long long kk,
                                          long long row_stride, long long col_stride) {
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
        const int r = col_stride == 1 ? i / kStep : i % kTile;
        const int k = col_stride == 1 ? i % kStep : i / kTile;
        const bool in = row0 + r < rows && k0 + k < kk;
        dst[k][r] = in ? ld(p + (row0 + r) * row_stride + (k0 + k) * col_stride) : 0.f;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) product_simt_kernel(const SsdProduct p) {
    __shared__ __align__(16) float as[kStep][kTile + 4], bs[kStep][kTile + 4];
    const long long m0 = (long long)blockIdx.x * kTile, n0 = (long long)blockIdx.y * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (long long k0 = 0; k0 < p.k; k0 += kStep) {
        load_tile(as, static_cast<const T *>(p.a), m0, p.m, k0, p.k, p.a_row, p.a_col);
        load_tile(bs, static_cast<const T *>(p.b), n0, p.n, k0, p.k, p.b_row, p.b_col);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            const float4 av = *reinterpret_cast<const float4 *>(&as[k][4 * ty]);
            const float4 bv = *reinterpret_cast<const float4 *>(&bs[k][4 * tx]);
            const float ar[4] = {av.x, av.y, av.z, av.w}, br[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(ar[i], br[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long m = m0 + 4 * ty + i;
        if (m >= p.m) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long n = n0 + 4 * tx + j;
            if (n >= p.n) break;
            float v = acc[i][j];
            if (p.a_scale) v *= p.a_scale[m] * p.b_scale[n];
            if (p.bias) v += p.bias[n];
            if (p.preact) st_any(p.preact, m * p.n + n, p.preact_type, v);
            v = ssd_act(v, p.act);
            if (p.residual) v += ld_any(p.residual, m * p.residual_row + n, p.out_type);
            st_any(p.out, m * p.out_row + n, p.out_type, v);
        }
    }
}

// dp = dy act'(p) and its column sums.  32 x 8 threads take 32 columns of the
// rows b, b + grid, ... ; the sums of each block of rows go to `partial`.
template <typename T>
__global__ void __launch_bounds__(256) act_bwd_kernel(const SsdActBwd a, float *partial) {
    __shared__ float part[8][33];
    const int j = blockIdx.x * 32 + threadIdx.x;
    float acc = 0.f;
    if (j < a.width) {
        for (long long r = (long long)blockIdx.y * 8 + threadIdx.y; r < a.rows;
             r += (long long)gridDim.y * 8) {
            float v = ssd_ld(static_cast<const T *>(a.dy) + r * a.dy_stride + j);
            if (a.preact)
                v *= ssd_act_slope(ssd_ld(static_cast<const T *>(a.preact) + r * a.width + j), a.act);
            if (a.dp) ssd_st(static_cast<T *>(a.dp) + r * a.width + j, v);
            acc += v;
        }
    }
    if (!partial) return;
    part[threadIdx.y][threadIdx.x] = acc;
    __syncthreads();
    if (threadIdx.y == 0 && j < a.width) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[i][threadIdx.x];
        partial[(size_t)blockIdx.y * a.width + j] = s;
    }
}

__global__ void __launch_bounds__(256)
column_sum_kernel(const float *__restrict__ partial, int n, int width, float *__restrict__ out) {
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= width) return;
    float s = 0.f;
    for (int r = 0; r < n; ++r) s += partial[(size_t)r * width + j];
    out[j] = s;
}

int act_bwd_rows(long long rows, int width, int sms) {
    const long long cols = (width + 31) / 32;
    const long long want = (8ll * sms + cols - 1) / cols, most = (rows + 7) / 8;
    return (int)(want < most ? want : most);
}

}  // namespace

cudaError_t ssd_launch_product_simt(const SsdProduct &p, cudaStream_t stream) {
    const dim3 grid((unsigned)((p.m + kTile - 1) / kTile), (unsigned)((p.n + kTile - 1) / kTile));
    switch (p.in) {
        case SSD_ELT_F32: product_simt_kernel<float><<<grid, 256, 0, stream>>>(p); break;
        case SSD_ELT_BF16: product_simt_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(p); break;
        default: product_simt_kernel<__nv_fp8_e4m3><<<grid, 256, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

size_t ssd_act_bwd_workspace(long long rows, int width, int sms) {
    return (size_t)act_bwd_rows(rows, width, sms) * width * sizeof(float);
}

cudaError_t ssd_launch_act_bwd(const SsdActBwd &a, float *partial, int sms, cudaStream_t stream) {
    const int n = act_bwd_rows(a.rows, a.width, sms);
    const dim3 grid((unsigned)((a.width + 31) / 32), (unsigned)n), block(32, 8);
    float *part = a.dbias ? partial : nullptr;
    if (a.type == SSD_ELT_F32) act_bwd_kernel<float><<<grid, block, 0, stream>>>(a, part);
    else act_bwd_kernel<__nv_bfloat16><<<grid, block, 0, stream>>>(a, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.dbias) return e;
    column_sum_kernel<<<(unsigned)((a.width + 255) / 256), 256, 0, stream>>>(partial, n, a.width,
                                                                            a.dbias);
    return cudaGetLastError();
}
