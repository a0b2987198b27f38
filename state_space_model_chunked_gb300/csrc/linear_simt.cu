// The matrix product in fp32 multiply-adds, for every type, stride and
// alignment: the path of fp32 inputs and of operands whose rows do not start
// on 16-byte boundaries; and the pass in front of the product's gradients.
//
//   out[m][n] = act(sum_k A(m,k) B(n,k) a_scale[m] b_scale[n] + bias[n]) + residual[m][n]
//
// A CTA's 64 x 64 tile takes 16 values of k a step through shared memory, each of
// 256 threads a 4 x 4 block of sums.  Simple rather than fast: one buffer and two
// barriers a step, scalar loads, no split of k.  Measured (time on the GPU): fp32
// 2048 x 2048 -> 2048 815 us (21 TFLOP/s), both its gradients 1638; 16 x 5120 -> 2560
// 570 us and 64 tokens 703, where 40 CTAs walk all of k; bf16 with unaligned rows 1000 x
// 1001 -> 1024 175 us (12 TFLOP/s), gradients 354.
#include <cuda_fp8.h>

#include <algorithm>

#include "act.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace {

constexpr int kTile = 64, kStep = 16;
constexpr int kActCtas = 5;     // CTAs an SM of the gradients' pass

__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ld(const __nv_fp8_e4m3 *p) { return float(*p); }

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
__global__ void __launch_bounds__(256)
product_simt_kernel(const SsdProduct p, const unsigned row_tiles) {
    __shared__ __align__(16) float as[kStep][kTile + 4], bs[kStep][kTile + 4];
    const long long m0 = (long long)(blockIdx.x % row_tiles) * kTile;
    const long long n0 = (long long)(blockIdx.x / row_tiles) * kTile;
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
            ssd_finish(p, m, n, acc[i][j]);
        }
    }
}

// dp = dy act'(p) and its column sums: bound by memory.  32 x 8 threads take
// 32 V columns of the rows b, b + grid, ... ; a thread's sums stay in registers,
// each block of rows' go to `partial`.  One wave of five CTAs an SM with two rows a
// thread under way in bf16: 65536 x 2560 with silu 158 us (0.94 of the measured
// bandwidth), 16376 x 2048 with gelu 40 us (0.74: the slope's arithmetic), the sums
// alone 16.6 us; four CTAs with four rows 168, 42 and 16.2 us, six with two 174, 45 and 16.8.
template <typename T, int V>
__global__ void __launch_bounds__(256, kActCtas)
act_bwd_kernel(const SsdActBwd a, float *partial, const bool beside) {
    constexpr int kAhead = 4 / (int)sizeof(T);      // rows under way in a thread
    __shared__ float part[8][32 * V + 1];
    if (!beside) ssdptx::griddep_wait();
    const int j = (blockIdx.x * 32 + threadIdx.x) * V;
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    if (j < a.width) {
        const T *dy = static_cast<const T *>(a.dy) + j, *pre = static_cast<const T *>(a.preact) + j;
        const long long step = (long long)gridDim.y * 8;
        for (long long r = (long long)blockIdx.y * 8 + threadIdx.y; r < a.rows; r += kAhead * step) {
            SsdRaw<T, V> d[kAhead], p[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const long long ru = r + u * step;
                d[u].zero();
                p[u].zero();
                if (ru >= a.rows) continue;
                d[u].load_cs(dy + ru * a.dy_stride);
                if (a.preact) p[u].load_cs(pre + ru * a.width);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const long long ru = r + u * step;
                if (ru >= a.rows) continue;
                float v[V];
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    v[k] = d[u].get(k);
                    if (a.preact) v[k] *= ssd_act_slope(p[u].get(k), a.act);
                    acc[k] += v[k];
                }
                if (a.dp) ssd_store_vec<V>(static_cast<T *>(a.dp) + ru * a.width + j, v);
            }
        }
    }
    if (!partial) return;       // (and then not beside another kernel)
#pragma unroll
    for (int k = 0; k < V; ++k) part[threadIdx.y][threadIdx.x * V + k] = acc[k];
    __syncthreads();
    for (int i = threadIdx.y * 32 + threadIdx.x; i < 32 * V; i += 256) {
        const int col = blockIdx.x * 32 * V + i;
        float s = 0.f;
#pragma unroll
        for (int y = 0; y < 8; ++y) s += part[y][i];
        if (col < a.width) partial[(size_t)blockIdx.y * a.width + col] = s;
    }
    if (beside) ssdptx::griddep_wait();
}

// out[j] = the sum over n partial rows in a fixed order: kRows x 32 threads take 32
// columns, each thread row every kRows-th partial row.  Beside a product, which
// leaves an SM few registers, 8 thread rows; else 32.
template <int kRows>
__global__ void __launch_bounds__(32 * kRows)
column_sum_kernel(const float *partial, int n, int width, float *out, const bool beside) {
    __shared__ float part[kRows][33];
    if (!beside) ssdptx::griddep_wait();
    const int j = blockIdx.x * 32 + threadIdx.x;
    float acc = 0.f;
    if (j < width) {
#pragma unroll 8
        for (int r = threadIdx.y; r < n; r += kRows)
            acc += __ldcg(partial + (size_t)r * width + j);
    }
    part[threadIdx.y][threadIdx.x] = acc;
    __syncthreads();
    if (threadIdx.y == 0 && j < width) {
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) v += part[r][threadIdx.x];
        out[j] = v;
    }
    if (beside) ssdptx::griddep_wait();
}

template <typename T>
cudaError_t launch_act_bwd(const SsdActBwd &a, float *partial, int n, SsdOrder order,
                           cudaStream_t stream) {
    const auto on_16 = [](const void *p, long long stride) {
        return !p || (((uintptr_t)p & 15u) == 0 && (stride * sizeof(T)) % 16 == 0);
    };
    const dim3 block(32, 8);
    const bool v8 =
        on_16(a.dy, a.dy_stride) && on_16(a.preact, a.width) && on_16(a.dp, a.width) &&
        a.width % 8 == 0;
    const auto kernel = v8 ? act_bwd_kernel<T, 8> : act_bwd_kernel<T, 1>;
    const dim3 grid((unsigned)((a.width + (v8 ? 255 : 31)) / (v8 ? 256 : 32)), (unsigned)n);
    return ssd_launch_early(kernel, grid, block, stream, a, partial, order == SsdOrder::beside);
}

}  // namespace

cudaError_t ssd_launch_product_simt(const SsdProduct &p, cudaStream_t stream) {
    // one dimension of tiles: the others of a grid end at 65535, which 2^22 features pass
    const long long rows = (p.m + kTile - 1) / kTile, tiles = rows * ((p.n + kTile - 1) / kTile);
    if (tiles >= (1ll << 31)) return cudaErrorInvalidValue;     // more than any memory holds
    const auto kernel = p.in == SSD_ELT_F32    ? product_simt_kernel<float>
                        : p.in == SSD_ELT_BF16 ? product_simt_kernel<__nv_bfloat16>
                                               : product_simt_kernel<__nv_fp8_e4m3>;
    kernel<<<(unsigned)tiles, 256, 0, stream>>>(p, (unsigned)rows);
    return cudaGetLastError();
}

// Blocks of rows: as many CTAs as the SMs hold, whatever vectors the arrays allow.
int ssd_act_bwd_rows(long long rows, int width, int sms) {
    const long long cols = (width + 255) / 256;
    const long long want = std::max(1ll, kActCtas * (long long)sms / cols), most = (rows + 7) / 8;
    return (int)std::min(want, most);
}

size_t ssd_act_bwd_workspace(long long rows, int width, int sms) {
    return (size_t)ssd_act_bwd_rows(rows, width, sms) * width * sizeof(float);
}

cudaError_t ssd_launch_act_bwd(const SsdActBwd &a, float *partial, int sms, SsdOrder order,
                               cudaStream_t stream) {
    const int n = ssd_act_bwd_rows(a.rows, a.width, sms);
    return a.type == SSD_ELT_F32 ? launch_act_bwd<float>(a, partial, n, order, stream)
                                 : launch_act_bwd<__nv_bfloat16>(a, partial, n, order, stream);
}

cudaError_t ssd_launch_column_sum(const float *partial, int n, int width, float *out,
                                  SsdOrder order, cudaStream_t stream) {
    const dim3 grid((unsigned)((width + 31) / 32));
    return order == SsdOrder::beside
               ? ssd_launch_early(column_sum_kernel<8>, grid, dim3(32, 8), stream, partial, n, width,
                                  out, true)
               : ssd_launch_early(column_sum_kernel<32>, grid, dim3(32, 32), stream, partial, n,
                                  width, out, false);
}
