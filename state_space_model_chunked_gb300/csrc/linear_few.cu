// The matrix product for few tokens, bf16 or E4M3 inputs: every weight is read
// once, so memory bounds it, and what counts is how many bytes are under way.
//
//   out[m][n] = act(sum_k x[m][k] w[n][k] a_scale[m] b_scale[n] + bias[n]) + residual[m][n]
//
// A CTA takes 16 features; its warps split k among themselves, and each lane
// reads its operands from global memory straight into the fragments of a
// 16 x 8 x 16 warp product (features x tokens x k, fp32 sums): a sum over k may
// take k in any order, so lane 4 g + t simply holds 16 consecutive bytes of
// features g and g + 8 and the same 16 bytes of token g.  Nothing is staged in
// shared memory and no barrier stands before the end, where the warps' sums are
// added in order.
//   Measured (time on the GPU): one token of 2560 to 15360 features in bf16 14.4 us
// (5.45 TB/s, 0.80 of the measured copy bandwidth), sixteen tokens of 5120 to 2560 in
// 8 bits 5.2 us, of which the weights' transfer is 2 (with at most two CTAs an SM a
// warp loads one step at a time: three trips to memory one after another, in bf16
// five, which take 9.4 us, and 7.0 for one token, against 3.9 for the transfer).  The tcgen05 tiles of
// linear_tc.cu, with their prologue, cluster barriers and tensor-memory round trip,
// took 18.2 and 10.9 us.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "act.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace {

constexpr int kRows = 16;       // features a CTA

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A 16-byte word as pairs of 16-bit values: itself for bf16; E4M3 values as f16
// (every one of them is exactly an f16).
template <bool kFp8>
struct Pairs {
    static constexpr int kN = kFp8 ? 8 : 4;
    uint32_t p[kN];
    __device__ __forceinline__ explicit Pairs(const uint4 &v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kFp8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
                        (__nv_fp8x2_storage_t)(w[i] >> (16 * h)), __NV_E4M3);
                    p[2 * i + h] = *reinterpret_cast<const uint32_t *>(&r);
                }
            } else {
                p[i] = w[i];
            }
        }
    }
};

// kNT: groups of 8 tokens.  kAhead: steps of two 16-byte words a row that a turn of
// the loop loads before it uses them; the compiler keeps fewer under way (for one
// group of tokens and five steps 54 registers, where the words alone would take 80).
template <bool kFp8, int kNT, int kWarps, int kAhead>
__global__ void __launch_bounds__(32 * kWarps) product_few_kernel(const SsdProduct p) {
    constexpr int kSize = kFp8 ? 1 : 2, kWord = 16 / kSize;
    constexpr int kStep = 8 * kWord;            // values of k a warp takes at once: 128 bytes a row
    __shared__ float part[kWarps][kNT * 8][kRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    ssdptx::griddep_wait();
    const long long n0 = (long long)blockIdx.x * kRows;
    const char *w = static_cast<const char *>(p.b), *x = static_cast<const char *>(p.a);
    // rows past the end read the last one; their sums are not used
    const char *wg = w + min(n0 + g, p.n - 1) * p.b_row * kSize + t * 16;
    const char *wh = w + min(n0 + g + 8, p.n - 1) * p.b_row * kSize + t * 16;
    const char *xt[kNT];
#pragma unroll
    for (int j = 0; j < kNT; ++j) xt[j] = x + min((long long)(j * 8 + g), p.m - 1) * p.a_row * kSize + t * 16;
    float acc[kNT][4];
#pragma unroll
    for (int j = 0; j < kNT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (long long k0 = (long long)warp * kStep; k0 < p.k; k0 += (long long)kAhead * kWarps * kStep) {
        uint4 a[kAhead][2][2];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // this lane's word of the step (k a multiple of a word: whole words only)
                const long long k = k0 + (long long)u * kWarps * kStep + h * 4 * kWord;
                const bool in = k + t * kWord < p.k;
                a[u][h][0] = in ? __ldcs(reinterpret_cast<const uint4 *>(wg + k * kSize)) : zero;
                a[u][h][1] = in ? __ldcs(reinterpret_cast<const uint4 *>(wh + k * kSize)) : zero;
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const long long k = k0 + (long long)u * kWarps * kStep + h * 4 * kWord;
                const bool in = k + t * kWord < p.k;
                const Pairs<kFp8> ag(a[u][h][0]), ah(a[u][h][1]);
#pragma unroll
                for (int j = 0; j < kNT; ++j) {
                    const Pairs<kFp8> b(in ? *reinterpret_cast<const uint4 *>(xt[j] + k * kSize)
                                           : zero);
#pragma unroll
                    for (int i = 0; i < Pairs<kFp8>::kN; i += 2) {
                        if constexpr (kFp8)
                            mma_f16(acc[j], ag.p[i], ah.p[i], ag.p[i + 1], ah.p[i + 1], b.p[i],
                                    b.p[i + 1]);
                        else
                            mma_bf16(acc[j], ag.p[i], ah.p[i], ag.p[i + 1], ah.p[i + 1], b.p[i],
                                     b.p[i + 1]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kNT; ++j) {
        part[warp][j * 8 + 2 * t][g] = acc[j][0];
        part[warp][j * 8 + 2 * t + 1][g] = acc[j][1];
        part[warp][j * 8 + 2 * t][g + 8] = acc[j][2];
        part[warp][j * 8 + 2 * t + 1][g + 8] = acc[j][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kNT * 8 * kRows; i += 32 * kWarps) {
        const int m = i / kRows, r = i % kRows;
        if (m >= p.m || n0 + r >= p.n) continue;
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) v += part[q][m][r];
        ssd_finish(p, m, n0 + r, v);
    }
}

template <bool kFp8, int kNT, int kWarps, int kAhead>
cudaError_t launch(const SsdProduct &p, cudaStream_t stream) {
    return ssd_launch_early(product_few_kernel<kFp8, kNT, kWarps, kAhead>,
                            dim3((unsigned)((p.n + kRows - 1) / kRows)), dim3(32 * kWarps), stream, p);
}

// Few CTAs an SM: many warps in each, so all of the SM's loads are under way;
// many CTAs: few warps, so each takes several steps between its start and its
// barrier, unless k is long (64 steps and more) and a lane's loads few.  us in
// bf16 by 16 / 8 / 4 warps for one token: 15360 features of 2560 (6.3 CTAs an SM)
// 20.0 / 17.4 / 14.6; 10240 of 5120 (4.2) - / 19.4 / 22.6; 2560 of 5120 (1.05)
// 7.9 / 11.7 / 21.0; for sixteen tokens 24.8 / 21.0 / 16.4, - / 33.7 / 24.0,
// 9.8 / 14.3 / 26.4.
template <bool kFp8, int kNT>
cudaError_t launch_warps(const SsdProduct &p, int sms, cudaStream_t stream) {
    const long long ctas = (p.n + kRows - 1) / kRows, steps = p.k * (kFp8 ? 1 : 2) / 128;
    if (ctas <= 2ll * sms) return launch<kFp8, kNT, 16, 1>(p, stream);
    if (ctas <= 4ll * sms || (kNT == 1 && steps >= 64)) return launch<kFp8, kNT, 8, 2>(p, stream);
    return launch<kFp8, kNT, 4, kFp8 || kNT == 1 ? 5 : 4>(p, stream);
}

}  // namespace

// K-major bf16 or E4M3 operands whose rows start on 16-byte boundaries, k a
// whole number of 16-byte words, at most 16 tokens.
bool ssd_product_few_handles(const SsdProduct &p) {
    if (p.in == SSD_ELT_F32 || p.m > 16 || p.a_col != 1 || p.b_col != 1) return false;
    const int size = p.in == SSD_ELT_E4M3 ? 1 : 2;
    return (p.k * size) % 16 == 0 && (p.a_row * size) % 16 == 0 && (p.b_row * size) % 16 == 0 &&
           ((uintptr_t)p.a & 15u) == 0 && ((uintptr_t)p.b & 15u) == 0;
}

cudaError_t ssd_launch_product_few(const SsdProduct &p, int sms, cudaStream_t stream) {
    if (p.in == SSD_ELT_E4M3)
        return p.m <= 8 ? launch_warps<true, 1>(p, sms, stream)
                        : launch_warps<true, 2>(p, sms, stream);
    return p.m <= 8 ? launch_warps<false, 1>(p, sms, stream)
                    : launch_warps<false, 2>(p, sms, stream);
}
