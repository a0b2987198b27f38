// Root-mean-square norm of s = x + residual, forward (with an 8-bit output
// and its row scales) and backward.
//
//   s = x + r,  rstd = (mean_j s_j^2 + eps)^(-1/2),  y_j = s_j rstd w_j
//   8 bits: scale = max_j |y_j| / 448 (1 where that is 0), q = e4m3(y / scale)
//   backward, with e_j = dy_j w_j:
//     ds_j = ds_out_j + rstd (e_j - s_j rstd^2 mean_i(e_i s_i))
//     dw_j = sum over rows of dy_j s_j rstd
//
// Both are bound by memory: every value is read once and written once, the
// sums stay in fp32, and each result is rounded once.  A CTA walks over rows,
// one at a time in registers (kC runs of V values a thread) with the next
// row's loads under way, and keeps its columns' weights in registers; the
// row's sum and its largest |s w| come from one pass and one barrier:
// max |y| = rstd max |s w|.
//   Measured (time on the GPU): 65536 rows of 2560, bf16 with a bf16 residual,
// to 8 bits 189 us (0.91 of the measured copy bandwidth); gradients of 16376
// rows of 1024 46 us (0.86); 16 rows 1.6 us, all of it the launch.  Without the next
// row's loads under way the first took 377 us and the second 89.
//   Widths that are no multiple of 8, and unaligned rows, move value by value: 16376
// rows of 1023 with an fp32 residual 47 us forward and 143 backward, of 2047 83 and 286
// (0.48 and 0.14 of the bandwidth), 65536 rows of 2559 to 8 bits 696.  Rows beyond a
// CTA's registers (above 8192 values, forward with vectors 16384) are read again for
// each pass over them: 4096 rows of 33000 417 us forward (0.38) and 672 backward (0.24),
// gradients at 16384 346 us (0.23).
#include "launch.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace {

constexpr float kE4m3Max = 448.f;
constexpr int kMostWarps = 16;      // a row's CTA: 128 registers a thread
// most runs a thread: of 8 values (forward, backward) and of one
constexpr int kRuns8 = 4, kBwdRuns8 = 2, kRuns1 = 16;
// runs wanted a thread where there are rows enough, and warps an SM holds.  us
// forward by (runs, warps): (4, 16) 190, (4, 24) 223, (2, 16) 288, (2, 32) 216,
// (1, 32) 262, (1, 48) 292; backward: (1, 16) 46.6, (1, 24) 51, (1, 32) 48.7, (2, 16) 47.0
constexpr int kFwdRuns = 4, kFwdWarpsSm = 16;
constexpr int kBwdRuns = 1, kBwdWarpsSm = 16;

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

template <typename TX, typename TR, typename TO, int V, int kC>
__global__ void __launch_bounds__(32 * kMostWarps) rmsnorm_fwd_kernel(const SsdNormFwd a) {
    ssdptx::griddep_wait();
    __shared__ float buf[2][2][32];
    constexpr bool kFp8 = sizeof(TO) == 1;
    const int nvec = a.width / V;
    const bool res = a.residual != nullptr;
    const TX *x = static_cast<const TX *>(a.x);
    const TR *r = static_cast<const TR *>(a.residual);
    Row<TX, V, kC> xr;
    Row<TR, V, kC> rr;
    long long row = blockIdx.x;
    xr.load(x + row * a.x_stride, nvec, true);
    rr.load(r + row * a.residual_stride, nvec, res);
    float w[kC][V];
    load_weight<V, kC>(a.weight, nvec, w);
    for (int turn = 0; row < a.rows; turn ^= 1) {
        float s[kC][V], sum = 0.f, mx = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                s[c][k] = xr.run[c].get(k);
                if (res) s[c][k] += rr.run[c].get(k);
                sum += s[c][k] * s[c][k];
            }
        }
        const long long next = row + gridDim.x;
        if (next < a.rows) {
            xr.load(x + next * a.x_stride, nvec, true);
            rr.load(r + next * a.residual_stride, nvec, res);
        }
        if (res) {
            TR *so = static_cast<TR *>(a.residual_out) + row * a.width;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int i = threadIdx.x + c * blockDim.x;
                if (i < nvec) ssd_store_vec<V>(so + (size_t)i * V, s[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < kC; ++c) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                s[c][k] *= w[c][k];
                if constexpr (kFp8) mx = fmaxf(mx, fabsf(s[c][k]));
            }
        }
        cta_sum_max<kFp8>(sum, mx, buf[turn]);
        const float rstd = rsqrtf(sum / (float)a.width + a.eps);
        const RowScale q(kFp8 ? mx * rstd : 0.f);
        if (threadIdx.x == 0) {
            a.rstd[row] = rstd;
            if constexpr (kFp8) a.scale[row] = q.scale;
        }
        TO *y = static_cast<TO *>(a.y) + row * a.width;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i >= nvec) continue;
            float o[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                o[k] = s[c][k] * rstd;
                if constexpr (kFp8) o[k] = q.apply(o[k]);
            }
            ssd_store_vec<V>(y + (size_t)i * V, o);
        }
        row = next;
    }
}

// Rows too wide for the registers of a CTA: two passes over the row, the
// second one out of L2.
template <typename TX, typename TR, typename TO>
__global__ void rmsnorm_fwd_wide_kernel(const SsdNormFwd a) {
    __shared__ float buf[2][32];
    constexpr bool kFp8 = sizeof(TO) == 1;
    const long long row = blockIdx.x;
    const TX *x = static_cast<const TX *>(a.x) + row * a.x_stride;
    const TR *r = a.residual ? static_cast<const TR *>(a.residual) + row * a.residual_stride
                             : nullptr;
    float sum = 0.f, mx = 0.f;
    for (int i = threadIdx.x; i < a.width; i += blockDim.x) {
        const float s = r ? ssd_ld(x + i) + ssd_ld(r + i) : ssd_ld(x + i);
        sum += s * s;
        if constexpr (kFp8) mx = fmaxf(mx, fabsf(s * a.weight[i]));
    }
    cta_sum_max<kFp8>(sum, mx, buf);
    const float rstd = rsqrtf(sum / (float)a.width + a.eps);
    const RowScale q(kFp8 ? mx * rstd : 0.f);
    if (threadIdx.x == 0) {
        a.rstd[row] = rstd;
        if constexpr (kFp8) a.scale[row] = q.scale;
    }
    TR *so = static_cast<TR *>(a.residual_out) + (r ? row * a.width : 0);
    TO *y = static_cast<TO *>(a.y) + row * a.width;
    for (int i = threadIdx.x; i < a.width; i += blockDim.x) {
        const float s = r ? ssd_ld(x + i) + ssd_ld(r + i) : ssd_ld(x + i);
        float o[1] = {s * rstd * a.weight[i]};
        if constexpr (kFp8) o[0] = q.apply(o[0]);
        ssd_store_vec<1>(y + i, o);
        if (r) ssd_st(so + i, s);
    }
}

// ------------------------------------------------------------------ backward
// A CTA walks the rows b, b + grid, ...; each thread keeps its columns' share
// of dw in registers over all of them and writes it once, as row b of the
// partial sums, which are then added in order.
template <typename T, typename TS, int V, int kC>
__global__ void __launch_bounds__(32 * kMostWarps)
rmsnorm_bwd_kernel(const SsdNormBwd a, float *__restrict__ partial) {
    ssdptx::griddep_wait();
    __shared__ float buf[2][2][32];
    const int nvec = a.width / V;
    const bool res = a.dresidual != nullptr;
    const T *dy = static_cast<const T *>(a.dy);
    const TS *st = static_cast<const TS *>(a.s), *dres = static_cast<const TS *>(a.dresidual);
    Row<T, V, kC> yr;
    Row<TS, V, kC> sr, dr;
    long long row = blockIdx.x;
    yr.load(dy + row * a.dy_stride, nvec, true);
    sr.load(st + row * a.s_stride, nvec, true);
    dr.load(dres + row * a.dresidual_stride, nvec, res);
    float rstd = a.rstd[row];
    float w[kC][V], dw[kC][V];
    load_weight<V, kC>(a.weight, nvec, w);
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int k = 0; k < V; ++k) dw[c][k] = 0.f;
    for (int turn = 0; row < a.rows; turn ^= 1) {
        // e = dy w, v = s rstd, and what came from elsewhere
        float e[kC][V], v[kC][V], d[kC][V], sum = 0.f, unused = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float dyv = yr.run[c].get(k);
                v[c][k] = sr.run[c].get(k) * rstd;
                d[c][k] = dr.run[c].get(k);
                e[c][k] = dyv * w[c][k];
                sum += e[c][k] * v[c][k];
                dw[c][k] += dyv * v[c][k];
            }
        }
        const float scale = rstd;
        const long long next = row + gridDim.x;
        if (next < a.rows) {
            yr.load(dy + next * a.dy_stride, nvec, true);
            sr.load(st + next * a.s_stride, nvec, true);
            dr.load(dres + next * a.dresidual_stride, nvec, res);
            rstd = a.rstd[next];
        }
        cta_sum_max<false>(sum, unused, buf[turn]);
        const float mean = sum / (float)a.width;
        T *dx = static_cast<T *>(a.dx) + row * a.width;
        TS *ds = a.ds ? static_cast<TS *>(a.ds) + row * a.width : nullptr;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i >= nvec) continue;
            float o[V];
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] = scale * (e[c][k] - v[c][k] * mean) + d[c][k];
            ssd_store_vec<V>(dx + (size_t)i * V, o);
            if (ds) ssd_store_vec<V>(ds + (size_t)i * V, o);
        }
        row = next;
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        const int i = threadIdx.x + c * blockDim.x;
        if (i < nvec) ssd_store_vec<V>(partial + (size_t)blockIdx.x * a.width + (size_t)i * V, dw[c]);
    }
}

// Rows too wide for a CTA's registers: the sums per row, then the columns.
template <typename T, typename TS>
__global__ void rmsnorm_bwd_wide_kernel(const SsdNormBwd a) {
    __shared__ float buf[2][32];
    const long long row = blockIdx.x;
    const T *dy = static_cast<const T *>(a.dy) + row * a.dy_stride;
    const TS *s = static_cast<const TS *>(a.s) + row * a.s_stride;
    const TS *dres = a.dresidual ? static_cast<const TS *>(a.dresidual) + row * a.dresidual_stride
                                 : nullptr;
    const float rstd = a.rstd[row];
    float sum = 0.f, unused = 0.f;
    for (int i = threadIdx.x; i < a.width; i += blockDim.x)
        sum += ssd_ld(dy + i) * a.weight[i] * ssd_ld(s + i);
    cta_sum_max<false>(sum, unused, buf);
    const float m = sum / (float)a.width * rstd * rstd;
    T *dx = static_cast<T *>(a.dx) + row * a.width;
    TS *ds = a.ds ? static_cast<TS *>(a.ds) + row * a.width : nullptr;
    for (int i = threadIdx.x; i < a.width; i += blockDim.x) {
        float o = rstd * (ssd_ld(dy + i) * a.weight[i] - ssd_ld(s + i) * m);
        if (dres) o += ssd_ld(dres + i);
        ssd_st(dx + i, o);
        if (ds) ssd_st(ds + i, o);
    }
}
template <typename T, typename TS>
__global__ void rmsnorm_dw_wide_kernel(const SsdNormBwd a, float *__restrict__ partial) {
    const int j = blockIdx.y * blockDim.x + threadIdx.x;
    if (j >= a.width) return;
    float acc = 0.f;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x)
        acc += ssd_ld(static_cast<const T *>(a.dy) + row * a.dy_stride + j) *
               (ssd_ld(static_cast<const TS *>(a.s) + row * a.s_stride + j) * a.rstd[row]);
    partial[(size_t)blockIdx.x * a.width + j] = acc;
}

// Threads and runs a thread for one row: at most `most_runs` runs of V values a
// thread (`want` where the warps allow it), a power of two of warps; 0 warps
// when the row does not fit.
struct RowShape {
    int warps, runs;
};
RowShape row_shape(int width, int V, int most_runs, int want) {
    const int nvec = (width + V - 1) / V;
    int w = 1;
    while (w < kMostWarps && (long long)w * 32 * want < nvec) w *= 2;
    const int runs = (nvec + w * 32 - 1) / (w * 32);
    return {runs <= most_runs ? w : 0, runs};
}

// CTAs of a walk over rows: as many as the SMs hold at once.
unsigned walkers(long long rows, int sms, int ctas) {
    const long long n = (long long)sms * ctas;
    return (unsigned)(rows < n ? rows : n);
}

bool vec8(const void *p, long long stride, int size) {
    return p == nullptr || (((uintptr_t)p & 15u) == 0 && (stride * size) % 16 == 0);
}

template <typename TX, typename TR, typename TO>
cudaError_t launch_fwd(const SsdNormFwd &a, int sms, cudaStream_t stream) {
    const bool v8 = a.width % 8 == 0 && vec8(a.weight, 0, 4) && vec8(a.x, a.x_stride, sizeof(TX)) &&
                    vec8(a.residual, a.residual_stride, sizeof(TR)) &&
                    vec8(a.residual_out, a.width, sizeof(TR)) && ((uintptr_t)a.y & 7u) == 0 &&
                    vec8(sizeof(TO) == 1 ? nullptr : a.y, a.width, sizeof(TO));
    // few rows leave SMs idle: one run a thread, so the row is read in one step
    const RowShape sh = row_shape(a.width, v8 ? 8 : 1, v8 ? kRuns8 : kRuns1,
                                  a.rows <= sms ? 1 : (v8 ? kFwdRuns : kRuns1));
    const unsigned rows = walkers(a.rows, sms, kFwdWarpsSm / (sh.warps ? sh.warps : 1));
    if (sh.warps == 0) {
        rmsnorm_fwd_wide_kernel<TX, TR, TO><<<(unsigned)a.rows, 1024, 0, stream>>>(a);
        return cudaGetLastError();
    }
    auto kernel = rmsnorm_fwd_kernel<TX, TR, TO, 1, kRuns1>;
    if (v8) {
        switch (sh.runs) {
            case 1: kernel = rmsnorm_fwd_kernel<TX, TR, TO, 8, 1>; break;
            case 2: kernel = rmsnorm_fwd_kernel<TX, TR, TO, 8, 2>; break;
            case 3: kernel = rmsnorm_fwd_kernel<TX, TR, TO, 8, 3>; break;
            default: kernel = rmsnorm_fwd_kernel<TX, TR, TO, 8, 4>; break;
        }
    }
    return ssd_launch_early(kernel, dim3(rows), dim3(32 * sh.warps), stream, a);
}

template <typename TX, typename TR>
cudaError_t launch_fwd_out(const SsdNormFwd &a, int sms, cudaStream_t stream) {
    switch (a.out) {
        case SSD_ELT_F32: return launch_fwd<TX, TR, float>(a, sms, stream);
        case SSD_ELT_BF16: return launch_fwd<TX, TR, __nv_bfloat16>(a, sms, stream);
        default: return launch_fwd<TX, TR, __nv_fp8_e4m3>(a, sms, stream);
    }
}

// CTAs, and so rows of partial sums, of the backward pass: by the warps that a
// row of this width takes with vectors (a row without them takes fewer CTAs).
int bwd_ctas(long long rows, int width, int sms) {
    const RowShape sh = row_shape(width, 8, kBwdRuns8, kBwdRuns);
    return (int)walkers(rows, sms, sh.warps ? kBwdWarpsSm / sh.warps : 2);
}

template <typename T, typename TS>
cudaError_t launch_bwd(const SsdNormBwd &a, float *partial, int sms, cudaStream_t stream) {
    const bool v8 = a.width % 8 == 0 && vec8(a.weight, 0, 4) && vec8(a.dy, a.dy_stride, sizeof(T)) &&
                    vec8(a.s, a.s_stride, sizeof(TS)) &&
                    vec8(a.dresidual, a.dresidual_stride, sizeof(TS)) &&
                    vec8(a.dx, a.width, sizeof(T)) && vec8(a.ds, a.width, sizeof(TS));
    const RowShape sh = row_shape(a.width, v8 ? 8 : 1, v8 ? kBwdRuns8 : kRuns1, v8 ? kBwdRuns : kRuns1);
    const int n = bwd_ctas(a.rows, a.width, sms);
    cudaError_t e;
    if (sh.warps == 0) {
        rmsnorm_bwd_wide_kernel<T, TS><<<(unsigned)a.rows, 1024, 0, stream>>>(a);
        const dim3 grid((unsigned)n, (unsigned)((a.width + 255) / 256));
        rmsnorm_dw_wide_kernel<T, TS><<<grid, 256, 0, stream>>>(a, partial);
        e = cudaGetLastError();
    } else {
        auto kernel = rmsnorm_bwd_kernel<T, TS, 1, kRuns1>;
        if (v8) kernel = sh.runs == 1 ? rmsnorm_bwd_kernel<T, TS, 8, 1> : rmsnorm_bwd_kernel<T, TS, 8, 2>;
        e = ssd_launch_early(kernel, dim3((unsigned)n), dim3(32 * sh.warps), stream, a, partial);
    }
    if (e != cudaSuccess) return e;
    return ssd_launch_column_sum(partial, n, a.width, a.dweight, SsdOrder::after, stream);
}

}  // namespace

cudaError_t ssd_launch_rmsnorm_fwd(const SsdNormFwd &a, int sms, cudaStream_t stream) {
    if (a.in == SSD_ELT_F32) return launch_fwd_out<float, float>(a, sms, stream);
    if (a.stream_type == SSD_ELT_F32) return launch_fwd_out<__nv_bfloat16, float>(a, sms, stream);
    return launch_fwd_out<__nv_bfloat16, __nv_bfloat16>(a, sms, stream);
}

size_t ssd_rmsnorm_bwd_workspace(long long rows, int width, int sms) {
    return (size_t)bwd_ctas(rows, width, sms) * (size_t)width * sizeof(float);
}

cudaError_t ssd_launch_rmsnorm_bwd(const SsdNormBwd &a, float *partial, int sms,
                                   cudaStream_t stream) {
    if (a.in == SSD_ELT_F32) return launch_bwd<float, float>(a, partial, sms, stream);
    if (a.stream_type == SSD_ELT_F32)
        return launch_bwd<__nv_bfloat16, float>(a, partial, sms, stream);
    return launch_bwd<__nv_bfloat16, __nv_bfloat16>(a, partial, sms, stream);
}
