// Layer norm of s = x + residual, forward (with an 8-bit output and its row scales) and
// backward.
//
//   s = x + r,  v_j = (s_j - mean) rstd,  rstd = (mean_j (s_j - mean)^2 + eps)^(-1/2)
//   y_j = v_j w_j + b_j
//   8 bits: scale = max_j |y_j| / 448 (1 where that is 0), q = e4m3(y / scale)
//   backward, with e_j = dy_j w_j:
//     ds_j = ds_out_j + rstd (e_j - mean_i e_i - v_j mean_i(e_i v_i))
//     dw_j = sum over rows of dy_j v_j,  db_j = sum over rows of dy_j
//
// Bound by memory: every value is read once and written once, the sums stay in fp32, and
// each result is rounded once.  As in the RMS norm a CTA walks over rows, one at a time in
// registers with the next row's loads under way, its columns' weights in registers too.
//   The mean and the sum of squares around it come from one pass and one barrier: every
// thread takes both over its own values (the squares around its own mean), and pairs are
// joined by
//     n = n1 + n2,  d = m2 - m1,  m = m1 + d n2 / n,  q = q1 + q2 + d^2 n1 n2 / n,
// which loses nothing where the mean is large against the spread, as sums of s^2 would,
// nor where one value is far from the others, as sums around a chosen value would.
//   16 rows of 2560: 2.6 us (latency: launch, one trip of loads, one barrier).  Gradients of
// 16376 rows of 1024: 46 us, 0.85 of a copy's rate, 2 of them the partial sums' second pass.
#include "norm_rows.cuh"
#include "ptx.cuh"

namespace {

using namespace ssdnorm;

constexpr int kRuns8 = 4, kBwdRuns8 = 2, kRuns1 = 16;
constexpr int kFwdRuns = 4, kFwdWarpsSm = 16;
constexpr int kBwdRuns = 1, kBwdWarpsSm = 16;

// A count of values, their mean, and the sum of squares around it.
struct Moments {
    float n, mean, q;
    __device__ __forceinline__ void join(float n2, float mean2, float q2) {
        // (none of its own: the other's, which a quotient near 1 would not be)
        const float all = n + n2, part = n > 0.f ? __fdividef(n2, all) : 1.f;
        const float d = mean2 - mean;
        mean += d * part;
        q += q2 + d * d * n * part;
        n = all;
    }
    __device__ __forceinline__ void join_lanes(int lanes) {
        for (int o = lanes / 2; o > 0; o >>= 1)
            join(__shfl_xor_sync(0xffffffffu, n, o), __shfl_xor_sync(0xffffffffu, mean, o),
                 __shfl_xor_sync(0xffffffffu, q, o));
    }
};

// The moments of the CTA's values in every thread.
__device__ __forceinline__ Moments cta_moments(Moments m, float (*buf)[32]) {
    m.join_lanes(32);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return m;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        buf[0][warp] = m.n;
        buf[1][warp] = m.mean;
        buf[2][warp] = m.q;
    }
    __syncthreads();
    const bool on = lane < warps;
    m = {on ? buf[0][lane] : 0.f, on ? buf[1][lane] : 0.f, on ? buf[2][lane] : 0.f};
    m.join_lanes(32);
    return m;
}

__device__ __forceinline__ float cta_max(float mx, float *buf) {
    mx = ssd_warp_max(mx);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return mx;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[warp] = mx;
    __syncthreads();
    return ssd_warp_max(lane < warps ? buf[lane] : 0.f);
}

// a and b summed over the CTA.
__device__ __forceinline__ void cta_sum2(float &a, float &b, float (*buf)[32]) {
    a = ssd_warp_sum(a);
    b = ssd_warp_sum(b);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        buf[0][warp] = a;
        buf[1][warp] = b;
    }
    __syncthreads();
    a = ssd_warp_sum(lane < warps ? buf[0][lane] : 0.f);
    b = ssd_warp_sum(lane < warps ? buf[1][lane] : 0.f);
}

template <typename TX, typename TR, typename TO, int V, int kC>
__global__ void __launch_bounds__(32 * kMostWarps) layernorm_fwd_kernel(const SsdLayerNormFwd a) {
    ssdptx::griddep_wait();
    __shared__ float buf[2][4][32];
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
    float w[kC][V], b[kC][V];
    load_weight<V, kC>(a.weight, nvec, w);
    load_weight<V, kC>(a.bias, a.bias ? nvec : 0, b);
    // this thread's runs, and its values' number
    int runs = 0;
#pragma unroll
    for (int c = 0; c < kC; ++c) runs += (int)(threadIdx.x + c * blockDim.x) < nvec;
    const float mine = (float)(runs * V);
    for (int turn = 0; row < a.rows; turn ^= 1) {
        float s[kC][V], sum = 0.f, mx = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                s[c][k] = xr.run[c].get(k);
                if (res) s[c][k] += rr.run[c].get(k);
                sum += s[c][k];
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
        // (divided, not by way of the reciprocal: a row of one bf16 value is its own mean exactly)
        Moments m{mine, runs ? sum / mine : 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            if ((int)(threadIdx.x + c * blockDim.x) >= nvec) continue;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float d = s[c][k] - m.mean;
                m.q += d * d;
            }
        }
        m = cta_moments(m, buf[turn]);
        const float rstd = rsqrtf(m.q / (float)a.width + a.eps);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                s[c][k] = (s[c][k] - m.mean) * rstd * w[c][k] + b[c][k];
                if constexpr (kFp8) mx = fmaxf(mx, fabsf(s[c][k]));
            }
        }
        if constexpr (kFp8) {
            // (values past the row have no weight and no bias: they are 0 here)
            mx = cta_max(mx, buf[turn][3]);
            if (rstd != rstd) mx = rstd;
        }
        const RowScale q(mx);
        if (threadIdx.x == 0) {
            a.mean[row] = m.mean;
            a.rstd[row] = rstd;
            if constexpr (kFp8) a.scale[row] = q.scale;
        }
        TO *y = static_cast<TO *>(a.y) + row * a.width;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i >= nvec) continue;
            if constexpr (kFp8) {
#pragma unroll
                for (int k = 0; k < V; ++k) s[c][k] = q.apply(s[c][k]);
            }
            ssd_store_vec<V>(y + (size_t)i * V, s[c]);
        }
        row = next;
    }
}

// Rows too wide for the registers of a CTA: passes over the row, the later ones out of L2.
template <typename TX, typename TR, typename TO>
__global__ void layernorm_fwd_wide_kernel(const SsdLayerNormFwd a) {
    __shared__ float buf[4][32];
    constexpr bool kFp8 = sizeof(TO) == 1;
    const long long row = blockIdx.x;
    const TX *x = static_cast<const TX *>(a.x) + row * a.x_stride;
    const TR *r = a.residual ? static_cast<const TR *>(a.residual) + row * a.residual_stride
                             : nullptr;
    const auto value = [&](int i) { return r ? ssd_ld(x + i) + ssd_ld(r + i) : ssd_ld(x + i); };
    Moments m{0.f, 0.f, 0.f};
    for (int i = threadIdx.x; i < a.width; i += blockDim.x) {
        const float s = value(i), d = s - m.mean;
        m.n += 1.f;
        m.mean += d / m.n;
        m.q += d * (s - m.mean);
    }
    m = cta_moments(m, buf);
    const float rstd = rsqrtf(m.q / (float)a.width + a.eps);
    const auto normed = [&](float s, int i) {
        return (s - m.mean) * rstd * a.weight[i] + (a.bias ? a.bias[i] : 0.f);
    };
    float mx = 0.f;
    if constexpr (kFp8) {
        for (int i = threadIdx.x; i < a.width; i += blockDim.x)
            mx = fmaxf(mx, fabsf(normed(value(i), i)));
        mx = cta_max(mx, buf[3]);
        if (rstd != rstd) mx = rstd;
    }
    const RowScale q(mx);
    if (threadIdx.x == 0) {
        a.mean[row] = m.mean;
        a.rstd[row] = rstd;
        if constexpr (kFp8) a.scale[row] = q.scale;
    }
    TR *so = static_cast<TR *>(a.residual_out) + (r ? row * a.width : 0);
    TO *y = static_cast<TO *>(a.y) + row * a.width;
    for (int i = threadIdx.x; i < a.width; i += blockDim.x) {
        const float s = value(i);
        float o[1] = {normed(s, i)};
        if constexpr (kFp8) o[0] = q.apply(o[0]);
        ssd_store_vec<1>(y + i, o);
        if (r) ssd_st(so + i, s);
    }
}

// ------------------------------------------------------------------ backward
// A CTA walks the rows b, b + grid, ...; each thread keeps its columns' share of dw and
// db in registers over all of them and writes it once, as row b of the partial sums,
// which are then added in order.
template <typename T, typename TS, int V, int kC>
__global__ void __launch_bounds__(32 * kMostWarps)
layernorm_bwd_kernel(const SsdLayerNormBwd a, float *partial) {
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
    float rstd = a.rstd[row], mean = a.mean[row];
    float w[kC][V], dw[kC][V], db[kC][V];
    load_weight<V, kC>(a.weight, nvec, w);
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int k = 0; k < V; ++k) dw[c][k] = db[c][k] = 0.f;
    for (int turn = 0; row < a.rows; turn ^= 1) {
        // e = dy w, v = (s - mean) rstd, and what came from elsewhere
        float e[kC][V], v[kC][V], d[kC][V], sum = 0.f, dot = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float dyv = yr.run[c].get(k);
                v[c][k] = (sr.run[c].get(k) - mean) * rstd;
                d[c][k] = dr.run[c].get(k);
                e[c][k] = dyv * w[c][k];
                sum += e[c][k];
                dot += e[c][k] * v[c][k];
                dw[c][k] += dyv * v[c][k];
                db[c][k] += dyv;
            }
        }
        const float scale = rstd;
        const long long next = row + gridDim.x;
        if (next < a.rows) {
            yr.load(dy + next * a.dy_stride, nvec, true);
            sr.load(st + next * a.s_stride, nvec, true);
            dr.load(dres + next * a.dresidual_stride, nvec, res);
            rstd = a.rstd[next];
            mean = a.mean[next];
        }
        cta_sum2(sum, dot, buf[turn]);
        const float c1 = sum / (float)a.width, c2 = dot / (float)a.width;
        T *dx = static_cast<T *>(a.dx) + row * a.width;
        TS *ds = a.ds ? static_cast<TS *>(a.ds) + row * a.width : nullptr;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i >= nvec) continue;
            float o[V];
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] = scale * (e[c][k] - c1 - v[c][k] * c2) + d[c][k];
            ssd_store_vec<V>(dx + (size_t)i * V, o);
            if (ds) ssd_store_vec<V>(ds + (size_t)i * V, o);
        }
        row = next;
    }
    float *const bias = partial + (size_t)gridDim.x * a.width;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        const int i = threadIdx.x + c * blockDim.x;
        if (i >= nvec) continue;
        const size_t at = (size_t)blockIdx.x * a.width + (size_t)i * V;
        ssd_store_vec<V>(partial + at, dw[c]);
        if (a.dbias) ssd_store_vec<V>(bias + at, db[c]);
    }
}

// Rows too wide for a CTA's registers: the sums per row, then the columns.
template <typename T, typename TS>
__global__ void layernorm_bwd_wide_kernel(const SsdLayerNormBwd a) {
    __shared__ float buf[2][32];
    const long long row = blockIdx.x;
    const T *dy = static_cast<const T *>(a.dy) + row * a.dy_stride;
    const TS *s = static_cast<const TS *>(a.s) + row * a.s_stride;
    const TS *dres = a.dresidual ? static_cast<const TS *>(a.dresidual) + row * a.dresidual_stride
                                 : nullptr;
    const float rstd = a.rstd[row], mean = a.mean[row];
    float sum = 0.f, dot = 0.f;
    for (int i = threadIdx.x; i < a.width; i += blockDim.x) {
        const float e = ssd_ld(dy + i) * a.weight[i];
        sum += e;
        dot += e * (ssd_ld(s + i) - mean) * rstd;
    }
    cta_sum2(sum, dot, buf);
    const float c1 = sum / (float)a.width, c2 = dot / (float)a.width;
    T *dx = static_cast<T *>(a.dx) + row * a.width;
    TS *ds = a.ds ? static_cast<TS *>(a.ds) + row * a.width : nullptr;
    for (int i = threadIdx.x; i < a.width; i += blockDim.x) {
        const float v = (ssd_ld(s + i) - mean) * rstd;
        float o = rstd * (ssd_ld(dy + i) * a.weight[i] - c1 - v * c2);
        if (dres) o += ssd_ld(dres + i);
        ssd_st(dx + i, o);
        if (ds) ssd_st(ds + i, o);
    }
}
template <typename T, typename TS>
__global__ void layernorm_dw_wide_kernel(const SsdLayerNormBwd a, float *partial) {
    const int j = blockIdx.y * blockDim.x + threadIdx.x;
    if (j >= a.width) return;
    float dw = 0.f, db = 0.f;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float dy = ssd_ld(static_cast<const T *>(a.dy) + row * a.dy_stride + j);
        const float s = ssd_ld(static_cast<const TS *>(a.s) + row * a.s_stride + j);
        dw += dy * ((s - a.mean[row]) * a.rstd[row]);
        db += dy;
    }
    partial[(size_t)blockIdx.x * a.width + j] = dw;
    if (a.dbias) partial[((size_t)gridDim.x + blockIdx.x) * a.width + j] = db;
}

// The sums of n partial rows, of dw (blockIdx.y 0) and of db (1), in a fixed order: 32 x 32
// threads take 32 columns, each thread row every 32nd partial row.
__global__ void __launch_bounds__(1024)
layernorm_sums_kernel(const float *partial, int n, int width, float *dweight, float *dbias) {
    __shared__ float part[32][33];
    ssdptx::griddep_wait();
    const int j = blockIdx.x * 32 + threadIdx.x;
    const float *rows = partial + (size_t)blockIdx.y * n * width;
    float acc = 0.f;
    if (j < width) {
#pragma unroll 8
        for (int r = threadIdx.y; r < n; r += 32) acc += __ldcg(rows + (size_t)r * width + j);
    }
    part[threadIdx.y][threadIdx.x] = acc;
    __syncthreads();
    if (threadIdx.y == 0 && j < width) {
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) v += part[r][threadIdx.x];
        (blockIdx.y ? dbias : dweight)[j] = v;
    }
}

template <typename TX, typename TR, typename TO>
cudaError_t launch_fwd(const SsdLayerNormFwd &a, int sms, cudaStream_t stream) {
    const bool v8 = a.width % 8 == 0 && vec8(a.weight, 0, 4) && vec8(a.bias, 0, 4) &&
                    vec8(a.x, a.x_stride, sizeof(TX)) &&
                    vec8(a.residual, a.residual_stride, sizeof(TR)) &&
                    vec8(a.residual_out, a.width, sizeof(TR)) && ((uintptr_t)a.y & 7u) == 0 &&
                    vec8(sizeof(TO) == 1 ? nullptr : a.y, a.width, sizeof(TO));
    // few rows leave SMs idle: one run a thread, so the row is read in one step
    const RowShape sh = row_shape(a.width, v8 ? 8 : 1, v8 ? kRuns8 : kRuns1,
                                  a.rows <= sms ? 1 : (v8 ? kFwdRuns : kRuns1));
    const unsigned rows = walkers(a.rows, sms, kFwdWarpsSm / (sh.warps ? sh.warps : 1));
    if (sh.warps == 0) {
        layernorm_fwd_wide_kernel<TX, TR, TO><<<(unsigned)a.rows, 1024, 0, stream>>>(a);
        return cudaGetLastError();
    }
    auto kernel = layernorm_fwd_kernel<TX, TR, TO, 1, kRuns1>;
    if (v8) {
        switch (sh.runs) {
            case 1: kernel = layernorm_fwd_kernel<TX, TR, TO, 8, 1>; break;
            case 2: kernel = layernorm_fwd_kernel<TX, TR, TO, 8, 2>; break;
            case 3: kernel = layernorm_fwd_kernel<TX, TR, TO, 8, 3>; break;
            default: kernel = layernorm_fwd_kernel<TX, TR, TO, 8, 4>; break;
        }
    }
    return ssd_launch_early(kernel, dim3(rows), dim3(32 * sh.warps), stream, a);
}

template <typename TX, typename TR>
cudaError_t launch_fwd_out(const SsdLayerNormFwd &a, int sms, cudaStream_t stream) {
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
cudaError_t launch_bwd(const SsdLayerNormBwd &a, float *partial, int sms, cudaStream_t stream) {
    const bool v8 = a.width % 8 == 0 && vec8(a.weight, 0, 4) && vec8(a.dy, a.dy_stride, sizeof(T)) &&
                    vec8(a.s, a.s_stride, sizeof(TS)) &&
                    vec8(a.dresidual, a.dresidual_stride, sizeof(TS)) &&
                    vec8(a.dx, a.width, sizeof(T)) && vec8(a.ds, a.width, sizeof(TS));
    const RowShape sh = row_shape(a.width, v8 ? 8 : 1, v8 ? kBwdRuns8 : kRuns1, v8 ? kBwdRuns : kRuns1);
    const int n = bwd_ctas(a.rows, a.width, sms);
    cudaError_t e;
    if (sh.warps == 0) {
        layernorm_bwd_wide_kernel<T, TS><<<(unsigned)a.rows, 1024, 0, stream>>>(a);
        const dim3 grid((unsigned)n, (unsigned)((a.width + 255) / 256));
        layernorm_dw_wide_kernel<T, TS><<<grid, 256, 0, stream>>>(a, partial);
        e = cudaGetLastError();
    } else {
        auto kernel = layernorm_bwd_kernel<T, TS, 1, kRuns1>;
        if (v8)
            kernel = sh.runs == 1 ? layernorm_bwd_kernel<T, TS, 8, 1> : layernorm_bwd_kernel<T, TS, 8, 2>;
        e = ssd_launch_early(kernel, dim3((unsigned)n), dim3(32 * sh.warps), stream, a, partial);
    }
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((a.width + 31) / 32), a.dbias ? 2u : 1u);
    return ssd_launch_early(layernorm_sums_kernel, grid, dim3(32, 32), stream,
                            (const float *)partial, n, a.width, a.dweight, a.dbias);
}

}  // namespace

cudaError_t ssd_launch_layernorm_fwd(const SsdLayerNormFwd &a, int sms, cudaStream_t stream) {
    if (a.in == SSD_ELT_F32) return launch_fwd_out<float, float>(a, sms, stream);
    if (a.stream_type == SSD_ELT_F32) return launch_fwd_out<__nv_bfloat16, float>(a, sms, stream);
    return launch_fwd_out<__nv_bfloat16, __nv_bfloat16>(a, sms, stream);
}

size_t ssd_layernorm_bwd_workspace(long long rows, int width, int sms) {
    return 2 * (size_t)bwd_ctas(rows, width, sms) * (size_t)width * sizeof(float);
}

cudaError_t ssd_launch_layernorm_bwd(const SsdLayerNormBwd &a, float *partial, int sms,
                                     cudaStream_t stream) {
    if (a.in == SSD_ELT_F32) return launch_bwd<float, float>(a, partial, sms, stream);
    if (a.stream_type == SSD_ELT_F32)
        return launch_bwd<__nv_bfloat16, float>(a, partial, sms, stream);
    return launch_bwd<__nv_bfloat16, __nv_bfloat16>(a, partial, sms, stream);
}
