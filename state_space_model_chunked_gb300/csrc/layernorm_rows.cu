// Layer norm forward of many rows to 8 bits, a row a warp (the formulas: layernorm.cu).
//
// With a CTA a row, a row waits for the barriers of its moments and of its largest value, and
// what an SM has under way does not cover that: 65536 rows of 2560 take 282 us.  A warp needs
// none.  Its next row is copied to shared memory while the present one is in registers (kC
// runs of 8 values a lane), from which the mean, the squares around it, the largest value and
// the output are taken by turns; weight and bias lie in shared memory too.  Bound by memory:
// each value is read and written once; 65536 rows of 2560 take 200 us, 0.86 of a copy's rate.
#include "norm_rows.cuh"
#include "ptx.cuh"

namespace {

using namespace ssdnorm;
using namespace ssdptx;

constexpr int kWarps = 8;
constexpr int kMostBytes = 232448, kSmBytes = 233472;      // shared memory of a CTA, and of an SM with 1 KB a CTA
constexpr int kCtasSm(int runs) { return runs <= 4 ? 4 : runs <= 10 ? 2 : 1; }

struct RowsLayout {
    uint32_t weight, x, r, row, bytes;      // row: bytes of a warp's row, x in front of r
};
RowsLayout rows_layout(const SsdLayerNormFwd &a) {
    const auto up = [](uint32_t n) { return (n + 127) / 128 * 128; };
    const uint32_t nx = a.in == SSD_ELT_F32 ? 4 : 2, nr = a.stream_type == SSD_ELT_F32 ? 4 : 2;
    RowsLayout l;
    l.weight = 128;
    l.x = l.weight + 2 * up(a.width * 4);
    l.r = up(a.width * nx);
    l.row = l.r + (a.residual ? up(a.width * nr) : 0);
    l.bytes = l.x + kWarps * l.row;
    return l;
}

// (withhold: the first warp's first copy is never complete)
struct Waits {
    unsigned long long limit;
    bool withhold;
    unsigned *err;
};

template <typename TX, typename TR, int kC>
__global__ void __launch_bounds__(32 * kWarps, kCtasSm(kC))
layernorm_rows_kernel(const SsdLayerNormFwd a, const RowsLayout l, const Waits wait) {
    extern __shared__ __align__(128) uint8_t rows_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nvec = a.width / 8;
    const uint32_t bar = smem_u32(rows_smem) + 8 * warp;
    uint8_t *const mine = rows_smem + l.x + warp * l.row;
    float *const weight = reinterpret_cast<float *>(rows_smem + l.weight), *const bias = weight + (l.x - l.weight) / 8;
    const bool res = a.residual != nullptr;
    if (lane == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    griddep_wait();
    const uint64_t once = l2_evict_first_policy();      // (207 -> 202 us at the size above)
    const auto fetch = [&](long long row) {
        const uint32_t bx = a.width * sizeof(TX), br = res ? a.width * sizeof(TR) : 0;
        mbar_arrive_expect_tx(bar, bx + br + (wait.withhold && row == 0 ? 16 : 0));
        bulk_load_evict_first(smem_u32(mine), static_cast<const TX *>(a.x) + row * a.x_stride, bx, bar, once);
        if (res)
            bulk_load_evict_first(smem_u32(mine + l.r), static_cast<const TR *>(a.residual) + row * a.residual_stride, br, bar, once);
    };
    const long long step = (long long)gridDim.x * kWarps;
    long long row = (long long)blockIdx.x * kWarps + warp;
    if (lane == 0 && row < a.rows) fetch(row);
    for (int i = threadIdx.x; i < a.width; i += 32 * kWarps) {
        weight[i] = a.weight[i];
        bias[i] = a.bias ? a.bias[i] : 0.f;
    }
    __syncthreads();
    const float share = 1.f / (float)a.width;
    for (uint32_t turn = 0; row < a.rows; turn ^= 1, row += step) {
        // (a warp that gives up asks for no more, and its copy lands before the CTA ends)
        if (!__all_sync(0xffffffffu, mbar_wait(bar, turn, wait.limit))) {
            ssd_report(wait.err, SSD_DEVERR_TIMEOUT);
            mbar_wait(bar, turn, kSsdDefaultWaitNs);
            return;
        }
        float s[kC][8], sum = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int i = lane + 32 * c;
            SsdRaw<TX, 8> x;
            SsdRaw<TR, 8> r;
            x.zero();
            r.zero();
            if (i < nvec) {
                x.load(reinterpret_cast<const TX *>(mine) + 8 * i);
                if (res) r.load(reinterpret_cast<const TR *>(mine + l.r) + 8 * i);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[c][k] = res ? x.get(k) + r.get(k) : x.get(k);
                sum += s[c][k];
            }
        }
        __syncwarp();
        if (lane == 0 && row + step < a.rows) fetch(row + step);
        if (res) {
            TR *const so = static_cast<TR *>(a.residual_out) + row * a.width;
#pragma unroll
            for (int c = 0; c < kC; ++c)
                if (lane + 32 * c < nvec) ssd_store_vec<8>(so + 8 * (lane + 32 * c), s[c]);
        }
        // (divided, not by way of the reciprocal: a row of one bf16 value is its own mean exactly)
        const float mean = ssd_warp_sum(sum) / (float)a.width;
        float squares = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            if (lane + 32 * c >= nvec) continue;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[c][k] -= mean;
                squares += s[c][k] * s[c][k];
            }
        }
        const float rstd = rsqrtf(ssd_warp_sum(squares) * share + a.eps);
        float mx = 0.f;
        __nv_fp8_e4m3 *const y = static_cast<__nv_fp8_e4m3 *>(a.y) + row * a.width;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int i = lane + 32 * c;
            if (i >= nvec) continue;
            SsdRaw<float, 8> w, b;
            w.load(weight + 8 * i);
            b.load(bias + 8 * i);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[c][k] = s[c][k] * rstd * w.get(k) + b.get(k);
                mx = fmaxf(mx, fabsf(s[c][k]));
            }
        }
        mx = ssd_warp_max(mx);
        if (rstd != rstd) mx = rstd;
        const RowScale q(mx);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int i = lane + 32 * c;
            if (i >= nvec) continue;
            if (q.tiny) {
#pragma unroll
                for (int k = 0; k < 8; ++k) s[c][k] = q.apply(s[c][k]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) s[c][k] *= q.inv;
            }
            ssd_store_vec<8>(y + 8 * i, s[c]);
        }
        if (lane == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
            a.scale[row] = q.scale;
        }
    }
}

template <typename TX, typename TR, int kC>
cudaError_t launch(const SsdLayerNormFwd &a, int sms, unsigned *err, cudaStream_t stream) {
    const RowsLayout l = rows_layout(a);
    const auto kernel = layernorm_rows_kernel<TX, TR, kC>;
    // (the most that any call takes: the attribute is the kernel's, and another thread may be
    // about to launch it with more than this call needs)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostBytes);
    if (e != cudaSuccess) return e;
    int ctas = (int)(kSmBytes / (l.bytes + 1024));
    if (ctas > kCtasSm(kC)) ctas = kCtasSm(kC);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(walkers((a.rows + kWarps - 1) / kWarps, sms, ctas));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = l.bytes;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const SsdDebug debug = ssd_debug_config();
    return cudaLaunchKernelEx(&cfg, kernel, a, l, Waits{debug.wait_ns, debug.fault == kSsdFaultWithholdSignal, err});
}

template <typename TX, typename TR>
cudaError_t launch_runs(const SsdLayerNormFwd &a, int sms, unsigned *err, cudaStream_t stream) {
    const int runs = (a.width + 255) / 256;
    if (runs <= 2) return launch<TX, TR, 2>(a, sms, err, stream);
    if (runs <= 4) return launch<TX, TR, 4>(a, sms, err, stream);
    if (runs <= 6) return launch<TX, TR, 6>(a, sms, err, stream);
    if (runs <= 8) return launch<TX, TR, 8>(a, sms, err, stream);
    if (runs <= 10) return launch<TX, TR, 10>(a, sms, err, stream);
    return launch<TX, TR, 16>(a, sms, err, stream);
}
}  // namespace

// Rows enough for the SMs' warps, in vectors, and few enough values for a warp's registers.
// Rows of 2560 to 8 bits, a warp each against a CTA each: 1216 rows 8.5 against 7.7 us, 2432 rows
// 11.6 against 12.9, 38912 rows 124 against 169.  To bf16, where no largest value is wanted, a
// CTA is as fast or faster (38912 rows: 126 against 133 us).
//   Other widths, us of 65536 rows (above 2560 columns, of as many values as those have), a warp
// each against a CTA each.  bf16 with a bf16 residual: 256 columns 29 and 30, 776 67 and 112,
// 1544 117 and 253, 2048 156 and 249, 2560 196 and 283, 2816 315 and 264, 3200 293 and 388, 4096
// 256 and 315.  In fp32: 512 72 and 71, 1024 142 and 175, 2048 280 and 365, 2560 360 and 409, 2816
// 404 and 398, 3200 397 and 503.  bf16 with an fp32 residual: 2048 242 and 301, 2560 367 and 317, 2816
// 421 and 302, 3200 398 and 436.  So a warp each where two CTAs of them fit on an SM; where only one
// does, if a CTA's row would take four runs a thread, which makes it slow, or the rows are fp32 of
// up to 2560 columns.
bool ssd_layernorm_rows_handles(const SsdLayerNormFwd &a, int sms) {
    if (a.out == SSD_ELT_F32 || a.out == SSD_ELT_BF16 || a.rows < 16ll * sms || a.width % 8 != 0 || a.width > 4096)
        return false;
    const int nx = a.in == SSD_ELT_F32 ? 4 : 2, nr = a.stream_type == SSD_ELT_F32 ? 4 : 2;
    const uint32_t bytes = rows_layout(a).bytes;
    const bool two = a.width <= 2560 && 2 * (bytes + 1024) <= kSmBytes;
    if (bytes > kMostBytes || !(two || row_shape(a.width, 8, 4, 4).runs == 4 || (nx == 4 && a.width <= 2560))) return false;
    return vec8(a.x, a.x_stride, nx) && vec8(a.residual, a.residual_stride, nr) && vec8(a.residual_out, a.width, nr) &&
           ((uintptr_t)a.y & 7u) == 0;
}

cudaError_t ssd_launch_layernorm_rows(const SsdLayerNormFwd &a, int sms, unsigned *err, cudaStream_t stream) {
    if (a.in == SSD_ELT_F32) return launch_runs<float, float>(a, sms, err, stream);
    if (a.stream_type == SSD_ELT_F32) return launch_runs<__nv_bfloat16, float>(a, sms, err, stream);
    return launch_runs<__nv_bfloat16, __nv_bfloat16>(a, sms, err, stream);
}
