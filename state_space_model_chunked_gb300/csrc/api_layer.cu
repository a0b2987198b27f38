// C ABI of the layer's steps around the scan (declarations and contracts:
// include/ssd.h): argument checks, workspace carve-outs and launches.  Like
// the rest of the ABI layer it allocates nothing and never synchronises.
#include <math.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "launch.h"

namespace {

constexpr size_t kBad = (size_t)-1;

bool float_type(ssd_dtype t) { return t == SSD_F32 || t == SSD_BF16; }
bool known_type(ssd_dtype t) { return float_type(t) || t == SSD_FP8_E4M3; }
SsdElt elt(ssd_dtype t) {
    return t == SSD_F32 ? SSD_ELT_F32 : (t == SSD_BF16 ? SSD_ELT_BF16 : SSD_ELT_E4M3);
}
size_t size_of(ssd_dtype t) { return t == SSD_F32 ? 4 : (t == SSD_BF16 ? 2 : 1); }

bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
// a required / an optional array of elements of `n` bytes
bool array(const void *p, size_t n) { return p && aligned(p, n); }
bool maybe(const void *p, size_t n) { return aligned(p, n); }

ssd_status launched(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

ssd_status check_workspace(const void *ws, size_t have, size_t need, size_t align) {
    if (need == 0) return SSD_OK;
    if (!ws || have < need) return SSD_ERR_WORKSPACE;
    return aligned(ws, align) ? SSD_OK : SSD_ERR_INVALID_ARG;
}

bool norm_sizes_ok(long long rows, int width) { return rows >= 0 && width > 0; }
bool norm_sizes_handled(long long rows, int width) {
    return rows < (1ll << 31) && width < (1 << 24);
}

ssd_status check_linear(ssd_dtype in, long long tokens, int features, int inner) {
    if (!known_type(in) || tokens < 0 || features <= 0 || inner <= 0) return SSD_ERR_INVALID_ARG;
    if (tokens >= (1ll << 31) - 256 || features >= (1 << 22)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

bool valid_activation(ssd_activation a) { return a >= SSD_ACT_NONE && a <= SSD_ACT_RELU; }

// The product on the path its types and alignments take.
bool on_tensor_cores(const SsdProduct &p) {
    return !ssd_product_few_handles(p) && !ssd_product_gemv_handles(p) && ssd_product_tc_handles(p);
}
cudaError_t launch_product(const SsdProduct &p, cudaStream_t stream) {
    if (ssd_product_few_handles(p)) return ssd_launch_product_few(p, ssd_sm_count(), stream);
    if (ssd_product_gemv_handles(p)) return ssd_launch_product_gemv(p, stream);
    if (ssd_product_tc_handles(p))
        return ssd_launch_product_tc(p, ssd_sm_count(), ssd_device_error_word(), stream);
    return ssd_launch_product_simt(p, stream);
}

// The sequences of a recurrence call.
ssd_status check_sequences(int nseq, int length, const int *host, const int *dev,
                           long long *tokens) {
    if (nseq <= 0 || (host == nullptr) != (dev == nullptr)) return SSD_ERR_INVALID_ARG;
    if (host) {
        if (!aligned(dev, 4) || host[0] != 0) return SSD_ERR_INVALID_ARG;
        for (int s = 0; s < nseq; ++s)
            if (host[s + 1] < host[s]) return SSD_ERR_INVALID_ARG;
        *tokens = host[nseq];
    } else {
        if (length < 0) return SSD_ERR_INVALID_ARG;
        *tokens = (long long)nseq * length;
    }
    return *tokens < (1ll << 31) - 2048 ? SSD_OK : SSD_ERR_UNSUPPORTED;
}

// Sizes the recurrence's grid can number (tiles of 64 tokens by blocks of 32 channels).
bool gated_handled(long long tokens, int width) {
    return width < (1 << 21) && (tokens / 64 + 1) * (width / 32 + 1) < (1ll << 31);
}

// What the recurrence's two directions share.
ssd_status gated_input(const void *x, const void *g, const void *z, ssd_dtype dtype, int nseq,
                       int length, const int *host, const int *dev, int width, long long x_stride,
                       long long g_stride, long long z_stride, const float *init, SsdGated *out) {
    if (!known_type(dtype) || width <= 0) return SSD_ERR_INVALID_ARG;
    if (!float_type(dtype)) return SSD_ERR_UNSUPPORTED;
    const ssd_status st = check_sequences(nseq, length, host, dev, &out->tokens);
    if (st != SSD_OK) return st;
    if (!gated_handled(out->tokens, width)) return SSD_ERR_UNSUPPORTED;
    const size_t n = size_of(dtype);
    if (out->tokens > 0 && (!array(x, n) || !array(g, n))) return SSD_ERR_INVALID_ARG;
    if (!maybe(z, n) || !maybe(init, 4)) return SSD_ERR_INVALID_ARG;
    if (x_stride < width || g_stride < width || (z && z_stride < width))
        return SSD_ERR_INVALID_ARG;
    out->x = x;
    out->g = g;
    out->z = z;
    out->init = init;
    out->bf16 = dtype == SSD_BF16;
    out->nseq = nseq;
    out->length = length;
    out->width = width;
    out->cu = dev;
    out->x_stride = x_stride;
    out->g_stride = g_stride;
    out->z_stride = z_stride;
    return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_rmsnorm_fwd(const void *x, const void *residual, const float *weight, float eps,
                           ssd_dtype x_dtype, ssd_dtype stream_dtype, ssd_dtype out_dtype,
                           long long rows, int width, long long x_stride,
                           long long residual_stride, void *y, void *residual_out, float *rstd,
                           float *scale, cudaStream_t stream) {
    if (!known_type(x_dtype) || !known_type(stream_dtype) || !known_type(out_dtype))
        return SSD_ERR_INVALID_ARG;
    if (!norm_sizes_ok(rows, width) || !(eps >= 0.f)) return SSD_ERR_INVALID_ARG;
    if (!float_type(x_dtype) || (stream_dtype != x_dtype && stream_dtype != SSD_F32))
        return SSD_ERR_UNSUPPORTED;
    if (!norm_sizes_handled(rows, width)) return SSD_ERR_UNSUPPORTED;
    if (rows == 0) return SSD_OK;
    const size_t nx = size_of(x_dtype), ns = size_of(stream_dtype);
    if (!array(x, nx) || !array(weight, 4) || !array(y, size_of(out_dtype)) || !array(rstd, 4))
        return SSD_ERR_INVALID_ARG;
    if (residual && (!aligned(residual, ns) || !array(residual_out, ns) || residual_stride < width))
        return SSD_ERR_INVALID_ARG;
    if (out_dtype == SSD_FP8_E4M3 && !array(scale, 4)) return SSD_ERR_INVALID_ARG;
    if (x_stride < width) return SSD_ERR_INVALID_ARG;
    SsdNormFwd a{x, residual, weight, eps, elt(x_dtype), elt(stream_dtype), elt(out_dtype),
                 rows, width, x_stride, residual_stride, y, residual ? residual_out : nullptr,
                 rstd, scale};
    return launched(ssd_launch_rmsnorm_fwd(a, ssd_sm_count(), stream));
}

size_t ssd_rmsnorm_bwd_workspace_bytes(long long rows, int width) {
    if (!norm_sizes_ok(rows, width) || !norm_sizes_handled(rows, width)) return kBad;
    return ssd_rmsnorm_bwd_workspace(rows, width, ssd_sm_count());
}

ssd_status ssd_rmsnorm_bwd(const void *dy, const void *s, const float *weight, const float *rstd,
                           const void *dresidual, ssd_dtype dtype, ssd_dtype stream_dtype,
                           long long rows, int width, long long dy_stride, long long s_stride,
                           long long dresidual_stride, void *dx, void *ds, float *dweight,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!known_type(dtype) || !known_type(stream_dtype)) return SSD_ERR_INVALID_ARG;
    if (!norm_sizes_ok(rows, width)) return SSD_ERR_INVALID_ARG;
    if (!float_type(dtype) || (stream_dtype != dtype && stream_dtype != SSD_F32))
        return SSD_ERR_UNSUPPORTED;
    if (!norm_sizes_handled(rows, width)) return SSD_ERR_UNSUPPORTED;
    if (!array(dweight, 4)) return SSD_ERR_INVALID_ARG;
    if (rows == 0)
        return launched(cudaMemsetAsync(dweight, 0, (size_t)width * sizeof(float), stream));
    const size_t n = size_of(dtype), ns = size_of(stream_dtype);
    if (!array(dy, n) || !array(s, ns) || !array(weight, 4) || !array(rstd, 4) || !array(dx, n) ||
        !maybe(dresidual, ns) || !maybe(ds, ns))
        return SSD_ERR_INVALID_ARG;
    if (dy_stride < width || s_stride < width || (dresidual && dresidual_stride < width))
        return SSD_ERR_INVALID_ARG;
    const int sms = ssd_sm_count();
    const ssd_status st = check_workspace(workspace, workspace_bytes,
                                          ssd_rmsnorm_bwd_workspace(rows, width, sms), 16);
    if (st != SSD_OK) return st;
    SsdNormBwd a{dy, s, dresidual, weight, rstd, elt(dtype), elt(stream_dtype), rows, width,
                 dy_stride, s_stride, dresidual_stride, dx, ds, dweight};
    return launched(ssd_launch_rmsnorm_bwd(a, static_cast<float *>(workspace), sms, stream));
}

ssd_status ssd_linear_fwd(const void *x, const float *x_scale, const void *w,
                          const float *w_scale, const float *bias, const void *residual,
                          ssd_activation activation, ssd_dtype in_dtype, ssd_dtype out_dtype,
                          long long tokens, int features, int inner, long long x_stride,
                          long long residual_stride, void *y, long long y_stride, void *preact,
                          cudaStream_t stream) {
    const ssd_status st = check_linear(in_dtype, tokens, features, inner);
    if (st != SSD_OK) return st;
    if (!known_type(out_dtype) || !valid_activation(activation)) return SSD_ERR_INVALID_ARG;
    if (!float_type(out_dtype) || (in_dtype == SSD_F32 && out_dtype != SSD_F32))
        return SSD_ERR_UNSUPPORTED;
    if (tokens == 0) return SSD_OK;
    const bool fp8 = in_dtype == SSD_FP8_E4M3;
    const size_t n = fp8 ? 4 : size_of(in_dtype), no = size_of(out_dtype);
    const size_t np = in_dtype == SSD_F32 ? 4 : 2;
    if (!array(x, n) || !array(w, n) || !array(y, no) || !maybe(residual, no) || !maybe(bias, 4) ||
        !maybe(preact, np))
        return SSD_ERR_INVALID_ARG;
    if (fp8 ? !array(x_scale, 4) || !array(w_scale, 4) : x_scale || w_scale)
        return SSD_ERR_INVALID_ARG;
    if (x_stride < inner || y_stride < features || (residual && residual_stride < features))
        return SSD_ERR_INVALID_ARG;
    SsdProduct p{x, w, elt(in_dtype), tokens, features, inner, x_stride, 1, inner, 1, x_scale,
                 w_scale, bias, residual, residual_stride, (SsdAct)(int)activation, y, preact,
                 elt(out_dtype), in_dtype == SSD_F32 ? SSD_ELT_F32 : SSD_ELT_BF16, y_stride};
    return launched(launch_product(p, stream));
}

namespace {
// Workspace of the product's gradients: dp (when the activation changes dy),
// then the partial column sums.
struct LinearBwdPlan {
    size_t dp, sums, total;
};
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
LinearBwdPlan linear_bwd_plan(ssd_dtype dtype, ssd_activation act, long long tokens, int features) {
    LinearBwdPlan p;
    p.dp = act == SSD_ACT_NONE ? 0 : up256((size_t)tokens * features * size_of(dtype));
    p.sums = up256(ssd_act_bwd_workspace(tokens, features, ssd_sm_count()));
    p.total = p.dp + p.sums;
    return p;
}
}  // namespace

size_t ssd_linear_bwd_workspace_bytes(ssd_dtype dtype, ssd_activation activation,
                                      long long tokens, int features, int inner) {
    if (check_linear(dtype, tokens, features, inner) != SSD_OK || inner >= (1 << 22) ||
        !float_type(dtype) || !valid_activation(activation))
        return kBad;
    return tokens == 0 ? 0 : linear_bwd_plan(dtype, activation, tokens, features).total;
}

ssd_status ssd_linear_bwd(const void *dy, const void *x, const void *w, const void *preact,
                          ssd_activation activation, ssd_dtype dtype, long long tokens,
                          int features, int inner, long long dy_stride, long long x_stride,
                          void *dx, void *dw, float *dbias, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream) {
    ssd_status st = check_linear(dtype, tokens, features, inner);
    if (st != SSD_OK) return st;
    if (!valid_activation(activation)) return SSD_ERR_INVALID_ARG;
    if (!float_type(dtype) || inner >= (1 << 22)) return SSD_ERR_UNSUPPORTED;
    const size_t n = size_of(dtype);
    if (!maybe(dx, n) || !maybe(dw, n) || !maybe(dbias, 4)) return SSD_ERR_INVALID_ARG;
    if (tokens == 0) {
        if (dw && cudaMemsetAsync(dw, 0, (size_t)features * inner * n, stream) != cudaSuccess)
            return SSD_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)features * 4, stream) != cudaSuccess)
            return SSD_ERR_CUDA;
        return SSD_OK;
    }
    if (!array(dy, n) || (dw && !array(x, n)) || (dx && !array(w, n))) return SSD_ERR_INVALID_ARG;
    if (activation == SSD_ACT_NONE ? preact != nullptr : !array(preact, n))
        return SSD_ERR_INVALID_ARG;
    if (dy_stride < features || (dw && x_stride < inner)) return SSD_ERR_INVALID_ARG;
    const LinearBwdPlan plan = linear_bwd_plan(dtype, activation, tokens, features);
    st = check_workspace(workspace, workspace_bytes, plan.total, 256);
    if (st != SSD_OK) return st;
    char *ws = static_cast<char *>(workspace);
    const int sms = ssd_sm_count();
    const SsdElt t = elt(dtype);
    const bool act = activation != SSD_ACT_NONE;
    const void *dp = act ? ws : dy;
    const long long dp_stride = act ? features : dy_stride;
    // The bias's gradient is summed in two passes, the second one beside the products;
    // without an activation, the first one too (dy is its input and theirs).
    const SsdActBwd pass{dy, preact, t, (SsdAct)(int)activation, tokens, features, dy_stride,
                         act ? ws : nullptr};
    float *partial = dbias ? reinterpret_cast<float *>(ws + plan.dp) : nullptr;
    const bool products = dx || dw;
    const bool first = act || (dbias && !products);
    if (first && ssd_launch_act_bwd(pass, partial, sms, SsdOrder::after, stream) != cudaSuccess)
        return SSD_ERR_CUDA;
    // dx[m][k] = sum_n dp[m][n] w[n][k], dw[n][k] = sum_m dp[m][n] x[m][k]
    const SsdProduct px{dp, w, t, tokens, inner, features, dp_stride, 1, 1, inner, nullptr, nullptr,
                        nullptr, nullptr, 0, SsdAct::none, dx, nullptr, t, t, inner};
    const SsdProduct pw{dp, x, t, features, inner, tokens, 1, dp_stride, 1, x_stride, nullptr,
                        nullptr, nullptr, nullptr, 0, SsdAct::none, dw, nullptr, t, t, inner};
    cudaError_t e = cudaSuccess;
    if (dx && dw && on_tensor_cores(px) && on_tensor_cores(pw)) {
        e = ssd_launch_product_two(px, pw, sms, ssd_device_error_word(), stream);
    } else {
        if (dx) e = launch_product(px, stream);
        if (dw && e == cudaSuccess) e = launch_product(pw, stream);
    }
    if (dbias && !first && e == cudaSuccess)
        e = ssd_launch_act_bwd(pass, partial, sms, SsdOrder::beside, stream);
    if (dbias && e == cudaSuccess)
        e = ssd_launch_column_sum(partial, ssd_act_bwd_rows(tokens, features, sms), features, dbias,
                                  first && products ? SsdOrder::beside : SsdOrder::after, stream);
    if (e != cudaSuccess) return SSD_ERR_CUDA;
    return SSD_OK;
}

int ssd_linear_path(ssd_product product, ssd_dtype in_dtype, long long tokens, int features,
                    int inner) {
    if (check_linear(in_dtype, tokens, features, inner) != SSD_OK || tokens == 0 ||
        product < SSD_PRODUCT_FORWARD || product > SSD_PRODUCT_GRADIENTS)
        return -1;
    if (product != SSD_PRODUCT_FORWARD && (!float_type(in_dtype) || inner >= (1 << 22))) return -1;
    const int sms = ssd_sm_count();
    if (sms <= 0) return -1;
    // operands as the calls have them, at an address that only its alignment is read of
    const void *at = reinterpret_cast<const void *>((uintptr_t)4096);
    const SsdElt t = elt(in_dtype);
    SsdProduct y{}, dx{}, dw{};
    y.a = y.b = dx.a = dx.b = dw.a = dw.b = at;
    y.in = dx.in = dw.in = t;
    y.m = tokens, y.n = features, y.k = inner;
    y.a_row = y.b_row = inner, y.a_col = y.b_col = 1;
    dx.m = tokens, dx.n = inner, dx.k = features;
    dx.a_row = features, dx.a_col = 1, dx.b_row = 1, dx.b_col = inner;
    dw.m = features, dw.n = inner, dw.k = tokens;
    dw.a_row = 1, dw.a_col = features, dw.b_row = 1, dw.b_col = inner;
    if (product == SSD_PRODUCT_GRADIENTS)
        return on_tensor_cores(dx) && on_tensor_cores(dw) ? ssd_product_two_path(dx, dw, sms)
                                                          : SSD_PATH_APART;
    const SsdProduct &p = product == SSD_PRODUCT_FORWARD ? y : product == SSD_PRODUCT_DX ? dx : dw;
    if (ssd_product_few_handles(p)) return SSD_PATH_FEW;
    if (ssd_product_gemv_handles(p)) return SSD_PATH_FP32_FEW;
    return ssd_product_tc_handles(p) ? ssd_product_tc_path(p, sms) : SSD_PATH_FP32;
}

size_t ssd_gated_scan_workspace_bytes(ssd_dtype dtype, long long tokens, int width) {
    if (!float_type(dtype) || tokens < 0 || tokens >= (1ll << 31) - 2048 || width <= 0 ||
        !gated_handled(tokens, width))
        return kBad;
    return ssd_gated_workspace(tokens, width);
}

ssd_status ssd_gated_scan_fwd(const void *x, const void *g, const void *z, ssd_dtype dtype,
                              int nseq, int length, const int *cu_seqlens_host,
                              const int *cu_seqlens_dev, int width, long long x_stride,
                              long long g_stride, long long z_stride, const float *init_state,
                              void *y, long long y_stride, float *final_state,
                              float *checkpoints, void *workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
    SsdGatedFwd a{};
    ssd_status st =
        gated_input(x, g, z, dtype, nseq, length, cu_seqlens_host, cu_seqlens_dev, width, x_stride,
                    g_stride, z_stride, init_state, &a.in);
    if (st != SSD_OK) return st;
    if (a.in.tokens > 0 && !array(y, size_of(dtype))) return SSD_ERR_INVALID_ARG;
    if (y_stride < width || !maybe(final_state, 4) || !maybe(checkpoints, 4))
        return SSD_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, ssd_gated_workspace(a.in.tokens, width), 256);
    if (st != SSD_OK) return st;
    a.y = y;
    a.y_stride = y_stride;
    a.final_state = final_state;
    a.checkpoints = checkpoints;
    return launched(ssd_launch_gated_fwd(a, ssd_sm_count(), workspace, ssd_device_error_word(), stream));
}

ssd_status ssd_gated_scan_bwd(const void *dy, const void *x, const void *g, const void *z,
                              ssd_dtype dtype, int nseq, int length, const int *cu_seqlens_host,
                              const int *cu_seqlens_dev, int width, long long dy_stride,
                              long long x_stride, long long g_stride, long long z_stride,
                              const float *init_state, const float *checkpoints,
                              const float *dfinal, void *dx, long long dx_stride, void *dg,
                              long long dg_stride, void *dz, long long dz_stride, float *dinit,
                              void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    SsdGatedBwd a{};
    ssd_status st =
        gated_input(x, g, z, dtype, nseq, length, cu_seqlens_host, cu_seqlens_dev, width, x_stride,
                    g_stride, z_stride, init_state, &a.in);
    if (st != SSD_OK) return st;
    const size_t n = size_of(dtype);
    if (a.in.tokens > 0 && (!array(dy, n) || !array(dx, n) || !array(dg, n) ||
                            (z && !array(dz, n)) || !array(checkpoints, 4)))
        return SSD_ERR_INVALID_ARG;
    if (dy_stride < width || dx_stride < width || dg_stride < width || (z && dz_stride < width) ||
        !maybe(dfinal, 4) || !maybe(dinit, 4))
        return SSD_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, ssd_gated_workspace(a.in.tokens, width), 256);
    if (st != SSD_OK) return st;
    a.dy = dy;
    a.dfinal = dfinal;
    a.checkpoints = checkpoints;
    a.dy_stride = dy_stride;
    a.dx_stride = dx_stride;
    a.dg_stride = dg_stride;
    a.dz_stride = dz_stride;
    a.dx = dx;
    a.dg = dg;
    a.dz = dz;
    a.dinit = dinit;
    return launched(ssd_launch_gated_bwd(a, ssd_sm_count(), workspace, ssd_device_error_word(), stream));
}

ssd_status ssd_gated_state_update(float *state, const void *x, const void *g, const void *z,
                                  ssd_dtype dtype, long long rows, int width, long long x_stride,
                                  long long g_stride, long long z_stride, void *y,
                                  cudaStream_t stream) {
    if (!known_type(dtype) || rows < 0 || width <= 0) return SSD_ERR_INVALID_ARG;
    if (!float_type(dtype) || rows >= (1ll << 31) || width >= (1 << 21) ||
        (size_t)rows * width >= ((size_t)1 << 38))
        return SSD_ERR_UNSUPPORTED;
    if (rows == 0) return SSD_OK;
    const size_t n = size_of(dtype);
    if (!array(state, 4) || !array(x, n) || !array(g, n) || !maybe(z, n) || !array(y, n))
        return SSD_ERR_INVALID_ARG;
    if (x_stride < width || g_stride < width || (z && z_stride < width))
        return SSD_ERR_INVALID_ARG;
    SsdGatedStep a{state, x, g, z, dtype == SSD_BF16, rows, width, x_stride, g_stride, z_stride, y};
    return launched(ssd_launch_gated_step(a, stream));
}

}  // extern "C"
