// Internal launchers behind the C ABI (include/ssd.h).  Arguments are
// validated by the ABI layer before any of these is called.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "common.cuh"

cudaError_t ssd_launch_decode(void *state, bool bf16_state, const void *x, const float *dt,
                              const float *A, const void *B, const void *C,
                              const float *D, void *y, bool bf16, int batch,
                              int H, int P, int N, int G, int num_sms, unsigned int *err,
                              const SsdFuse &fuse, cudaStream_t stream);

// ntok consecutive tokens per (batch, head) in one launch (state read and
// written once); headdim must not exceed ssd_decode_multi_max_headdim(N)
// (0 for an unsupported dstate).
cudaError_t ssd_launch_decode_multi(void *state, bool bf16_state, const void *x, const float *dt,
                                    const float *A, const void *B, const void *C,
                                    const float *D, void *y, bool bf16, int batch, int ntok,
                                    int H, int P, int N, int G, int num_sms, const SsdFuse &fuse,
                                    cudaStream_t stream);
int ssd_decode_multi_max_headdim(int N);

size_t ssd_simt_smem_bytes(int N);

// fp8 (E4M3) -> bfloat16 widening of up to three arrays in one launch; every
// pointer 16-byte aligned (the ABI checks the sources, the workspace
// carve-out aligns the destinations).
struct SsdWidenJob {
    const void *src;
    void *dst;
    size_t n;
};
struct SsdWidenJobs {
    SsdWidenJob job[3];
    int count;
};
struct SsdWidenFirst {     // first CTA of each job in the widening launch
    size_t cta[3];
};
cudaError_t ssd_launch_widen_fp8(const SsdWidenJobs &jobs, cudaStream_t stream);

// Sequence split over GPUs by tokens: a token range's log-decay A_h * sum dt
// ([batch][H], dt transformed as the scan does), and the chain of R ranges'
// contributions into each range's entering state ([R][batch][H][P][N]).
cudaError_t ssd_launch_range_log_decay(const float *dt, const float *A, int batch, int L, int H,
                                       const SsdFuse &fuse, float *out, cudaStream_t stream);
cudaError_t ssd_launch_chain_states(const float *contrib, const float *log_decay,
                                    const float *init, int R, int batch, int H, int P, int N,
                                    float *entering, cudaStream_t stream);

// Test hooks of the ABI layer: the fault to inject (0 = none) and the limit
// of every bounded device wait, read by the launchers at each launch.
struct SsdDebug {
    int fault;
    unsigned long long wait_ns;
};
SsdDebug ssd_debug_config();

// Events recorded around the kernel that writes y (null = none).
struct SsdProfileEvents {
    cudaEvent_t before, after;
};

// Records a profiling event on `stream`; inside stream capture it becomes an
// event-record node of the graph (an external record), not a capture-internal
// dependency.
inline cudaError_t ssd_record_event(cudaEvent_t ev, cudaStream_t stream) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(stream, &st);
    if (e != cudaSuccess) return e;
    if (st == cudaStreamCaptureStatusActive)
        return cudaEventRecordWithFlags(ev, stream, cudaEventRecordExternal);
    return cudaEventRecord(ev, stream);
}

cudaError_t ssd_launch_scan_simt(const void *x, const float *dt, const float *A,
                                 const void *B, const void *C, const float *D,
                                 const float *init, void *y, float *fin, bool bf16,
                                 int batch, int L, int H, int P, int N, int G,
                                 const SsdFuse &fuse, const int *cu, SsdProfileEvents prof,
                                 cudaStream_t stream);

// The driver's cuTensorMapEncodeTiled (null when it has none).
PFN_cuTensorMapEncodeTiled_v12000 ssd_tensor_map_encoder();

// Tensor-core (tcgen05/TMEM/TMA) chunked scan.
struct SsdTcPlan {
    bool supported;
    int tiles;            // 128-token tiles per sequence (last may be ragged)
    int heads_per_cta;    // heads sharing one C.B^T product
    int seg_tiles;        // tiles per segment (the unit of sequence parallelism)
    int nseg;             // segments per sequence
    int seg_heads;        // heads per CTA of the segment-contribution kernel
    int seg_split;        // batched, seg_heads 4: segments launched at four heads per
                          // CTA (the rest at two, in a second launch); 0 = one launch
    size_t workspace;     // bytes of workspace required
    int launches;         // kernels enqueued per call
    // work items: sequences, segment contributions (every segment but each
    // sequence's last) and scan segments; batched plans have nseqs equal
    // sequences of `tiles` tiles, packed plans (varlen) per-sequence lengths
    bool varlen;
    int nseqs, nslots, items;
    size_t dt_offset;     // workspace bytes before the transformed step sizes
};

SsdTcPlan ssd_tc_plan(int batch, int L, int H, int P, int N, int G, int num_sms);
// Plan for nseq packed sequences, token offsets cu_host[0..nseq] (host copy).
SsdTcPlan ssd_tc_plan_varlen(int nseq, const int *cu_host, int H, int P, int N, int G,
                             int num_sms);

cudaError_t ssd_launch_scan_tc(const SsdTcPlan &plan, const void *x, const float *dt,
                               const float *A, const void *B, const void *C,
                               const float *D, const float *init, void *y, float *fin,
                               int batch, int L, int H, int P, int N, int G,
                               void *workspace, unsigned int *err, const SsdFuse &fuse,
                               SsdProfileEvents prof, cudaStream_t stream,
                               const int *cu_dev = nullptr);

// ------------------------------------------------ the steps around the scan
// What the layer's other kernels share with the ABI layer: the current
// device's error word and its number of SMs.
unsigned int *ssd_device_error_word();
int ssd_sm_count();

// Element types of the layer's operators.
enum SsdElt { SSD_ELT_F32 = 0, SSD_ELT_BF16 = 1, SSD_ELT_E4M3 = 2 };

// Root-mean-square norm (rmsnorm.cu).  `in`: the type of x (forward) and of dy
// and dx (backward); `stream_type`: that of the residual stream.
struct SsdNormFwd {
    const void *x, *residual;
    const float *weight;
    float eps;
    SsdElt in, stream_type, out;
    long long rows;
    int width;
    long long x_stride, residual_stride;
    void *y, *residual_out;
    float *rstd, *scale;
};
cudaError_t ssd_launch_rmsnorm_fwd(const SsdNormFwd &a, int sms, cudaStream_t stream);

struct SsdNormBwd {
    const void *dy, *s, *dresidual;
    const float *weight, *rstd;
    SsdElt in, stream_type;
    long long rows;
    int width;
    long long dy_stride, s_stride, dresidual_stride;
    void *dx, *ds;
    float *dweight;
};
size_t ssd_rmsnorm_bwd_workspace(long long rows, int width, int sms);
cudaError_t ssd_launch_rmsnorm_bwd(const SsdNormBwd &a, float *partial, int sms,
                                   cudaStream_t stream);

// Layer norm (layernorm.cu), with the RMS norm's types and strides.
struct SsdLayerNormFwd {
    const void *x, *residual;
    const float *weight, *bias;
    float eps;
    SsdElt in, stream_type, out;
    long long rows;
    int width;
    long long x_stride, residual_stride;
    void *y, *residual_out;
    float *mean, *rstd, *scale;
};
cudaError_t ssd_launch_layernorm_fwd(const SsdLayerNormFwd &a, int sms, cudaStream_t stream);
// Many rows, a row a warp (layernorm_rows.cu).
bool ssd_layernorm_rows_handles(const SsdLayerNormFwd &a, int sms);
cudaError_t ssd_launch_layernorm_rows(const SsdLayerNormFwd &a, int sms, unsigned *err, cudaStream_t stream);

struct SsdLayerNormBwd {
    const void *dy, *s, *dresidual;
    const float *weight, *mean, *rstd;
    SsdElt in, stream_type;
    long long rows;
    int width;
    long long dy_stride, s_stride, dresidual_stride;
    void *dx, *ds;
    float *dweight, *dbias;
};
size_t ssd_layernorm_bwd_workspace(long long rows, int width, int sms);
cudaError_t ssd_launch_layernorm_bwd(const SsdLayerNormBwd &a, float *partial, int sms,
                                     cudaStream_t stream);

// Embedding (embedding.cu): rows of a table by tokens, and its gradient.
struct SsdEmbedding {
    const void *tokens;
    bool wide;                  // tokens of 64 bits
    const void *table;
    SsdElt table_type, out_type;
    long long count;
    int vocab, width;
    float scale;
    void *y;
};
cudaError_t ssd_launch_embedding(const SsdEmbedding &a, int sms, cudaStream_t stream);
struct SsdEmbeddingBwd {
    const void *tokens;
    bool wide;
    const void *dy;
    long long dy_stride;
    SsdElt in, out_type;
    long long count;
    int vocab, width;
    float scale;
    void *dtable;
};
size_t ssd_embedding_bwd_workspace(long long count, int vocab, int width);
cudaError_t ssd_launch_embedding_bwd(const SsdEmbeddingBwd &a, void *ws, int sms,
                                     cudaStream_t stream);

// Gated delta rule over sequences as the gated recurrence has them (delta_simt.cu).
constexpr int kSsdDeltaChunk = 64;      // tokens between the states that are kept
struct SsdDelta {
    const void *q, *k, *v;
    const float *g, *beta;
    bool bf16;
    long long tokens;
    int nseq, length;
    const int *cu;
    int heads, groups, p, n;
    long long q_stride, k_stride, v_stride;     // of a token
    float scale;
};
// The place of the state before a sequence's 64 * c-th token among the kept ones, for a
// sequence that begins at token `first`.
__host__ __device__ inline long long ssd_delta_slot(long long first, int seq, long long c) {
    return first / kSsdDeltaChunk + seq + c;
}
__host__ __device__ inline long long ssd_delta_slots(long long tokens, int nseq) {
    return tokens / kSsdDeltaChunk + nseq;
}
struct SsdDeltaFwd {
    SsdDelta in;
    const float *init;
    void *o;
    long long o_stride;
    float *final_state, *checkpoints;
};
cudaError_t ssd_launch_delta_fwd_simt(const SsdDeltaFwd &a, int sms, cudaStream_t stream);
struct SsdDeltaBwd {
    SsdDelta in;
    const void *dout;
    const float *checkpoints, *dfinal;
    long long do_stride, dq_stride, dk_stride, dv_stride;
    void *dq, *dk, *dv;
    float *dg, *dbeta, *dinit;
};
size_t ssd_delta_bwd_simt_workspace(const SsdDelta &d);
cudaError_t ssd_launch_delta_bwd_simt(const SsdDeltaBwd &a, void *ws, cudaStream_t stream);
// One token (delta_step.cu): state_out may be state.
struct SsdDeltaStep {
    const void *state;
    void *state_out;
    bool bf16_state;
    const void *q, *k, *v;
    const float *g, *beta;
    bool bf16;
    int batch, heads, groups, p, n;
    long long q_stride, k_stride, v_stride;
    float scale;
    void *o;
};
cudaError_t ssd_launch_delta_step(const SsdDeltaStep &a, int sms, cudaStream_t stream);

// Gated linear recurrence (gated_scan.cu) over `tokens` tokens laid end to
// end: nseq sequences of `length` tokens each, or, with cu (device, nseq + 1
// offsets), of any lengths.
constexpr int kSsdCheckpointTokens = 64;
struct SsdGated {
    const void *x, *g, *z;
    const float *init;
    bool bf16;
    long long tokens;
    int nseq, length, width;
    const int *cu;
    long long x_stride, g_stride, z_stride;
};
struct SsdGatedFwd {
    SsdGated in;
    void *y;
    long long y_stride;
    float *final_state, *checkpoints;
};
struct SsdGatedBwd {
    SsdGated in;
    const void *dy;
    const float *dfinal, *checkpoints;
    long long dy_stride, dx_stride, dg_stride, dz_stride;
    void *dx, *dg, *dz;
    float *dinit;
};
// ws: ssd_gated_workspace bytes; err: the device error word of bounded waits.
size_t ssd_gated_workspace(long long tokens, int width);
cudaError_t ssd_launch_gated_fwd(const SsdGatedFwd &a, int sms, void *ws, unsigned *err,
                                 cudaStream_t stream);
cudaError_t ssd_launch_gated_bwd(const SsdGatedBwd &a, int sms, void *ws, unsigned *err,
                                 cudaStream_t stream);
struct SsdGatedStep {
    float *state;
    const void *x, *g, *z;
    bool bf16;
    long long rows;
    int width;
    long long x_stride, g_stride, z_stride;
    void *y;
};
cudaError_t ssd_launch_gated_step(const SsdGatedStep &a, cudaStream_t stream);

// Matrix product with a fused epilogue: out[m][n] = act(sum_k A(m,k) B(n,k)
// * a_scale[m] * b_scale[n] + bias[n]) + residual[m][n].
enum class SsdAct { none = 0, silu = 1, gelu = 2, relu = 3 };
struct SsdProduct {
    // element (row, k) of A at a[row * a_row + k * a_col]; one of the two
    // strides is 1.  B likewise by its rows n.
    const void *a, *b;
    SsdElt in;
    long long m, n, k;
    long long a_row, a_col, b_row, b_col;
    const float *a_scale, *b_scale, *bias;
    const void *residual;        // of the output's type
    long long residual_row;
    SsdAct act;
    void *out, *preact;          // preact: of type preact_type, rows of n values, or null
    SsdElt out_type, preact_type;
    long long out_row;
};
cudaError_t ssd_launch_product_simt(const SsdProduct &p, cudaStream_t stream);
bool ssd_product_few_handles(const SsdProduct &p);
cudaError_t ssd_launch_product_few(const SsdProduct &p, int sms, cudaStream_t stream);
bool ssd_product_gemv_handles(const SsdProduct &p);
cudaError_t ssd_launch_product_gemv(const SsdProduct &p, cudaStream_t stream);
bool ssd_product_tc_handles(const SsdProduct &p);
cudaError_t ssd_launch_product_tc(const SsdProduct &p, int sms, unsigned *err,
                                  cudaStream_t stream);
// Which way it takes (the header's ssd_path): of ssd_product_tc_handles products, one
// alone and a gradient's two.
int ssd_product_tc_path(const SsdProduct &p, int sms);
int ssd_product_two_path(const SsdProduct &dx, const SsdProduct &dw, int sms);
// A gradient's two products on the tensor cores: `dx` of a K-major A and a B with its
// rows contiguous, `dw` with both operands' rows contiguous.
cudaError_t ssd_launch_product_two(const SsdProduct &dx, const SsdProduct &dw, int sms,
                                   unsigned *err, cudaStream_t stream);

// dp = dy act'(preact) (dp null: not stored) and the column sums of dp by blocks of
// rows (`partial` holds ssd_act_bwd_workspace bytes; null: none).
struct SsdActBwd {
    const void *dy, *preact;
    SsdElt type;
    SsdAct act;
    long long rows;
    int width;
    long long dy_stride;
    void *dp;
};
// A launch that may start while the kernel in front of it in the stream still runs:
// the kernel calls griddep_wait before it touches anything that one may, so what
// overlaps is the launch and the set-up.  It reads with ordinary loads: those of the
// read-only cache are defined for memory that nobody writes while the kernel lives.
template <typename... P, typename... A>
cudaError_t ssd_launch_early(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t stream,
                             A... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// How a kernel stands to the one in front of it in the stream: after it, or beside it,
// where it reads nothing of that kernel's and only ends after it.
enum class SsdOrder { after, beside };
// out[j] = the sum of column j over n rows of `width` floats (linear_simt.cu).
cudaError_t ssd_launch_column_sum(const float *partial, int n, int width, float *out,
                                  SsdOrder order, cudaStream_t stream);
size_t ssd_act_bwd_workspace(long long rows, int width, int sms);
cudaError_t ssd_launch_act_bwd(const SsdActBwd &a, float *partial, int sms, SsdOrder order,
                               cudaStream_t stream);
// How many rows of sums it leaves in `partial`.
int ssd_act_bwd_rows(long long rows, int width, int sms);

// The delta rule on the tensor cores (delta_tc.cu): whether the sizes allow it, and the
// addresses too; ws: ssd_delta_tc_workspace bytes (0 for other sizes).
bool ssd_delta_tc_sizes(const SsdDelta &d);
bool ssd_delta_tc_inputs(const SsdDelta &d);
bool ssd_delta_tc_handles(const SsdDeltaFwd &a);
size_t ssd_delta_tc_workspace(const SsdDelta &d, int sms);
cudaError_t ssd_launch_delta_fwd_tc(const SsdDeltaFwd &a, void *ws, int sms, unsigned *err,
                                    cudaStream_t stream);
// Its gradients (delta_tc_bwd.cu); ws: ssd_delta_tc_bwd_workspace bytes.
bool ssd_delta_tc_bwd_handles(const SsdDeltaBwd &b);
size_t ssd_delta_tc_bwd_workspace(const SsdDelta &d, int sms);
cudaError_t ssd_launch_delta_bwd_tc(const SsdDeltaBwd &a, void *ws, int sms, unsigned *err, cudaStream_t stream);
// dq and dk from the sums of `parts` neighbours of [token][groups * parts][N] (delta_simt.cu).
cudaError_t ssd_launch_delta_group_sums(const float *dq_parts, void *dq, long long dq_stride, const float *dk_parts,
                                        void *dk, long long dk_stride, const SsdDelta &d, int parts, cudaStream_t stream);
