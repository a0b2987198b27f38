/*
 * ssd.h -- C ABI of libssd.so, the GB300 (sm_103a) Mamba-2 state-space-duality
 * (SSD) hot path: the chunked scan for prefill and the single-token state
 * update for decode.
 *
 * Where the operations come from:
 *   - "Mamba-Family State-Space Model Kernels on a Programmable CGLA",
 *     section III.A (Mamba-2 layer with three kernel shapes): SSD Step-1 is
 *     GEMM1 (reduction over the state size N) -> Hadamard mask -> GEMM2
 *     (reduction over the chunk length Q); Step-3 updates the recurrent state
 *     h sequentially across chunks, with an input-dependent diagonal
 *     transition A_c; section III.C: the per-chunk recurrence is an N x d
 *     product (128 x 64 for Mamba-370M).
 *   - "Compiler-First State Space Duality and Portable O(1) Autoregressive
 *     Caching for Inference", abstract: diagonal per-head dynamics,
 *     fixed-size chunking, and an O(1) cached decode step.
 *   - "Mambalaya: Einsum-Based Fusion Optimizations on State-Space Models",
 *     abstract and Figures 4-5: fuse neighbouring Einsums so intermediates
 *     do not round-trip off-chip memory.
 *
 * The recurrence, for each batch row b and head h (group g = h / (H / G)):
 *     h_t = exp(dt_t * A_h) * h_{t-1} + dt_t * B_t x_t^T      (state N x P)
 *     y_t = C_t . h_t + D_h * x_t                             (uses updated h)
 * with h_{-1} = init_state (or zero) and final_state = h_{L-1}.  dt is used
 * exactly as given unless a call passes a dt transform (ssd_dt_transform);
 * the fused entry points can also gate y by silu(z).
 *
 * Layouts (row-major, contiguous, element strides implied by the sizes):
 *     x, y            [batch][seqlen][nheads][headdim]          in_dtype
 *     dt              [batch][seqlen][nheads]                    float
 *     A, D            [nheads]                                   float
 *     B, C            [batch][seqlen][ngroups][dstate]           in_dtype
 *     init_state, final_state, decode state
 *                     [batch][nheads][headdim][dstate]           float
 *                     (a decode state may be bfloat16: ssd_state_update_fused)
 * For decode, drop the seqlen dimension.  Packed variable-length batches
 * (ssd_scan_fwd_varlen) drop the batch dimension of the token arrays.
 *
 * fp8 inputs (in_dtype SSD_FP8_E4M3, prefill entry points only): x, B and C
 * hold one byte per value in the E4M3 encoding -- sign bit, 4 exponent bits
 * with bias 7, 3 significand bits; exponent field 0 encodes the subnormals
 * m * 2^-9; no infinities; S.1111.111 is NaN; the largest finite value is
 * 448.  Every E4M3 value is exactly a bfloat16 value, so each call widens x,
 * B and C once into bfloat16 copies in its workspace (one elementwise kernel,
 * ssd_fp8_e4m3_to_bf16) and runs the bf16 path on the copies: the result is
 * the bf16 path's on the exactly decoded inputs.  y and the gate's z are
 * bfloat16 in such a call.  The pages name reduced precision as future work
 * (CGLA sections V.A and VI) without fixing a format; E4M3 is the common
 * 8-bit one.  The decode entry points return SSD_ERR_UNSUPPORTED for it.
 *
 * Ownership: every pointer is a DEVICE pointer owned by the caller, except
 * where an entry point says otherwise.  The library allocates no memory;
 * scratch memory is the caller's workspace, sized by
 * ssd_scan_workspace_bytes().
 *
 * Asynchrony: work is enqueued on `stream` and the call returns without
 * synchronising.  Argument errors are detected on the host before anything
 * is enqueued and are returned synchronously.  Device-side faults the kernels
 * detect themselves (a bounded wait that ran out, a misaligned shared-memory
 * carve-out) set a device error word read by ssd_last_device_error().
 *
 * Aliasing: y and final_state must not overlap any input.  The decode state
 * is updated in place.
 */
#ifndef SSD_GB300_H
#define SSD_GB300_H

#include <stddef.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SSD_OK = 0,
    SSD_ERR_INVALID_ARG = 1,   /* null pointer, size <= 0, H % G != 0, misaligned pointer */
    SSD_ERR_UNSUPPORTED = 2,   /* a valid shape the requested kernel does not handle */
    SSD_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed */
    SSD_ERR_TIMEOUT = 4,       /* a bounded device-side wait ran out (read via ssd_last_device_error) */
    SSD_ERR_WORKSPACE = 5      /* workspace pointer null or smaller than ssd_scan_workspace_bytes() */
} ssd_status;

typedef enum { SSD_F32 = 0, SSD_BF16 = 1, SSD_FP8_E4M3 = 2 } ssd_dtype;

/* Which kernels ssd_scan_fwd_algo uses, and the delta rule's calls that end in
 * _algo.  AUTO takes the tensor-core path when the shape allows it and the SIMT
 * path otherwise; both run on the GPU. */
typedef enum {
    SSD_ALGO_AUTO = 0,
    SSD_ALGO_SIMT = 1,      /* exact-fp32 FFMA chunked scan, any shape */
    SSD_ALGO_TCGEN05 = 2    /* tcgen05/TMEM/TMA chunked scan: bf16 inputs, headdim 64,
                               dstate 128 */
} ssd_algo;

/* Bytes of device workspace ssd_scan_fwd / ssd_scan_fwd_algo need for this
 * shape on the CURRENT device (the segment plan depends on its SM count), for
 * either input dtype (fp32 inputs need none; the figure is that of bf16
 * inputs): the segment states and decays of the tensor-core path.  Returns 0
 * when the shape needs none, and (size_t)-1 for invalid sizes. */
size_t ssd_scan_workspace_bytes(int batch, int seqlen, int nheads, int headdim,
                                int dstate, int ngroups, int chunk);

/* The exact workspace of a call with this input dtype and, when
 * with_dt_transform != 0, a dt transform (ssd_scan_fwd_dt, ssd_scan_fwd_fused):
 * on the tensor-core path a transform adds batch x seqlen x nheads floats for
 * the transformed step sizes.  SSD_FP8_E4M3 adds the bfloat16 copies of x, B
 * and C (2 bytes per value, each copy rounded up to 256 bytes) in front of
 * the workspace of the bf16 call.  (size_t)-1 for invalid sizes. */
size_t ssd_scan_fused_workspace_bytes(int batch, int seqlen, int nheads, int headdim,
                                      int dstate, int ngroups, int chunk,
                                      ssd_dtype in_dtype, int with_dt_transform);

/* Number of kernel launches ssd_scan_fwd enqueues for this shape on the
 * current device (for launch accounting and CUDA-graph planning); -1 for
 * invalid sizes.  A dt transform on the tensor-core path adds one (the
 * elementwise pass that transforms every dt once), and so do fp8 inputs (the
 * widening of x, B and C). */
int ssd_scan_kernel_launches(int batch, int seqlen, int nheads, int headdim,
                             int dstate, int ngroups, int chunk,
                             ssd_dtype in_dtype);

/* Prefill: the chunked SSD scan over a whole sequence (section III.A of the
 * CGLA page: Step-1 intra-chunk dual form, chunk states, Step-3 inter-chunk
 * recurrence, plus the off-diagonal output and the D skip).
 *
 *   x, B, C     in_dtype device arrays (layouts above; SSD_FP8_E4M3 as
 *               described there, with its workspace from
 *               ssd_scan_fused_workspace_bytes).
 *   dt, A       float.  D: float [nheads] or NULL (no skip term).
 *   chunk       the chunk length Q: one of 16, 32, 64, 128, 256, validated
 *               and otherwise UNUSED.  The result does not depend on Q (the
 *               chunked form is an exact re-association of the recurrence);
 *               the kernels tile the sequence in their own block sizes (128
 *               tokens on the tensor-core path, 64 on the SIMT path).
 *   dt          any sign is accepted.  dt >= 0 (a time step) is the intended
 *               use; with dt < 0 the recurrence grows instead of decaying,
 *               and the tensor-core path stays exact only while that growth
 *               inside one 128-token tile is below about e^60 (its mask
 *               factors are fp32); the SIMT path has no such limit.
 *   init_state  float [batch][nheads][headdim][dstate] or NULL (zeros).
 *   y           in_dtype output (bfloat16 for fp8 inputs).  final_state:
 *               float output or NULL.
 *   workspace   device scratch of at least ssd_scan_workspace_bytes() bytes
 *               (may be NULL when that is 0), 256-byte aligned; its contents
 *               need no initialisation.
 * Requirements: all sizes > 0, nheads % ngroups == 0, dstate % 4 == 0,
 * dstate <= 256, base pointers 16-byte aligned.  seqlen may be any length
 * (the last block is ragged). */
ssd_status ssd_scan_fwd(const void *x, const float *dt, const float *A,
                        const void *B, const void *C, const float *D,
                        ssd_dtype in_dtype, int batch, int seqlen, int nheads,
                        int headdim, int dstate, int ngroups, int chunk,
                        const float *init_state, void *y, float *final_state,
                        void *workspace, size_t workspace_bytes,
                        cudaStream_t stream);

/* Same as ssd_scan_fwd with an explicit kernel choice.  SSD_ALGO_TCGEN05
 * returns SSD_ERR_UNSUPPORTED for shapes it does not handle. */
ssd_status ssd_scan_fwd_algo(ssd_algo algo, const void *x, const float *dt,
                             const float *A, const void *B, const void *C,
                             const float *D, ssd_dtype in_dtype, int batch,
                             int seqlen, int nheads, int headdim, int dstate,
                             int ngroups, int chunk, const float *init_state,
                             void *y, float *final_state, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream);

/* Optional transform of the raw step size, applied to every dt the kernels
 * read (the pages take the step Delta from the input projection, CGLA
 * section III.A, without spelling out how it is made positive; this is the
 * usual bias + softplus parameterisation).  The fp32 and decode kernels apply
 * it where they read dt; the tensor-core path transforms every dt once, in an
 * elementwise pass into the workspace, before its kernels run:
 *
 *   dt <- min(max(sp(dt_raw + dt_bias[h]), dt_min), dt_max)
 *   sp(u) = log(1 + e^u) when softplus != 0, else sp(u) = u.
 *
 * dt_bias: float [nheads] device array or NULL (no bias).  dt_min <= dt_max
 * (NaN rejected); use -INFINITY / INFINITY for no clamp.  The sign rule of
 * ssd_scan_fwd applies to the transformed dt (softplus, or dt_min >= 0, makes
 * it a non-negative time step).  The caller owns dt_bias; it is read during
 * the call's kernels. */
typedef struct ssd_dt_transform {
    const float *dt_bias;
    int softplus;
    float dt_min, dt_max;
} ssd_dt_transform;

/* ssd_scan_fwd_algo with a dt transform (NULL = identity: exactly
 * ssd_scan_fwd_algo).  Returns SSD_ERR_INVALID_ARG when dt_min > dt_max or
 * either is NaN.  With a transform the workspace is
 * ssd_scan_fused_workspace_bytes(..., in_dtype, 1). */
ssd_status ssd_scan_fwd_dt(ssd_algo algo, const void *x, const float *dt,
                           const float *A, const void *B, const void *C,
                           const float *D, const ssd_dt_transform *dt_transform,
                           ssd_dtype in_dtype, int batch, int seqlen, int nheads,
                           int headdim, int dstate, int ngroups, int chunk,
                           const float *init_state, void *y, float *final_state,
                           void *workspace, size_t workspace_bytes,
                           cudaStream_t stream);

/* Packed variable-length sequences: the scan of ssd_scan_fwd_dt run on each
 * of nseq independent sequences laid end to end on one token axis (each
 * sequence is its own recurrence with its own initial and final state, as
 * the pages define the scan per sequence; the packing is this library's
 * layout, not the pages').  Sequence s is tokens cu[s] .. cu[s+1]-1 of
 * T = cu[nseq] tokens:
 *   x, y   in_dtype [T][nheads][headdim];  dt float [T][nheads];
 *   B, C   in_dtype [T][ngroups][dstate];
 *   init_state, final_state  float [nseq][nheads][headdim][dstate] or NULL.
 *   cu_seqlens_host  int [nseq + 1] HOST array: cu[0] = 0, non-decreasing.
 *                    Empty sequences are allowed (final = initial state, or
 *                    zeros); with T = 0 the token arrays may be NULL.  It
 *                    sizes the grid and the workspace.
 *   cu_seqlens_dev   the same nseq + 1 values in a DEVICE int array, read by
 *                    the kernels; the two copies must agree (not checked).
 *   z      in_dtype [T][nheads][headdim] (bfloat16 for fp8 inputs) or
 *          NULL: the output gate of ssd_scan_fwd_fused.
 * Other arguments and requirements as ssd_scan_fwd_dt.  The workspace is
 * sized by ssd_scan_varlen_workspace_bytes() for the same offsets.
 * Returns SSD_ERR_INVALID_ARG for offsets that do not start at 0 or decrease. */
ssd_status ssd_scan_fwd_varlen(ssd_algo algo, const void *x, const float *dt,
                               const float *A, const void *B, const void *C,
                               const float *D, const ssd_dt_transform *dt_transform,
                               const void *z, ssd_dtype in_dtype, int nseq,
                               const int *cu_seqlens_host,
                               const int *cu_seqlens_dev, int nheads, int headdim,
                               int dstate, int ngroups, int chunk,
                               const float *init_state, void *y,
                               float *final_state, void *workspace,
                               size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes and kernel launches of ssd_scan_fwd_varlen for these
 * offsets on the current device ((size_t)-1 / -1 for invalid arguments).  The
 * workspace figure covers a call with a dt transform (total tokens x nheads
 * floats for the transformed step sizes on the tensor-core path); a call
 * without one uses that much less of it. */
size_t ssd_scan_varlen_workspace_bytes(int nseq, const int *cu_seqlens_host,
                                       int nheads, int headdim, int dstate,
                                       int ngroups, int chunk, ssd_dtype in_dtype);
int ssd_scan_varlen_kernel_launches(int nseq, const int *cu_seqlens_host,
                                    int nheads, int headdim, int dstate,
                                    int ngroups, int chunk, ssd_dtype in_dtype);

/* Output gate of the layer step after the scan, fused into the kernels that
 * write y (the fusion of neighbouring layer steps into the scan that the
 * compiler-first SSD page and the Mambalaya cascade describe; the gate's
 * form is the usual Mamba-2 one, not spelled out on the pages):
 *
 *   y <- y * silu(z),   silu(z) = z / (1 + e^-z),
 *
 * applied after the D skip, before y is rounded to its dtype.  z: a device
 * array of y's dtype and layout, 16-byte aligned, or NULL (no gate).  The
 * normalisation that may follow the gate in a layer is not fused (it reduces
 * over all heads of a token).  Everything else as ssd_scan_fwd_dt. */
ssd_status ssd_scan_fwd_fused(ssd_algo algo, const void *x, const float *dt,
                              const float *A, const void *B, const void *C,
                              const float *D, const ssd_dt_transform *dt_transform,
                              const void *z, ssd_dtype in_dtype, int batch,
                              int seqlen, int nheads, int headdim, int dstate,
                              int ngroups, int chunk, const float *init_state,
                              void *y, float *final_state, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream);

/* Profiling hook (process-wide, not for concurrent callers): while both
 * events are non-NULL, every following ssd_scan_fwd / ssd_scan_fwd_algo
 * records `before` immediately before and `after` immediately after the
 * kernel that writes y, on the call's stream, so cudaEventElapsedTime gives
 * that kernel's device time.  Works inside stream capture (the records become
 * graph nodes).  Pass NULL, NULL to stop.  Always returns SSD_OK. */
ssd_status ssd_scan_profile_events(cudaEvent_t before, cudaEvent_t after);

/* Size of the scratch array built into the library for ssd_scan_fwd_static. */
#define SSD_STATIC_SCRATCH_BYTES (64u << 20)

/* ssd_scan_fwd for callers that cannot allocate device memory (the pages
 * have no counterpart: this exists for callers whose memory is fixed at
 * start-up, such as an engine plugin handed only its inputs and outputs, or a
 * runtime that forbids device allocation after initialisation).  Same
 * arguments and results as ssd_scan_fwd without the workspace: the scratch is
 * a fixed array of SSD_STATIC_SCRATCH_BYTES inside the library, held on every
 * GPU that loads the library until the process exits.  Allocates nothing.
 *   - Returns SSD_ERR_WORKSPACE when the shape needs more scratch than
 *     SSD_STATIC_SCRATCH_BYTES (ssd_scan_workspace_bytes() tells how much).
 *     The 2.7B-shaped 65536-token layer (80 heads, 23 MB of bf16 segment
 *     states on a 152-SM GB300) fits.
 *   - The first call on each device looks up the scratch address for that
 *     device; make that first call before any stream capture.
 *   - All calls share the one scratch array: calls whose work overlaps on the
 *     GPU (unordered streams) race.  No scratch contents need clearing. */
ssd_status ssd_scan_fwd_static(const void *x, const float *dt, const float *A,
                               const void *B, const void *C, const float *D,
                               ssd_dtype in_dtype, int batch, int seqlen,
                               int nheads, int headdim, int dstate,
                               int ngroups, int chunk,
                               const float *init_state, void *y,
                               float *final_state, cudaStream_t stream);

/* Decode: one token of the recurrence for every (batch, head), the O(1)
 * cached step of the compiler-first SSD page.
 *   state  float [batch][nheads][headdim][dstate], read and updated IN PLACE.
 *   x      in_dtype [batch][nheads][headdim];  dt float [batch][nheads];
 *   B, C   in_dtype [batch][ngroups][dstate];  A, D float [nheads] (D may be NULL).
 *   y      in_dtype [batch][nheads][headdim], computed from the updated state.
 * A stack of layers can be updated in one call by treating (layer, head) as
 * the head index and giving every layer its own group (ngroups = layers).
 * Requirements: sizes > 0, nheads % ngroups == 0, dstate a power of two in
 * [4, 256], 16-byte aligned state / B / C. */
ssd_status ssd_state_update(float *state, const void *x, const float *dt,
                            const float *A, const void *B, const void *C,
                            const float *D, ssd_dtype in_dtype, int batch,
                            int nheads, int headdim, int dstate, int ngroups,
                            void *y, cudaStream_t stream);

/* ssd_state_update with a dt transform (see ssd_dt_transform; NULL =
 * identity). */
ssd_status ssd_state_update_dt(float *state, const void *x, const float *dt,
                               const float *A, const void *B, const void *C,
                               const float *D, const ssd_dt_transform *dt_transform,
                               ssd_dtype in_dtype, int batch, int nheads,
                               int headdim, int dstate, int ngroups, void *y,
                               cudaStream_t stream);

/* ssd_state_update_dt with the output gate of ssd_scan_fwd_fused and a
 * choice of state storage.
 *   state        [batch][nheads][headdim][dstate] of state_dtype, in place.
 *                SSD_BF16 stores the state as bfloat16 (half the bytes of
 *                the HBM-bound update): each step reads it, updates it in
 *                fp32 and writes it rounded to nearest even; y is computed
 *                from the fp32 update before that rounding.  The pages name
 *                reduced precision as future work (CGLA sections IV and VI)
 *                without fixing a format; this is the plainest one.  bf16
 *                states need in_dtype SSD_BF16 (else SSD_ERR_UNSUPPORTED).
 *   z            in_dtype [batch][nheads][headdim] (y's layout), 16-byte
 *                aligned, or NULL: the output gate y <- y * silu(z). */
ssd_status ssd_state_update_fused(void *state, ssd_dtype state_dtype, const void *x,
                                  const float *dt, const float *A, const void *B,
                                  const void *C, const float *D,
                                  const ssd_dt_transform *dt_transform, const void *z,
                                  ssd_dtype in_dtype, int batch, int nheads, int headdim,
                                  int dstate, int ngroups, void *y, cudaStream_t stream);

/* Decode of `ntokens` consecutive tokens per (batch, head) in one call: the
 * on-device multi-step loop of the O(1) cached decode (compiler-first SSD
 * page, abstract).  Equivalent to ntokens calls of ssd_state_update_fused in
 * token order, except that a bf16 state is rounded once, when it is written
 * back after the last token, not after every token (the state stays fp32 on
 * chip in between).  Each state is read once and written once per call, so
 * its HBM traffic per token falls by ntokens.
 *   state        [batch][nheads][headdim][dstate] of state_dtype, in place.
 *   x, y, z      in_dtype [batch][ntokens][nheads][headdim] (z may be NULL).
 *   dt           float [batch][ntokens][nheads].
 *   B, C         in_dtype [batch][ntokens][ngroups][dstate].
 *   A, D, dt_transform as ssd_state_update_fused.
 * The token arrays have the layouts of ssd_scan_fwd with seqlen = ntokens.
 * Requirements: those of ssd_state_update_fused, ntokens > 0, and headdim at
 * most 512 for dstate 4 to 16, 8192 / dstate for dstate 32 to 128 (256, 128,
 * 64) and 64 for dstate 256, else SSD_ERR_UNSUPPORTED. */
ssd_status ssd_state_update_multi(void *state, ssd_dtype state_dtype, const void *x,
                                  const float *dt, const float *A, const void *B,
                                  const void *C, const float *D,
                                  const ssd_dt_transform *dt_transform, const void *z,
                                  ssd_dtype in_dtype, int batch, int ntokens, int nheads,
                                  int headdim, int dstate, int ngroups, void *y,
                                  cudaStream_t stream);

/* Widens n E4M3 values (the fp8 encoding described at the top) to bfloat16,
 * exactly: the conversion every fp8 prefill call runs on x, B and C, exported
 * for callers that keep fp8 copies of other tensors.  NaN codes give a
 * bfloat16 NaN.  src: n bytes, dst: n bfloat16 values, both device pointers,
 * 16-byte aligned, not overlapping.  n == 0 enqueues nothing.  Returns
 * SSD_ERR_INVALID_ARG for a null or misaligned pointer (n > 0). */
ssd_status ssd_fp8_e4m3_to_bf16(const void *src, void *dst, size_t n, cudaStream_t stream);

/* One long sequence split over GPUs by tokens (GPU r holds a contiguous
 * range of its tokens): the exchange step.  Step-3 of the recurrence at the
 * granularity of a range (CGLA section III.A: the state is carried
 * sequentially, with the input-dependent diagonal decay):
 *     H_in[0] = init,   H_in[r+1] = exp(a_r) H_in[r] + F_r,
 * with a_r the range's log-decay and F_r the state the range reaches from a
 * zero state (its ssd_scan_fwd with init_state = NULL).  Each GPU scans its
 * range from zero for F_r, the pairs (a_r, F_r) are gathered from every GPU,
 * each chains them to its own H_in and scans its range again from H_in for
 * y; the last range's final state is the sequence's.  The pages do not build
 * this split (their runs are on one device); the all-gather is the caller's
 * (torch.distributed in the Python package).
 *
 * ssd_range_log_decay: log_decay[b][h] = A[h] * sum over the range's tokens
 * of dt[b][t][h] (after the dt transform, when one is given, as the scan
 * applies it), summed in double precision.  dt [batch][seqlen][nheads],
 * A [nheads], log_decay [batch][nheads]: float device arrays.
 * SSD_ERR_INVALID_ARG for null pointers, sizes <= 0 or an invalid transform. */
ssd_status ssd_range_log_decay(const float *dt, const float *A,
                               const ssd_dt_transform *dt_transform, int batch, int seqlen,
                               int nheads, float *log_decay, cudaStream_t stream);

/* ssd_chain_states: entering[r] = H_in[r] for r = 0 .. nranges-1 from the
 * ranges' contributions contrib[r] = F_r and log-decays log_decay[r] = a_r,
 * starting from init (zeros when NULL).  contrib, entering
 * [nranges][batch][nheads][headdim][dstate]; log_decay
 * [nranges][batch][nheads]; init [batch][nheads][headdim][dstate]: float
 * device arrays; entering must not overlap the inputs.  SSD_ERR_INVALID_ARG
 * for null required pointers or sizes <= 0. */
ssd_status ssd_chain_states(const float *contrib, const float *log_decay, const float *init,
                            int nranges, int batch, int nheads, int headdim, int dstate,
                            float *entering, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * The steps of a layer around such a recurrence: the root-mean-square norm
 * with the residual's addition, the matrix product with bias, activation and
 * residual in its epilogue, and a gated linear recurrence that is elementwise
 * over the channels.  Each is given forward and backward.  The pages do not
 * build them; the formulas below are their definition.
 *
 * Matrices are row-major with unit-stride columns; an argument `name_stride`
 * is the distance of two rows in elements (at least the row's width), so a
 * column range of a wider matrix can be passed as it lies.  Arrays without a
 * stride argument are contiguous.  Outputs must not overlap inputs unless an
 * entry point says so.  Pointers need the alignment of their element type (4
 * bytes for E4M3 rows read by ssd_linear_fwd); 16-byte aligned pointers and
 * strides take the vector paths.  Sums, statistics, states and gradients in
 * flight are fp32; each output is rounded once.
 *
 * Root-mean-square norm of the residual stream s = x + residual:
 *     s = x + residual            (s = x when residual is NULL)
 *     rstd = (mean_j s_j^2 + eps)^(-1/2)          over the row's `width` values
 *     y_j = s_j rstd weight_j
 * computed from the unrounded s.
 *   x             x_dtype (SSD_F32 or SSD_BF16) [rows][width], x_stride.
 *   residual      stream_dtype [rows][width], residual_stride, or NULL.
 *                 stream_dtype is x_dtype or SSD_F32.
 *   weight        float [width].  eps >= 0.
 *   y             out_dtype [rows][width]: SSD_F32, SSD_BF16, or SSD_FP8_E4M3
 *                 with one scale a row: scale = max_j |y_j| / 448 (1 where that
 *                 is 0 in fp32), y holds y_j / scale, computed in fp32 as
 *                 y_j (1 / scale), rounded to nearest even.
 *   residual_out  stream_dtype [rows][width]: s.  Required with a residual
 *                 (may be the residual itself), ignored without.
 *   rstd          float [rows].  scale: float [rows], required for 8-bit
 *                 outputs, ignored otherwise.
 * rows == 0 enqueues nothing.  SSD_ERR_INVALID_ARG for null pointers, width
 * <= 0, rows < 0, strides below width, eps < 0 or NaN; SSD_ERR_UNSUPPORTED
 * for other types, rows >= 2^31 or width >= 2^24. */
ssd_status ssd_rmsnorm_fwd(const void *x, const void *residual, const float *weight, float eps,
                           ssd_dtype x_dtype, ssd_dtype stream_dtype, ssd_dtype out_dtype,
                           long long rows, int width, long long x_stride,
                           long long residual_stride, void *y, void *residual_out, float *rstd,
                           float *scale, cudaStream_t stream);

/* Gradients of ssd_rmsnorm_fwd.  With e_j = dy_j weight_j:
 *     ds_j = dresidual_j + rstd (e_j - s_j rstd^2 mean_i(e_i s_i))
 *     dweight_j = sum over rows of dy_j s_j rstd
 * ds is the gradient of x and of the residual alike.  An 8-bit output is
 * treated as the unrounded one: dy is the gradient of y.
 *   dy          dtype (SSD_F32 or SSD_BF16) [rows][width], dy_stride.
 *   s           stream_dtype (dtype or SSD_F32) [rows][width], s_stride: the
 *               residual_out of the forward call (or its x).
 *   rstd        float [rows], of the forward call.
 *   dresidual   stream_dtype [rows][width], dresidual_stride: the gradient
 *               that reached residual_out from elsewhere, or NULL.
 *   dx          dtype [rows][width].  ds: stream_dtype [rows][width], or NULL.
 *   dweight     float [width]; the sum's order is fixed for given sizes.
 *   workspace   ssd_rmsnorm_bwd_workspace_bytes() bytes, 16-byte aligned.
 * Errors as ssd_rmsnorm_fwd, and SSD_ERR_WORKSPACE.  rows == 0 writes zeros
 * to dweight. */
ssd_status ssd_rmsnorm_bwd(const void *dy, const void *s, const float *weight, const float *rstd,
                           const void *dresidual, ssd_dtype dtype, ssd_dtype stream_dtype,
                           long long rows, int width, long long dy_stride, long long s_stride,
                           long long dresidual_stride, void *dx, void *ds, float *dweight,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream);
/* Workspace of ssd_rmsnorm_bwd on the current device; (size_t)-1 for invalid sizes. */
size_t ssd_rmsnorm_bwd_workspace_bytes(long long rows, int width);

/* The activation of ssd_linear_fwd: p, p / (1 + e^-p), p (1 + erf(p / sqrt 2)) / 2, max(p, 0). */
typedef enum {
    SSD_ACT_NONE = 0,
    SSD_ACT_SILU = 1,
    SSD_ACT_GELU = 2,
    SSD_ACT_RELU = 3
} ssd_activation;

/* Matrix product with its epilogue:
 *     p[m][n] = (sum_k x[m][k] w[n][k]) x_scale[m] w_scale[n] + bias[n]
 *     y[m][n] = act(p[m][n]) + residual[m][n]
 *   x           in_dtype [tokens][inner], x_stride.
 *   w           in_dtype [features][inner].
 *   x_scale     float [tokens], w_scale float [features]: required for
 *               SSD_FP8_E4M3 (ssd_rmsnorm_fwd writes such rows), NULL otherwise.
 *   bias        float [features] or NULL.
 *   residual    out_dtype [tokens][features], residual_stride, or NULL.
 *   y           out_dtype [tokens][features], y_stride.  out_dtype: SSD_BF16
 *               or SSD_F32 for bf16 and fp8 inputs, SSD_F32 for fp32 inputs.
 *               y may be the residual itself (same pointer and stride).
 *   preact      p, contiguous, SSD_F32 for fp32 inputs and SSD_BF16 otherwise,
 *               or NULL: what ssd_linear_bwd needs of the forward call.
 * bf16 and fp8 inputs whose rows start on 16-byte boundaries run on the
 * tensor cores (products of the inputs as they are, fp32 sums); fp32 inputs
 * and other alignments in fp32 multiply-adds.  tokens == 0 enqueues nothing.
 * SSD_ERR_INVALID_ARG for null pointers, sizes, strides or enums out of range;
 * SSD_ERR_UNSUPPORTED for type combinations not listed and for sizes of 2^31 - 256
 * tokens or 2^22 features or more. */
ssd_status ssd_linear_fwd(const void *x, const float *x_scale, const void *w,
                          const float *w_scale, const float *bias, const void *residual,
                          ssd_activation activation, ssd_dtype in_dtype, ssd_dtype out_dtype,
                          long long tokens, int features, int inner, long long x_stride,
                          long long residual_stride, void *y, long long y_stride, void *preact,
                          cudaStream_t stream);

/* Gradients of ssd_linear_fwd (fp32 or bf16 inputs).  With dp = dy act'(preact):
 *     dx[m][k] = sum_n dp[m][n] w[n][k]
 *     dw[n][k] = sum_m dp[m][n] x[m][k]
 *     dbias[n] = sum_m dp[m][n]
 * (the residual's gradient is dy itself).  dp is rounded to dtype before the
 * two products and not before dbias.
 *   dy          dtype [tokens][features], dy_stride.
 *   preact      dtype [tokens][features], contiguous; NULL with SSD_ACT_NONE.
 *   dx          dtype [tokens][inner], contiguous, or NULL: not wanted.
 *   dw          dtype [features][inner], contiguous, or NULL.
 *   dbias       float [features] or NULL.
 *   workspace   ssd_linear_bwd_workspace_bytes() bytes, 256-byte aligned.
 * tokens == 0 writes zeros to dw and dbias.  Sums run in an order fixed for
 * given sizes.  Errors as ssd_linear_fwd, and SSD_ERR_WORKSPACE; here inner
 * too stays below 2^22. */
ssd_status ssd_linear_bwd(const void *dy, const void *x, const void *w, const void *preact,
                          ssd_activation activation, ssd_dtype dtype, long long tokens,
                          int features, int inner, long long dy_stride, long long x_stride,
                          void *dx, void *dw, float *dbias, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream);
size_t ssd_linear_bwd_workspace_bytes(ssd_dtype dtype, ssd_activation activation,
                                      long long tokens, int features, int inner);

/* The kernel that a product takes on the CURRENT device, whose SM count the choice
 * depends on, when its operands are contiguous and 16-byte aligned. */
typedef enum {
    SSD_PRODUCT_FORWARD = 0,        /* ssd_linear_fwd */
    SSD_PRODUCT_DX = 1,             /* ssd_linear_bwd, dx alone */
    SSD_PRODUCT_DW = 2,             /* dw alone */
    SSD_PRODUCT_GRADIENTS = 3       /* both */
} ssd_product;
typedef enum {
    SSD_PATH_FP32 = 0,              /* fp32 multiply-adds, 64 x 64 tiles */
    SSD_PATH_FP32_FEW = 1,          /* the same for at most 4 tokens */
    SSD_PATH_FEW = 2,               /* warp products, at most 16 tokens */
    SSD_PATH_FEW_SPLIT = 3,         /* tcgen05 with the tokens as columns, k split over a cluster */
    SSD_PATH_WHOLE = 4,             /* tcgen05, 128 x 128 tiles */
    SSD_PATH_PAIRS = 5,             /* 256 x 256 tiles of CTA pairs */
    SSD_PATH_SPLIT = 6,             /* 128 x 128 tiles, k split over a cluster */
    SSD_PATH_SPLIT_PAIRS = 7,       /* 256 x 256 tiles, k split over pairs */
    SSD_PATH_PAIRS_AND_SPLIT = 8,   /* whole rounds of pairs' tiles, those left over split */
    SSD_PATH_TOGETHER = 9,          /* both gradients in one launch of pairs */
    SSD_PATH_APART = 10             /* the gradients one after the other, each on its own path */
} ssd_path;
/* An ssd_path (for launch accounting and tests); -1 for invalid sizes or enums,
 * gradients of 8-bit inputs, or without a device. */
int ssd_linear_path(ssd_product product, ssd_dtype in_dtype, long long tokens, int features,
                    int inner);

/* Gated linear recurrence, elementwise over `width` channels:
 *     f_t = sigmoid(g_t)
 *     h_t = f_t h_{t-1} + (1 - f_t) x_t
 *     y_t = h_t silu(z_t)                  (y_t = h_t when z is NULL)
 * over nseq sequences laid end to end on one axis of `tokens` tokens.
 *   x, g, z, y   dtype (SSD_F32 or SSD_BF16) [tokens][width], each with its
 *                row stride.
 *   length       tokens of each sequence (tokens = nseq * length), when
 *                cu_seqlens_host is NULL.
 *   cu_seqlens_host, cu_seqlens_dev   offsets of sequences of any lengths
 *                (nseq + 1 ints, host and device copies) as in
 *                ssd_scan_fwd_varlen; both or neither.  `length` is then ignored.
 *   init_state   float [nseq][width] or NULL (zeros).
 *   final_state  float [nseq][width] or NULL.  An empty sequence's final state
 *                is its initial one.
 *   checkpoints  float [ceil(tokens / 64)][width] or NULL: the state before
 *                tokens 0, 64, 128, ... of the token axis (a sequence's first
 *                token has its initial state there): what ssd_gated_scan_bwd
 *                needs of the forward call.
 *   workspace    ssd_gated_scan_workspace_bytes() bytes, 256-byte aligned (may
 *                be NULL when that is 0); no initialisation needed.
 * SSD_ERR_INVALID_ARG for null pointers, sizes <= 0 (length 0 is allowed),
 * strides below width or offsets that do not start at 0 or decrease;
 * SSD_ERR_UNSUPPORTED for other types, width >= 2^21, 2^31 - 2048 tokens or
 * more, or tokens * width of about 2^42 or more.  A call of more than 64 tokens
 * joins its parts on the device by waits that are bounded in time; one that
 * runs out is reported by ssd_last_device_error().  In which grouping the parts'
 * fp32 states are joined follows their progress, so two equal calls of more than 64
 * tokens may differ in the last fp32 bits of their results (and so in single bf16
 * values); the same holds for ssd_gated_scan_bwd. */
ssd_status ssd_gated_scan_fwd(const void *x, const void *g, const void *z, ssd_dtype dtype,
                              int nseq, int length, const int *cu_seqlens_host,
                              const int *cu_seqlens_dev, int width, long long x_stride,
                              long long g_stride, long long z_stride, const float *init_state,
                              void *y, long long y_stride, float *final_state,
                              float *checkpoints, void *workspace, size_t workspace_bytes,
                              cudaStream_t stream);
size_t ssd_gated_scan_workspace_bytes(ssd_dtype dtype, long long tokens, int width);

/* Gradients of ssd_gated_scan_fwd.  With dh_t = dy_t silu(z_t), plus dfinal at
 * a sequence's last token, and lam_t = dh_t + f_{t+1} lam_{t+1} inside it:
 *     dx_t = (1 - f_t) lam_t
 *     dg_t = lam_t (h_{t-1} - x_t) f_t (1 - f_t)
 *     dz_t = dy_t h_t silu'(z_t)
 *     dinit = f_0 lam_0                     (dfinal for an empty sequence)
 * x, g, z, init_state, offsets and checkpoints as in (and of) the forward call.
 *   dy, dx, dg, dz   dtype [tokens][width] with row strides; dz is required
 *                    with z and ignored without.
 *   dfinal, dinit    float [nseq][width] or NULL.
 *   workspace        ssd_gated_scan_workspace_bytes() bytes.
 * h is recomputed in fp32 from the checkpoints. */
ssd_status ssd_gated_scan_bwd(const void *dy, const void *x, const void *g, const void *z,
                              ssd_dtype dtype, int nseq, int length, const int *cu_seqlens_host,
                              const int *cu_seqlens_dev, int width, long long dy_stride,
                              long long x_stride, long long g_stride, long long z_stride,
                              const float *init_state, const float *checkpoints,
                              const float *dfinal, void *dx, long long dx_stride, void *dg,
                              long long dg_stride, void *dz, long long dz_stride, float *dinit,
                              void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* One token of the gated recurrence: state float [rows][width], read and
 * updated in place; x, g, z (or NULL) and y dtype [rows][width], x, g and z
 * with row strides.  y may be x, g or z itself when that is contiguous.  rows
 * == 0 enqueues nothing. */
ssd_status ssd_gated_state_update(float *state, const void *x, const void *g, const void *z,
                                  ssd_dtype dtype, long long rows, int width, long long x_stride,
                                  long long g_stride, long long z_stride, void *y,
                                  cudaStream_t stream);

/* Layer norm of the residual stream s = x + residual:
 *     mean = mean_j s_j,   rstd = (mean_j (s_j - mean)^2 + eps)^(-1/2)
 *     y_j = (s_j - mean) rstd weight_j + bias_j
 * computed from the unrounded s.  x, residual, weight, y, residual_out, rstd, scale, types
 * and strides as in ssd_rmsnorm_fwd (an 8-bit row's scale is that of its y); bias float
 * [width] or NULL (zeros); mean float [rows].  A row that holds a NaN or an infinity gives
 * NaN.  Errors as ssd_rmsnorm_fwd. */
ssd_status ssd_layernorm_fwd(const void *x, const void *residual, const float *weight,
                             const float *bias, float eps, ssd_dtype x_dtype,
                             ssd_dtype stream_dtype, ssd_dtype out_dtype, long long rows, int width,
                             long long x_stride, long long residual_stride, void *y,
                             void *residual_out, float *mean, float *rstd, float *scale,
                             cudaStream_t stream);

/* Gradients of ssd_layernorm_fwd.  With v_j = (s_j - mean) rstd and e_j = dy_j weight_j:
 *     ds_j = dresidual_j + rstd (e_j - mean_i(e_i) - v_j mean_i(e_i v_i))
 *     dweight_j = sum over rows of dy_j v_j,   dbias_j = sum over rows of dy_j
 * Arguments as in ssd_rmsnorm_bwd; mean and rstd of the forward call; dbias float [width]
 * or NULL: not wanted; workspace ssd_layernorm_bwd_workspace_bytes() bytes, 16-byte
 * aligned.  The sums' order is fixed for given sizes.  rows == 0 writes zeros to dweight
 * and dbias. */
ssd_status ssd_layernorm_bwd(const void *dy, const void *s, const float *weight, const float *mean,
                             const float *rstd, const void *dresidual, ssd_dtype dtype,
                             ssd_dtype stream_dtype, long long rows, int width, long long dy_stride,
                             long long s_stride, long long dresidual_stride, void *dx, void *ds,
                             float *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                             cudaStream_t stream);
/* Workspace of ssd_layernorm_bwd on the current device; (size_t)-1 for invalid sizes. */
size_t ssd_layernorm_bwd_workspace_bytes(long long rows, int width);

/* Embedding: rows of a table by tokens,
 *     y[t][j] = table[tokens[t]][j] scale
 *   tokens   SSD_I32 or SSD_I64 [count].  A token below 0 or not below vocab stands for
 *            padding: its row of y is zeros, and it has no part in the gradient.
 *   table    table_dtype (SSD_F32 or SSD_BF16) [vocab][width], contiguous.
 *   y        out_dtype (SSD_F32 or SSD_BF16) [count][width]; each value is rounded once.
 * count == 0 enqueues nothing.  SSD_ERR_INVALID_ARG for null or misaligned pointers, sizes
 * out of range, a scale that is not finite; SSD_ERR_UNSUPPORTED for other types, 2^31 - 2048
 * tokens, 2^30 rows of the table or 2^24 columns or more. */
typedef enum { SSD_I32 = 0, SSD_I64 = 1 } ssd_index;
ssd_status ssd_embedding_fwd(const void *tokens, ssd_index token_type, const void *table,
                             ssd_dtype table_dtype, ssd_dtype out_dtype, long long count, int vocab,
                             int width, float scale, void *y, cudaStream_t stream);

/* The table's gradient, dense:
 *     dtable[v][j] = scale * sum over the t with tokens[t] = v of dy[t][j]
 *   dy       dtype (SSD_F32 or SSD_BF16) [count][width], dy_stride.
 *   dtable   out_dtype (SSD_F32 or SSD_BF16) [vocab][width]: every row is written, rows
 *            without a token as zeros.  Sums are fp32 and rounded once.
 *   workspace  ssd_embedding_bwd_workspace_bytes() bytes, 256-byte aligned.
 * The tokens are sorted on the device and each row's sum runs in an order fixed for given
 * tokens, so equal calls give equal bits.  count == 0 writes zeros.  Errors as
 * ssd_embedding_fwd, and SSD_ERR_WORKSPACE. */
ssd_status ssd_embedding_bwd(const void *dy, const void *tokens, ssd_index token_type,
                             ssd_dtype dtype, ssd_dtype out_dtype, long long count, int vocab,
                             int width, long long dy_stride, float scale, void *dtable,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream);
/* (size_t)-1 for invalid sizes. */
size_t ssd_embedding_bwd_workspace_bytes(long long count, int vocab, int width);

/* Gated delta rule: a linear recurrence whose state is corrected towards each token's value,
 * for every head with its state S [headdim][dstate]:
 *     S' = exp(g_t) S_{t-1}
 *     u_t = beta_t (v_t - S' k_t)
 *     S_t = S' + u_t k_t^T
 *     o_t = scale S_t q_t
 * over nseq sequences laid end to end on one axis of `tokens` tokens (length, or
 * cu_seqlens_host and cu_seqlens_dev, as in ssd_gated_scan_fwd).
 *   q, k         dtype (SSD_F32 or SSD_BF16) [tokens][ngroups][dstate]; head h uses group
 *                h / (nheads / ngroups).  q_stride and k_stride: distance of two tokens.
 *   v, o         dtype [tokens][nheads][headdim], with v_stride and o_stride.
 *   g            float [tokens][nheads]: the logarithm of the decay (<= 0 in use; -infinity
 *                forgets the state, values below -200 count as that).
 *   beta         float [tokens][nheads]: how much of the value is written (0 to 1 in use,
 *                with keys of unit length).
 *   init_state, final_state   float [nseq][nheads][headdim][dstate] or NULL (zeros / not
 *                wanted); they may be the same array.  An empty sequence's final state is its
 *                initial one.
 *   checkpoints  float [tokens / 64 + nseq][nheads][headdim][dstate] or NULL: what
 *                ssd_delta_scan_bwd needs of the forward call.  The state before a sequence's
 *                tokens 0, 64, 128, ... lies at first / 64 + s + 0, 1, 2, ... (s: the
 *                sequence, first: its first token on the axis); other places are not written.
 *   workspace    ssd_delta_scan_workspace_bytes() bytes, 256-byte aligned (may be NULL
 *                when that is 0); no initialisation needed.
 * bf16 inputs with dstate <= 128, dstate and headdim multiples of 8, and tokens and states that
 * start on 16-byte boundaries run on the tensor cores, in chunks of 64 tokens, with factors that are
 * no bf16 values held to 16 bits (final states, checkpoints and the fp32 gradients are 3e-6 to
 * 6e-6 of their size off); others in fp32 multiply-adds, token by token (1e-7), which
 * ssd_delta_scan_fwd_algo asks for whatever the sizes.  On the tensor cores a long sequence of few heads goes in
 * parts side by side, whose number follows from the sizes and the device's SMs.  Equal calls
 * give equal bits.  A token's NaN or infinity reaches what the formula says, and on the tensor
 * cores also outputs of earlier tokens of its chunk (of a sequence's tokens 64 c to 64 c + 63);
 * nothing of earlier chunks, of other sequences, or of heads that do not read it.
 * Requirements: dstate <= 256, headdim <= 2^14, nheads <= 2^16 a multiple of ngroups.
 * SSD_ERR_INVALID_ARG for null or misaligned pointers, sizes <= 0 (length 0 is allowed),
 * strides below a token's values, bad offsets or a scale that is not finite;
 * SSD_ERR_UNSUPPORTED for other types and sizes beyond those, or beyond a grid (2^31
 * runs of 64 tokens by heads by 32 rows); SSD_ERR_WORKSPACE.  The tensor-core kernels' waits
 * are bounded in time; one that runs out is reported by ssd_last_device_error(). */
ssd_status ssd_delta_scan_fwd(const void *q, const void *k, const void *v, const float *g,
                              const float *beta, ssd_dtype dtype, int nseq, int length,
                              const int *cu_seqlens_host, const int *cu_seqlens_dev, int nheads,
                              int headdim, int dstate, int ngroups, long long q_stride,
                              long long k_stride, long long v_stride, float scale,
                              const float *init_state, void *o, long long o_stride,
                              float *final_state, float *checkpoints, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream);
/* 0 where the call needs none; (size_t)-1 for invalid sizes. */
size_t ssd_delta_scan_workspace_bytes(ssd_dtype dtype, long long tokens, int nseq, int nheads,
                                      int headdim, int dstate, int ngroups);

/* Same as ssd_delta_scan_fwd with an explicit kernel choice: SSD_ALGO_SIMT takes the fp32
 * multiply-adds for every size and alignment (no workspace); SSD_ALGO_TCGEN05 returns
 * SSD_ERR_UNSUPPORTED for types, sizes and alignments that the tensor-core kernels do not
 * take (0 as the workspace of such sizes). */
ssd_status ssd_delta_scan_fwd_algo(ssd_algo algo, const void *q, const void *k, const void *v,
                                   const float *g, const float *beta, ssd_dtype dtype, int nseq,
                                   int length, const int *cu_seqlens_host, const int *cu_seqlens_dev,
                                   int nheads, int headdim, int dstate, int ngroups, long long q_stride,
                                   long long k_stride, long long v_stride, float scale,
                                   const float *init_state, void *o, long long o_stride,
                                   float *final_state, float *checkpoints, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream);
size_t ssd_delta_scan_workspace_bytes_algo(ssd_algo algo, ssd_dtype dtype, long long tokens, int nseq,
                                           int nheads, int headdim, int dstate, int ngroups);

/* Gradients of ssd_delta_scan_fwd.  With L_t the gradient of S_t, which begins with dfinal
 * behind a sequence's last token:
 *     L_t += scale do_t q_t^T,   w_t = L_t k_t,   dv_t = beta_t w_t
 *     L' = L_t - dv_t k_t^T,     L_{t-1} = exp(g_t) L'        (dinit: before the first token)
 *     dbeta_t = w_t (v_t - S' k_t),   dg_t = <L', S'>
 *     dq_t = scale S_t^T do_t,   dk_t = L_t^T u_t - S'^T dv_t     (summed over a group's heads)
 *   dout         dtype [tokens][nheads][headdim], do_stride: the gradient of o.
 *   q, k, v, g, beta, scale and sequences as given to the forward call; checkpoints: what
 *                it left.
 *   dfinal, dinit   float [nseq][nheads][headdim][dstate] or NULL (zeros / not wanted).
 *   dq, dk, dv   dtype, laid out as q, k and v, with their own token strides.
 *   dg, dbeta    float [tokens][nheads].
 *   workspace    ssd_delta_scan_bwd_workspace_bytes() bytes, 256-byte aligned: enough for
 *                either kind of kernels, since those that run follow from the addresses too.
 *                A call needs what ssd_delta_scan_bwd_workspace_bytes_algo() says of the kind
 *                that it takes: on the tensor cores about 34 KB + 32 KB + 512 bytes a column of
 *                the state (dstate <= 64: of 64, else of 128) for every 64 tokens of a head, and
 *                8 dstate bytes a token and head where heads share keys; in fp32
 *                multiply-adds 8 (headdim + dstate * ceil(headdim / 64)) bytes a token and head
 *                (by 32 rows where headdim <= 32 or dstate > 128).
 * Sums are fp32 in an order fixed for given sizes and the device's SMs; each result is
 * rounded once.  dg is had as sums over a token's 64, of terms as large as dout_t . o_t and
 * dv_t . v_t: its error goes by their size (fp32 multiply-adds: 1e-7 of it), also where a strong
 * decay leaves dg itself much smaller.  bf16 inputs as for ssd_delta_scan_fwd with
 * headdim <= 128 run on the tensor cores, others in fp32 multiply-adds.  A NaN or an infinity of dout reaches all gradients
 * of its token's 64 (as above) and what the formula says in front of them.  dq, dk and dv
 * overlap none of the inputs. */
ssd_status ssd_delta_scan_bwd(const void *dout, const void *q, const void *k, const void *v,
                              const float *g, const float *beta, ssd_dtype dtype, int nseq,
                              int length, const int *cu_seqlens_host, const int *cu_seqlens_dev,
                              int nheads, int headdim, int dstate, int ngroups, long long do_stride,
                              long long q_stride, long long k_stride, long long v_stride, float scale,
                              const float *checkpoints, const float *dfinal, void *dq,
                              long long dq_stride, void *dk, long long dk_stride, void *dv,
                              long long dv_stride, float *dg, float *dbeta, float *dinit,
                              void *workspace, size_t workspace_bytes, cudaStream_t stream);
/* (size_t)-1 for invalid sizes. */
size_t ssd_delta_scan_bwd_workspace_bytes(ssd_dtype dtype, long long tokens, int nseq, int nheads,
                                          int headdim, int dstate, int ngroups);

/* Same as ssd_delta_scan_bwd with an explicit kernel choice, as ssd_delta_scan_fwd_algo; the
 * checkpoints may be of either choice. */
ssd_status ssd_delta_scan_bwd_algo(ssd_algo algo, const void *dout, const void *q, const void *k,
                                   const void *v, const float *g, const float *beta, ssd_dtype dtype,
                                   int nseq, int length, const int *cu_seqlens_host,
                                   const int *cu_seqlens_dev, int nheads, int headdim, int dstate,
                                   int ngroups, long long do_stride, long long q_stride,
                                   long long k_stride, long long v_stride, float scale,
                                   const float *checkpoints, const float *dfinal, void *dq,
                                   long long dq_stride, void *dk, long long dk_stride, void *dv,
                                   long long dv_stride, float *dg, float *dbeta, float *dinit,
                                   void *workspace, size_t workspace_bytes, cudaStream_t stream);
size_t ssd_delta_scan_bwd_workspace_bytes_algo(ssd_algo algo, ssd_dtype dtype, long long tokens,
                                               int nseq, int nheads, int headdim, int dstate,
                                               int ngroups);

/* One token of the delta rule: state [batch][nheads][headdim][dstate] of state_dtype (SSD_F32,
 * or SSD_BF16 with bf16 inputs, rounded once) gives state_out, which may be the state itself;
 * q, k [batch][ngroups][dstate], v [batch][nheads][headdim] of dtype with strides of a batch
 * row; g, beta float [batch][nheads]; o dtype [batch][nheads][headdim].  batch == 0 enqueues
 * nothing.  Requirements and errors as ssd_delta_scan_fwd. */
ssd_status ssd_delta_state_update(const void *state, ssd_dtype state_dtype, void *state_out,
                                  const void *q, const void *k, const void *v, const float *g,
                                  const float *beta, ssd_dtype dtype, int batch, int nheads,
                                  int headdim, int dstate, int ngroups, long long q_stride,
                                  long long k_stride, long long v_stride, float scale, void *o,
                                  cudaStream_t stream);

/* Human-readable name of a status code (static storage). */
const char *ssd_status_string(ssd_status s);

/* Reads and clears the device error word on the current device
 * (synchronises the device).  SSD_OK when no kernel reported a fault. */
ssd_status ssd_last_device_error(void);

/* Test hook for the bounded device-side waits (the pages have no
 * counterpart).  Every later launch of the tensor-core scan, of the gated
 * recurrence, of the tensor-core product, of the tensor-core delta rule and of
 * the layer norm of many rows to 8 bits reads the setting; it is process-wide
 * and not synchronised with calls in flight on other host threads.
 *   fault          SSD_FAULT_NONE: normal operation.  SSD_FAULT_WITHHOLD_SIGNAL:
 *                  in the CTAs of each sequence's first segment, the barrier
 *                  that signals "decay factors ready" waits for one arrival
 *                  more than the warp computing them gives, so the first wait
 *                  for it runs out; the CTA then lets its issued copies and
 *                  tensor-core products complete, frees its tensor memory and
 *                  exits, and the device error word reads SSD_ERR_TIMEOUT.
 *                  The outputs of that call are undefined.
 *                  In ssd_gated_scan_fwd / _bwd calls of more than one tile the
 *                  first tile of the walk publishes nothing, so the tiles behind
 *                  it give up after wait_limit_ns each, with the same report.
 *                  In the tensor-core product the first CTA's (or pair of CTAs')
 *                  first accumulator is never announced, with the same end.  In
 *                  the layer norm of many rows the first row's copy is never
 *                  complete: its warp gives up, waits once more and ends.
 *   wait_limit_ns  limit of every bounded wait in those kernels but those for a
 *                  CTA's own copies and products in flight, at its end or where
 *                  nothing else is waited for (always the default); 0 restores
 *                  the default (2 s).
 * Returns SSD_ERR_INVALID_ARG for an unknown fault. */
typedef enum { SSD_FAULT_NONE = 0, SSD_FAULT_WITHHOLD_SIGNAL = 1 } ssd_fault;
ssd_status ssd_debug_inject_fault(ssd_fault fault, unsigned long long wait_limit_ns);

#ifdef __cplusplus
}
#endif

#endif /* SSD_GB300_H */
