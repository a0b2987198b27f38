// Gated delta rule on the tensor cores (bf16 inputs, up to 128 state columns), by chunks of
// 64 tokens.  With G_i the sum of g over the chunk's tokens up to i, and S the state before
// the chunk, the corrections u_i of all its tokens solve one triangular system:
//
//   A_ij = beta_i exp(G_i - G_j) k_i . k_j   (j < i),      T = (1 + A)^-1
//   R = V - diag(exp G) K S^T,                             U = T diag(beta) R
//   P_ij = scale exp(G_i - G_j) q_i . k_j    (j <= i)
//   O = scale diag(exp G) Q S^T + P U
//   S <- exp(G_end) S + U^T diag(exp(G_end - G)) K
//
// Two kernels.  The first makes T diag(beta) and P of every chunk, all of them side by
// side.  The second walks a sequence's chunks, one CTA a head and 128 rows of its state,
// with the state's rows as the tensor core's lanes: S, R and U are transposed products'
// left operands in tensor memory, so what one product leaves in a thread's lane is
// scaled, rounded and put back as the next one's operand without leaving the lane.
//
// K, Q and V are bf16 values as they are.  T, P, S, R and U are held in two bf16 parts
// (16 bits), the product of two second parts left out: with one part the state, which is
// handed on in fp32, would be off by 3e-3 of itself, with two it is by 7e-6.
#include <mutex>

#include "delta_tc.cuh"
#include "vec.cuh"

namespace {

using namespace ssddelta;

// ------------------------------------------------------------- chunk matrices
// One CTA a chunk and key group, all of the group's heads after each other.  The 64 queries
// over the 64 keys, times the keys, are one product of M = 128, N = 64: a thread's lane is
// then a row of Q K^T (threads 0 .. 63) or of K K^T (64 .. 127).  The triangle is inverted
// in fp32: blocks of 16 by substitution, a thread a column, then twice
//     (T11  0; T21  T22),   T21 = -T22 (A21 T11)
// for blocks of 32 and of 64 (substituting all 64 rows in one thread took five times as
// long: 2016 dependent steps, and more code than the instruction cache holds).
constexpr int kPrepThreads = 128;
constexpr int kTw = 36;         // floats a row of a 32 x 32 block
struct PrepSmem {
    // at 0: Q over K by panels, then the images
    static constexpr uint32_t kA = 4 * kPanel;              // A's columns, fp32 (W above the diagonal)
    static constexpr uint32_t kRows = kA + kC * kC * 4;     // T11 and T22 by rows
    static constexpr uint32_t kCols = kRows + 2 * 32 * kTw * 4;     // and by columns
    static constexpr uint32_t kSums = kCols + 2 * 32 * kTw * 4;     // G in two floats, beta, decay to token 31
    static constexpr uint32_t kBars = kSums + 4 * kC * 4;
    static constexpr uint32_t kBytes = kBars + 64;
};

struct Prep {
    SsdDelta d;
    uint8_t *records;
    unsigned *err;
};

// a + b of numbers in two floats each, the second one what the first does not hold.
__device__ __forceinline__ float2 add_two(float2 a, float2 b) {
    const float s = a.x + b.x, v = s - a.x;
    const float e = (a.x - (s - v)) + (b.x - v) + a.y + b.y;
    const float hi = s + e;
    return make_float2(hi, e - (hi - s));
}

// (1 + A)^-1 of `columns` (A[r][c] at 64 c + r), all 128 threads: its diagonal blocks of 32
// to `rows` and `cols`, and rows 32 + r0, + 1 by columns c0 .. c0 + 3 of the block below.
__device__ __forceinline__ void invert(float *columns, float *rows, float *cols, int r0, int c0, float (&below)[2][4]) {
    const int t = threadIdx.x;
    if (t < 64) {       // blocks of 16
        const int b = t >> 4, c = t & 15;
        float acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
        float *const row = rows + (b >> 1) * 32 * kTw, *const col = cols + (b >> 1) * 32 * kTw;
        const int off = (b & 1) * 16;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float x = i == c ? 1.f : -acc[i];
            const float4 *a = reinterpret_cast<const float4 *>(columns + (16 * b + i) * kC + 16 * b);
#pragma unroll
            for (int v = (i + 1) / 4; v < 4; ++v) {
                const float4 y = a[v];
                if (4 * v > i) acc[4 * v] += y.x * x;
                if (4 * v + 1 > i) acc[4 * v + 1] += y.y * x;
                if (4 * v + 2 > i) acc[4 * v + 2] += y.z * x;
                acc[4 * v + 3] += y.w * x;
            }
            row[(off + i) * kTw + off + c] = x;
            col[(off + c) * kTw + off + i] = x;
        }
    } else {            // above them nothing
        for (int i = t - 64; i < 2 * 256; i += 64) {
            const int b = i >> 8, r = (i >> 4) & 15, c = i & 15;
            rows[b * 32 * kTw + r * kTw + 16 + c] = 0.f;
            cols[b * 32 * kTw + (16 + c) * kTw + r] = 0.f;
        }
    }
    __syncthreads();
    {                   // blocks of 32: 64 threads each, a row's four columns
        const int b = t >> 6, r = (t >> 2) & 15, c = (t & 3) * 4;
        float *const row = rows + b * 32 * kTw, *const col = cols + b * 32 * kTw;
        float *const w = columns + (32 + r) * kC + 16 * b;      // a row of W
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float a = columns[(32 * b + k) * kC + 32 * b + 16 + r];
            const float4 y = *reinterpret_cast<const float4 *>(row + k * kTw + c);
            x.x += a * y.x;
            x.y += a * y.y;
            x.z += a * y.z;
            x.w += a * y.w;
        }
        *reinterpret_cast<float4 *>(w + c) = x;
        __syncthreads();
        float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float a = -row[(16 + r) * kTw + 16 + k];
            const float4 y = *reinterpret_cast<const float4 *>(columns + (32 + k) * kC + 16 * b + c);
            z.x += a * y.x;
            z.y += a * y.y;
            z.z += a * y.z;
            z.w += a * y.w;
        }
        *reinterpret_cast<float4 *>(row + (16 + r) * kTw + c) = z;
        col[c * kTw + 16 + r] = z.x;
        col[(c + 1) * kTw + 16 + r] = z.y;
        col[(c + 2) * kTw + 16 + r] = z.z;
        col[(c + 3) * kTw + 16 + r] = z.w;
    }
    __syncthreads();
    // the block of 32 below: two rows by four columns a thread
    float w[2][4] = {};
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
        const float2 a = *reinterpret_cast<const float2 *>(columns + k * kC + 32 + r0);
        const float4 y = *reinterpret_cast<const float4 *>(rows + k * kTw + c0);
        w[0][0] += a.x * y.x, w[0][1] += a.x * y.y, w[0][2] += a.x * y.z, w[0][3] += a.x * y.w;
        w[1][0] += a.y * y.x, w[1][1] += a.y * y.y, w[1][2] += a.y * y.z, w[1][3] += a.y * y.w;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
        *reinterpret_cast<float4 *>(columns + (32 + r0 + j) * kC + c0) = make_float4(w[j][0], w[j][1], w[j][2], w[j][3]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) below[j][i] = 0.f;
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
        const float2 a = *reinterpret_cast<const float2 *>(cols + (32 + k) * kTw + r0);
        const float4 y = *reinterpret_cast<const float4 *>(columns + (32 + k) * kC + c0);
        below[0][0] -= a.x * y.x, below[0][1] -= a.x * y.y, below[0][2] -= a.x * y.z, below[0][3] -= a.x * y.w;
        below[1][0] -= a.y * y.x, below[1][1] -= a.y * y.y, below[1][2] -= a.y * y.z, below[1][3] -= a.y * y.w;
    }
}

// Eight values of a row as the two parts' vectors in the images at `to`.
__device__ __forceinline__ void put_parts(uint8_t *image, uint32_t at, const float *v) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Split s = split2(v[2 * i], v[2 * i + 1]);
        hi[i] = s.hi;
        lo[i] = s.lo;
    }
    *reinterpret_cast<uint4 *>(image + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(image + kPanel + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

template <int kPanels>
__global__ void __launch_bounds__(kPrepThreads)
delta_chunk_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK, const Prep a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const SsdDelta &d = a.d;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) {
        if (threadIdx.x == 0) ssd_report(a.err, SSD_DEVERR_SMEM_ALIGN);
        return;
    }
    const long long slot = blockIdx.x / d.groups;
    const int group = (int)(blockIdx.x % d.groups);
    const ChunkAt at = chunk_at(d, slot);
    if (!at.live) return;
    const int valid = min(kC, at.len - at.chunk * kC);
    const long long token = at.first + (long long)at.chunk * kC;
    const uint32_t full = base + PrepSmem::kBars, done = full + 8;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + PrepSmem::kBars + 16);
    if (threadIdx.x == 0) {
        mbar_init(full, 1);
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tslot), 64);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    if (threadIdx.x == 0) {
        mbar_arrive_expect_tx(full, kPanels * 2 * kPanel);
#pragma unroll
        for (int p = 0; p < kPanels; ++p) {
            tma_load_3d(base + p * 2 * kPanel, &mapQ, full, 64 * p, group, (int)token);
            tma_load_3d(base + p * 2 * kPanel + kPanel, &mapK, full, 64 * p, group, (int)token);
        }
    }
    // (waits for the CTA's own copies and product)
    if (!mbar_wait(full, 0, kSsdDefaultWaitNs)) ssd_report(a.err, SSD_DEVERR_TIMEOUT);
    if (warp == 1 && elect_one()) {
        constexpr uint32_t kId = idesc_bf16_f32(128, 64, false, false);
#pragma unroll
        for (int p = 0; p < kPanels; ++p) {
            const uint64_t ad = smem_desc(base + p * 2 * kPanel, 16, 1024, kSwizzle128B);
            const uint64_t bd = smem_desc(base + p * 2 * kPanel + kPanel, 16, 1024, kSwizzle128B);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ss(tmem, ad + 2 * k, bd + 2 * k, kId, p + k > 0);
        }
        mma_commit(done);
    }
    __syncwarp();
    if (!mbar_wait(done, 0, kSsdDefaultWaitNs)) ssd_report(a.err, SSD_DEVERR_TIMEOUT);
    tc_fence_after();
    float *const sum_hi = reinterpret_cast<float *>(smem + PrepSmem::kSums), *const sum_lo = sum_hi + kC;
    float *const betas = sum_lo + kC, *const to_half = betas + kC;
    float *const columns = reinterpret_cast<float *>(smem + PrepSmem::kA);
    float *const rows = reinterpret_cast<float *>(smem + PrepSmem::kRows);
    float *const cols = reinterpret_cast<float *>(smem + PrepSmem::kCols);
    const int wide = d.heads / d.groups, row = threadIdx.x & 63;
    const bool keys = warp >= 2;
    for (int h = 0; h < wide; ++h) {
        const int head = group * wide + h;
        uint8_t *const record = a.records + ((size_t)slot * d.heads + head) * kRecord;
        // sums of g in two floats: a later token's decay is the difference of two of them,
        // which an early strong decay must not round away
        if (warp < 2) {
            const bool on = row < valid;
            const size_t i = (size_t)(token + row) * d.heads + head;
            float g = on ? d.g[i] : 0.f;
            g = g < -200.f ? -200.f : g;
            float2 s = make_float2(g, 0.f);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float2 n = make_float2(__shfl_up_sync(0xffffffffu, s.x, o), __shfl_up_sync(0xffffffffu, s.y, o));
                if (lane >= o) s = add_two(n, s);
            }
            sum_hi[row] = s.x;
            sum_lo[row] = s.y;
            betas[row] = on ? d.beta[i] : 0.f;
        }
        // the images of the head in front have been read, its blocks used
        if (threadIdx.x == 0 && h > 0) bulk_wait_read<0>();
        __syncthreads();
        const float2 half = make_float2(sum_hi[31], sum_lo[31]);
        float2 mine = make_float2(sum_hi[row], sum_lo[row]);
        if (row >= 32) mine = add_two(half, mine);
        const float2 end = add_two(half, make_float2(sum_hi[63], sum_lo[63]));
        // over the middle, decays are products: of the row's from it and the column's to it
        const float from_half = row < 32 ? 0.f : __expf((mine.x - half.x) + (mine.y - half.y));
        __syncthreads();
        if (threadIdx.x < kC) {
            float *gates = reinterpret_cast<float *>(record + kRecGates);
            gates[row] = __expf(mine.x + mine.y);
            gates[kC + row] = __expf((end.x - mine.x) + (end.y - mine.y));
            if (row < 32) {
                to_half[row] = __expf((half.x - mine.x) + (half.y - mine.y));
            } else {
                sum_hi[row] = mine.x;
                sum_lo[row] = mine.y;
            }
        }
        __syncthreads();
        const float factor = keys ? betas[row] : d.scale;
#pragma unroll 1
        for (int c0 = 0; c0 < kC; c0 += 16) {
            float v[16];
            if (c0 > 16 && row < 32) {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = 0.f;
            } else {
                uint32_t r[16];
                tmem_ld16(tmem + ((uint32_t)(warp * 32) << 16) + c0, r);
                const bool over = c0 < 32 && row >= 32;
                float e[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    e[j] = over ? from_half * to_half[c0 + j]
                                : __expf((mine.x - sum_hi[c0 + j]) + (mine.y - sum_lo[c0 + j]));
                tmem_ld_wait(r);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const bool in = row < valid && (keys ? c0 + j < row : c0 + j <= row);
                    v[j] = in ? factor * e[j] * __uint_as_float(r[j]) : 0.f;
                }
            }
            if (keys) {
                // (above the diagonal block the array is another's)
                if (c0 < 32 || row >= 32) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) columns[(c0 + j) * kC + row] = v[j];
                }
            } else {
                put_parts(smem + kRecP, panel_at(row, c0), v);
                put_parts(smem + kRecP, panel_at(row, c0 + 8), v + 8);
            }
        }
        __syncthreads();
        const int r0 = (threadIdx.x >> 3) * 2, c0 = (threadIdx.x & 7) * 4;
        float below[2][4];
        invert(columns, rows, cols, r0, c0, below);
        // T diag(beta)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const Split x = split2(below[j][0] * betas[c0], below[j][1] * betas[c0 + 1]);
            const Split y = split2(below[j][2] * betas[c0 + 2], below[j][3] * betas[c0 + 3]);
            const uint32_t to = kRecT + panel_at(32 + r0 + j, c0);
            *reinterpret_cast<uint2 *>(smem + to) = make_uint2(x.hi, y.hi);
            *reinterpret_cast<uint2 *>(smem + kPanel + to) = make_uint2(x.lo, y.lo);
        }
        for (int i = threadIdx.x; i < 64 * 4; i += kPrepThreads) {
            const int r = i >> 2, c = (i & 3) * 8, b = r >> 5;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = rows[(b * 32 + (r & 31)) * kTw + c + j] * betas[32 * b + c + j];
            put_parts(smem + kRecT, panel_at(r, 32 * b + c), v);
        }
        {
            const uint32_t to = kRecT + panel_at(threadIdx.x >> 2, 32 + (threadIdx.x & 3) * 8);
            *reinterpret_cast<uint4 *>(smem + to) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(smem + kPanel + to) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (threadIdx.x == 0) {
            bulk_store(record, base, 4 * kPanel);
            bulk_commit();
        }
    }
    if (threadIdx.x == 0) bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 64);
}

// ------------------------------------------------------------------ the walk
// Tensor memory, 512 columns: the state in fp32 and in two bf16 parts; what a product
// leaves for the next step (K S^T, then U); the output's two products after each other;
// R, then U, in two parts; U weighted by the decay to the chunk's end, in two parts.
constexpr uint32_t kColS = 0, kColSh = 128, kColSl = 192, kColX = 256, kColO = 320, kColR = 384, kColRl = 416,
                   kColW = 448, kColWl = 480;
// 16 warps on the chain, 8 on the output, one for the copies, one for the products
constexpr int kChainWarps = 16, kOutWarps = 8;
constexpr int kLoadWarp = kChainWarps + kOutWarps, kMmaWarp = kLoadWarp + 1, kWalkThreads = 32 * (kMmaWarp + 1);

template <int kPanels>
struct WalkSmem {
    static constexpr uint32_t kK = 0, kQ = kPanels * kPanel, kRec = 2 * kPanels * kPanel;
    static constexpr uint32_t kV = kRec + kRecord;      // [token][128], as they lie
    static constexpr uint32_t kStage = (kV + 64 * 256 + 1023) / 1024 * 1024;
    static constexpr uint32_t kO = 2 * kStage;          // [token][128]: the output on its way
    static constexpr uint32_t kCtl = kO + 64 * 256;
    static constexpr uint32_t kBytes = kCtl + 256;
};

struct WalkTc {
    SsdDelta d;
    const uint8_t *records;
    const float *init;
    __nv_bfloat16 *o;
    long long o_stride;
    float *final_state, *checkpoints;
    int blocks;                 // of 128 rows a head
    bool o_vectors;             // whether the output's rows start on 16 bytes
    unsigned *err;
    unsigned long long wait_ns;
    bool withhold;
};

enum WalkBar {
    kFull = 0, kEmpty = 2,      // two stages each
    kKs = 4, kU, kS, kQs, kPu, kDrain,              // products done
    kSh, kSl, kRh, kRl, kWh, kWl,                   // operands' parts written by the chain
    kUReady, kQsRead, kPuRead,                      // and by the output's warps, or read
    kBars
};

template <int kPanels>
__global__ void __launch_bounds__(kWalkThreads, 1)
delta_walk_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                     const __grid_constant__ CUtensorMap mapV, const WalkTc a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using Lay = WalkSmem<kPanels>;
    constexpr int kN = 64 * kPanels;
    const SsdDelta &d = a.d;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) {
        if (threadIdx.x == 0) ssd_report(a.err, SSD_DEVERR_SMEM_ALIGN);
        return;
    }
    const int head = (int)(blockIdx.x % d.heads), block = (int)(blockIdx.x / d.heads % a.blocks);
    const int seq = (int)(blockIdx.x / d.heads / a.blocks), group = head / (d.heads / d.groups);
    const long long first = d.cu ? d.cu[seq] : (long long)seq * d.length;
    const int len = d.cu ? d.cu[seq + 1] - d.cu[seq] : d.length;
    const int chunks = (len + kC - 1) / kC, p0 = block * 128;
    const size_t state = ((size_t)seq * d.heads + head) * d.p * d.n;
    if (chunks == 0) {
        if (a.final_state)
            for (long long i = threadIdx.x; i < (long long)min(128, d.p - p0) * d.n; i += kWalkThreads)
                a.final_state[state + (size_t)p0 * d.n + i] = a.init ? a.init[state + (size_t)p0 * d.n + i] : 0.f;
        return;
    }
    const auto bar = [&](int i) { return base + Lay::kCtl + 8u * (uint32_t)i; };
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + Lay::kCtl + 8 * kBars);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + Lay::kCtl + 8 * kBars + 4);
    const Waiter wait{abort, a.err, a.wait_ns};
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(kFull + s), 1);
            mbar_init(bar(kEmpty + s), 1 + kChainWarps + kOutWarps);
        }
        for (int i : {kKs, kU, kS, kQs, kPu, kDrain}) mbar_init(bar(i), 1);
        for (int i : {kSh, kSl, kRh, kRl, kWh, kWl}) mbar_init(bar(i), kChainWarps);
        for (int i : {kQsRead, kUReady, kPuRead}) mbar_init(bar(i), kOutWarps);
        fence_mbar_init();
        *abort = 0;
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tslot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const long long slot0 = ssd_delta_slot(first, seq, 0);
    int loaded = 0;

    if (warp == kLoadWarp) {
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            if (c >= 2 && !wait.warp(bar(kEmpty + s), ((c >> 1) - 1) & 1)) break;
            if (elect_one()) {
                const uint32_t to = base + s * Lay::kStage;
                const int token = (int)(first + (long long)c * kC);
                mbar_arrive_expect_tx(bar(kFull + s), 2 * kPanels * kPanel + kRecord + 64 * 256);
#pragma unroll
                for (int p = 0; p < kPanels; ++p) {
                    tma_load_3d(to + Lay::kK + p * kPanel, &mapK, bar(kFull + s), 64 * p, group, token);
                    tma_load_3d(to + Lay::kQ + p * kPanel, &mapQ, bar(kFull + s), 64 * p, group, token);
                }
                bulk_load(to + Lay::kRec, a.records + ((size_t)(slot0 + c) * d.heads + head) * kRecord, kRecord,
                          bar(kFull + s));
                tma_load_3d(to + Lay::kV, &mapV, bar(kFull + s), p0, head, token);
            }
            __syncwarp();
            loaded = c + 1;
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t kId64 = idesc_bf16_f32(128, 64, false, false);
        constexpr uint32_t kIdS = idesc_bf16_f32(128, kN, false, true);
        const bool one = elect_one();
        // D (+)= A rows' K part . B^T over a panel pair's columns, one part of A
        const auto over_n = [&](uint32_t dcol, uint32_t acol, uint32_t tile, bool add) {
#pragma unroll
            for (int p = 0; p < kPanels; ++p) {
                const uint64_t bd = smem_desc(tile + p * kPanel, 16, 1024, kSwizzle128B);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ts(tmem + dcol, tmem + acol + 32 * p + 8 * k, bd + 2 * k, kId64, add || p + k > 0);
            }
        };
        // D (+)= A . M^T of a lower triangular M, without the columns that are zero
        const auto triangle = [&](uint32_t dcol, uint32_t acol, uint32_t tile, bool add) {
            const uint64_t bd = smem_desc(tile, 16, 1024, kSwizzle128B);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_ts(tmem + dcol + 16 * k, tmem + acol + 8 * k, bd + 2 * k + 128 * k,
                       idesc_bf16_f32(128, 64 - 16 * k, false, false), add || k > 0);
        };
        // An operand's rounded part is used while the chain still writes what rounding left.
        // A commit covers all that was issued before it: with K S^T of a chunk done, so is
        // P U of the one in front, with the state's update Q S^T.
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            const uint32_t at = base + s * Lay::kStage;
            if (!wait.warp(bar(kFull + s), (c >> 1) & 1) || !wait.warp(bar(kSh), c & 1)) break;
            tc_fence_after();
            if (one) over_n(kColX, kColSh, at + Lay::kK, false);
            __syncwarp();
            if (!wait.warp(bar(kSl), c & 1)) break;
            tc_fence_after();
            if (one) {
                over_n(kColX, kColSl, at + Lay::kK, true);
                if (!(a.withhold && blockIdx.x == 0 && c == 0)) mma_commit(bar(kKs));
            }
            __syncwarp();
            if (c > 0 && !wait.warp(bar(kPuRead), (c - 1) & 1)) break;
            tc_fence_after();
            if (one) over_n(kColO, kColSh, at + Lay::kQ, false);
            __syncwarp();
            if (!wait.warp(bar(kRh), c & 1)) break;
            tc_fence_after();
            if (one) {
                triangle(kColX, kColR, at + Lay::kRec + kRecT, false);
                triangle(kColX, kColR, at + Lay::kRec + kRecT + kPanel, true);
            }
            __syncwarp();
            if (!wait.warp(bar(kRl), c & 1)) break;
            tc_fence_after();
            if (one) {
                triangle(kColX, kColRl, at + Lay::kRec + kRecT, true);
                mma_commit(bar(kU));
                over_n(kColO, kColSl, at + Lay::kQ, true);
                mma_commit(bar(kQs));
            }
            __syncwarp();
            const uint64_t keys = smem_desc(at + Lay::kK, kPanel, 1024, kSwizzle128B);
            if (!wait.warp(bar(kWh), c & 1)) break;
            tc_fence_after();
            if (one) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ts(tmem + kColS, tmem + kColW + 8 * k, keys + 128 * k, kIdS, 1);
            }
            __syncwarp();
            if (!wait.warp(bar(kWl), c & 1)) break;
            tc_fence_after();
            if (one) {
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ts(tmem + kColS, tmem + kColWl + 8 * k, keys + 128 * k, kIdS, 1);
                mma_commit(bar(kS));
            }
            __syncwarp();
            if (!wait.warp(bar(kUReady), c & 1) || !wait.warp(bar(kQsRead), c & 1)) break;
            tc_fence_after();
            if (one) {
                triangle(kColO, kColR, at + Lay::kRec + kRecP, false);
                triangle(kColO, kColR, at + Lay::kRec + kRecP + kPanel, true);
                triangle(kColO, kColRl, at + Lay::kRec + kRecP, true);
                mma_commit(bar(kPu));
                mma_commit(bar(kEmpty + s));
            }
            __syncwarp();
        }
        // what was issued completes before the CTA gives its tensor memory back
        if (one) mma_commit(bar(kDrain));
        __syncwarp();
        if (!mbar_wait(bar(kDrain), 0, kSsdDefaultWaitNs)) ssd_report(a.err, SSD_DEVERR_TIMEOUT);
    } else if (warp >= kChainWarps) {
        // the output: U's parts for P U, scale exp(G) (Q S^T) + P U; half of the tokens each
        const int q = warp & 3, half = (warp - kChainWarps) >> 2;
        const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
        __nv_bfloat16 *const out = reinterpret_cast<__nv_bfloat16 *>(smem + Lay::kO);
        const int tid = threadIdx.x - 32 * kChainWarps;
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1, tokens = min(kC, len - c * kC);
            const float *gates = reinterpret_cast<const float *>(smem + s * Lay::kStage + Lay::kRec + kRecGates) + 32 * half;
            if (!wait.warp(bar(kFull + s), (c >> 1) & 1) || !wait.warp(bar(kU), c & 1)) break;
            tc_fence_after();
            {
                uint32_t r[32], hi[16], lo[16];
                tmem_ld32(tq + kColX + 32 * half, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const Split x = split2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                    hi[i] = x.hi;
                    lo[i] = x.lo;
                }
                tmem_st16(tq + kColR + 16 * half, hi);
                tmem_st16(tq + kColRl + 16 * half, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kUReady));
            if (!wait.warp(bar(kQs), c & 1)) break;
            tc_fence_after();
            uint32_t y[32];
            tmem_ld32(tq + kColO + 32 * half, y);
            tmem_ld_wait(y);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kQsRead));
            if (!wait.warp(bar(kPu), c & 1)) break;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[16];
                tmem_ld16(tq + kColO + 32 * half + 16 * h, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    y[16 * h + i] = __float_as_uint(__uint_as_float(r[i]) +
                                                    d.scale * gates[16 * h + i] * __uint_as_float(y[16 * h + i]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kPuRead));
                mbar_arrive(bar(kEmpty + s));
            }
            // by way of shared memory: a lane has a channel, memory wants a token's together
#pragma unroll
            for (int i = 0; i < 32; ++i) out[(32 * half + i) * 128 + 32 * q + lane] = __float2bfloat16_rn(__uint_as_float(y[i]));
            named_bar_sync(1, 32 * kOutWarps);
            __nv_bfloat16 *const to = a.o + (size_t)(first + (long long)c * kC) * a.o_stride + (size_t)head * d.p + p0;
            if (a.o_vectors) {
                for (int i = tid; i < tokens * 16; i += 32 * kOutWarps) {
                    const int t = i >> 4, at = (i & 15) * 8;
                    if (p0 + at < d.p)
                        *reinterpret_cast<uint4 *>(to + (size_t)t * a.o_stride + at) =
                            *reinterpret_cast<const uint4 *>(out + t * 128 + at);
                }
            } else {
                for (int i = tid; i < tokens * 128; i += 32 * kOutWarps) {
                    const int t = i >> 7, at = i & 127;
                    if (p0 + at < d.p) to[(size_t)t * a.o_stride + at] = out[t * 128 + at];
                }
            }
            named_bar_sync(1, 32 * kOutWarps);
        }
    } else {
        // the chain: a thread has a row of the state and of V^T, R^T and U^T; the four groups
        // of four warps have a quarter of the columns each
        const int q = warp & 3, part = warp >> 2, row = 32 * q + lane, p = p0 + row;
        const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
        constexpr int kMine = kN / 4;
        const int n0 = part * kMine;
        const bool vec = d.n % 4 == 0;
        const auto to_memory = [&](float *m, const float (&v)[kMine]) {
            if (p >= d.p) return;
            float *to = m + (size_t)p * d.n;
#pragma unroll
            for (int i = 0; i < kMine; i += 4) {
                const int n = n0 + i;
                if (vec) {
                    if (n < d.n) *reinterpret_cast<float4 *>(to + n) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                } else {
                    for (int j = 0; j < 4; ++j)
                        if (n + j < d.n) to[n + j] = v[i + j];
                }
            }
        };
        // what this thread wrote to tensor memory is there for the products
        const auto ready = [&](int which) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(which));
        };
        // the state before chunk c: its parts, and in fp32 decayed over the chunk
        const auto put = [&](int c, const float (&v)[kMine], float decay) {
            uint32_t hi[kMine / 2];
#pragma unroll
            for (int i = 0; i < kMine / 2; ++i) hi[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            if constexpr (kMine == 32) tmem_st16(tq + kColSh + n0 / 2, hi);
            else tmem_st8(tq + kColSh + n0 / 2, hi);
            ready(kSh);
#pragma unroll
            for (int i = 0; i < kMine / 2; ++i) hi[i] = rest2(v[2 * i], v[2 * i + 1], hi[i]);
            if constexpr (kMine == 32) tmem_st16(tq + kColSl + n0 / 2, hi);
            else tmem_st8(tq + kColSl + n0 / 2, hi);
            ready(kSl);
            // (waited for before the chunk's kWh)
#pragma unroll
            for (int h = 0; h < kMine / 16; ++h) {
                uint32_t f[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 x = fmul2(make_float2(v[16 * h + 2 * i], v[16 * h + 2 * i + 1]), make_float2(decay, decay));
                    f[2 * i] = __float_as_uint(x.x);
                    f[2 * i + 1] = __float_as_uint(x.y);
                }
                tmem_st16(tq + kColS + n0 + 16 * h, f);
            }
            if (a.checkpoints) to_memory(a.checkpoints + ((size_t)(slot0 + c) * d.heads + head) * d.p * d.n, v);
        };
        const auto stage = [&](int c) { return smem + (c & 1) * Lay::kStage; };
        // keys behind the sequence's end are another's, or nothing: zeros
        const auto clean = [&](int c) {
            const int tokens = len - c * kC;
            if (tokens >= kC) return;
            uint4 *k = reinterpret_cast<uint4 *>(stage(c) + Lay::kK);
            for (int i = threadIdx.x; i < kPanels * (kC - tokens) * 8; i += 32 * kChainWarps) {
                const int panel = i / ((kC - tokens) * 8), at = i % ((kC - tokens) * 8);
                k[panel * (kPanel / 16) + tokens * 8 + at] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
        };
        bool on = wait.warp(bar(kFull), 0);
        if (on) {
            clean(0);
            float v[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                v[i] = a.init && p < d.p && n0 + i < d.n ? a.init[state + (size_t)p * d.n + n0 + i] : 0.f;
            put(0, v, reinterpret_cast<const float *>(stage(0) + Lay::kRec + kRecGates)[kC - 1]);
        }
        for (int c = 0; on && c < chunks; ++c) {
            const int s = c & 1, tokens = min(kC, len - c * kC) - 16 * part;
            const float4 *gates = reinterpret_cast<const float4 *>(stage(c) + Lay::kRec + kRecGates) + 4 * part;
            float x[16], f[16];
            {
                const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(stage(c) + Lay::kV) + 16 * part * 128 + row;
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __bfloat162float(v[i * 128]);
#pragma unroll
                for (int i = 0; i < 4; ++i) *reinterpret_cast<float4 *>(f + 4 * i) = gates[i];
            }
            if (!wait.warp(bar(kKs), c & 1)) break;
            tc_fence_after();
            uint32_t r[16], hi[8];
            tmem_ld16(tq + kColX + 16 * part, r);
            tmem_ld_wait(r);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 y = ffma2(make_float2(-f[i], -f[i + 1]),
                                       make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                                       make_float2(x[i], x[i + 1]));
                x[i] = y.x;
                x[i + 1] = y.y;
            }
            if (tokens < 16) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i >= tokens) x[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) hi[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            tmem_st8(tq + kColR + 8 * part, hi);
            ready(kRh);
#pragma unroll
            for (int i = 0; i < 8; ++i) hi[i] = rest2(x[2 * i], x[2 * i + 1], hi[i]);
            tmem_st8(tq + kColRl + 8 * part, hi);
            ready(kRl);
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float4 *>(f + 4 * i) = gates[kC / 4 + i];
            if (!wait.warp(bar(kU), c & 1)) break;
            tc_fence_after();
            tmem_ld16(tq + kColX + 16 * part, r);
            tmem_ld_wait(r);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 y = fmul2(make_float2(f[i], f[i + 1]),
                                       make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])));
                x[i] = y.x;
                x[i + 1] = y.y;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) hi[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            tmem_st8(tq + kColW + 8 * part, hi);
            ready(kWh);
#pragma unroll
            for (int i = 0; i < 8; ++i) hi[i] = rest2(x[2 * i], x[2 * i + 1], hi[i]);
            tmem_st8(tq + kColWl + 8 * part, hi);
            ready(kWl);
            if (lane == 0) mbar_arrive(bar(kEmpty + s));
            const bool more = c + 1 < chunks;
            if (more && !wait.warp(bar(kFull + (s ^ 1)), ((c + 1) >> 1) & 1)) break;
            if (more) clean(c + 1);
            const float decay = more ? reinterpret_cast<const float *>(stage(c + 1) + Lay::kRec + kRecGates)[kC - 1] : 1.f;
            if (!wait.warp(bar(kS), c & 1)) break;
            tc_fence_after();
            uint32_t m[kMine];
            if constexpr (kMine == 32) tmem_ld32(tq + kColS + n0, m);
            else tmem_ld16(tq + kColS + n0, m);
            tmem_ld_wait(m);
            float y[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i) y[i] = __uint_as_float(m[i]);
            if (more) put(c + 1, y, decay);
            else if (a.final_state) to_memory(a.final_state + state, y);
        }
    }
    // copies in flight land before the CTA ends
    if (warp == kLoadWarp) {
        for (int c = loaded > 2 ? loaded - 2 : 0; c < loaded; ++c)
            if (!mbar_wait(bar(kFull + (c & 1)), (c >> 1) & 1, kSsdDefaultWaitNs)) ssd_report(a.err, SSD_DEVERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// [tokens][heads][width] bf16 by boxes of `cols` values of one head and 64 tokens.
bool make_map(CUtensorMap *m, const void *p, int width, int heads, long long tokens, long long stride, int cols,
              bool swizzle) {
    const auto enc = ssd_tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {(cuuint32_t)cols, 1, (cuuint32_t)kC}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kPanels>
cudaError_t launch_fwd(const SsdDeltaFwd &f, void *ws, unsigned *err, cudaStream_t stream) {
    const SsdDelta &d = f.in;
    CUtensorMap q, k, v;
    if (!make_map(&q, d.q, d.n, d.groups, d.tokens, d.q_stride, 64, true) ||
        !make_map(&k, d.k, d.n, d.groups, d.tokens, d.k_stride, 64, true) ||
        !make_map(&v, d.v, d.p, d.heads, d.tokens, d.v_stride, 128, false))
        return cudaErrorInvalidValue;
    const SsdDebug debug = ssd_debug_config();
    uint8_t *records = static_cast<uint8_t *>(ws);
    const long long slots = ssd_delta_slots(d.tokens, d.nseq);
    cudaError_t e = cudaFuncSetAttribute(delta_chunk_kernel<kPanels>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PrepSmem::kBytes);
    if (e != cudaSuccess) return e;
    delta_chunk_kernel<kPanels><<<(unsigned)(slots * d.groups), kPrepThreads, PrepSmem::kBytes, stream>>>(
        q, k, Prep{d, records, err});
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    using Lay = WalkSmem<kPanels>;
    static_assert(Lay::kBytes <= 232448, "more than 227 KB of shared memory");
    e = cudaFuncSetAttribute(delta_walk_tc_kernel<kPanels>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kBytes);
    if (e != cudaSuccess) return e;
    const int blocks = (d.p + 127) / 128;
    const WalkTc w{d, records, f.init, static_cast<__nv_bfloat16 *>(f.o), f.o_stride, f.final_state, f.checkpoints, blocks,
                   ((uintptr_t)f.o & 15u) == 0 && f.o_stride % 8 == 0, err, debug.wait_ns, debug.fault == kSsdFaultWithholdSignal};
    delta_walk_tc_kernel<kPanels><<<(unsigned)((long long)d.nseq * d.heads * blocks), kWalkThreads, Lay::kBytes, stream>>>(
        q, k, v, w);
    return cudaGetLastError();
}

}  // namespace

// Types and sizes that these kernels take, and alignments: the copies' rows start on 16 bytes.
bool ssd_delta_tc_sizes(const SsdDelta &d) {
    return d.bf16 && d.n <= 128 && d.n % 8 == 0 && d.p % 8 == 0 && d.tokens > 0;
}
bool ssd_delta_tc_handles(const SsdDelta &d) {
    const auto rows_ok = [](const void *p, long long stride) { return ((uintptr_t)p & 15u) == 0 && stride % 8 == 0; };
    return ssd_delta_tc_sizes(d) && rows_ok(d.q, d.q_stride) && rows_ok(d.k, d.k_stride) && rows_ok(d.v, d.v_stride) &&
           ssd_tensor_map_encoder() != nullptr;
}

size_t ssd_delta_tc_workspace(const SsdDelta &d) {
    return ssd_delta_tc_sizes(d) ? (size_t)ssd_delta_slots(d.tokens, d.nseq) * d.heads * kRecord : 0;
}

cudaError_t ssd_launch_delta_fwd_tc(const SsdDeltaFwd &a, void *ws, unsigned *err, cudaStream_t stream) {
    return a.in.n <= 64 ? launch_fwd<1>(a, ws, err, stream) : launch_fwd<2>(a, ws, err, stream);
}
