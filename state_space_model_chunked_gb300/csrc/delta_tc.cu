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
// then a row of Q K^T (threads 0 .. 63) or of K K^T (64 .. 127).
constexpr int kPrepThreads = 128;
struct PrepSmem {
    // at 0: Q over K by panels, then the images
    static constexpr uint32_t kA = 4 * kPanel;              // A's columns, fp32
    static constexpr uint32_t kSums = kA + kC * kC * 4;     // G in two floats, beta
    static constexpr uint32_t kBars = kSums + 3 * kC * 4;
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

// T's column `col`, solved row by row: what row i of T gives is taken off all rows behind
// it.  `first`: the first row that is not zero in any of the warp's columns.
template <int kFirst>
__device__ __forceinline__ void solve_column(const float *columns, int col, float beta, uint8_t *hi, uint8_t *lo) {
    float acc[kC];
#pragma unroll
    for (int i = 0; i < kC; ++i) acc[i] = 0.f;
#pragma unroll
    for (int i = kFirst; i < kC; ++i) {
        const float t = i == col ? 1.f : -acc[i];
        const float4 *a = reinterpret_cast<const float4 *>(columns + i * kC);
#pragma unroll
        for (int v = (i + 1) / 4; v < kC / 4; ++v) {
            const float4 x = a[v];
            if (4 * v > i) acc[4 * v] += x.x * t;
            if (4 * v + 1 > i) acc[4 * v + 1] += x.y * t;
            if (4 * v + 2 > i) acc[4 * v + 2] += x.z * t;
            acc[4 * v + 3] += x.w * t;
        }
        const float tb = t * beta;
        const __nv_bfloat16 h = __float2bfloat16_rn(tb);
        *reinterpret_cast<__nv_bfloat16 *>(hi + panel_at(i, col)) = h;
        *reinterpret_cast<__nv_bfloat16 *>(lo + panel_at(i, col)) = __float2bfloat16_rn(tb - __bfloat162float(h));
    }
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
        *reinterpret_cast<uint16_t *>(hi + panel_at(i, col)) = 0;
        *reinterpret_cast<uint16_t *>(lo + panel_at(i, col)) = 0;
    }
}

template <int kPanels>
__global__ void __launch_bounds__(kPrepThreads)
delta_chunk_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK, const Prep a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const SsdDelta &d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    float *const betas = sum_lo + kC, *const columns = reinterpret_cast<float *>(smem + PrepSmem::kA);
    const int wide = d.heads / d.groups, row = threadIdx.x & 63;
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
        // the images of the head in front have been read, its columns used
        if (threadIdx.x == 0 && h > 0) bulk_wait_read<0>();
        __syncthreads();
        const float2 half = make_float2(sum_hi[31], sum_lo[31]);
        float2 mine = make_float2(sum_hi[row], sum_lo[row]);
        if (row >= 32) mine = add_two(half, mine);
        const float2 end = add_two(half, make_float2(sum_hi[63], sum_lo[63]));
        __syncthreads();
        if (threadIdx.x >= 32 && threadIdx.x < 64) {
            sum_hi[row] = mine.x;
            sum_lo[row] = mine.y;
        }
        if (threadIdx.x < kC) {
            float *gates = reinterpret_cast<float *>(record + kRecGates);
            gates[row] = __expf(mine.x + mine.y);
            gates[kC + row] = __expf((end.x - mine.x) + (end.y - mine.y));
        }
        __syncthreads();
        const bool keys = warp >= 2;
        const float factor = keys ? betas[row] : d.scale;
        for (int c0 = 0; c0 < kC; c0 += 32) {
            uint32_t r[32];
            tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16) + c0, r);
            tmem_ld_wait(r);
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const int col = c0 + j;
                const float e = __expf((mine.x - sum_hi[col]) + (mine.y - sum_lo[col]));
                const bool in = row < valid && (keys ? col < row : col <= row);
                v[j] = in ? factor * e * __uint_as_float(r[j]) : 0.f;
            }
            if (keys) {
#pragma unroll
                for (int j = 0; j < 32; ++j) columns[(c0 + j) * kC + row] = v[j];
            } else {
#pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const Split s = split2(v[j + 2 * i], v[j + 2 * i + 1]);
                        hi[i] = s.hi;
                        lo[i] = s.lo;
                    }
                    const uint32_t to = kRecP + panel_at(row, c0 + j);
                    *reinterpret_cast<uint4 *>(smem + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(smem + to + kPanel) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
        }
        if (keys) {
            named_bar_sync(1, 64);
            if (warp == 2) solve_column<0>(columns, row, betas[row], smem + kRecT, smem + kRecT + kPanel);
            else solve_column<32>(columns, row, betas[row], smem + kRecT, smem + kRecT + kPanel);
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
constexpr int kWalkThreads = 14 * 32;       // 8 warps on the chain, 4 on the output, copies, products
constexpr int kOutWarp = 8, kLoadWarp = 12, kMmaWarp = 13;

template <int kPanels>
struct WalkSmem {
    static constexpr uint32_t kK = 0, kQ = kPanels * kPanel, kRec = 2 * kPanels * kPanel;
    static constexpr uint32_t kV = kRec + kRecord;      // [token][128], as they lie
    static constexpr uint32_t kStage = (kV + 64 * 256 + 1023) / 1024 * 1024;
    static constexpr uint32_t kCtl = 2 * kStage;
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
    unsigned *err;
    unsigned long long wait_ns;
    bool withhold;
};

enum WalkBar {
    kFull = 0, kEmpty = 2,      // two stages each
    kKs = 4, kRReady, kU, kWReady, kS, kSReady, kQs, kQsRead, kUReady, kPu, kPuRead, kDrain, kBars
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
            mbar_init(bar(kEmpty + s), 1 + 8 + 4);
        }
        for (int i : {kKs, kU, kS, kQs, kPu, kDrain}) mbar_init(bar(i), 1);
        for (int i : {kRReady, kWReady, kSReady}) mbar_init(bar(i), 8);
        for (int i : {kQsRead, kUReady, kPuRead}) mbar_init(bar(i), 4);
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
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            const uint32_t at = base + s * Lay::kStage;
            if (!wait.warp(bar(kFull + s), (c >> 1) & 1) || !wait.warp(bar(kSReady), c & 1)) break;
            tc_fence_after();
            if (one) {
                over_n(kColX, kColSh, at + Lay::kK, false);
                over_n(kColX, kColSl, at + Lay::kK, true);
                if (!(a.withhold && blockIdx.x == 0 && c == 0)) mma_commit(bar(kKs));
            }
            __syncwarp();
            if (c > 0 && !wait.warp(bar(kPuRead), (c - 1) & 1)) break;
            tc_fence_after();
            if (one) over_n(kColO, kColSh, at + Lay::kQ, false);
            __syncwarp();
            if (!wait.warp(bar(kRReady), c & 1)) break;
            tc_fence_after();
            if (one) {
                triangle(kColX, kColR, at + Lay::kRec + kRecT, false);
                triangle(kColX, kColR, at + Lay::kRec + kRecT + kPanel, true);
                triangle(kColX, kColRl, at + Lay::kRec + kRecT, true);
                mma_commit(bar(kU));
                over_n(kColO, kColSl, at + Lay::kQ, true);
                mma_commit(bar(kQs));
            }
            __syncwarp();
            if (!wait.warp(bar(kWReady), c & 1)) break;
            tc_fence_after();
            if (one) {
                const uint64_t bd = smem_desc(at + Lay::kK, kPanel, 1024, kSwizzle128B);
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ts(tmem + kColS, tmem + kColW + 8 * k, bd + 128 * k, kIdS, 1);
#pragma unroll
                for (int k = 0; k < 4; ++k) mma_ts(tmem + kColS, tmem + kColWl + 8 * k, bd + 128 * k, kIdS, 1);
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
    } else if (warp >= kOutWarp) {
        // the output: U's parts for P U, scale exp(G) (Q S^T) + P U
        const int q = warp & 3, p = p0 + 32 * q + lane;
        const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1, tokens = min(kC, len - c * kC);
            const float *gates = reinterpret_cast<const float *>(smem + s * Lay::kStage + Lay::kRec + kRecGates);
            if (!wait.warp(bar(kFull + s), (c >> 1) & 1) || !wait.warp(bar(kU), c & 1)) break;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[32], hi[16], lo[16];
                tmem_ld32(tq + kColX + 32 * h, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const Split x = split2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                    hi[i] = x.hi;
                    lo[i] = x.lo;
                }
                tmem_st16(tq + kColR + 16 * h, hi);
                tmem_st16(tq + kColRl + 16 * h, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kUReady));
            if (!wait.warp(bar(kQs), c & 1)) break;
            tc_fence_after();
            float y[64];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
                tmem_ld32(tq + kColO + 32 * h, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 32; ++i) y[32 * h + i] = d.scale * gates[32 * h + i] * __uint_as_float(r[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kQsRead));
                mbar_arrive(bar(kEmpty + s));
            }
            if (!wait.warp(bar(kPu), c & 1)) break;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
                tmem_ld32(tq + kColO + 32 * h, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 32; ++i) y[32 * h + i] += __uint_as_float(r[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kPuRead));
            if (p < d.p) {
                __nv_bfloat16 *to = a.o + (size_t)(first + (long long)c * kC) * a.o_stride + (size_t)head * d.p + p;
#pragma unroll
                for (int i = 0; i < kC; ++i)
                    if (i < tokens) to[(size_t)i * a.o_stride] = __float2bfloat16_rn(y[i]);
            }
        }
    } else {
        // the chain: a thread has a row of the state and of V^T, R^T and U^T; the two groups
        // of four warps have half of the columns each
        const int q = warp & 3, half = warp >> 2, row = 32 * q + lane, p = p0 + row;
        const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
        constexpr int kMine = kN / 2;
        const int n0 = half * kMine;
        // the state's columns n0 + 32 b ..: two parts, and fp32 decayed over the next chunk
        const auto put = [&](int b, float (&v)[32], float decay) {
            uint32_t hi[16], lo[16], f[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const Split x = split2(v[2 * i], v[2 * i + 1]);
                hi[i] = x.hi;
                lo[i] = x.lo;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = __float_as_uint(v[i] * decay);
            tmem_st16(tq + kColSh + n0 / 2 + 16 * b, hi);
            tmem_st16(tq + kColSl + n0 / 2 + 16 * b, lo);
            tmem_st32(tq + kColS + n0 + 32 * b, f);
        };
        const bool vec = d.n % 4 == 0;
        const auto to_memory = [&](float *m, int b, const float (&v)[32]) {
            if (p >= d.p) return;
            float *to = m + (size_t)p * d.n;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const int n = n0 + 32 * b + i;
                if (vec) {
                    if (n < d.n) *reinterpret_cast<float4 *>(to + n) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                } else {
                    for (int j = 0; j < 4; ++j)
                        if (n + j < d.n) to[n + j] = v[i + j];
                }
            }
        };
        const auto stage = [&](int c) { return smem + (c & 1) * Lay::kStage; };
        // keys behind the sequence's end are another's, or nothing: zeros
        const auto clean = [&](int c) {
            const int tokens = len - c * kC;
            if (tokens >= kC) return;
            uint4 *k = reinterpret_cast<uint4 *>(stage(c) + Lay::kK);
            for (int i = threadIdx.x; i < kPanels * (kC - tokens) * 8; i += 256) {
                const int panel = i / ((kC - tokens) * 8), at = i % ((kC - tokens) * 8);
                k[panel * (kPanel / 16) + tokens * 8 + at] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
        };
        bool on = wait.warp(bar(kFull), 0);
        if (on) {
            clean(0);
            const float decay = reinterpret_cast<const float *>(stage(0) + Lay::kRec + kRecGates)[kC - 1];
#pragma unroll
            for (int b = 0; b < kMine / 32; ++b) {
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int n = n0 + 32 * b + i;
                    v[i] = a.init && p < d.p && n < d.n ? a.init[state + (size_t)p * d.n + n] : 0.f;
                }
                put(b, v, decay);
                if (a.checkpoints) to_memory(a.checkpoints + ((size_t)slot0 * d.heads + head) * d.p * d.n, b, v);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kSReady));
        }
        for (int c = 0; on && c < chunks; ++c) {
            const int s = c & 1, tokens = min(kC, len - c * kC);
            const float *gates = reinterpret_cast<const float *>(stage(c) + Lay::kRec + kRecGates);
            const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(stage(c) + Lay::kV) + row;
            if (!wait.warp(bar(kKs), c & 1)) break;
            // (P U of the chunk in front has read U's parts, where R's go)
            if (c > 0 && !wait.warp(bar(kPu), (c - 1) & 1)) break;
            tc_fence_after();
            {
                uint32_t r[32], hi[16], lo[16];
                tmem_ld32(tq + kColX + 32 * half, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int t = 32 * half + 2 * i + j;
                        x[j] = __bfloat162float(v[t * 128]) - gates[t] * __uint_as_float(r[2 * i + j]);
                        if (t >= tokens) x[j] = 0.f;
                    }
                    const Split y = split2(x[0], x[1]);
                    hi[i] = y.hi;
                    lo[i] = y.lo;
                }
                tmem_st16(tq + kColR + 16 * half, hi);
                tmem_st16(tq + kColRl + 16 * half, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kRReady));
            if (!wait.warp(bar(kU), c & 1)) break;
            tc_fence_after();
            {
                uint32_t r[32], hi[16], lo[16];
                tmem_ld32(tq + kColX + 32 * half, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int t = kC + 32 * half + 2 * i;
                    const Split y = split2(gates[t] * __uint_as_float(r[2 * i]), gates[t + 1] * __uint_as_float(r[2 * i + 1]));
                    hi[i] = y.hi;
                    lo[i] = y.lo;
                }
                tmem_st16(tq + kColW + 16 * half, hi);
                tmem_st16(tq + kColWl + 16 * half, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kWReady));
                mbar_arrive(bar(kEmpty + s));
            }
            const bool more = c + 1 < chunks;
            if (more && !wait.warp(bar(kFull + (s ^ 1)), ((c + 1) >> 1) & 1)) break;
            if (more) clean(c + 1);
            // (Q S^T has read the state's parts)
            if (!wait.warp(bar(kQs), c & 1) || !wait.warp(bar(kS), c & 1)) break;
            tc_fence_after();
            const float decay = more ? reinterpret_cast<const float *>(stage(c + 1) + Lay::kRec + kRecGates)[kC - 1] : 1.f;
#pragma unroll
            for (int b = 0; b < kMine / 32; ++b) {
                uint32_t r[32];
                float x[32];
                tmem_ld32(tq + kColS + n0 + 32 * b, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
                if (more) {
                    put(b, x, decay);
                    if (a.checkpoints)
                        to_memory(a.checkpoints + ((size_t)(slot0 + c + 1) * d.heads + head) * d.p * d.n, b, x);
                } else if (a.final_state) {
                    to_memory(a.final_state + state, b, x);
                }
            }
            if (!more) break;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kSReady));
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
                   err, debug.wait_ns, debug.fault == kSsdFaultWithholdSignal};
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
