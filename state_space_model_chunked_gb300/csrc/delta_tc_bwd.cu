// Gradients of the gated delta rule on the tensor cores, by the chunks of 64 tokens of
// delta_tc.cu.  With S the state before a chunk (kept by the forward pass), dS the gradient
// of the state behind it, and T, P, R, U as there:
//
//   dU = P^T dO + diag(exp(G_end - G)) K dS^T
//   Z  = (T diag(beta))^T dU                       (the gradient of V; its diagonal's part in fp32)
//   dS <- exp(G_end) dS + (diag(scale exp G) dO)^T Q - (diag(exp G) Z)^T K
//
// is a walk over the chunks, from the last one on (the first kernel: one CTA a head, the
// state's rows as the tensor core's lanes, as in the forward walk; it leaves Z and every
// chunk's dS), and with M1 = dO U^T, M2 = Z U^T (64 x 64) and D_ij = exp(G_i - G_j)
//
//   dP_ij = scale D_ij M1_ij (j <= i)       dA_ij = -D_ij M2_ij (j < i)
//   dQ = scale diag(exp G) dO S + dP K
//   dK = -diag(exp G) Z S + diag(exp(G_end - G)) U dS + dP^T Q + dA K + dA^T K
//   dbeta_i = z_i . u_i / beta_i^2
//   dg_t = exp(G_end) <S, dS> + sum_(i >= t) (what token i reads of S, dotted with it)
//        + sum_(j < t) (what token j leaves in dS) + sum_(i >= t > j) (dP o QK + dA o KK)_ij
//
// of every chunk by itself (the second kernel, a chunk and head a CTA).  Where one sum
// over pairs i >= t > j is wanted, it is taken as the running sum of row sums less column
// sums of the same fp32 values, so what cancels does so exactly.
//   As forward, factors that are no bf16 values are held in two bf16 parts.
//   A long sequence of few heads is walked in parts, as forward but from the last one on: 25600
// tokens, one head 1626 -> 284 us, 32 heads 2790 -> 2130.
//   8 x 2047 tokens, 16 heads of 128 x 128: 570 us, of which the chunk matrices 59, the walk 137
// (dS and Z leave at 3.0 TB/s beside 2.4 TB/s of loads) and the second kernel 367: 25000 cycles a
// chunk and head for six products in turn, each between two barriers, with 47% of the issue
// slots, and 220 KB of tiles an SM that leave no room for a second CTA.
#include "delta_tc.cuh"

namespace {

using namespace ssddelta;

// MMA helpers: one kind::f16 product of M = 128 over 16 columns or rows of K a call.
// A panel's descriptor moves by 32 bytes along a row (K-major) and by 16 rows (MN-major).
constexpr uint64_t kStepK = 2, kStepMn = 128;

// ------------------------------------------------------------------ the walk
// Tensor memory: dS in fp32 and in two parts; K dS^T, then Z; P^T dO; dU, then Z weighted,
// in two parts; dO weighted, in two parts.
constexpr uint32_t kColS = 0, kColSh = 128, kColSl = 192, kColX = 256, kColY = 320, kColR = 384, kColRl = 416,
                   kColD = 448, kColDl = 480;
constexpr int kChainWarps = 16, kOutWarps = 8;
constexpr int kLoadWarp = kChainWarps + kOutWarps, kMmaWarp = kLoadWarp + 1, kBackThreads = 32 * (kMmaWarp + 1);

constexpr uint32_t kTall = 2 * kPanel;              // a panel of 128 rows
constexpr uint32_t kImageRows = 32 * 128;           // a warp's rows of one
static_assert(kOutWarps * kImageRows >= kChainWarps * kStageRows && 4 * kPanel >= kChainWarps * kStageRows, "one place for both");
// A chunk's dS, for every head: its two parts, each [128 of P][N] by tall panels.
constexpr uint32_t state_image(int panels) { return 2 * panels * kTall; }
// And its Z in fp32, by tiles of 32 tokens x 32 rows of a state, as the warps have them.
constexpr size_t kZTile = 64 * 128;
__device__ __forceinline__ size_t z_at(size_t record, int token, int row) {
    return record * kZTile + (size_t)((token >> 5) * 4 + (row >> 5)) * 1024 + (token & 31) * 32 + (row & 31);
}

template <int kPanels>
struct BackSmem {
    static constexpr uint32_t kK = 0, kQ = kPanels * kPanel, kDo = 2 * kPanels * kPanel, kRec = kDo + 2 * kPanel;
    static constexpr uint32_t kStage = (kRec + kRecord + 1023) / 1024 * 1024;
    static constexpr uint32_t kOut = 2 * kStage;        // [token][128]: dV on its way
    static constexpr uint32_t kRows = kOut + 64 * 256;  // by warps: dfinal, then images of dS and Z on their way out
    static constexpr uint32_t kCtl = kRows + kOutWarps * kImageRows;
    static constexpr uint32_t kBytes = kCtl + 256;
};

struct BackTc {
    SsdDelta d;
    const uint8_t *records;
    const float *dfinal;
    __nv_bfloat16 *dv;
    long long dv_stride;
    bool dv_vectors;
    float *dinit;
    float *z;               // [slot][head] tiles
    uint8_t *dstate;        // [slot][head] images
    // in parts (segments > 1), as the forward walk: `d` has them for sequences; before that, from
    // the last one on, their ends for `starts` [seq][segment from the last][head][P][N], and maps
    int segments, half;
    float *starts, *maps;
    unsigned *err;
    unsigned long long wait_ns;
    bool withhold;
};

enum BackBar {
    kFull = 0, kEmpty = 2,
    kE = 4, kZ, kS, kDrain,                 // products done
    kSh, kSl, kRh, kRl, kWh, kWl,           // operands' parts written by the chain
    kD, kZRead, kSRead,                     // by the output's warps, and read by them
    kStaged, kStored,                       // dV in shared memory, and out of it
    kBars
};

template <int kPanels, bool kEnds>
__global__ void __launch_bounds__(kBackThreads, 1)
delta_back_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                     const __grid_constant__ CUtensorMap mapDo, const BackTc a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using Lay = BackSmem<kPanels>;
    constexpr int kN = 64 * kPanels;
    const SsdDelta &d = a.d;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) {
        if (threadIdx.x == 0) ssd_report(a.err, SSD_DEVERR_SMEM_ALIGN);
        return;
    }
    // kEnds: parts for their ends or (map) for their maps, without output
    const unsigned maps = kEnds ? (unsigned)d.nseq * (a.segments - 2) * d.heads : 0;
    const bool map = kEnds && blockIdx.x < maps;
    const unsigned job = blockIdx.x - (map ? 0 : maps);
    const int head = (int)(job % d.heads), group = head / (d.heads / d.groups), rows = map ? d.n : d.p;
    int seq = (int)(job / d.heads), back = 0;       // back: the part's number from the last one
    if constexpr (kEnds) {
        back = a.segments - 2 - seq / d.nseq;
        seq %= d.nseq;
    } else {
        seq = sequence_of(d, seq, reinterpret_cast<volatile int *>(smem + Lay::kCtl + 8 * kBars + 8));
    }
    long long first = d.cu ? d.cu[seq] : (long long)seq * d.length;
    int len = d.cu ? d.cu[seq + 1] - d.cu[seq] : d.length;
    if constexpr (kEnds) {
        const int at = part_start(len, a.segments - 1 - back, a.segments, a.half);
        len = part_start(len, a.segments - back, a.segments, a.half) - at;
        first += at;
    }
    const int chunks = (len + kC - 1) / kC;
    const size_t size = (size_t)rows * d.n;
    // where dS comes from (null: zeros, or a map's unit matrix) and goes to
    const auto source = [&]() -> const float * {
        if (kEnds) return back == 0 && a.dfinal ? a.dfinal + ((size_t)seq * d.heads + head) * size : nullptr;
        if (a.segments == 1) return a.dfinal ? a.dfinal + ((size_t)seq * d.heads + head) * size : nullptr;
        const int whole = seq / a.segments, i = a.segments - 1 - seq % a.segments;
        return a.starts + (((size_t)whole * a.segments + i) * d.heads + head) * size;
    };
    const auto target = [&]() -> float * {
        if (map) return a.maps + (((size_t)seq * (a.segments - 2) + back - 1) * d.heads + head) * size;
        if (kEnds) return a.starts + (((size_t)seq * a.segments + back + 1) * d.heads + head) * size;
        if (!a.dinit || seq % a.segments) return nullptr;
        return a.dinit + ((size_t)(seq / a.segments) * d.heads + head) * size;
    };
    if (chunks == 0) {
        const float *from = source();
        if (float *const to = target())
            for (int i = threadIdx.x; i < (int)size; i += kBackThreads)
                to[i] = from ? from[i] : map && i / d.n == i % d.n ? 1.f : 0.f;
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
        for (int i : {kE, kZ, kS, kDrain}) mbar_init(bar(i), 1);
        for (int i : {kSh, kSl, kRh, kRl, kWh, kWl}) mbar_init(bar(i), kChainWarps);
        for (int i : {kD, kZRead, kSRead, kStaged, kStored}) mbar_init(bar(i), kOutWarps);
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
    const long long slot0 = ssd_delta_slot(first, kEnds ? seq : seq / a.segments, 0);
    int loaded = 0;

    // step `it` of the walk is chunk chunks - 1 - it, in stage it & 1
    if (warp == kLoadWarp) {
        for (int it = 0; it < chunks; ++it) {
            const int s = it & 1, c = chunks - 1 - it;
            if (it >= 2 && !wait.warp(bar(kEmpty + s), ((it >> 1) - 1) & 1)) break;
            if (elect_one()) {
                const uint32_t to = base + s * Lay::kStage;
                const int token = (int)(first + (long long)c * kC);
                mbar_arrive_expect_tx(bar(kFull + s), (map ? kPanels : 2 * kPanels + 2) * kPanel + kRecord);
#pragma unroll
                for (int p = 0; p < kPanels; ++p) {
                    tma_load_3d(to + Lay::kK + p * kPanel, &mapK, bar(kFull + s), 64 * p, group, token);
                    if (!map) tma_load_3d(to + Lay::kQ + p * kPanel, &mapQ, bar(kFull + s), 64 * p, group, token);
                }
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    if (!map) tma_load_3d(to + Lay::kDo + p * kPanel, &mapDo, bar(kFull + s), 64 * p, head, token);
                bulk_load(to + Lay::kRec, a.records + ((size_t)(slot0 + c) * d.heads + head) * kRecord, kRecord,
                          bar(kFull + s));
            }
            __syncwarp();
            loaded = it + 1;
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t kId64 = idesc_bf16_f32(128, 64, false, false);
        constexpr uint32_t kIdS = idesc_bf16_f32(128, kN, false, true);
        const bool one = elect_one();
        const auto keys = [&](uint32_t acol, uint32_t tile, bool add) {
#pragma unroll
            for (int p = 0; p < kPanels; ++p) {
                const uint64_t bd = smem_desc(tile + p * kPanel, 16, 1024, kSwizzle128B);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ts(tmem + kColX, tmem + acol + 32 * p + 8 * k, bd + kStepK * k, kId64, add || p + k > 0);
            }
        };
        // D (+)= A . M of a lower triangular M, whose rows from 16 k on end at column 16 k + 15
        const auto triangle = [&](uint32_t acol, uint32_t tile, bool add) {
            const uint64_t bd = smem_desc(tile, kPanel, 1024, kSwizzle128B);
#pragma unroll
            for (int k = 3; k >= 0; --k)
                mma_ts(tmem + kColX, tmem + acol + 8 * k, bd + kStepMn * k, idesc_bf16_f32(128, 16 * k + 16, false, true),
                       add || k < 3);
        };
        const auto state_update = [&](uint32_t acol, uint32_t tile) {
            const uint64_t bd = smem_desc(tile, kPanel, 1024, kSwizzle128B);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ts(tmem + kColS, tmem + acol + 8 * k, bd + kStepMn * k, kIdS, 1);
        };
        const auto from_output = [&](uint32_t at) {
            const uint64_t ad = smem_desc(at + Lay::kDo, kPanel, 1024, kSwizzle128B);
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                const uint64_t bd = smem_desc(at + Lay::kRec + kRecP + part * kPanel, kPanel, 1024, kSwizzle128B);
#pragma unroll
                for (int k = 3; k >= 0; --k)
                    mma_ss(tmem + kColY, ad + kStepMn * k, bd + kStepMn * k, idesc_bf16_f32(128, 16 * k + 16, true, true),
                           part > 0 || k < 3);
            }
        };
        for (int it = 0; it < chunks; ++it) {
            const int s = it & 1;
            const uint32_t at = base + s * Lay::kStage;
            if (!wait.warp(bar(kFull + s), (it >> 1) & 1) || !wait.warp(bar(kSh), it & 1)) break;
            // (Z of the step in front has been read)
            if (!kEnds && it > 0 && !wait.warp(bar(kZRead), (it - 1) & 1)) break;
            tc_fence_after();
            if (one) {
                // the last chunk's rows behind the sequence's end are clean only now
                if (it == 0 && !map) from_output(at);
                keys(kColSh, at + Lay::kK, false);
            }
            __syncwarp();
            if (!wait.warp(bar(kSl), it & 1)) break;
            tc_fence_after();
            if (one) {
                keys(kColSl, at + Lay::kK, true);
                if (!(a.withhold && blockIdx.x == 0 && it == 0)) mma_commit(bar(kE));
            }
            __syncwarp();
            if (!wait.warp(bar(kRh), it & 1)) break;
            tc_fence_after();
            if (one) {
                triangle(kColR, at + Lay::kRec + kRecT, true);
                triangle(kColR, at + Lay::kRec + kRecT + kPanel, true);
            }
            __syncwarp();
            if (!wait.warp(bar(kRl), it & 1)) break;
            tc_fence_after();
            if (one) {
                triangle(kColRl, at + Lay::kRec + kRecT, true);
                mma_commit(bar(kZ));
            }
            __syncwarp();
            if (!map) {
                if (!wait.warp(bar(kD), it & 1)) break;
                tc_fence_after();
                if (one) {
                    state_update(kColD, at + Lay::kQ);
                    state_update(kColDl, at + Lay::kQ);
                }
                __syncwarp();
            }
            if (!wait.warp(bar(kWh), it & 1)) break;
            tc_fence_after();
            if (one) state_update(kColR, at + Lay::kK);
            __syncwarp();
            if (!wait.warp(bar(kWl), it & 1)) break;
            tc_fence_after();
            if (one) {
                state_update(kColRl, at + Lay::kK);
                mma_commit(bar(kS));
                mma_commit(bar(kEmpty + s));
            }
            __syncwarp();
            if (it + 1 < chunks && !map) {
                if (!wait.warp(bar(kFull + (s ^ 1)), ((it + 1) >> 1) & 1)) break;
                if (one) from_output(base + (s ^ 1) * Lay::kStage);
                __syncwarp();
            }
        }
        // what was issued completes before the CTA gives its tensor memory back
        if (one) mma_commit(bar(kDrain));
        __syncwarp();
        if (!mbar_wait(bar(kDrain), 0, kSsdDefaultWaitNs)) ssd_report(a.err, SSD_DEVERR_TIMEOUT);
    } else if (warp >= kChainWarps) {
        // dO's weighted parts, and Z on its way out: half of the tokens each
        const int q = warp & 3, half = (warp - kChainWarps) >> 2, row = 32 * q + lane;
        const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
        __nv_bfloat16 *const out = reinterpret_cast<__nv_bfloat16 *>(smem + Lay::kOut);
        const int tid = threadIdx.x - 32 * kChainWarps;
        for (int it = 0; it < chunks; ++it) {
            const int s = it & 1, c = chunks - 1 - it, tokens = min(kC, len - c * kC);
            const uint8_t *stage = smem + s * Lay::kStage;
            const float *gates = reinterpret_cast<const float *>(stage + Lay::kRec + kRecGates) + 32 * half;
            if (!wait.warp(bar(kFull + s), (it >> 1) & 1)) break;
            if (map) {
                if (lane == 0) mbar_arrive(bar(kEmpty + s));
                continue;
            }
            // (the step in front has used its parts)
            if (it > 0 && !wait.warp(bar(kS), (it - 1) & 1)) break;
            tc_fence_after();
            {
                const uint8_t *from = stage + Lay::kDo + (row >> 6) * kPanel;
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int t = 32 * half + 2 * i + j;
                        const float o = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(from + panel_at(t, row & 63)));
                        x[j] = t < tokens ? o * (d.scale * gates[2 * i + j]) : 0.f;
                    }
                    const Split y = split2(x[0], x[1]);
                    hi[i] = y.hi;
                    lo[i] = y.lo;
                }
                tmem_st16(tq + kColD + 16 * half, hi);
                tmem_st16(tq + kColDl + 16 * half, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kD));
                mbar_arrive(bar(kEmpty + s));
            }
            if (kEnds) continue;
            // dS, as the products have it, for the chunk's other gradients: a panel's 32 rows
            // of a part are 4 KB in one piece
            if (!wait.warp(bar(kSl), it & 1)) break;
            tc_fence_after();
            uint8_t *const rows = smem + Lay::kRows + (warp - kChainWarps) * kImageRows;
            if (half < kPanels) {
                uint8_t *const image = a.dstate + ((size_t)(slot0 + c) * d.heads + head) * state_image(kPanels);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    uint32_t r[32];
                    tmem_ld32(tq + (part ? kColSl : kColSh) + 32 * half, r);
                    tmem_ld_wait(r);
                    if (lane == 0) bulk_wait_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(rows + lane * 128 + ((i ^ lane) & 7) * 16) =
                            make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        bulk_store(image + (part * kPanels + half) * kTall + q * kImageRows, smem_u32(rows), kImageRows);
                        bulk_commit();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kSRead));
            if (!wait.warp(bar(kZ), it & 1)) break;
            tc_fence_after();
            uint32_t z[32];
            tmem_ld32(tq + kColX + 32 * half, z);
            tmem_ld_wait(z);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kZRead));
            if (32 * q < d.p) {
                // (the image's last part has left this place)
                if (lane == 0) bulk_wait_read<0>();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 32; ++i) reinterpret_cast<uint32_t *>(rows)[32 * i + lane] = z[i];
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bulk_store(a.z + z_at((size_t)(slot0 + c) * d.heads + head, 32 * half, 32 * q), smem_u32(rows), kImageRows);
                    bulk_commit();
                }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) out[(32 * half + i) * 128 + row] = __float2bfloat16_rn(__uint_as_float(z[i]));
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kStaged));
            if (!wait.warp(bar(kStaged), it & 1)) break;
            __nv_bfloat16 *const to = a.dv + (size_t)(first + (long long)c * kC) * a.dv_stride + (size_t)head * d.p;
            if (a.dv_vectors) {
                for (int i = tid; i < tokens * 16; i += 32 * kOutWarps) {
                    const int t = i >> 4, at = (i & 15) * 8;
                    if (at < d.p)
                        *reinterpret_cast<uint4 *>(to + (size_t)t * a.dv_stride + at) =
                            *reinterpret_cast<const uint4 *>(out + t * 128 + at);
                }
            } else {
                for (int i = tid; i < tokens * 128; i += 32 * kOutWarps) {
                    const int t = i >> 7, at = i & 127;
                    if (at < d.p) to[(size_t)t * a.dv_stride + at] = out[t * 128 + at];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kStored));
            if (!wait.warp(bar(kStored), it & 1)) break;
        }
        if (lane == 0) bulk_wait_all();
    } else {
        // the chain: a thread has a row of dS and of dU^T and Z^T
        const int q = warp & 3, part = warp >> 2;
        const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
        constexpr int kMine = kN / 4;
        const int n0 = part * kMine;
        const auto ready = [&](int which) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(which));
        };
        // the gradient of the state behind a chunk: its parts, and in fp32 decayed over the chunk
        const auto put = [&](const float (&v)[kMine], float decay) {
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
            // (waited for before the chunk's kRh)
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
        };
        const auto stage = [&](int it) { return smem + (it & 1) * Lay::kStage; };
        const auto decay_of = [&](int it) { return reinterpret_cast<const float *>(stage(it) + Lay::kRec + kRecGates)[kC - 1]; };
        float v[kMine];
        if (const float *from = source()) {
            load_rows<kMine>(reinterpret_cast<float *>(smem + Lay::kRows + warp * kStageRows), v,
                             from + (size_t)(32 * q) * d.n + n0, d.n, rows - 32 * q, d.n - n0);
        } else {
#pragma unroll
            for (int i = 0; i < kMine; ++i) v[i] = map && n0 + i == 32 * q + lane ? 1.f : 0.f;
        }
        const bool on = wait.warp(bar(kFull), 0);
        if (on) {
            const int tokens = len - (chunks - 1) * kC;
            if (tokens < kC) {
                clean_rows(smem, kPanel, 2 * kPanels + 2, tokens, threadIdx.x, 32 * kChainWarps);     // (never a map's)
                fence_proxy_async_smem();
            }
            put(v, decay_of(0));
        }
        for (int it = 0; on && it < chunks; ++it) {
            const int s = it & 1, c = chunks - 1 - it, tokens = min(kC, len - c * kC) - 16 * part;
            const float4 *gates = reinterpret_cast<const float4 *>(stage(it) + Lay::kRec + kRecGates) + 4 * part;
            float x[16], f[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float4 *>(f + 4 * i) = gates[kGateW / 4 + i];
            if (!wait.warp(bar(kE), it & 1)) break;
            tc_fence_after();
            uint32_t r[16], y[16], hi[8];
            tmem_ld16(tq + kColX + 16 * part, r);
            if (!map) tmem_ld16(tq + kColY + 16 * part, y);
            tmem_ld_wait(r);
            tmem_ld_wait(y);
            if (map) {
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = 0;
            }
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 u = ffma2(make_float2(f[i], f[i + 1]), make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                                       make_float2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])));
                x[i] = u.x;
                x[i + 1] = u.y;
            }
            if (tokens < 16) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i >= tokens) x[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) hi[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            tmem_st8(tq + kColR + 8 * part, hi);
            // Z's own term, beta dU, where the product adds the later tokens'
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float4 *>(f + 4 * i) = gates[kGateBeta / 4 + i];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 u = fmul2(make_float2(x[i], x[i + 1]), make_float2(f[i], f[i + 1]));
                r[i] = __float_as_uint(u.x);
                r[i + 1] = __float_as_uint(u.y);
            }
            tmem_st16(tq + kColX + 16 * part, r);
            ready(kRh);
#pragma unroll
            for (int i = 0; i < 8; ++i) hi[i] = rest2(x[2 * i], x[2 * i + 1], hi[i]);
            tmem_st8(tq + kColRl + 8 * part, hi);
            ready(kRl);
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float4 *>(f + 4 * i) = gates[i];
            if (!wait.warp(bar(kZ), it & 1)) break;
            tc_fence_after();
            tmem_ld16(tq + kColX + 16 * part, r);
            tmem_ld_wait(r);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 u = fmul2(make_float2(-f[i], -f[i + 1]), make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])));
                x[i] = u.x;
                x[i + 1] = u.y;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) hi[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            tmem_st8(tq + kColR + 8 * part, hi);
            ready(kWh);
#pragma unroll
            for (int i = 0; i < 8; ++i) hi[i] = rest2(x[2 * i], x[2 * i + 1], hi[i]);
            tmem_st8(tq + kColRl + 8 * part, hi);
            ready(kWl);
            if (lane == 0) mbar_arrive(bar(kEmpty + s));
            const bool more = it + 1 < chunks;
            if (more && !wait.warp(bar(kFull + (s ^ 1)), ((it + 1) >> 1) & 1)) break;
            const float decay = more ? decay_of(it + 1) : 1.f;
            // (dS's parts have been read by the output's warps)
            if (!wait.warp(bar(kS), it & 1) || (!kEnds && !wait.warp(bar(kSRead), it & 1))) break;
            tc_fence_after();
            uint32_t m[kMine];
            if constexpr (kMine == 32) tmem_ld32(tq + kColS + n0, m);
            else tmem_ld16(tq + kColS + n0, m);
            tmem_ld_wait(m);
            float v[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i) v[i] = __uint_as_float(m[i]);
            if (more) put(v, decay);
            else if (float *const to = target())        // (by way of the last chunk's keys, queries and dO, which are used up)
                store_rows<kMine>(reinterpret_cast<float *>(stage(it) + warp * kStageRows), v,
                                  to + (size_t)(32 * q) * d.n + n0, d.n, rows - 32 * q, d.n - n0);
        }
    }
    // copies in flight land before the CTA ends
    if (warp == kLoadWarp) {
        for (int it = loaded > 2 ? loaded - 2 : 0; it < loaded; ++it)
            if (!mbar_wait(bar(kFull + (it & 1)), (it >> 1) & 1, kSsdDefaultWaitNs)) ssd_report(a.err, SSD_DEVERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------ a chunk's other gradients
// Steps of products and of elementwise work by turns, all warps together: with 224 KB of
// tiles one CTA an SM.  What is loaded first (a state, Z) is asked for at once, and what the
// CTA that comes next on this SM will load is brought into L2 meanwhile.
constexpr int kGradWarps = 16, kGradThreads = 32 * kGradWarps;
template <int kPanels>
struct GradSmem {
    static constexpr uint32_t kQk = 0;                          // panels of queries over keys
    static constexpr uint32_t kAh = kQk + kPanels * kTall;      // dO over Z's rounded part, then dS's
    static constexpr uint32_t kAl = kAh + 2 * kTall;            // nothing over what rounding left of Z, or of dS
    static constexpr uint32_t kU = kAl + 2 * kTall;             // U's parts
    static constexpr uint32_t kSs = kU + 4 * kPanel;            // the parts of S, [P][N]; then scratch
    static constexpr uint32_t kW = kSs + 4 * kTall;             // V and T; then the parts of dP and of dA
    static constexpr uint32_t kCtl = kW + 4 * kPanel;
    static constexpr uint32_t kGatesAt = kCtl + 64;
    static constexpr uint32_t kShareAt = kGatesAt + kGates * 4;     // of beta in the record's (kLeastBeta), by tokens
    static constexpr uint32_t kBytes = kShareAt + kC * 4;
    // scratch, where S was (floats)
    static constexpr int kRowSum = 0, kColSum = 512, kAhead = 768, kBehind = 1024, kDbeta = 1280, kWhole = 1536;
};

struct GradTc {
    SsdDelta d;
    const uint8_t *records;
    const float *checkpoints, *z;
    const uint8_t *dstate;
    __nv_bfloat16 *dq, *dk;             // where a group is one head; else sums by head:
    float *dq_heads, *dk_heads;         // [token][head][N]
    long long dq_stride, dk_stride;
    bool vectors;                       // whether their rows start on 16 bytes
    float *dg, *dbeta;
    int ahead;                          // how many CTAs on the next on an SM is
    unsigned *err;
};

// The sums over the warp's lanes of kCount (16 or 32) values a lane: lane l's answer is that
// of value l % kCount.
template <int kCount>
__device__ __forceinline__ float lanes_transposed_sum(float (&v)[kCount], int lane) {
    if constexpr (kCount == 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
    }
#pragma unroll
    for (int o = kCount / 2; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    return v[0];
}

template <int kPanels>
__global__ void __launch_bounds__(kGradThreads, 1)
delta_grad_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                     const __grid_constant__ CUtensorMap mapV, const __grid_constant__ CUtensorMap mapDo, const GradTc a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using Lay = GradSmem<kPanels>;
    const SsdDelta &d = a.d;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int q = warp & 3, c0 = 16 * (warp >> 2);      // lanes of tensor memory, and the warp's columns
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) {
        if (threadIdx.x == 0) ssd_report(a.err, SSD_DEVERR_SMEM_ALIGN);
        return;
    }
    const long long slot = blockIdx.x / d.heads;
    const int head = (int)(blockIdx.x % d.heads), group = head / (d.heads / d.groups);
    const ChunkAt at = chunk_at(d, slot);
    if (!at.live) return;
    const int valid = min(kC, at.len - at.chunk * kC);
    const long long token = at.first + (long long)at.chunk * kC;
    const size_t record = (size_t)slot * d.heads + head, size = (size_t)d.p * d.n;
    const uint32_t full = base + Lay::kCtl, done = full + 8, second = full + 16;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + Lay::kCtl + 24);
    if (threadIdx.x == 0) {
        mbar_init(full, 1);
        mbar_init(done, 1);
        mbar_init(second, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(full, kPanels * kTall + 2 * kPanel + 64 * 256 + 2 * kPanel + kGates * 4);
        const int t = (int)token;
#pragma unroll
        for (int p = 0; p < kPanels; ++p) {
            tma_load_3d(base + Lay::kQk + p * kTall, &mapQ, full, 64 * p, group, t);
            tma_load_3d(base + Lay::kQk + p * kTall + kPanel, &mapK, full, 64 * p, group, t);
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) tma_load_3d(base + Lay::kAh + p * kTall, &mapDo, full, 64 * p, head, t);
        tma_load_3d(base + Lay::kW, &mapV, full, 0, head, t);
        bulk_load(base + Lay::kW + 2 * kPanel, a.records + record * kRecord + kRecT, 2 * kPanel, full);
        bulk_load(base + Lay::kGatesAt, a.records + record * kRecord + kRecGates, kGates * 4, full);
    }
    // A token whose beta is below kLeastBeta has that in its record, so that dbeta can be had of
    // Z and U; what reaches other tokens and the gradients of q, k and g is its beta's share of U.
    if (threadIdx.x < kC) {
        const float beta = threadIdx.x < valid ? d.beta[(size_t)(token + threadIdx.x) * d.heads + head] : 1.f;
        reinterpret_cast<float *>(smem + Lay::kShareAt)[threadIdx.x] = fabsf(beta) < kLeastBeta ? fabsf(beta) / kLeastBeta : 1.f;
    }
    // a state's row by a warp: lane l has the columns 4 l .. 4 l + 3; a part's panel is tall
    const bool mine = 4 * lane < d.n;
    const auto load_state = [&](const float *m, int row) {
        return mine && row < d.p ? __ldcs(reinterpret_cast<const float4 *>(m + (size_t)row * d.n + 4 * lane))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    const uint32_t state_panel = Lay::kSs + (uint32_t)(lane >> 4) * kTall;
    const auto store_state = [&](int row, float4 v) {
        if (64 * kPanels <= 4 * lane) return;
        const uint32_t to = state_panel + panel_at(row, (4 * lane) & 63);
        const Split x = split2(v.x, v.y), y = split2(v.z, v.w);
        *reinterpret_cast<uint2 *>(smem + to) = make_uint2(x.hi, y.hi);
        *reinterpret_cast<uint2 *>(smem + to + kPanels * kTall) = make_uint2(x.lo, y.lo);
    };
    {
        float4 v[8], z[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = load_state(a.checkpoints + record * size, 8 * warp + i);
        // Z, a token a row
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * warp + i, p = 4 * lane;
            z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < valid && p < d.p)       // (P is a multiple of 8)
                z[i] = *reinterpret_cast<const float4 *>(a.z + z_at(record, t, p));
        }
        if (warp == 1) {
            tmem_alloc(smem_u32(tslot), 512);
            tmem_relinquish();
        }
        const long long next = (long long)blockIdx.x + a.ahead;
        if (warp == 2 && next < gridDim.x) {
            const long long slot2 = next / d.heads;
            const int head2 = (int)(next % d.heads), group2 = head2 / (d.heads / d.groups);
            const ChunkAt at2 = chunk_at(d, slot2);
            if (at2.live && elect_one()) {
                const int t = (int)(at2.first + (long long)at2.chunk * kC);
                bulk_prefetch_l2(a.checkpoints + (size_t)next * size, (uint32_t)(size * 4));
                bulk_prefetch_l2(a.dstate + (size_t)next * state_image(kPanels), state_image(kPanels));
                bulk_prefetch_l2(a.records + (size_t)next * kRecord, kRecord);
                bulk_prefetch_l2(a.z + (size_t)next * kZTile, kZTile * 4);
#pragma unroll
                for (int p = 0; p < kPanels; ++p) {
                    tma_prefetch_l2_3d(&mapQ, 64 * p, group2, t);
                    tma_prefetch_l2_3d(&mapK, 64 * p, group2, t);
                }
#pragma unroll
                for (int p = 0; p < 2; ++p) tma_prefetch_l2_3d(&mapDo, 64 * p, head2, t);
                tma_prefetch_l2_3d(&mapV, 0, head2, t);
            }
            __syncwarp();
        }
        for (int i = threadIdx.x; i < 1024; i += kGradThreads)
            *reinterpret_cast<uint4 *>(smem + Lay::kAl + (i >> 9) * kTall + (i & 511) * 16) = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) store_state(8 * warp + i, v[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t to = (uint32_t)(lane >> 4) * kTall + panel_at(64 + 4 * warp + i, (4 * lane) & 63);
            const Split x = split2(z[i].x, z[i].y), y = split2(z[i].z, z[i].w);
            *reinterpret_cast<uint2 *>(smem + Lay::kAh + to) = make_uint2(x.hi, y.hi);
            *reinterpret_cast<uint2 *>(smem + Lay::kAl + to) = make_uint2(x.lo, y.lo);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot, tq = tmem + ((uint32_t)(32 * q) << 16);
    // (waits for the CTA's own copies and products)
    if (!mbar_wait(full, 0, kSsdDefaultWaitNs)) ssd_report(a.err, SSD_DEVERR_TIMEOUT);
    clean_rows(smem + Lay::kQk, kPanel, 2 * kPanels, valid, threadIdx.x, kGradThreads);
    clean_rows(smem + Lay::kAh, kTall, 2, valid, threadIdx.x, kGradThreads);
    const bool issuer = warp == 0;
    uint32_t phase = 0;
    // what all threads wrote is there for the products, and what the products leave for all
    const auto before = [&] {
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    const auto after = [&] {
        __syncwarp();
        if (!mbar_wait(done, phase, kSsdDefaultWaitNs)) ssd_report(a.err, SSD_DEVERR_TIMEOUT);
        phase ^= 1;
        tc_fence_after();
    };
    constexpr uint32_t kId = idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t kColU = 0, kColQk = 64, kColM = 128, kColDoS = 192, kColZs = 256, kColPk = 320, kColSum = 384,
                       kColUs = 448, kColR = 448, kColRl = 480;
    static_assert(kColZs == kColDoS + 64, "one product of 128 columns");
    const uint32_t sh = base + Lay::kSs, sl = sh + kPanels * kTall, ah = base + Lay::kAh, al = base + Lay::kAl;
    const uint32_t uh = base + Lay::kU, ul = uh + 2 * kPanel, w = base + Lay::kW, qk = base + Lay::kQk;
    // D (+)= A B^T over `panels` of 64 columns: A by tall panels, B by panels `bstep` apart
    const auto rows_rows = [&](uint32_t dcol, uint32_t at_a, uint32_t at_b, uint32_t bstep, int panels, bool add) {
        for (int p = 0; p < panels; ++p) {
            const uint64_t ad = smem_desc(at_a + p * kTall, 16, 1024, kSwizzle128B);
            const uint64_t bd = smem_desc(at_b + p * bstep, 16, 1024, kSwizzle128B);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ss(tmem + dcol, ad + kStepK * k, bd + kStepK * k, kId, add || p + k > 0);
        }
    };
    // D (+)= A^T B^T: A [128 of P][N] by tall panels of N, B [rows][P] by panels `bstep` apart
    const auto cols_rows = [&](uint32_t dcol, uint32_t at_a, uint32_t at_b, uint32_t bstep, uint32_t id, bool add) {
        const uint64_t ad = smem_desc(at_a, kTall, 1024, kSwizzle128B);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint64_t bd = smem_desc(at_b + p * bstep, 16, 1024, kSwizzle128B);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ss(tmem + dcol, ad + kStepMn * (4 * p + k), bd + kStepK * k, id, add || p + k > 0);
        }
    };
    constexpr uint32_t kIdMn = idesc_bf16_f32(128, 64, true, false), kIdMnWide = idesc_bf16_f32(128, 128, true, false);
    // D (+)= A^T M^T (columns of D from 16 k on) and A^T M (up to 16 k + 15) of a lower
    // triangular M [64][64], A [64][N]
    const auto tokens_lower = [&](uint32_t dcol, uint32_t at_a, uint32_t at_m, bool add) {
        const uint64_t ad = smem_desc(at_a, kTall, 1024, kSwizzle128B), bd = smem_desc(at_m, 16, 1024, kSwizzle128B);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mma_ss(tmem + dcol + 16 * k, ad + kStepMn * k, bd + kStepK * k + kStepMn * k,
                   idesc_bf16_f32(128, 64 - 16 * k, true, false), add || k > 0);
    };
    const auto tokens_upper = [&](uint32_t dcol, uint32_t at_a, uint32_t at_m, bool add) {
        const uint64_t ad = smem_desc(at_a, kTall, 1024, kSwizzle128B), bd = smem_desc(at_m, kPanel, 1024, kSwizzle128B);
#pragma unroll
        for (int k = 3; k >= 0; --k)
            mma_ss(tmem + dcol, ad + kStepMn * k, bd + kStepMn * k, idesc_bf16_f32(128, 16 * k + 16, true, true), add || k < 3);
    };
    const float *gates = reinterpret_cast<const float *>(smem + Lay::kGatesAt);
    // the gates of the warp's 16 tokens (kGates: their betas' shares)
    static_assert(Lay::kShareAt == Lay::kGatesAt + kGates * 4, "behind the gates");
    const auto gates_of = [&](int which, float (&f)[16]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4 *>(f + 4 * i) = *reinterpret_cast<const float4 *>(gates + which + c0 + 4 * i);
    };
    float *const scratch = reinterpret_cast<float *>(smem + Lay::kSs);

    // K S^T by the state's rows; Q K^T over K K^T
    before();
    if (issuer && elect_one()) {
        rows_rows(kColU, sh, qk + kPanel, kTall, kPanels, false);
        rows_rows(kColU, sl, qk + kPanel, kTall, kPanels, true);
        rows_rows(kColQk, qk, qk + kPanel, kTall, kPanels, false);
        mma_commit(done);
    }
    const int row = 32 * q + lane;
    // Z as it is, for its products with U: dbeta (their parts' product would lose some of it)
    float zu[16], own;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        zu[i] = c0 + i < valid && row < d.p ? a.z[z_at(record, c0 + i, row)] : 0.f;
    after();
    // R, as the left operand of U (a token's share of it), and beta R, to which that product is added
    {
        uint32_t r[16], hi[8], lo[8];
        tmem_ld16(tq + kColU + c0, r);
        tmem_ld_wait(r);
        const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(smem + Lay::kW) + c0 * 128 + row;
        float gamma[16], beta[16], share[16];
        gates_of(0, gamma);
        gates_of(kGateBeta, beta);
        gates_of(kGates, share);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = 2 * i + j;
                x[j] = __bfloat162float(v[t * 128]) - gamma[t] * __uint_as_float(r[t]);
                if (c0 + t >= valid) x[j] = 0.f;
                r[t] = __float_as_uint(x[j] * beta[t]);
            }
            const Split y = split2(x[0] * share[2 * i], x[1] * share[2 * i + 1]);
            hi[i] = y.hi;
            lo[i] = y.lo;
        }
        tmem_st8(tq + kColR + c0 / 2, hi);
        tmem_st8(tq + kColRl + c0 / 2, lo);
        tmem_st16(tq + kColU + c0, r);
        tmem_st_wait();
    }
    before();
    if (issuer && elect_one()) {
        const auto triangle = [&](uint32_t acol, uint32_t tile) {
            const uint64_t bd = smem_desc(tile, 16, 1024, kSwizzle128B);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_ts(tmem + kColU + 16 * k, tmem + acol + 8 * k, bd + kStepK * k + kStepMn * k,
                       idesc_bf16_f32(128, 64 - 16 * k, false, false), 1);
        };
        triangle(kColR, w + 2 * kPanel);
        triangle(kColR, w + 3 * kPanel);
        triangle(kColRl, w + 2 * kPanel);
        mma_commit(done);
        // (dO S)^T beside (Z S)^T, while U goes to shared memory
        cols_rows(kColDoS, sh, ah, kTall, kIdMnWide, false);
        cols_rows(kColDoS, sl, ah, kTall, kIdMnWide, true);
        cols_rows(kColZs, sh, al + kPanel, kTall, kIdMn, true);
    }
    after();
    // U by tokens
    {
        uint32_t r[16];
        tmem_ld16(tq + kColU + c0, r);
        tmem_ld_wait(r);
        uint8_t *const to = smem + Lay::kU + (row >> 6) * kPanel;
        float share[16];
        gates_of(kGates, share);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const Split x = split2(__uint_as_float(r[i]) * share[i], __uint_as_float(r[i + 1]) * share[i + 1]);
            zu[i] *= __uint_as_float(r[i]);
            zu[i + 1] *= __uint_as_float(r[i + 1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t o = panel_at(c0 + i + j, row & 63);
                *reinterpret_cast<uint16_t *>(to + o) = (uint16_t)(x.hi >> (16 * j));
                *reinterpret_cast<uint16_t *>(to + 2 * kPanel + o) = (uint16_t)(x.lo >> (16 * j));
            }
        }
        own = lanes_transposed_sum(zu, lane);
    }
    before();
    if (issuer && elect_one()) {
        // M1 over M2
        rows_rows(kColM, ah, uh, kPanel, 2, false);
        rows_rows(kColM, ah, ul, kPanel, 2, true);
        rows_rows(kColM, al, uh, kPanel, 2, true);
        mma_commit(done);
    }
    after();
    // dS in the place of dO and Z
    if (threadIdx.x == 0) {
        const uint8_t *from = a.dstate + record * state_image(kPanels);
        mbar_arrive_expect_tx(second, state_image(kPanels));
        bulk_load(ah, from, kPanels * kTall, second);
        bulk_load(al, from + kPanels * kTall, kPanels * kTall, second);
    }
    // dP (lanes 0 .. 63) and dA (64 .. 127), a row a lane; and what pairs of tokens add to dg
    float sum = 0.f, col;
    float2 both = make_float2(0.f, 0.f);
    {
        const int r = row & 63;
        const bool keys = q >= 2;
        uint32_t m[16], x[16];
        tmem_ld16(tq + kColM + c0, m);
        tmem_ld16(tq + kColQk + c0, x);
        const float2 *sums = reinterpret_cast<const float2 *>(gates + kGateSums);
        const float2 mine_ = sums[r], whole = sums[31];
        const bool over = r >= 32 && c0 < 32;       // from the first half of the tokens to the second
        const int last = r < valid ? (keys ? r - 1 : r) : -1;
        const float factor = keys ? -1.f : d.scale;
        tmem_ld_wait(m);
        tmem_ld_wait(x);
        float v[16], e[16];
        const float4 *const columns = reinterpret_cast<const float4 *>(sums + c0);
        const float2 less = make_float2(-1.f, -1.f), by = make_float2(factor, factor);
        // (over: what the row has summed up and what is left of the first half behind the column)
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const float4 c = columns[j / 2];
            const float2 from = over ? whole : mine_;
            float2 g0 = ffma2(make_float2(c.x, c.y), less, from), g1 = ffma2(make_float2(c.z, c.w), less, from);
            const float more = over ? mine_.x + mine_.y : 0.f;
            const float2 m2 = fmul2(fmul2(make_float2(ex2_approx(more + (g0.x + g0.y)), ex2_approx(more + (g1.x + g1.y))), by),
                                    make_float2(__uint_as_float(m[j]), __uint_as_float(m[j + 1])));
            const float2 e2 = fmul2(m2, make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])));
            v[j] = c0 + j <= last ? m2.x : 0.f;
            v[j + 1] = c0 + j + 1 <= last ? m2.y : 0.f;
            e[j] = c0 + j <= last && c0 + j < r ? e2.x : 0.f;
            e[j + 1] = c0 + j + 1 <= last && c0 + j + 1 < r ? e2.y : 0.f;
            sum += e[j] + e[j + 1];
        }
        uint8_t *const to = smem + Lay::kW + (keys ? 2 * kPanel : 0);
        put_parts(to, panel_at(r, c0), v);
        put_parts(to, panel_at(r, c0 + 8), v + 8);
        col = lanes_transposed_sum(e, lane);
    }
    // <S, dS>: both lie alike
    if (!mbar_wait(second, 0, kSsdDefaultWaitNs)) ssd_report(a.err, SSD_DEVERR_TIMEOUT);
    for (uint32_t i = threadIdx.x * 16; i < kPanels * kTall; i += kGradThreads * 16) {
        const auto pairs = [&](uint32_t hi, uint32_t lo, float2 (&x)[4]) {
            const uint4 h = *reinterpret_cast<const uint4 *>(smem + hi + i), l = *reinterpret_cast<const uint4 *>(smem + lo + i);
            const uint32_t a_[4] = {h.x, h.y, h.z, h.w}, b_[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = fadd2(make_float2(__uint_as_float(a_[j] << 16), __uint_as_float(a_[j] & 0xffff0000u)),
                             make_float2(__uint_as_float(b_[j] << 16), __uint_as_float(b_[j] & 0xffff0000u)));
        };
        float2 x[4], y[4];
        pairs(Lay::kSs, Lay::kSs + kPanels * kTall, x);
        pairs(Lay::kAh, Lay::kAl, y);
#pragma unroll
        for (int j = 0; j < 4; ++j) both = ffma2(x[j], y[j], both);
    }
    float dot = both.x + both.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    before();
    if (issuer && elect_one()) {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const uint32_t dp = w + part * kPanel, da = w + (2 + part) * kPanel;
            tokens_lower(kColPk, qk + kPanel, dp, part > 0);
            tokens_upper(kColSum, qk, dp, part > 0);
            tokens_lower(kColSum, qk + kPanel, da, true);
            tokens_upper(kColSum, qk + kPanel, da, true);
        }
        cols_rows(kColUs, ah, uh, kPanel, kIdMn, false);
        cols_rows(kColUs, al, uh, kPanel, kIdMn, true);
        cols_rows(kColUs, ah, ul, kPanel, kIdMn, true);
        mma_commit(done);
    }
    // (S is used up: scratch)
    scratch[Lay::kRowSum + (q >= 2 ? 256 : 0) + 4 * c0 + (row & 63)] = sum;
    if (lane < 16) {
        scratch[Lay::kColSum + (q >= 2 ? 128 : 0) + 64 * (q & 1) + c0 + lane] = col;
        scratch[Lay::kDbeta + 64 * q + c0 + lane] = own;
    }
    if (lane == 0) scratch[Lay::kWhole + warp] = dot;
    // meanwhile what tokens read of S, dotted with them: a lane is a column of dQ and dK
    const bool on = row < d.n;
    const uint8_t *const keys = smem + Lay::kQk + (row >> 6) * kTall;
    float dots[32], dq[16], dk[16];
    {
        uint32_t x[16], y[16];
        float gamma[16];
        gates_of(0, gamma);
        tmem_ld16(tq + kColDoS + c0, x);
        tmem_ld16(tq + kColZs + c0, y);
        tmem_ld_wait(x);
        tmem_ld_wait(y);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            dq[i] = d.scale * gamma[i] * __uint_as_float(x[i]);
            dk[i] = -gamma[i] * __uint_as_float(y[i]);
            dots[i] = dots[16 + i] = 0.f;
            if (on) {
                const uint32_t o = panel_at(c0 + i, row & 63);
                const float qv = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(keys + o));
                const float kv = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(keys + kPanel + o));
                dots[i] = dq[i] * qv + dk[i] * kv;
                dots[16 + i] = kv;
            }
        }
    }
    after();
    {
        uint32_t x[16], y[16];
        float w[16];
        gates_of(kGateW, w);
        tmem_ld16(tq + kColUs + c0, x);
        tmem_ld16(tq + kColPk + c0, y);
        tmem_ld_wait(x);
        tmem_ld_wait(y);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float u = w[i] * __uint_as_float(x[i]);
            dk[i] += u;
            dots[16 + i] = on ? dots[16 + i] * u : 0.f;
            dq[i] += __uint_as_float(y[i]);
        }
        tmem_ld16(tq + kColSum + c0, x);
        tmem_ld_wait(x);
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[i] += __uint_as_float(x[i]);
        // by way of shared memory, in the places of dS's parts, which are used up
        if (on && a.dq == nullptr) {
            float *const to = reinterpret_cast<float *>(smem + Lay::kAh) + c0 * 128 + row;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                to[i * 128] = dq[i];
                to[i * 128 + kTall / 2] = dk[i];
            }
        } else if (on) {
            __nv_bfloat16 *const to = reinterpret_cast<__nv_bfloat16 *>(smem + Lay::kAh) + c0 * 128 + row;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                to[i * 128] = __float2bfloat16_rn(dq[i]);
                to[i * 128 + kTall / 2] = __float2bfloat16_rn(dk[i]);
            }
        }
        const float sum = lanes_transposed_sum(dots, lane);
        scratch[(lane < 16 ? Lay::kAhead : Lay::kBehind) + 64 * q + c0 + (lane & 15)] = sum;
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp >= kGradWarps - 4) {
        // the rows of dQ, then of dK
        const auto rows = [&](int i, auto store) {
            const int t = i & 63;
            if (t >= valid) return;
            if (a.dq == nullptr)
                store((i < 64 ? a.dq_heads : a.dk_heads) + ((size_t)(token + t) * d.heads + head) * d.n,
                      Lay::kAh + (uint32_t)i * 512, d.n * 4);
            else
                store((i < 64 ? a.dq + (size_t)(token + t) * a.dq_stride : a.dk + (size_t)(token + t) * a.dk_stride) + group * d.n,
                      Lay::kAh + (uint32_t)i * 256, d.n * 2);
        };
        if (a.vectors) {
            rows(threadIdx.x & 127, [&](void *to, uint32_t from, uint32_t bytes) { bulk_store(to, base + from, bytes); });
            bulk_commit();
            bulk_wait_read<0>();
        } else {
            for (int i = warp & 3; i < 128; i += 4)
                rows(i, [&](void *to, uint32_t from, uint32_t bytes) {
                    for (uint32_t j = lane; j < bytes / 2; j += 32)
                        static_cast<uint16_t *>(to)[j] = reinterpret_cast<const uint16_t *>(smem + from)[j];
                });
        }
    }
    if (warp == 0) {
        // lane l: tokens 2 l and 2 l + 1
        float whole = lane < kGradWarps ? scratch[Lay::kWhole + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) whole += __shfl_xor_sync(0xffffffffu, whole, o);
        float from[2], into[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float *s = scratch + 2 * lane + i;
            float rows = 0.f, cols = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) rows += s[Lay::kRowSum + 64 * j];
#pragma unroll
            for (int j = 0; j < 4; ++j) cols += s[Lay::kColSum + 64 * j];
            from[i] = (rows - cols) + ((s[Lay::kAhead] + s[Lay::kAhead + 64]) + (s[Lay::kAhead + 128] + s[Lay::kAhead + 192]));
            into[i] = (s[Lay::kBehind] + s[Lay::kBehind + 64]) + (s[Lay::kBehind + 128] + s[Lay::kBehind + 192]);
        }
        // of `from` the sum from the token on, of `into` that of the tokens before it
        float ahead = from[0] + from[1], behind = into[0] + into[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_down_sync(0xffffffffu, ahead, o), y = __shfl_up_sync(0xffffffffu, behind, o);
            if (lane + o < 32) ahead += x;
            if (lane >= o) behind += y;
        }
        const float next = __shfl_down_sync(0xffffffffu, ahead, 1), before_ = __shfl_up_sync(0xffffffffu, behind, 1);
        const float past = lane ? before_ : 0.f, rest = lane < 31 ? next : 0.f;
        const float dg[2] = {ahead + past, (rest + from[1]) + (past + into[0])};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            if (t >= valid) continue;
            const size_t o = (size_t)(token + t) * d.heads + head;
            const float *b = scratch + Lay::kDbeta + t, be = gates[kGateBeta + t];
            a.dg[o] = dg[i] + gates[kC - 1] * whole;
            a.dbeta[o] = ((b[0] + b[64]) + (b[128] + b[192])) / be / be;
        }
    }
    if (warp == 1) tmem_dealloc(tmem, 512);
}

struct Plan {
    size_t records, z, dstate, dq, dk, parts, total;
};
Plan plan_of(const SsdDelta &d, int sms) {
    const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t slots = (size_t)ssd_delta_slots(d.tokens, d.nseq), tokens = (size_t)d.tokens;
    Plan p;
    p.records = 0;
    p.z = up(slots * d.heads * kRecord);
    p.dstate = p.z + up(slots * d.heads * kZTile * 4);
    p.dq = p.dstate + up(slots * d.heads * state_image(d.n <= 64 ? 1 : 2));
    p.dk = p.dq + (d.heads == d.groups ? 0 : up(tokens * d.heads * d.n * 4));
    p.parts = p.dk + (d.heads == d.groups ? 0 : up(tokens * d.heads * d.n * 4));
    p.total = p.parts + parts_of(d, segments_of(d, sms).parts, nullptr).bytes;
    return p;
}

template <int kPanels>
cudaError_t launch(const SsdDeltaBwd &b, void *ws, int sms, unsigned *err, cudaStream_t stream) {
    const SsdDelta &d = b.in;
    CUtensorMap q, k, v, o;
    if (!make_map(&q, d.q, d.n, d.groups, d.tokens, d.q_stride, 64, true) ||
        !make_map(&k, d.k, d.n, d.groups, d.tokens, d.k_stride, 64, true) ||
        !make_map(&v, d.v, d.p, d.heads, d.tokens, d.v_stride, 128, false) ||
        !make_map(&o, b.dout, d.p, d.heads, d.tokens, b.do_stride, 64, true))
        return cudaErrorInvalidValue;
    const SsdDebug debug = ssd_debug_config();
    const Plan plan = plan_of(d, sms);
    const auto at = [&](size_t offset) { return static_cast<char *>(ws) + offset; };
    uint8_t *records = reinterpret_cast<uint8_t *>(at(plan.records));
    float *z = reinterpret_cast<float *>(at(plan.z));
    uint8_t *dstate = reinterpret_cast<uint8_t *>(at(plan.dstate));
    cudaError_t e = launch_chunks(d, records, true, sms, err, stream);
    if (e != cudaSuccess) return e;
    using Back = BackSmem<kPanels>;
    using Grad = GradSmem<kPanels>;
    static_assert(Back::kBytes <= 232448 && Grad::kBytes <= 232448, "more than 227 KB of shared memory");
    e = cudaFuncSetAttribute(delta_back_tc_kernel<kPanels, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Back::kBytes);
    if (e != cudaSuccess) return e;
    const InParts segments = segments_of(d, sms);
    const Parts parts = parts_of(d, segments.parts, reinterpret_cast<uint8_t *>(at(plan.parts)));
    BackTc w{d, records, b.dfinal, static_cast<__nv_bfloat16 *>(b.dv), b.dv_stride,
             ((uintptr_t)b.dv & 15u) == 0 && b.dv_stride % 8 == 0, b.dinit, z, dstate,
             segments.parts, -segments.half, parts.starts, parts.maps, err, debug.wait_ns,
             debug.fault == kSsdFaultWithholdSignal};
    const long long walks = (long long)d.nseq * d.heads;
    if (segments.parts > 1) {
        e = cudaFuncSetAttribute(delta_back_tc_kernel<kPanels, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Back::kBytes);
        if (e != cudaSuccess) return e;
        const long long jobs = walks * (2 * segments.parts - 3);
        delta_back_tc_kernel<kPanels, true><<<(unsigned)jobs, kBackThreads, Back::kBytes, stream>>>(q, k, o, w);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = launch_join(d, b.dfinal, segments, w.half, parts, sms, err, stream)) != cudaSuccess) return e;
        w.d.cu = parts.cu;
        w.d.nseq *= segments.parts;
    }
    delta_back_tc_kernel<kPanels, false><<<(unsigned)(walks * segments.parts), kBackThreads, Back::kBytes, stream>>>(q, k, o, w);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = cudaFuncSetAttribute(delta_grad_tc_kernel<kPanels>, cudaFuncAttributeMaxDynamicSharedMemorySize, Grad::kBytes);
    if (e != cudaSuccess) return e;
    const bool one = d.heads == d.groups;
    const GradTc g{d, records, b.checkpoints, z, dstate, one ? static_cast<__nv_bfloat16 *>(b.dq) : nullptr,
                   one ? static_cast<__nv_bfloat16 *>(b.dk) : nullptr, reinterpret_cast<float *>(at(plan.dq)),
                   reinterpret_cast<float *>(at(plan.dk)), b.dq_stride, b.dk_stride,
                   !one || (on_16(b.dq) && on_16(b.dk) && b.dq_stride % 8 == 0 && b.dk_stride % 8 == 0), b.dg, b.dbeta, sms, err};
    const long long ctas = ssd_delta_slots(d.tokens, d.nseq) * d.heads;
    delta_grad_tc_kernel<kPanels><<<(unsigned)ctas, kGradThreads, Grad::kBytes, stream>>>(q, k, v, o, g);
    if ((e = cudaGetLastError()) != cudaSuccess || one) return e;
    return ssd_launch_delta_group_sums(g.dq_heads, b.dq, b.dq_stride, g.dk_heads, b.dk, b.dk_stride, d, d.heads / d.groups, stream);
}

}  // namespace

bool ssd_delta_tc_bwd_sizes(const SsdDelta &d) { return ssd_delta_tc_sizes(d) && d.p <= 128; }
bool ssd_delta_tc_bwd_handles(const SsdDeltaBwd &b) {
    return ssd_delta_tc_bwd_sizes(b.in) && ssd_delta_tc_inputs(b.in) && on_16(b.dout) && b.do_stride % 8 == 0 &&
           on_16(b.checkpoints) && on_16(b.dfinal) && on_16(b.dinit);
}
size_t ssd_delta_tc_bwd_workspace(const SsdDelta &d, int sms) {
    return ssd_delta_tc_bwd_sizes(d) ? plan_of(d, sms).total : 0;
}

cudaError_t ssd_launch_delta_bwd_tc(const SsdDeltaBwd &a, void *ws, int sms, unsigned *err, cudaStream_t stream) {
    return a.in.n <= 64 ? launch<1>(a, ws, sms, err, stream) : launch<2>(a, ws, sms, err, stream);
}
