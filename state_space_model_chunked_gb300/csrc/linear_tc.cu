// The matrix product on the 5th-generation tensor cores, bf16 or E4M3 inputs:
//
//   out[m][n] = act(sum_k A(m,k) B(n,k) a_scale[m] b_scale[n] + bias[n]) + residual[m][n]
//
// A CTA computes tiles of 128 x kBN: a producer warp brings 128-byte-wide
// blocks of both operands into a ring of shared-memory stages by TMA (rows
// past an end read as zero), an issuer warp multiplies them into a TMEM
// accumulator, and eight epilogue warps read that back, one TMEM lane (a row
// of A) a thread, and apply scales, bias, activation and residual on the way
// to global memory.
//   Operands lie with k contiguous (K-major) or with their rows contiguous
// (MN-major, the gradients' transposed operands); both use 128-byte swizzled
// tiles.  kSwap takes the weights as A and the tokens as B, for few tokens:
// then a lane is a feature, and the rows of B are only as many as needed.
//   Without kSplit a CTA walks over tiles with two accumulators, so a tile's
// epilogue runs under the next one's products.  With kSplit the k axis of one
// tile is split over a cluster of CTAs and their sums are joined through
// distributed shared memory, in rank order.  That exchange is bound by the
// distributed reads, about 20 bytes a clock into an SM.
//   Measured (time on the GPU): 65536 x 5120 -> 2560 in bf16 with bias, silu and
// residual 1065 to 1090 us (1.6 PFLOP/s, under the power limit; 0.94 of a library
// product's sustained rate), both gradients of 16376 x 1024 -> 2048 86 us (1.6 PFLOP/s),
// 4001 x 768 -> 1536 in 8 bits 14.3 us, 512 x 2560 -> 2560 in bf16 12.9 us.  A product of
// few tiles has a fixed cost: 1 us before the first load, which the kernel in front
// in the stream hides, 1.2 us for its data, 0.6 us at the end, and with k split about 4 us
// for the exchange.  Where tiles take few k blocks the epilogue bounds them, with and
// without an activation: 21375 x 688 -> 9632 263 us with silu and 275 without (a library
// product's burst rate would make it 147), 4096 x 688 -> 4096 26 us.
#include <cuda.h>

#include <algorithm>
#include <limits>

#include "../../include/ssd.h"
#include "act.cuh"
#include "answers.h"
#include "launch.h"
#include "ptx.cuh"
#include "vec.cuh"

using namespace ssdptx;

namespace {

constexpr int kBM = 128;
constexpr int kRowBytes = 128;                  // a block's k extent
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);  // producer, issuer, epilogue
constexpr uint32_t kABytes = kBM * kRowBytes;
constexpr uint32_t kRingBytes = 196608;
constexpr uint32_t kCtrlBytes = 1024;
constexpr int kMaxStages = 12;

constexpr uint32_t stage_bytes(int bn) { return kABytes + bn * kRowBytes; }
constexpr int stages(int bn) {
    return kRingBytes / stage_bytes(bn) < kMaxStages ? kRingBytes / stage_bytes(bn) : kMaxStages;
}
constexpr uint32_t tmem_cols(int bn, bool split) {
    const int want = split ? bn : 2 * bn;
    return want <= 32 ? 32 : want <= 64 ? 64 : want <= 128 ? 128 : want <= 256 ? 256 : 512;
}

struct Args {
    SsdProduct p;           // rows of A are p.m, or (kSwap) p.n
    int row_tiles, col_tiles, kblocks;
    int tile0, tile1;       // the tiles of this launch
    bool vec;               // rows of out, preact and residual on 16 bytes
    unsigned *err;
    unsigned long long wait_ns;
    bool withhold;          // test hook: the first CTA's (pair's) first accumulator is not announced
};

struct Ctrl {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort;
    uint32_t other_abort;   // the flag of the pair's other CTA (alone: this one's) in the cluster
    uint32_t issued;        // a pair: blocks that this CTA's producer has issued
};
static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block");

// A wait that another role's failure, in either CTA of a pair, also ends; the first to
// run out reports.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Ctrl *ctl, const Args &a) {
    const uint32_t b = smem_u32(bar);
    if (mbar_try_wait(b, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait(b, parity)) return true;
        if (*reinterpret_cast<volatile int *>(&ctl->abort)) return false;
        if (globaltimer_ns() - t0 > a.wait_ns) {
            *reinterpret_cast<volatile int *>(&ctl->abort) = 1;
            cluster_st_u32(ctl->other_abort, 1u);
            cluster_fence();
            ssd_report(a.err, SSD_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// The same by a whole warp, which goes on or gives up as one.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Ctrl *ctl, const Args &a) {
    return __all_sync(0xffffffffu, wait(bar, parity, ctl, a));
}

// Where a role has given up, copies may be on their way that nobody has waited for.  A
// CTA ends only after they have landed: the last blocks' of `issued`, with the default
// limit, since the one in force may be shorter than a copy takes.
__device__ __forceinline__ void await_copies(Ctrl *ctl, uint32_t issued, uint32_t stages) {
    for (uint32_t i = issued > stages ? issued - stages : 0; i < issued; ++i)
        mbar_wait(smem_u32(&ctl->full[i % stages]), (i / stages) & 1, kSsdDefaultWaitNs);
}

// Tiles in groups of 8 row tiles, column by column: the CTAs that run at one
// time share rows of both operands in L2.
__device__ __forceinline__ void tile_at(const Args &a, int t, int &row, int &col) {
    constexpr int kGroup = 8;
    const int per = kGroup * a.col_tiles, g = t / per, first = g * kGroup;
    const int rows = min(kGroup, a.row_tiles - first);
    row = first + (t - g * per) % rows;
    col = (t - g * per) / rows;
}

template <SsdAct kAct, int N>
__device__ __forceinline__ void act_each(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = ssd_act(v[i], kAct);
}
template <int N>
__device__ __forceinline__ void act_all(float (&v)[N], SsdAct act) {
    switch (act) {
        case SsdAct::silu: act_each<SsdAct::silu>(v); break;
        case SsdAct::gelu: act_each<SsdAct::gelu>(v); break;
        case SsdAct::relu: act_each<SsdAct::relu>(v); break;
        default: break;
    }
}

// The bias and scale of a warp's half of a tile's columns (32 of every 64), in
// shared memory of its own, so that no barrier stands between it and the others.
struct Columns {
    alignas(16) float bias[128], scale[128];
};
constexpr uint32_t kColumnBytes = kEpiWarps * sizeof(Columns);
constexpr uint32_t smem_bytes(int bn) {
    return kCtrlBytes + stages(bn) * stage_bytes(bn) + kColumnBytes;
}

// The warp fetches its columns before the tile's products are complete; zeros past
// the last column.
template <int kBN>
__device__ __forceinline__ void fetch_columns(const Args &a, Columns *cols, int half, long long n0) {
    if (!a.p.bias && !a.p.a_scale) return;
    const int lane = threadIdx.x & 31;
    __syncwarp();               // the tile before has been read
#pragma unroll
    for (int k = 0; k < kBN / 64; ++k) {
        const long long n = n0 + half * 32 + k * 64 + lane;
        const bool in = n < a.p.n;
        cols->bias[k * 32 + lane] = a.p.bias && in ? a.p.bias[n] : 0.f;
        cols->scale[k * 32 + lane] = a.p.a_scale && in ? a.p.b_scale[n] : 0.f;
    }
    __syncwarp();
}

// N columns n .. n + N - 1 of row m: vectors of 8 where the rows of out, preact and
// residual have 16-byte vectors, value by value where not and in the last columns.
// `residual` holds its whole vectors.  Value by value through one out-of-line
// function, which the last 16 of 944 columns took, was 20.5 against 7.6 us for 388 x
// 560 -> 944, and 41 against 22 us with all rows unaligned (1000 x 1024 -> 1001).
template <typename TO, int N>
struct RowPart {
    SsdRaw<TO, 8> residual[N / 8];
    int left, vectors;          // columns in range, and how many vectors of them
    __device__ __forceinline__ void ask(const Args &a, long long m, long long n) {
        left = (int)max(0ll, min((long long)N, a.p.n - n));
        vectors = a.vec ? left / 8 : 0;
        if (m >= a.p.m || !a.p.residual) return;
        const TO *res = static_cast<const TO *>(a.p.residual) + m * a.p.residual_row + n;
#pragma unroll
        for (int j = 0; j < N / 8; ++j)
            if (j < vectors) residual[j].load(res + 8 * j);
    }
    template <typename T>
    __device__ __forceinline__ void store(T *out, const float (&v)[N]) const {
#pragma unroll
        for (int j = 0; j < N / 8; ++j) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = v[8 * j + i];
            if (j < vectors) ssd_store_vec<8>(out + 8 * j, o);
        }
        if (8 * vectors == left) return;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float o[1] = {v[i]};
            if (i >= 8 * vectors && i < left) ssd_store_vec<1>(out + i, o);
        }
    }
    // bias(i), scale(i): column n + i's
    template <typename B, typename S>
    __device__ __forceinline__ void finish(const Args &a, long long m, long long n, float row_scale,
                                           B &&bias, S &&scale, float (&v)[N]) {
        const SsdProduct &p = a.p;
        if (left == 0 || m >= p.m) return;
        if (p.a_scale) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = v[i] * row_scale * scale(i);
        }
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += bias(i);
        }
        if (p.preact) store(static_cast<__nv_bfloat16 *>(p.preact) + m * p.n + n, v);
        act_all(v, p.act);
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < 8 * vectors) v[i] += residual[i / 8].get(i % 8);
            if (8 * vectors < left) {
                const TO *res = static_cast<const TO *>(p.residual) + m * p.residual_row + n;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    SsdRaw<TO, 1> one;
                    one.zero();
                    if (i >= 8 * vectors && i < left) one.load(res + i);
                    v[i] += one.get(0);
                }
            }
        }
        store(static_cast<TO *>(p.out) + m * p.out_row + n, v);
    }
};

// A warp's half of the columns of an accumulator tile (acc: the tile's first
// column in the warp's lanes) to global memory, row m of the output a lane.
// `ready` waits for the accumulator, `read` runs once it may be written again.
// One copy of the code for all columns: unrolled, the epilogue outgrows the
// instruction cache (1320 against 1120 us for 65536 x 5120 -> 2560).  Laying the
// rows out in shared memory for coalesced stores took longer, not shorter (1000
// against 977 us for the same product, whose 80 k blocks hide the epilogue; not timed
// where k is short).
template <typename TO, int kBN, typename F, typename G>
__device__ __forceinline__ bool drain(const Args &a, const Columns *cols, uint32_t acc, int half,
                                      long long m, long long n0, F &&ready, G &&read) {
    const float scale = a.p.a_scale && m < a.p.m ? a.p.a_scale[m] : 1.f;
    RowPart<TO, 32> part;
    part.ask(a, m, n0 + half * 32);
    if (!ready()) return false;
    tc_fence_after();
#pragma unroll 1
    for (int c = half * 32; c < kBN; c += 64) {
        if (c >= 64) part.ask(a, m, n0 + c);
        __syncwarp();           // rows past the end part here, the load is the whole warp's
        uint32_t r[32];
        tmem_ld32(acc + c, r);
        tmem_ld_wait(r);
        if (c + 64 >= kBN) {
            tc_fence_before();
            __syncwarp();
            read();
        }
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
        const auto at = [&](const float *q) {
            return [=](int i) {
                const float4 w = reinterpret_cast<const float4 *>(q + c / 64 * 32)[i / 4];
                return i % 4 == 0 ? w.x : i % 4 == 1 ? w.y : i % 4 == 2 ? w.z : w.w;
            };
        };
        part.finish(a, m, n0 + c, scale, at(cols->bias), at(cols->scale), v);
    }
    return true;
}
template <int kBN, typename F, typename G>
__device__ __forceinline__ bool drain_accumulator(const Args &a, Columns *cols, uint32_t acc,
                                                  int half, long long m, long long n0, F &&ready,
                                                  G &&read) {
    fetch_columns<kBN>(a, cols, half, n0);
    return a.p.out_type == SSD_ELT_F32
               ? drain<float, kBN>(a, cols, acc, half, m, n0, ready, read)
               : drain<__nv_bfloat16, kBN>(a, cols, acc, half, m, n0, ready, read);
}

// ------------------------------------------------------------ split of k: the exchange
// A rank's partial sums over the ring, four columns of a row together: column c of
// row r is component c % 4 of vector c / 4 * kBM + r, so that a warp's accesses,
// here and in another rank's shared memory, are whole vectors without conflicts.
template <int kBN>
__device__ __forceinline__ void store_sums(uint8_t *ring, uint32_t acc, int r, int half) {
    float4 *part = reinterpret_cast<float4 *>(ring);
    tc_fence_after();
#pragma unroll 1
    for (int c = half * 16; c < kBN; c += 32) {
        uint32_t v[16];
        tmem_ld16(acc + c, v);
        tmem_ld_wait(v);
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            part[(c + i) / 4 * kBM + r] =
                make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                            __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
    }
    tc_fence_before();
}

// N columns of row r (c its first one), N a multiple of 4: their sums over the ranks,
// in order, four ranks' loads under way.
template <int N>
__device__ __forceinline__ void sum_ranks(const uint32_t (&peer)[8], int ranks, int r, int c,
                                          float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll
    for (int k0 = 0; k0 < 8; k0 += 4) {
        if (k0 >= ranks) break;
        float4 q[4][N / 4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < N / 4; ++j)
                if (k0 + k < ranks)
                    q[k][j] = cluster_ld_f32x4(peer[k0 + k] + ((c / 4 + j) * kBM + r) * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < N / 4; ++j)
                if (k0 + k < ranks) {
                    v[4 * j] += q[k][j].x, v[4 * j + 1] += q[k][j].y;
                    v[4 * j + 2] += q[k][j].z, v[4 * j + 3] += q[k][j].w;
                }
    }
}

// Rank `rank` of `ranks` adds its share of the columns over all ranks, in order,
// and finishes them.  Rank k's sums lie at `ring` in the cluster's CTA
// k * stride + offset.  r: this thread's row of the tile, row0 and col0 its first row
// and column (with kSwap: first feature and token).  Rows and columns past the end are
// not fetched.  (Fetching of the last columns' vectors only those in range took longer:
// 512 x 2560 -> 2560 13.4 against 12.5 us.)
template <int kBN, bool kSwap>
__device__ __forceinline__ void finish_split(const Args &a, uint32_t ring, int r, int half,
                                             int rank, int ranks, int stride, int offset,
                                             long long row0, long long col0) {
    uint32_t peer[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) peer[k] = cluster_map(ring, (k < ranks ? k : 0) * stride + offset);
    if constexpr (kSwap) {
        const long long n = row0 + r;
        if (n >= a.p.n) return;
#pragma unroll 1
        for (int c = (rank * 2 + half) * 4; c < kBN; c += 8 * ranks) {
            const long long m = col0 + c;
            if (m >= a.p.m) break;
            float v[4];
            sum_ranks(peer, ranks, r, c, v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (m + i < a.p.m) ssd_finish(a.p, m + i, n, v[i]);
        }
    } else {
        constexpr int kPart = 16;
        const long long m = row0 + r;
        if (m >= a.p.m) return;
        const float scale = a.p.a_scale ? a.p.a_scale[m] : 1.f;
#pragma unroll 1
        for (int c = (rank * 2 + half) * kPart; c < kBN; c += 2 * kPart * ranks) {
            const long long n = col0 + c;
            if (n >= a.p.n) break;
            float v[kPart];
            sum_ranks(peer, ranks, r, c, v);
            const auto last = [&](auto part) {
                part.ask(a, m, n);
                const auto at = [&](const float *q) {
                    return [=](int i) { return i < part.left ? q[n + i] : 0.f; };
                };
                part.finish(a, m, n, scale, at(a.p.bias), at(a.p.b_scale), v);
            };
            if (a.p.out_type == SSD_ELT_F32) last(RowPart<float, kPart>{});
            else last(RowPart<__nv_bfloat16, kPart>{});
        }
    }
}

// One k block of both operands into a stage.  Coordinates are (k, row) for a
// K-major operand and (row, k) for an MN-major one, whose 64 x 64 boxes lie
// one after another.
template <int kBN, bool kAmn, bool kBmn, bool kFp8>
__device__ __forceinline__ void load_stage(const CUtensorMap *ma, const CUtensorMap *mb,
                                           uint32_t dst, uint32_t bar, int kb, int row, int col) {
    constexpr int kK = kFp8 ? 128 : 64;
    mbar_arrive_expect_tx(bar, stage_bytes(kBN));
    if constexpr (kAmn) {
#pragma unroll
        for (int i = 0; i < kBM / 64; ++i)
            tma_load_2d(dst + i * 8192, ma, bar, row * kBM + i * 64, kb * kK);
    } else {
        tma_load_2d(dst, ma, bar, kb * kK, row * kBM);
    }
    if constexpr (kBmn) {
#pragma unroll
        for (int i = 0; i < kBN / 64; ++i)
            tma_load_2d(dst + kABytes + i * 8192, mb, bar, col * kBN + i * 64, kb * kK);
    } else {
        tma_load_2d(dst + kABytes, mb, bar, kb * kK, col * kBN);
    }
}

template <int kBN, bool kAmn, bool kBmn, bool kFp8, bool kSwap, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
product_tc_kernel(const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_b, const __grid_constant__ Args a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int kStages = stages(kBN);
    constexpr uint32_t kStage = stage_bytes(kBN), kCols = tmem_cols(kBN, kSplit);
    Ctrl *ctl = reinterpret_cast<Ctrl *>(smem);
    const uint32_t ring = smem_u32(smem) + kCtrlBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool misplaced = (ring & 1023u) != 0u;    // the same in every CTA of the grid
    if (misplaced) {
        griddep_wait();
        if (threadIdx.x == 0) ssd_report(a.err, SSD_DEVERR_SMEM_ALIGN);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&ctl->full[i]), 1);
            mbar_init(smem_u32(&ctl->empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl->acc_full[i]), 1);
            mbar_init(smem_u32(&ctl->acc_empty[i]), kEpiWarps);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort = 0;
        ctl->other_abort = smem_u32(&ctl->abort);
        fence_mbar_init();
    }
    if (threadIdx.x == 64) {
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&ctl->tmem), kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    griddep_wait();                     // the kernel in front: its results may be operands
    griddep_launch_dependents();        // what may run beside this product may start

    // this CTA's tiles and, with kSplit, its part of the k blocks
    const int ntiles = a.row_tiles * a.col_tiles;
    const int rank = kSplit ? (int)cluster_rank() : 0, ranks = kSplit ? (int)cluster_size() : 1;
    const int first = kSplit ? (int)blockIdx.x / ranks : (int)blockIdx.x;
    const int step = kSplit ? ntiles : (int)gridDim.x;
    const int kb0 = kSplit ? (int)((long long)a.kblocks * rank / ranks) : 0;
    const int kb1 = kSplit ? (int)((long long)a.kblocks * (rank + 1) / ranks) : a.kblocks;

    uint32_t n = 0;                     // the producer's: blocks issued so far
    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            for (int t = first; ok && t < ntiles; t += step) {
                int row, col;
                tile_at(a, t, row, col);
                for (int kb = kb0; kb < kb1; ++kb, ++n) {
                    const uint32_t s = n % kStages, turn = n / kStages;
                    if (turn > 0 && !wait(&ctl->empty[s], (turn - 1) & 1, ctl, a)) {
                        ok = false;
                        break;
                    }
                    load_stage<kBN, kAmn, kBmn, kFp8>(&map_a, &map_b, ring + s * kStage,
                                                      smem_u32(&ctl->full[s]), kb, row, col);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t kId = kFp8 ? idesc_e4m3_f32(kBM, kBN)
                                          : idesc_bf16_f32(kBM, kBN, kAmn, kBmn);
            const uint64_t ad = kAmn ? smem_desc(ring, 8192, 1024, kSwizzle128B)
                                     : smem_desc(ring, 16, 1024, kSwizzle128B);
            const uint64_t bd = kBmn ? smem_desc(ring + kABytes, 8192, 1024, kSwizzle128B)
                                     : smem_desc(ring + kABytes, 16, 1024, kSwizzle128B);
            // a step's 32 bytes of k in a K-major row; 16 rows of k when MN-major
            constexpr uint64_t kAStep = kAmn ? 2048 >> 4 : 32 >> 4;
            constexpr uint64_t kBStep = kBmn ? 2048 >> 4 : 32 >> 4;
            uint32_t n = 0, tiles = 0;
            bool ok = true;
            for (int t = first; ok && t < ntiles; t += step, ++tiles) {
                const uint32_t buf = tiles & 1, turn = tiles >> 1;
                const uint32_t d = tmem + (kSplit ? 0 : buf * kBN);
                if (turn > 0 && !wait(&ctl->acc_empty[buf], (turn - 1) & 1, ctl, a)) break;
                tc_fence_after();
                for (int kb = kb0; kb < kb1; ++kb, ++n) {
                    const uint32_t s = n % kStages;
                    if (!wait(&ctl->full[s], (n / kStages) & 1, ctl, a)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t off = (uint64_t)(s * kStage) >> 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (kFp8)
                            mma_ss_fp8(d, ad + off + i * kAStep, bd + off + i * kBStep, kId,
                                       kb > kb0 || i > 0);
                        else
                            mma_ss(d, ad + off + i * kAStep, bd + off + i * kBStep, kId,
                                   kb > kb0 || i > 0);
                    }
                    mma_commit(smem_u32(&ctl->empty[s]));
                }
                if (ok && !(a.withhold && blockIdx.x == 0 && tiles == 0))
                    mma_commit(smem_u32(&ctl->acc_full[buf]));
            }
            // every product has ended before the accumulators are freed
            mma_commit(smem_u32(&ctl->drain));
            mbar_wait(smem_u32(&ctl->drain), 0, kSsdDefaultWaitNs);
        }
    } else {
        // a warp reads the 32 TMEM lanes of its number modulo 4; the two warps
        // of a quarter share its columns
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        Columns *cols =
            reinterpret_cast<Columns *>(smem + kCtrlBytes + kStages * kStage) + (warp - 2);
        if constexpr (!kSplit) {
            uint32_t tiles = 0;
            for (int t = first; t < ntiles; t += step, ++tiles) {
                const uint32_t buf = tiles & 1, turn = tiles >> 1;
                int row, col;
                tile_at(a, t, row, col);
                if (!drain_accumulator<kBN>(
                        a, cols, tmem + lanes + buf * kBN, half,
                        (long long)row * kBM + quarter * 32 + lane, (long long)col * kBN,
                        [&]() { return wait_warp(&ctl->acc_full[buf], turn & 1, ctl, a); },
                        [&]() {
                            if (lane == 0) mbar_arrive(smem_u32(&ctl->acc_empty[buf]));
                        }))
                    break;
            }
        } else {
            // every copy into the ring has been read: the last product waited for them
            if (wait_warp(&ctl->acc_full[0], 0, ctl, a))
                store_sums<kBN>(smem + kCtrlBytes, tmem + lanes, quarter * 32 + lane, half);
        }
    }
    if constexpr (kSplit) {
        __syncwarp();
        cluster_sync_all();
        if (warp >= 2 && !ctl->abort) {
            int row, col;
            tile_at(a, first, row, col);
            finish_split<kBN, kSwap>(a, smem_u32(smem) + kCtrlBytes, (warp & 3) * 32 + lane,
                                     (warp - 2) >> 2, rank, ranks, 1, 0, (long long)row * kBM,
                                     (long long)col * kBN);
        }
        __syncwarp();
        cluster_sync_all();         // nobody leaves before its sums have been read
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (ctl->abort) {
        if (threadIdx.x == 0) await_copies(ctl, n, kStages);
        __syncthreads();
    }
    if (warp == 1) tmem_dealloc(tmem, kCols);
}

// A pair of CTAs computes tiles of 256 x 256: each brings its 128 rows of A and of
// B, so an SM takes in 32 KB of operands a k block where a 128 x 256 tile of its
// own takes 48: the SM's 64 bytes a clock from L2 then last as long as the products
// (512 clocks a block), instead of half as long again.  The even CTA's issuer
// multiplies for both; its `full` barriers count both CTAs' bytes, its
// `acc_empty` ones both CTAs' epilogue warps.
constexpr int kPairBN = 256;
constexpr uint32_t kPairStage = 2 * kABytes;
constexpr int kPairStages = kRingBytes / kPairStage;
static_assert(kPairStages <= kMaxStages, "stages");

struct Job {
    CUtensorMap map_a, map_b;
    Args a;
};
// One product, or (kTwo) two whose tiles one launch computes: the pairs take the
// first one's tiles in turn, then the second one's.  The first `late` pairs have one
// more of the first product's tiles than the others, so those begin with `extra`
// of the second's for themselves; then all take them in turn.
template <bool kTwo>
struct Jobs {
    Job job[kTwo ? 2 : 1];
    int late, extra;
    int amn;                // kTwo: which product's A is MN-major
};
struct Place {
    int job, row, col;
};
// Tile number j of pair `pair` of `pairs`; false past its last one.
template <bool kTwo>
__device__ __forceinline__ bool place(const Jobs<kTwo> &jobs, int pair, int pairs, int j, Place &at) {
    const Args &one = jobs.job[0].a;
    int t = one.tile0 + pair + j * pairs;
    at.job = 0;
    if (t >= one.tile1) {
        if constexpr (!kTwo) return false;
        const Args &two = jobs.job[kTwo ? 1 : 0].a;
        at.job = 1;
        j -= (one.tile1 - pair + pairs - 1) / pairs;
        const int own = jobs.extra * (pairs - jobs.late);
        if (pair < jobs.late) t = own + j * pairs + pair;
        else if (j < jobs.extra) t = j * (pairs - jobs.late) + pair - jobs.late;
        else t = own + (j - jobs.extra) * pairs + pair;
        if (t >= two.tile1) return false;
    }
    tile_at(jobs.job[at.job].a, t, at.row, at.col);
    return true;
}

template <bool kAmn, bool kBmn, bool kFp8, bool kSplit, bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
product_pair_kernel(const __grid_constant__ Jobs<kTwo> jobs) {
    const Args &a = jobs.job[0].a;
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int kK = kFp8 ? 128 : 64;
    Ctrl *ctl = reinterpret_cast<Ctrl *>(smem);
    const uint32_t ring = smem_u32(smem) + kCtrlBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the pair's place in the cluster (its part of k), this CTA's in the pair
    const int in_cluster = (int)cluster_rank(), leader = in_cluster & ~1, rank = in_cluster & 1;
    const int part = in_cluster / 2, parts = kSplit ? (int)cluster_size() / 2 : 1;
    const bool misplaced = (ring & 1023u) != 0u;    // the same in every CTA of the grid
    if (misplaced) {
        griddep_wait();
        if (threadIdx.x == 0) ssd_report(a.err, SSD_DEVERR_SMEM_ALIGN);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(smem_u32(&ctl->full[i]), 1);
            mbar_init(smem_u32(&ctl->empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ctl->acc_full[i]), 1);
            mbar_init(smem_u32(&ctl->acc_empty[i]), 2 * kEpiWarps);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort = 0;
        ctl->other_abort = cluster_map(smem_u32(&ctl->abort), in_cluster ^ 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 64) {
        for (const Job &job : jobs.job) {
            tma_prefetch_desc(&job.map_a);
            tma_prefetch_desc(&job.map_b);
        }
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl->tmem), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();         // both CTAs' barriers and tensor memory stand
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    griddep_wait();                     // the kernel in front: its results may be operands
    griddep_launch_dependents();        // what may run beside this product may start
    // this pair's tiles: one with kSplit, and of that a part of the k blocks
    const int pair = (int)blockIdx.x / (2 * parts), pairs = (int)gridDim.x / (2 * parts);
    const auto tile = [&](int j, Place &at) {
        return (!kSplit || j == 0) && place(jobs, pair, pairs, j, at);
    };
    const auto blocks = [&](const Place &at, int &kb0, int &kb1) {
        const int n = jobs.job[at.job].a.kblocks;
        kb0 = kSplit ? (int)((long long)n * part / parts) : 0;
        kb1 = kSplit ? (int)((long long)n * (part + 1) / parts) : n;
    };

    // block number i of this CTA's share of a tile's operands into its stage
    const auto issue = [&](const Place &at, int kb, uint32_t i) {
        const CUtensorMap *map_a = &jobs.job[at.job].map_a, *map_b = &jobs.job[at.job].map_b;
        const int ar = at.row * 256 + rank * 128, br = at.col * 256 + rank * 128;
        const uint32_t s = i % kPairStages;
        const uint32_t own = smem_u32(&ctl->full[s]), bar = cluster_map(own, leader);
        const uint32_t dst = ring + s * kPairStage;
        if (rank == 0) mbar_arrive_expect_tx(own, 2 * kPairStage);
        if (kTwo ? at.job == jobs.amn : kAmn) {
            tma_load_2d_pair(dst, map_a, bar, ar, kb * kK);
            tma_load_2d_pair(dst + 8192, map_a, bar, ar + 64, kb * kK);
        } else {
            tma_load_2d_pair(dst, map_a, bar, kb * kK, ar);
        }
        if constexpr (kBmn) {
            tma_load_2d_pair(dst + kABytes, map_b, bar, br, kb * kK);
            tma_load_2d_pair(dst + kABytes + 8192, map_b, bar, br + 64, kb * kK);
        } else {
            tma_load_2d_pair(dst + kABytes, map_b, bar, kb * kK, br);
        }
    };
    uint32_t n = 0;                     // the producer's: blocks issued so far

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            Place at;
            for (int j = 0; ok && tile(j, at); ++j) {
                int kb, kb1;
                for (blocks(at, kb, kb1); kb < kb1; ++kb, ++n) {
                    const uint32_t turn = n / kPairStages;
                    if (turn > 0 && !wait(&ctl->empty[n % kPairStages], (turn - 1) & 1, ctl, a)) {
                        ok = false;
                        break;
                    }
                    issue(at, kb, n);
                }
            }
            // the last stages too have been handed back: no arrival at these barriers is
            // on its way when the CTA ends
            for (uint32_t i = n > kPairStages ? n - kPairStages : 0; ok && i < n; ++i)
                ok = wait(&ctl->empty[i % kPairStages], (i / kPairStages) & 1, ctl, a);
            ctl->issued = n;
            cluster_fence();
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint64_t bd = smem_desc(ring + kABytes, kBmn ? 8192 : 16, 1024, kSwizzle128B);
            constexpr uint64_t kBStep = kBmn ? 2048 >> 4 : 32 >> 4;
            const uint16_t both = (uint16_t)(3u << leader);
            uint32_t n = 0;
            bool ok = true;
            Place at;
            int j = 0;
            for (; ok && tile(j, at); ++j) {
                const uint32_t buf = j & 1, turn = (uint32_t)j >> 1;
                const uint32_t d = tmem + buf * kPairBN;
                const bool amn = kTwo ? at.job == jobs.amn : kAmn;
                const uint32_t id = kFp8 ? idesc_e4m3_f32(256, kPairBN)
                                         : idesc_bf16_f32(256, kPairBN, amn, kBmn);
                const uint64_t ad = smem_desc(ring, amn ? 8192 : 16, 1024, kSwizzle128B);
                const uint64_t a_step = amn ? 2048 >> 4 : 32 >> 4;
                if (turn > 0 && !wait(&ctl->acc_empty[buf], (turn - 1) & 1, ctl, a)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                int kb, kb1;
                bool more = false;      // the tile's first product writes, the others add
                for (blocks(at, kb, kb1); kb < kb1; ++kb, ++n) {
                    const uint32_t s = n % kPairStages;
                    if (!wait(&ctl->full[s], (n / kPairStages) & 1, ctl, a)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t off = (uint64_t)(s * kPairStage) >> 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_ss_pair<kFp8>(d, ad + off + i * a_step, bd + off + i * kBStep, id,
                                          more || i > 0);
                    more = true;
                    mma_commit_pair(smem_u32(&ctl->empty[s]), both);
                }
                if (ok && !(a.withhold && blockIdx.x == 0 && j == 0))
                    mma_commit_pair(smem_u32(&ctl->acc_full[buf]), both);
            }
            // both CTAs' epilogues have handed back the last accumulators: their arrivals
            // at these barriers are not on their way when this CTA ends
            if constexpr (!kSplit) {
                for (int i = j > 2 ? j - 2 : 0; ok && i < j; ++i)
                    ok = wait(&ctl->acc_empty[i & 1], (i >> 1) & 1, ctl, a);
            }
            // every product has ended before the accumulators are freed
            mma_commit_pair(smem_u32(&ctl->drain), both);
            mbar_wait(smem_u32(&ctl->drain), 0, kSsdDefaultWaitNs);
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        Columns *cols =
            reinterpret_cast<Columns *>(smem + kCtrlBytes + kPairStages * kPairStage) + (warp - 2);
        if constexpr (kSplit) {
            if (wait_warp(&ctl->acc_full[0], 0, ctl, a))
                store_sums<kPairBN>(smem + kCtrlBytes, tmem + lanes, quarter * 32 + lane, half);
        }
        Place at;
        for (int j = 0; !kSplit && tile(j, at); ++j) {
            const uint32_t buf = j & 1, turn = (uint32_t)j >> 1;
            if (!drain_accumulator<kPairBN>(
                    jobs.job[at.job].a, cols, tmem + lanes + buf * kPairBN, half,
                    (long long)at.row * 256 + rank * 128 + quarter * 32 + lane,
                    (long long)at.col * kPairBN,
                    [&]() { return wait_warp(&ctl->acc_full[buf], turn & 1, ctl, a); },
                    [&]() {
                        if (lane == 0)
                            mbar_arrive_cluster_relaxed(cluster_map(smem_u32(&ctl->acc_empty[buf]), leader));
                    }))
                break;
        }
    }
    if constexpr (kSplit) {
        __syncwarp();
        cluster_sync_all();
        Place at;
        if (warp >= 2 && !ctl->abort && tile(0, at))
            finish_split<kPairBN, false>(a, smem_u32(smem) + kCtrlBytes, (warp & 3) * 32 + lane,
                                         (warp - 2) >> 2, part, parts, 2, rank,
                                         (long long)at.row * 256 + rank * 128,
                                         (long long)at.col * kPairBN);
    }
    __syncwarp();
    tc_fence_before();
    // no CTA leaves while others use its barriers or operands, nor before its sums have
    // been read: only an arrival that releases waits for the loads of them
    if constexpr (kSplit) cluster_sync_all();
    else cluster_sync_relaxed();
    // the issuer's last commit has arrived in the odd CTA too
    if (warp == 1 && lane == 0 && rank == 1) mbar_wait(smem_u32(&ctl->drain), 0, kSsdDefaultWaitNs);
    __syncwarp();
    if (ctl->abort) {           // in both CTAs or in neither
        // The even CTA's barriers count both CTAs' copies: each issues what the other has
        // (any block will do, nobody reads it), and the even one waits for all.
        if (threadIdx.x == 0) {
            const uint32_t all =
                max(n, cluster_ld_u32(cluster_map(smem_u32(&ctl->issued), in_cluster ^ 1)));
            for (; n < all; ++n) issue(Place{0, 0, 0}, 0, n);
            if (rank == 0) await_copies(ctl, all, kPairStages);
        }
        __syncwarp();
    }
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
    __syncwarp();
    cluster_sync_relaxed();     // nor before both have freed the tensor memory they share
}

// ------------------------------------------------------------------ host
// A 2-D map of an operand: `rows` rows of k values.  K-major: boxes of 128
// bytes of k by `box_rows`; MN-major: 64 rows by 64 values of k.
bool operand_map(CUtensorMap *map, const void *base, bool fp8, bool mn, long long rows,
                 long long k, long long stride, int box_rows) {
    const auto enc = ssd_tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t size = fp8 ? 1 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)(mn ? rows : k), (cuuint64_t)(mn ? k : rows)};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * size};
    const cuuint32_t box[2] = {(cuuint32_t)(mn ? 64 : kRowBytes / size),
                               (cuuint32_t)(mn ? 64 : box_rows)};
    const cuuint32_t es[2] = {1, 1};
    return enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool on_16(const void *p, long long stride, int size) {
    return ((uintptr_t)p & 15u) == 0 && (stride * size) % 16 == 0;
}

Args args_of(const SsdProduct &p, int bm, int bn, bool fp8, unsigned *err) {
    Args a{};
    a.p = p;
    a.row_tiles = (int)((p.m + bm - 1) / bm);
    a.col_tiles = (int)((p.n + bn - 1) / bn);
    a.kblocks = (int)((p.k + (fp8 ? 127 : 63)) / (fp8 ? 128 : 64));
    const int so = p.out_type == SSD_ELT_F32 ? 4 : 2;
    a.vec = on_16(p.out, p.out_row, so) && (!p.residual || on_16(p.residual, p.residual_row, so)) &&
            (!p.preact || on_16(p.preact, p.n, 2));
    a.err = err;
    const SsdDebug dbg = ssd_debug_config();
    a.wait_ns = dbg.wait_ns;
    a.withhold = dbg.fault == kSsdFaultWithholdSignal;
    return a;
}

// Clusters of r CTAs that the current device holds at once.  They do not span the SMs'
// groups, so that can be fewer than the SMs over r, which stand in where the device
// does not answer.  Every kernel here takes an SM to itself, so one answer of a device
// serves them all.
template <typename Kernel>
int clusters_at_once(Kernel kernel, cudaLaunchConfig_t cfg, int r, int sms) {
    static SsdAnswers<9> answers;
    int device = -1;
    if (cudaGetDevice(&device) != cudaSuccess) device = -1;
    const int n = answers.get(device, r, [&]() {
        int found = 0;
        cfg.gridDim = dim3((unsigned)r);
        cfg.attrs->val.clusterDim.x = r;
        if (cudaOccupancyMaxActiveClusters(&found, kernel, &cfg) == cudaSuccess) return found;
        (void)cudaGetLastError();
        return -1;
    });
    return n >= 0 ? n : sms / r;
}

// Ranks of a split: the largest cluster of which there is one for every tile at
// once (with 20 tiles, seven ranks took two waves), of at least two k blocks a
// rank, at most eight (portable cluster size).
template <typename Kernel>
int split_ranks(Kernel kernel, const cudaLaunchConfig_t &cfg, long long tiles, long long kblocks,
                int sms) {
    for (int r = 8; r > 1; --r)
        if (kblocks >= 2 * r && tiles <= clusters_at_once(kernel, cfg, r, sms)) return r;
    return 1;
}

template <int kBN, bool kAmn, bool kBmn, bool kFp8, bool kSwap, bool kSplit>
cudaError_t launch(const SsdProduct &p, int sms, unsigned *err, cudaStream_t stream) {
    constexpr uint32_t kSmem = smem_bytes(kBN);
    const long long rows = kSwap ? p.n : p.m, cols = kSwap ? p.m : p.n;
    const void *rp = kSwap ? p.b : p.a, *cp = kSwap ? p.a : p.b;
    const long long rs = kSwap ? p.b_row : (kAmn ? p.a_col : p.a_row);
    const long long cs = kSwap ? p.a_row : (kBmn ? p.b_col : p.b_row);
    Args a = args_of(p, kBM, kBN, kFp8, err);
    if (kSwap) {
        a.row_tiles = (int)((rows + kBM - 1) / kBM);
        a.col_tiles = (int)((cols + kBN - 1) / kBN);
    }
    CUtensorMap ma, mb;
    if (!operand_map(&ma, rp, kFp8, kAmn, rows, p.k, rs, kBM) ||
        !operand_map(&mb, cp, kFp8, kBmn, cols, p.k, cs, kBN))
        return cudaErrorInvalidValue;
    const auto kernel = product_tc_kernel<kBN, kAmn, kBmn, kFp8, kSwap, kSplit>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)a.row_tiles * a.col_tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const int ranks = kSplit ? split_ranks(kernel, cfg, tiles, a.kblocks, sms) : 1;
    attr[0].val.clusterDim.x = ranks;
    cfg.gridDim = dim3((unsigned)(kSplit ? tiles * ranks : (tiles < sms ? tiles : sms)));
    return cudaLaunchKernelEx(&cfg, kernel, ma, mb, a);
}

// A product's operands and tiles tile0 .. tile1 - 1 (row by row of groups, as
// tile_at has them; tile1 < 0: to the last) for pairs.
bool pair_job(Job *job, const SsdProduct &p, bool amn, bool bmn, bool fp8, int tile0, int tile1,
              unsigned *err) {
    job->a = args_of(p, 256, kPairBN, fp8, err);
    job->a.tile0 = tile0;
    job->a.tile1 = tile1 < 0 ? job->a.row_tiles * job->a.col_tiles : tile1;
    return operand_map(&job->map_a, p.a, fp8, amn, p.m, p.k, amn ? p.a_col : p.a_row, kBM) &&
           operand_map(&job->map_b, p.b, fp8, bmn, p.n, p.k, bmn ? p.b_col : p.b_row, 128);
}

// The launch of a kernel of pairs, `cfg` and its attributes (the first: the cluster's
// size) but for the grid.
template <typename Kernel>
cudaError_t pair_config(Kernel kernel, cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr,
                        cudaStream_t stream) {
    constexpr uint32_t kSmem = kCtrlBytes + kPairStages * kPairStage + kColumnBytes;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    *cfg = {};
    cfg->blockDim = dim3(kThreads);
    cfg->dynamicSmemBytes = kSmem;
    cfg->stream = stream;
    cfg->attrs = attr;
    cfg->numAttrs = 2;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
}

template <bool kAmn, bool kBmn, bool kFp8, bool kSplit>
cudaError_t launch_pair(const SsdProduct &p, int tile0, int tile1, int sms, unsigned *err,
                        cudaStream_t stream) {
    Jobs<false> jobs{};
    if (!pair_job(&jobs.job[0], p, kAmn, kBmn, kFp8, tile0, tile1, err)) return cudaErrorInvalidValue;
    const Args &a = jobs.job[0].a;
    const auto kernel = product_pair_kernel<kAmn, kBmn, kFp8, kSplit, false>;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    const cudaError_t e = pair_config(kernel, &cfg, attr, stream);
    if (e != cudaSuccess) return e;
    const long long tiles = a.tile1 - a.tile0;
    int parts = kSplit ? 4 : 1;
    while (parts > 1 &&
           (a.kblocks < 2 * parts || tiles > clusters_at_once(kernel, cfg, 2 * parts, sms)))
        --parts;
    const long long pairs =
        kSplit ? tiles : std::min<long long>(tiles, std::max(1, clusters_at_once(kernel, cfg, 2, sms)));
    attr[0].val.clusterDim.x = 2 * parts;
    cfg.gridDim = dim3((unsigned)(2 * parts * pairs));
    return cudaLaunchKernelEx(&cfg, kernel, jobs);
}

template <bool kFp8>
cudaError_t few_tokens(const SsdProduct &p, int sms, unsigned *err, cudaStream_t stream) {
    if (p.m <= 32) return launch<32, false, false, kFp8, true, true>(p, sms, err, stream);
    return launch<64, false, false, kFp8, true, true>(p, sms, err, stream);
}

// Tiles of 128 x 128 or pairs' 256 x 256, whole or with k split, by the time each
// would take, in units of 64 ns.  A k block takes as long as its operands take into
// the SM, 32 KB for either: 4 units; the epilogue of a tile, which the next tile's
// products hide if they last as long, counts for 20 and 40; a split's barriers and
// exchange of sums 50.  These order the ways rather than tell their times: a pair
// tile's epilogue takes two to three times the 2.6 us of its 40 units, so products of
// few k blocks last about twice what is estimated, in either shape of tile (whole and
// pairs: 21375 x 688 -> 9632 359 and 263 us, 16376 x 1024 -> 2048 with gelu 84 and 54,
// 16376 x 512 -> 4096 118 and 112; 4001 x 768 -> 1536 in 8 bits 14.3 and 15.3; the better
// one was chosen each time).  Whole tiles run in rounds of as many
// as the SMs take; a split has as many ranks as 7/8 of the SMs allow (clusters do
// not fill all of them).  Or whole rounds of the pairs' tiles, and the few left over
// split, in a launch of their own for another 100 units (gradients at 2635 x 7664 x
// 1952: 147 against 164 us; at 16376 x 2048 x 1024, where it does not pay, 103
// against 98).
constexpr long long kBlockCost = 4, kPairEpilogue = 40, kLaunchCost = 100;
enum class Way {
    whole = SSD_PATH_WHOLE,
    pairs = SSD_PATH_PAIRS,
    split = SSD_PATH_SPLIT,
    split_pairs = SSD_PATH_SPLIT_PAIRS,
    pairs_and_split = SSD_PATH_PAIRS_AND_SPLIT
};
struct Choice {
    Way way;
    long long cost;
    int full;               // tiles of whole rounds of pairs
};
long long tiles_of(const SsdProduct &p, int rows, int cols) {
    return (p.m + rows - 1) / rows * ((p.n + cols - 1) / cols);
}
long long kblocks_of(const SsdProduct &p, bool fp8) {
    return (p.k + (fp8 ? 127 : 63)) / (fp8 ? 128 : 64);
}
Choice choose(const SsdProduct &p, bool fp8, int sms) {
    const long long kb = kblocks_of(p, fp8), never = std::numeric_limits<long long>::max();
    const auto whole = [&](long long n, int slots, long long epilogue) {
        return (n + slots - 1) / slots * std::max(kBlockCost * kb, epilogue) + epilogue;
    };
    const auto split = [&](long long n, int ctas, int most) {
        const long long r = std::min({sms * 7ll / 8 / (ctas * n), kb / 2, (long long)most});
        return r < 2 ? never : (kb + r - 1) / r * kBlockCost + 50;
    };
    const int pairs = sms / 2;
    const long long small = tiles_of(p, 128, 128), large = tiles_of(p, 256, 256);
    const long long full = large / pairs * pairs;
    const long long rest = full > 0 && full < large ? split(large - full, 2, 4) : never;
    const long long t[5] = {whole(small, sms, 20), whole(large, pairs, kPairEpilogue),
                            split(small, 1, 8), split(large, 2, 4),
                            rest == never ? never
                                          : whole(full, pairs, kPairEpilogue) + rest + kLaunchCost};
    const int best = (int)(std::min_element(t, t + 5) - t);
    return {(Way)((int)Way::whole + best), t[best], (int)full};
}

template <bool kAmn, bool kBmn, bool kFp8>
cudaError_t many(const SsdProduct &p, int sms, unsigned *err, cudaStream_t stream) {
    const Choice c = choose(p, kFp8, sms);
    switch (c.way) {
        case Way::whole: return launch<128, kAmn, kBmn, kFp8, false, false>(p, sms, err, stream);
        case Way::pairs: return launch_pair<kAmn, kBmn, kFp8, false>(p, 0, -1, sms, err, stream);
        case Way::split: return launch<128, kAmn, kBmn, kFp8, false, true>(p, sms, err, stream);
        case Way::split_pairs: return launch_pair<kAmn, kBmn, kFp8, true>(p, 0, -1, sms, err, stream);
        default: break;
    }
    const cudaError_t e = launch_pair<kAmn, kBmn, kFp8, false>(p, 0, c.full, sms, err, stream);
    return e != cudaSuccess ? e : launch_pair<kAmn, kBmn, kFp8, true>(p, c.full, -1, sms, err, stream);
}

// Two products in one launch of `pairs` pairs: how its tiles are dealt (Jobs), and
// its cost in the units above.
struct Deal {
    int late, extra;
    long long cost;
};
Deal deal(const SsdProduct &one, const SsdProduct &two, long long pairs) {
    const long long n1 = tiles_of(one, 256, 256), n2 = tiles_of(two, 256, 256);
    const long long c1 = std::max(kBlockCost * kblocks_of(one, false), kPairEpilogue);
    const long long c2 = std::max(kBlockCost * kblocks_of(two, false), kPairEpilogue);
    const long long rounds = n1 / pairs, late = n1 % pairs, early = pairs - late;
    Deal best{(int)late, 0, std::numeric_limits<long long>::max()};
    for (long long extra = 0; extra <= (c1 + c2 - 1) / c2 && extra <= n2; ++extra) {
        // tiles taken in turn, and those that go past the last whole turn: to the late pairs first
        const long long shared = std::max(0ll, n2 - extra * early);
        const long long turns = shared / pairs, over = shared % pairs;
        const long long of_late = turns + (over > 0), of_early = turns + (over > late);
        const long long own = extra * early <= n2 ? extra : (n2 + early - 1) / early;
        const long long cost = std::max(late ? (rounds + 1) * c1 + of_late * c2 : 0,
                                        rounds * c1 + (own + of_early) * c2) + kPairEpilogue;
        if (cost < best.cost) best = {(int)late, (int)extra, cost};
    }
    return best;
}

}  // namespace

// Both operands' rows on 16-byte boundaries, sizes within a map's and a grid's range.
bool ssd_product_tc_handles(const SsdProduct &p) {
    if (p.in == SSD_ELT_F32) return false;
    const int size = p.in == SSD_ELT_E4M3 ? 1 : 2;
    const bool amn = p.a_row == 1 && p.a_col != 1, bmn = p.b_row == 1 && p.b_col != 1;
    if (size == 1 && (amn || bmn)) return false;
    if (amn && !bmn) return false;      // no caller multiplies so
    const long long as = amn ? p.a_col : p.a_row, bs = bmn ? p.b_col : p.b_row;
    if (!on_16(p.a, as, size) || !on_16(p.b, bs, size)) return false;
    const long long tiles = ((p.m + 127) / 128) * ((p.n + 127) / 128);
    return tiles < (1ll << 27) && as < (1ll << 36) && bs < (1ll << 36) && p.k < (1ll << 31);
}

// At most 64 tokens (of a forward product) are a tile's columns.
static bool tokens_as_columns(const SsdProduct &p) {
    return p.m <= 64 && !(p.b_row == 1 && p.b_col != 1);
}

int ssd_product_tc_path(const SsdProduct &p, int sms) {
    return tokens_as_columns(p) ? SSD_PATH_FEW_SPLIT : (int)choose(p, p.in == SSD_ELT_E4M3, sms).way;
}

cudaError_t ssd_launch_product_tc(const SsdProduct &p, int sms, unsigned *err,
                                  cudaStream_t stream) {
    const bool amn = p.a_row == 1 && p.a_col != 1, bmn = p.b_row == 1 && p.b_col != 1;
    if (amn) return many<true, true, false>(p, sms, err, stream);
    if (bmn) return many<false, true, false>(p, sms, err, stream);
    const bool few = tokens_as_columns(p);
    if (p.in == SSD_ELT_E4M3)
        return few ? few_tokens<true>(p, sms, err, stream)
                   : many<false, false, true>(p, sms, err, stream);
    return few ? few_tokens<false>(p, sms, err, stream)
               : many<false, false, false>(p, sms, err, stream);
}

// The gradients dx and dw: how one launch would deal them, and whether it is taken.
struct Two {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    bool dw_first, together;
    long long pairs;
    Deal deal;
};
static cudaError_t plan_two(const SsdProduct &dx, const SsdProduct &dw, int sms,
                            cudaStream_t stream, Two *t) {
    const auto kernel = product_pair_kernel<false, true, false, false, true>;
    const cudaError_t e = pair_config(kernel, &t->cfg, t->attr, stream);
    if (e != cudaSuccess) return e;
    t->dw_first = dw.k > dx.k;
    const SsdProduct &one = t->dw_first ? dw : dx, &two = t->dw_first ? dx : dw;
    const long long tiles = tiles_of(one, 256, 256) + tiles_of(two, 256, 256);
    t->pairs = std::min<long long>(tiles, std::max(1, clusters_at_once(kernel, t->cfg, 2, sms)));
    t->deal = deal(one, two, t->pairs);
    const long long apart =
        choose(dx, false, sms).cost + choose(dw, false, sms).cost + kLaunchCost;
    t->together = apart >= t->deal.cost + t->deal.cost / 10;
    return cudaSuccess;
}

int ssd_product_two_path(const SsdProduct &dx, const SsdProduct &dw, int sms) {
    Two t;
    if (plan_two(dx, dw, sms, nullptr, &t) != cudaSuccess) return -1;
    return t.together ? SSD_PATH_TOGETHER : SSD_PATH_APART;
}

// In one launch, if that is cheaper than a launch each, the
// product of the longer k first: pairs that have no tile of its last round begin with
// the other's.  Tiles of two products at a time share less of what they read, about a
// tenth of the time.  us of both in one launch and in two: tokens x features x inner
// 2635 x 7664 x 1952 104 and 126, 16376 x 2048 x 1024 86 and 96, 300 x 1024 x 1024
// 11.7 and 13.5; where it is not taken, 8000 x 10240 x 2560, 538 and 512.
cudaError_t ssd_launch_product_two(const SsdProduct &dx, const SsdProduct &dw, int sms,
                                   unsigned *err, cudaStream_t stream) {
    Two t;
    const cudaError_t e = plan_two(dx, dw, sms, stream, &t);
    if (e != cudaSuccess) return e;
    if (!t.together) {
        const cudaError_t first = many<false, true, false>(dx, sms, err, stream);
        return first != cudaSuccess ? first : many<true, true, false>(dw, sms, err, stream);
    }
    Jobs<true> jobs{};
    jobs.late = t.deal.late;
    jobs.extra = t.deal.extra;
    jobs.amn = t.dw_first ? 0 : 1;
    if (!pair_job(&jobs.job[0], t.dw_first ? dw : dx, t.dw_first, true, false, 0, -1, err) ||
        !pair_job(&jobs.job[1], t.dw_first ? dx : dw, !t.dw_first, true, false, 0, -1, err))
        return cudaErrorInvalidValue;
    t.cfg.gridDim = dim3((unsigned)(2 * t.pairs));
    return cudaLaunchKernelEx(&t.cfg, product_pair_kernel<false, true, false, false, true>, jobs);
}
