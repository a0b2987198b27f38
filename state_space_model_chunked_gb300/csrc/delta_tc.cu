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
// (U's largest part is beta_i r_i, from T's diagonal: that is added in fp32.)
//
// Two kernels.  The first makes T diag(beta) and P of every chunk, all of them side by
// side.  The second walks a sequence's chunks, one CTA a head and 128 rows of its state,
// with the state's rows as the tensor core's lanes: S, R and U are transposed products'
// left operands in tensor memory, so what one product leaves in a thread's lane is
// scaled, rounded and put back as the next one's operand without leaving the lane.
//
// A long sequence of few heads is walked in parts (segments_of).
//
// K, Q and V are bf16 values as they are.  T, P, S, R and U are held in two bf16 parts
// (16 bits), the product of two second parts left out: with one part the state, which is
// handed on in fp32, would be off by 3e-3 of itself, with two it is by 4e-6.
//
// 65536 tokens, 32 heads of 128 x 128: 1743 us, of which the chunk matrices 368 (their records
// of 34 KB a chunk and head are written at 3.0 TB/s; 50% of the issue slots, ten barriers a
// head, five CTAs an SM), the parts' ends and maps 650, their joining 18, the walks 700.  47
// sequences of 1394 on average, 24 heads of 64 x 128: 717 us, of which 262 and 450.  A walk is
// bound by latency: a chunk takes 2.1 us without output and 2.4 with it, for five products that
// wait for one another (1300 cycles of them) and the steps between them.
#include <mutex>

#include "delta_tc.cuh"
#include "vec.cuh"

namespace {

using namespace ssddelta;

// ------------------------------------------------------------- chunk matrices
// One CTA a chunk and key group, the group's heads after each other (or, where that would
// be few CTAs, a share of them).  The 64 queries over the 64 keys, times the keys, are one
// product of M = 128, N = 64: a thread's lane is then a row of Q K^T (threads 0 .. 63) or of
// K K^T (64 .. 127).  The triangle is inverted to fp32's precision: blocks of 16 by
// substitution, a thread a column, then twice
//     (T11  0; T21  T22),   T21 = -T22 (A21 T11)
// for blocks of 32 (in fp32) and of 64 (TF32 products of two parts each, 22 bits).
constexpr int kPrepThreads = 128;
constexpr int kTw = 36;         // floats a row of a 32 x 32 block
constexpr int kAw = 68;         // and a column of A
struct PrepSmem {
    // At 0 the tiles, Q over K by panels; then A by columns (and W above its diagonal
    // blocks), and in its place at last T's images; P's images behind them.
    static constexpr uint32_t kP = kC * kAw * 4;
    static constexpr uint32_t kRows = kP + 2 * kPanel;              // T11 and T22 by rows
    static constexpr uint32_t kSums = kRows + 2 * 32 * kTw * 4;     // of g, beta, decay to token 31
    static constexpr uint32_t kBars = kSums + 4 * kC * 4;
    static constexpr uint32_t kBytes = kBars + 64;
};
static_assert(PrepSmem::kP % 1024 == 0 && PrepSmem::kRows >= 4 * kPanel, "images and tiles");

struct Prep {
    SsdDelta d;
    uint8_t *records;
    int split;          // CTAs that share a group's heads
    bool least_beta;
    unsigned *err;
};

// a + b of numbers in two floats each, the second one what the first does not hold.
__device__ __forceinline__ float2 add_two(float2 a, float2 b) {
    const float s = a.x + b.x, v = s - a.x;
    const float e = (a.x - (s - v)) + (b.x - v) + a.y + b.y;
    const float hi = s + e;
    return make_float2(hi, e - (hi - s));
}

// D += A B for tiles of 16 x 8 and 8 x 8, each in two TF32 parts, without the product of
// both second ones.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
template <int kCount>
__device__ __forceinline__ void split_tf32(const float (&x)[kCount], uint32_t (&hi)[kCount], uint32_t (&lo)[kCount]) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
        asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi[i]) : "f"(x[i]));
        lo[i] = __float_as_uint(x[i] - __uint_as_float(hi[i]));
    }
}
// d = a b for the warp's 16 x 16 of 32 x 32 matrices, over k from 8 k0 to 8 k1; a(r, k), b(k, c).
template <typename A, typename B>
__device__ __forceinline__ void product_tf32(float (&d)[2][4], int m0, int n0, int k0, int k1, A a, B b) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j][i] = 0.f;
#pragma unroll 2
    for (int k = 8 * k0; k < 8 * k1; k += 8) {
        const float x[4] = {a(m0 + g, k + t), a(m0 + g + 8, k + t), a(m0 + g, k + t + 4), a(m0 + g + 8, k + t + 4)};
        uint32_t ah[4], al[4];
        split_tf32(x, ah, al);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float y[2] = {b(k + t, n0 + 8 * j + g), b(k + t + 4, n0 + 8 * j + g)};
            uint32_t bh[2], bl[2];
            split_tf32(y, bh, bl);
            mma_tf32(d[j], al, bh);
            mma_tf32(d[j], ah, bl);
            mma_tf32(d[j], ah, bh);
        }
    }
}

// s + a y of four values, by pairs.
__device__ __forceinline__ void fma4(float4 &s, float a, const float4 &y) {
    const float2 aa = make_float2(a, a);
    const float2 lo = ffma2(aa, make_float2(y.x, y.y), make_float2(s.x, s.y));
    const float2 hi = ffma2(aa, make_float2(y.z, y.w), make_float2(s.z, s.w));
    s = make_float4(lo.x, lo.y, hi.x, hi.y);
}
// (1 + A)^-1 of `columns` (A[r][c] at kAw c + r), by all 128 threads: its diagonal blocks of
// 32 to `rows`, and of the block below the warp's 16 x 16 (rows m0, columns n0 of it).
__device__ __forceinline__ void invert(float *columns, float *rows, int m0, int n0, float (&below)[2][4]) {
    const int t = threadIdx.x;
    if (t < 64) {       // blocks of 16
        const int b = t >> 4, c = t & 15;
        float4 acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        float *const row = rows + ((b >> 1) * 32 + (b & 1) * 16) * kTw + (b & 1) * 16 + c;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float at[4] = {acc[i / 4].x, acc[i / 4].y, acc[i / 4].z, acc[i / 4].w};
            const float x = i == c ? 1.f : -at[i % 4];
            const float4 *a = reinterpret_cast<const float4 *>(columns + (16 * b + i) * kAw + 16 * b);
#pragma unroll
            for (int v = (i + 1) / 4; v < 4; ++v) fma4(acc[v], x, a[v]);      // (used sums get more, unread)
            row[i * kTw] = x;
        }
    } else {            // above them nothing
        for (int i = t - 64; i < 2 * 64; i += 64) {
            const int b = i >> 6, r = (i >> 2) & 15, c = (i & 3) * 4;
            *reinterpret_cast<float4 *>(rows + (b * 32 + r) * kTw + 16 + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    __syncthreads();
    {                   // blocks of 32: 64 threads each, a row's four columns
        const int b = t >> 6, r = (t >> 2) & 15, c = (t & 3) * 4;
        float *const row = rows + b * 32 * kTw;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float a = columns[(32 * b + k) * kAw + 32 * b + 16 + r];
            fma4(x, a, *reinterpret_cast<const float4 *>(row + k * kTw + c));
        }
        *reinterpret_cast<float4 *>(columns + (32 + r) * kAw + 16 * b + c) = x;     // W
        __syncthreads();
        float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float a = row[(16 + r) * kTw + 16 + k];
            fma4(z, -a, *reinterpret_cast<const float4 *>(columns + (32 + k) * kAw + 16 * b + c));
        }
        *reinterpret_cast<float4 *>(row + (16 + r) * kTw + c) = z;
    }
    __syncthreads();
    // the block of 32 below (T11's columns from 16 on begin at row 16, T22's first 16 rows
    // end at column 16)
    const int g = (t & 31) >> 2, u = t & 3;
    product_tf32(below, m0, n0, n0 / 8, 4, [&](int r, int k) { return columns[k * kAw + 32 + r]; },
                 [&](int k, int c) { return rows[k * kTw + c]; });
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float *const w = columns + (32 + m0 + g) * kAw + n0 + 8 * j + 2 * u;
        *reinterpret_cast<float2 *>(w) = make_float2(below[j][0], below[j][1]);
        *reinterpret_cast<float2 *>(w + 8 * kAw) = make_float2(below[j][2], below[j][3]);
    }
    __syncthreads();
    product_tf32(below, m0, n0, 0, (m0 + 16) / 8, [&](int r, int k) { return rows[(32 + r) * kTw + k]; },
                 [&](int k, int c) { return -columns[(32 + k) * kAw + c]; });
}

template <int kPanels>
__global__ void __launch_bounds__(kPrepThreads, 5)
delta_chunk_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK, const Prep a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const SsdDelta &d = a.d;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) {
        if (threadIdx.x == 0) ssd_report(a.err, SSD_DEVERR_SMEM_ALIGN);
        return;
    }
    const int share = (int)(blockIdx.x % a.split), group = (int)(blockIdx.x / a.split % d.groups);
    const long long slot = blockIdx.x / a.split / d.groups;
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
    const int all = d.heads / d.groups, row = threadIdx.x & 63;
    const int head0 = group * all + all * share / a.split, wide = group * all + all * (share + 1) / a.split - head0;
    // the first head's gates on their way beside the copies
    const bool on = warp < 2 && row < valid;
    const size_t gate0 = (size_t)(token + row) * d.heads + head0;
    float g = on ? d.g[gate0] : 0.f, beta = on ? d.beta[gate0] : 0.f;
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
    float2 *const sums = reinterpret_cast<float2 *>(smem + PrepSmem::kSums);
    float *const betas = reinterpret_cast<float *>(sums + kC), *const to_half = betas + kC;
    float *const columns = reinterpret_cast<float *>(smem);
    float *const rows = reinterpret_cast<float *>(smem + PrepSmem::kRows);
    const bool keys = warp >= 2;
    const int upper = warp & 1;         // which half of the 64 tokens the warp's rows are
    // P's upper right quarter, for all heads
    for (int i = threadIdx.x; i < 2 * 32 * 4; i += kPrepThreads)
        *reinterpret_cast<uint4 *>(smem + PrepSmem::kP + (i >> 7) * kPanel + panel_at((i >> 2) & 31, 32 + (i & 3) * 8)) =
            make_uint4(0, 0, 0, 0);
    for (int h = 0; h < wide; ++h) {
        uint8_t *const record = a.records + ((size_t)slot * d.heads + head0 + h) * kRecord;
        // The images of the head in front have been read, its sums used.  Each half's sums of
        // log2(e) g are held in two floats: a later token's decay is the difference of two of
        // them, which an early strong decay must not round away.
        if (threadIdx.x == 0 && h > 0) bulk_wait_read<0>();
        __syncthreads();
        float2 s = make_float2(0.f, 0.f);
        if (warp < 2) {
            constexpr float kLog2e = 1.4426950408889634f, kRest = 1.9259629911266175e-8f;
            g = g < -200.f ? -200.f : g;
            s.x = g * kLog2e;
            s.y = fmaf(g, kLog2e, -s.x) + g * kRest;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float2 n = make_float2(__shfl_up_sync(0xffffffffu, s.x, o), __shfl_up_sync(0xffffffffu, s.y, o));
                if (lane >= o) s = add_two(n, s);
            }
            sums[row] = s;
            if (a.least_beta && fabsf(beta) < kLeastBeta) beta = copysignf(kLeastBeta, beta);
            betas[row] = beta;
            if (h + 1 < wide) {
                g = on ? d.g[gate0 + h + 1] : 0.f;
                beta = on ? d.beta[gate0 + h + 1] : 0.f;
            }
        }
        __syncthreads();
        const float2 half = sums[31], rest = sums[63], mine = sums[row];
        const float upto = mine.x + mine.y;
        if (warp < 2) {
            float *gates = reinterpret_cast<float *>(record + kRecGates);
            const float2 whole = upper ? rest : half;
            const float behind = (whole.x - mine.x) + (whole.y - mine.y);
            gates[row] = ex2_approx(upper ? half.x + upto : upto);
            gates[kGateW + row] = ex2_approx(upper ? behind : behind + rest.x);
            gates[kGateBeta + row] = betas[row];
            *reinterpret_cast<float2 *>(gates + kGateSums + 2 * row) = mine;
            if (!upper) to_half[row] = ex2_approx(behind);
        }
        __syncthreads();
        // rows behind the sequence's end stay empty
        const int last = row < valid ? (keys ? row - 1 : row) : -1;
        const float factor = keys ? betas[row] : d.scale, from_half = factor * ex2_approx(upto);
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
#pragma unroll 1
        for (int c0 = 0; c0 < kC; c0 += 16) {
            float v[16];
            if (!upper && c0 >= 32) break;      // (zeros)
            uint32_t r[16];
            tmem_ld16(lanes + c0, r);
            float2 by;
            if (upper && c0 < 32) {
#pragma unroll
                for (int j = 0; j < 16; j += 4) *reinterpret_cast<float4 *>(v + j) = *reinterpret_cast<const float4 *>(to_half + c0 + j);
                by = make_float2(from_half, from_half);
            } else {
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float4 c = *reinterpret_cast<const float4 *>(sums + c0 + j);
                    const float2 less = make_float2(-1.f, -1.f);
                    const float2 x = ffma2(make_float2(c.x, c.y), less, mine), y = ffma2(make_float2(c.z, c.w), less, mine);
                    v[j] = ex2_approx(x.x + x.y);
                    v[j + 1] = ex2_approx(y.x + y.y);
                }
                by = make_float2(factor, factor);
            }
            tmem_ld_wait(r);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const float2 x = fmul2(fmul2(make_float2(v[j], v[j + 1]), by),
                                       make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])));
                v[j] = c0 + j <= last ? x.x : 0.f;
                v[j + 1] = c0 + j + 1 <= last ? x.y : 0.f;
            }
            if (keys) {
#pragma unroll
                for (int j = 0; j < 16; ++j) columns[(c0 + j) * kAw + row] = v[j];
            } else {
                put_parts(smem + PrepSmem::kP, panel_at(row, c0), v);
                put_parts(smem + PrepSmem::kP, panel_at(row, c0 + 8), v + 8);
            }
        }
        __syncthreads();
        const int m0 = (warp >> 1) * 16, n0 = (warp & 1) * 16;
        float below[2][4];
        invert(columns, rows, m0, n0, below);
        __syncthreads();
        // T diag(beta) without its diagonal, in A's place
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = n0 + 8 * j + 2 * (lane & 3), r = 32 + m0 + (lane >> 2);
            const float2 be = *reinterpret_cast<const float2 *>(betas + c);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const Split x = split2(below[j][2 * i] * be.x, below[j][2 * i + 1] * be.y);
                const uint32_t to = panel_at(r + 8 * i, c);
                *reinterpret_cast<uint32_t *>(smem + to) = x.hi;
                *reinterpret_cast<uint32_t *>(smem + kPanel + to) = x.lo;
            }
        }
        for (int i = threadIdx.x; i < 64 * 4; i += kPrepThreads) {
            const int r = i >> 2, c = (i & 3) * 8, b = r & 32;
            const float4 *from = reinterpret_cast<const float4 *>(rows + r * kTw + c);
            const float4 *be = reinterpret_cast<const float4 *>(betas + b + c);
            float v[8];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 x = from[j], y = be[j];
                v[4 * j] = x.x * y.x;
                v[4 * j + 1] = x.y * y.y;
                v[4 * j + 2] = x.z * y.z;
                v[4 * j + 3] = x.w * y.w;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j == (r & 31)) v[j] = 0.f;
            put_parts(smem, panel_at(r, b + c), v);
        }
        {
            const uint32_t to = panel_at(threadIdx.x >> 2, 32 + (threadIdx.x & 3) * 8);
            *reinterpret_cast<uint4 *>(smem + to) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(smem + kPanel + to) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (threadIdx.x == 0) {
            bulk_store(record + kRecT, base, 2 * kPanel);
            bulk_store(record + kRecP, base + PrepSmem::kP, 2 * kPanel);
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
// 16 warps on the chain, 8 on the output, one for the copies, one for the products.  (With 4 on
// the output, or the copies issued by the products' warp, the chain gets 80 registers a thread
// and spills nothing, and a chunk takes 8% longer; so it does where setmaxnreg shares them out.)
constexpr int kChainWarps = 16, kOutWarps = 8;
constexpr int kLoadWarp = kChainWarps + kOutWarps, kMmaWarp = kLoadWarp + 1, kWalkThreads = 32 * (kMmaWarp + 1);

template <int kPanels>
struct WalkSmem {
    static constexpr uint32_t kK = 0, kQ = kPanels * kPanel, kRec = 2 * kPanels * kPanel;
    static constexpr uint32_t kV = kRec + kRecord;      // [token][128], as they lie
    static constexpr uint32_t kStage = (kV + 64 * 256 + 1023) / 1024 * 1024;
    static constexpr uint32_t kO = 2 * kStage;          // [token][128]: the output on its way
    static constexpr uint32_t kRows = kO + 64 * 256;    // states on their way, by warps
    static constexpr uint32_t kCtl = kRows + kChainWarps * kStageRows;
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
    // A sequence in parts that are walked side by side (segments > 1): `d` has the parts for
    // sequences.  For the states they start from, `starts` [seq][segment][head][P][N], come
    // first: every part but the last from a state of zeros (the first from its own), for its
    // end; and for all of these but the first what they make of the rows of a unit matrix,
    // `maps` [seq][segment - 1][head][N][N].
    int segments, half;
    float *starts, *maps;
    unsigned *err;
    unsigned long long wait_ns;
    bool withhold;
};

enum WalkBar {
    kFull = 0, kEmpty = 2,      // two stages each
    kKs = 4, kU, kS, kQs, kPu, kDrain,              // products done
    kSh, kSl, kRh, kRl, kWh, kWl,                   // operands' parts written by the chain
    kUReady, kQsRead, kPuRead,                      // and by the output's warps, or read
    kStaged, kStored,                               // the output in shared memory, and out of it
    kBars
};

template <int kPanels, bool kEnds>
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
    // kEnds: parts for their ends or (map) for their maps, without output
    // (first parts last, for where there are too many jobs for the SMs)
    const unsigned maps = kEnds ? (unsigned)d.nseq * (a.segments - 2) * d.heads : 0;
    const bool map = kEnds && blockIdx.x < maps;
    const unsigned job = blockIdx.x - (map ? 0 : maps);
    const int blocks = map ? 1 : a.blocks, rows = map ? d.n : d.p;
    const int head = (int)(job % d.heads), block = (int)(job / d.heads % blocks);
    int seq = (int)(job / d.heads / blocks), segment = 0;
    if constexpr (kEnds) {
        segment = a.segments - 2 - seq / d.nseq;
        seq %= d.nseq;
    } else {
        seq = sequence_of(d, seq, reinterpret_cast<volatile int *>(smem + Lay::kCtl + 8 * kBars + 8));
    }
    const int group = head / (d.heads / d.groups);
    long long first = d.cu ? d.cu[seq] : (long long)seq * d.length;
    int len = d.cu ? d.cu[seq + 1] - d.cu[seq] : d.length;
    if constexpr (kEnds) {
        const int at = part_start(len, segment, a.segments, a.half);
        len = part_start(len, segment + 1, a.segments, a.half) - at;
        first += at;
    }
    const int chunks = (len + kC - 1) / kC, p0 = block * 128;
    const size_t one = (size_t)rows * d.n;
    // where the state comes from (null: zeros, or a map's unit matrix) and goes to
    const auto source = [&]() -> const float * {
        return a.init && segment == 0 ? a.init + ((size_t)seq * d.heads + head) * one : nullptr;
    };
    const auto target = [&]() -> float * {
        if (map) return a.maps + (((size_t)seq * (a.segments - 2) + segment - 1) * d.heads + head) * one;
        if (kEnds) return a.starts + (((size_t)seq * a.segments + segment + 1) * d.heads + head) * one;
        if (!a.final_state || (seq + 1) % a.segments) return nullptr;
        return a.final_state + ((size_t)(seq / a.segments) * d.heads + head) * one;
    };
    if (chunks == 0) {
        const float *init = source();
        if (float *const final_state = target())
            for (long long i = threadIdx.x; i < (long long)min(128, rows - p0) * d.n; i += kWalkThreads)
                final_state[(size_t)p0 * d.n + i] = init ? init[(size_t)p0 * d.n + i]
                                                    : map && i / d.n == i % d.n ? 1.f : 0.f;
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
        for (int i : {kQsRead, kUReady, kPuRead, kStaged, kStored}) mbar_init(bar(i), kOutWarps);
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

    if (warp == kLoadWarp) {
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            if (c >= 2 && !wait.warp(bar(kEmpty + s), ((c >> 1) - 1) & 1)) break;
            if (elect_one()) {
                const uint32_t to = base + s * Lay::kStage;
                const int token = (int)(first + (long long)c * kC);
                mbar_arrive_expect_tx(bar(kFull + s), (kEnds ? 1 : 2) * kPanels * kPanel + kRecord + (map ? 0 : 64 * 256));
#pragma unroll
                for (int p = 0; p < kPanels; ++p) {
                    tma_load_3d(to + Lay::kK + p * kPanel, &mapK, bar(kFull + s), 64 * p, group, token);
                    if (!kEnds) tma_load_3d(to + Lay::kQ + p * kPanel, &mapQ, bar(kFull + s), 64 * p, group, token);
                }
                bulk_load(to + Lay::kRec, a.records + ((size_t)(slot0 + c) * d.heads + head) * kRecord, kRecord,
                          bar(kFull + s));
                if (!map) tma_load_3d(to + Lay::kV, &mapV, bar(kFull + s), p0, head, token);
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
            if (!kEnds) {
                if (c > 0 && !wait.warp(bar(kPuRead), (c - 1) & 1)) break;
                tc_fence_after();
                if (one) over_n(kColO, kColSh, at + Lay::kQ, false);
                __syncwarp();
            }
            if (!wait.warp(bar(kRh), c & 1)) break;
            tc_fence_after();
            if (one) {
                triangle(kColX, kColR, at + Lay::kRec + kRecT, true);
                triangle(kColX, kColR, at + Lay::kRec + kRecT + kPanel, true);
            }
            __syncwarp();
            if (!wait.warp(bar(kRl), c & 1)) break;
            tc_fence_after();
            if (one) {
                triangle(kColX, kColRl, at + Lay::kRec + kRecT, true);
                mma_commit(bar(kU));
                if (!kEnds) {
                    over_n(kColO, kColSl, at + Lay::kQ, true);
                    mma_commit(bar(kQs));
                }
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
                if (kEnds) mma_commit(bar(kEmpty + s));
            }
            __syncwarp();
            if (kEnds) continue;
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
            if (!wait.warp(bar(kFull + s), (c >> 1) & 1)) break;
            if (kEnds) {
                if (lane == 0) mbar_arrive(bar(kEmpty + s));
                continue;
            }
            if (!wait.warp(bar(kU), c & 1)) break;
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
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kStaged));
            if (!wait.warp(bar(kStaged), c & 1)) break;
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
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kStored));
            if (!wait.warp(bar(kStored), c & 1)) break;
        }
    } else {
        // the chain: a thread has a row of the state and of V^T, R^T and U^T; the four groups
        // of four warps have a quarter of the columns each
        const int q = warp & 3, part = warp >> 2, row = 32 * q + lane, p = p0 + row;
        const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
        constexpr int kMine = kN / 4;
        const int n0 = part * kMine;
        const auto to_memory = [&](float *m, const float (&v)[kMine]) {
            store_rows<kMine>(reinterpret_cast<float *>(smem + Lay::kRows + warp * kStageRows), v,
                              m + (size_t)(p0 + 32 * q) * d.n + n0, d.n, rows - (p0 + 32 * q), d.n - n0);
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
            if (!kEnds && a.checkpoints) to_memory(a.checkpoints + ((size_t)(slot0 + c) * d.heads + head) * one, v);
        };
        const auto stage = [&](int c) { return smem + (c & 1) * Lay::kStage; };
        const auto clean = [&](int c) {
            if (len - c * kC >= kC) return;
            clean_rows(stage(c) + Lay::kK, kPanel, kPanels, len - c * kC, threadIdx.x, 32 * kChainWarps);
            fence_proxy_async_smem();
        };
        float v[kMine];
        if (const float *init = source()) {
            load_rows<kMine>(reinterpret_cast<float *>(smem + Lay::kRows + warp * kStageRows), v,
                             init + (size_t)(p0 + 32 * q) * d.n + n0, d.n, rows - (p0 + 32 * q), d.n - n0);
        } else {
#pragma unroll
            for (int i = 0; i < kMine; ++i) v[i] = map && n0 + i == p ? 1.f : 0.f;
        }
        const bool on = wait.warp(bar(kFull), 0);
        if (on) {
            clean(0);
            put(0, v, reinterpret_cast<const float *>(stage(0) + Lay::kRec + kRecGates)[kC - 1]);
        }
        for (int c = 0; on && c < chunks; ++c) {
            const int s = c & 1, tokens = min(kC, len - c * kC) - 16 * part;
            const float4 *gates = reinterpret_cast<const float4 *>(stage(c) + Lay::kRec + kRecGates) + 4 * part;
            float x[16], f[16];
            {
                const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(stage(c) + Lay::kV) + 16 * part * 128 + row;
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = map ? 0.f : __bfloat162float(v[i * 128]);
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
            // U's own term, beta R, where the product adds the earlier tokens'
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float4 *>(f + 4 * i) = gates[kGateBeta / 4 + i];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 y = fmul2(make_float2(x[i], x[i + 1]), make_float2(f[i], f[i + 1]));
                r[i] = __float_as_uint(y.x);
                r[i + 1] = __float_as_uint(y.y);
            }
            tmem_st16(tq + kColX + 16 * part, r);
            ready(kRh);
#pragma unroll
            for (int i = 0; i < 8; ++i) hi[i] = rest2(x[2 * i], x[2 * i + 1], hi[i]);
            tmem_st8(tq + kColRl + 8 * part, hi);
            ready(kRl);
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float4 *>(f + 4 * i) = gates[kGateW / 4 + i];
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
            else if (float *const final_state = target()) to_memory(final_state, y);
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

// The states that a sequence's parts start from: of the first what its own is; of the second
// that one's end; E_s <- E_s + E_(s-1) M_(s-1) from there on.  A thread has a column of kR of a
// CTA's 2 kR rows; the maps are copied to shared memory one ahead.  Bound by that memory's
// reads, with few rows by each step's latency.  And the offsets of the parts.
constexpr uint32_t kJoinMap = 128 * 128 * 4;
constexpr uint32_t join_bytes(int r) { return 2 * kJoinMap + 2 * 128 * 2 * r * 4 + 16; }
template <int kR>
__global__ void __launch_bounds__(256)
delta_join_kernel(const SsdDelta d, const float *init, int segments, int part_half, int *cu, float *starts,
                  const float *maps, unsigned *err) {
    extern __shared__ __align__(128) uint8_t join_smem[];
    const int seq = (int)(blockIdx.x / d.heads), head = (int)(blockIdx.x % d.heads), n = d.n;
    constexpr int kJoinRows = 2 * kR;
    const int r0 = blockIdx.y * kJoinRows, col = threadIdx.x & 127, half = threadIdx.x >> 7;
    const size_t one = (size_t)d.p * n;
    const uint32_t bars = smem_u32(join_smem) + join_bytes(kR) - 16;
    if (threadIdx.x == 0) {
        mbar_init(bars, 1);
        mbar_init(bars + 8, 1);
        fence_mbar_init();
    }
    __syncthreads();
    const auto fetch = [&](int s) {     // the map of part s - 1
        if (threadIdx.x != 0 || s >= segments) return;
        const float *map = maps + (((size_t)seq * (segments - 2) + s - 2) * d.heads + head) * n * n;
        mbar_arrive_expect_tx(bars + 8 * (s & 1), n * n * 4);
        bulk_load(smem_u32(join_smem) + (s & 1) * kJoinMap, map, n * n * 4, bars + 8 * (s & 1));
    };
    fetch(2);
    fetch(3);
    if (head == 0 && blockIdx.y == 0 && threadIdx.x <= segments) {
        const int first = d.cu ? d.cu[seq] : seq * d.length, len = d.cu ? d.cu[seq + 1] - first : d.length;
        cu[seq * segments + threadIdx.x] =
            first + part_start(len, threadIdx.x, segments, part_half);     // (a sequence's end twice)
    }
    // states by columns, 2 kR rows each, of a part and of the one in front of it
    float *const states = reinterpret_cast<float *>(join_smem + 2 * kJoinMap);
    const int row = r0 + kR * half;
    float *const own = starts + ((size_t)seq * segments * d.heads + head) * one + (size_t)row * n + col;
    const float *const from = init ? init + ((size_t)seq * d.heads + head) * one + (size_t)row * n + col : nullptr;
    const auto on = [&](int i) { return col < n && row + i < d.p; };
    {
        float first[kR], second[kR];
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            first[i] = from && on(i) ? from[(size_t)i * n] : 0.f;
            second[i] = on(i) ? own[(size_t)d.heads * one + (size_t)i * n] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            if (on(i)) own[(size_t)i * n] = first[i];
            states[128 * kJoinRows + col * kJoinRows + kR * half + i] = second[i];
        }
    }
    for (int s = 2; s < segments; ++s) {
        float *const to = own + (size_t)s * d.heads * one;
        float v[kR];
#pragma unroll
        for (int i = 0; i < kR; ++i) v[i] = on(i) ? to[(size_t)i * n] : 0.f;
        // (the states in front are there; a CTA that gives up asks for no more maps, and those under
        // way land before it ends)
        if (!__syncthreads_and(mbar_wait(bars + 8 * (s & 1), ((s >> 1) - 1) & 1, kSsdDefaultWaitNs))) {
            if (threadIdx.x == 0) ssd_report(err, SSD_DEVERR_TIMEOUT);
            for (int t = s; t < segments && t < s + 2; ++t) mbar_wait(bars + 8 * (t & 1), ((t >> 1) - 1) & 1, kSsdDefaultWaitNs);
            return;
        }
        const float *map = reinterpret_cast<const float *>(join_smem + (s & 1) * kJoinMap) + col;
        const float *e = states + ((s - 1) & 1) * 128 * kJoinRows + kR * half;
        if (col < n) {
#pragma unroll 8
            for (int k = 0; k < n; ++k) {
                const float m = map[k * n];
#pragma unroll
                for (int i = 0; i < kR; i += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(e + k * kJoinRows + i);
                    v[i] += x.x * m;
                    v[i + 1] += x.y * m;
                    v[i + 2] += x.z * m;
                    v[i + 3] += x.w * m;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            if (on(i)) to[(size_t)i * n] = v[i];
            states[(s & 1) * 128 * kJoinRows + col * kJoinRows + kR * half + i] = v[i];
        }
        __syncthreads();        // (the map has been read)
        fetch(s + 2);
    }
}

size_t records_bytes(const SsdDelta &d) {
    return ((size_t)ssd_delta_slots(d.tokens, d.nseq) * d.heads * kRecord + 255) / 256 * 256;
}

template <int kPanels>
cudaError_t launch_chunks_of(const SsdDelta &d, uint8_t *records, bool least_beta, int sms, unsigned *err,
                             cudaStream_t stream) {
    CUtensorMap q, k;
    if (!make_map(&q, d.q, d.n, d.groups, d.tokens, d.q_stride, 64, true) ||
        !make_map(&k, d.k, d.n, d.groups, d.tokens, d.k_stride, 64, true))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(delta_chunk_kernel<kPanels>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PrepSmem::kBytes);
    if (e != cudaSuccess) return e;
    // CTAs for some rounds of five an SM
    const long long ctas = ssd_delta_slots(d.tokens, d.nseq) * d.groups, want = 20ll * sms;
    const int wide = d.heads / d.groups;
    const int split = (int)(ctas >= want ? 1 : (want + ctas - 1) / ctas < wide ? (want + ctas - 1) / ctas : wide);
    if (ctas * split >= (1ll << 31)) return cudaErrorInvalidValue;
    delta_chunk_kernel<kPanels><<<(unsigned)(ctas * split), kPrepThreads, PrepSmem::kBytes, stream>>>(
        q, k, Prep{d, records, split, least_beta, err});
    return cudaGetLastError();
}

template <int kPanels>
cudaError_t launch_fwd(const SsdDeltaFwd &f, void *ws, int sms, unsigned *err, cudaStream_t stream) {
    const SsdDelta &d = f.in;
    CUtensorMap q, k, v;
    if (!make_map(&q, d.q, d.n, d.groups, d.tokens, d.q_stride, 64, true) ||
        !make_map(&k, d.k, d.n, d.groups, d.tokens, d.k_stride, 64, true) ||
        !make_map(&v, d.v, d.p, d.heads, d.tokens, d.v_stride, 128, false))
        return cudaErrorInvalidValue;
    const SsdDebug debug = ssd_debug_config();
    uint8_t *records = static_cast<uint8_t *>(ws);
    cudaError_t e = launch_chunks(d, records, false, sms, err, stream);
    if (e != cudaSuccess) return e;
    using Lay = WalkSmem<kPanels>;
    static_assert(Lay::kBytes <= 232448, "more than 227 KB of shared memory");
    e = cudaFuncSetAttribute(delta_walk_tc_kernel<kPanels, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kBytes);
    if (e != cudaSuccess) return e;
    const int blocks = (d.p + 127) / 128;
    const InParts segments = segments_of(d, sms);
    WalkTc w{d, records, f.init, static_cast<__nv_bfloat16 *>(f.o), f.o_stride, f.final_state, f.checkpoints, blocks,
             on_16(f.o) && f.o_stride % 8 == 0, segments.parts, segments.half, nullptr, nullptr, err, debug.wait_ns,
             debug.fault == kSsdFaultWithholdSignal};
    if (w.segments > 1) {
        const Parts parts = parts_of(d, w.segments, records + records_bytes(d));
        w.starts = parts.starts;
        w.maps = parts.maps;
        e = cudaFuncSetAttribute(delta_walk_tc_kernel<kPanels, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kBytes);
        if (e != cudaSuccess) return e;
        const long long walks = (long long)d.nseq * d.heads;
        const long long jobs = walks * blocks * (w.segments - 1) + walks * (w.segments - 2);
        delta_walk_tc_kernel<kPanels, true><<<(unsigned)jobs, kWalkThreads, Lay::kBytes, stream>>>(q, k, v, w);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = launch_join(d, f.init, segments, w.half, parts, sms, err, stream)) != cudaSuccess) return e;
        w.d.cu = parts.cu;
        w.d.nseq *= w.segments;
        w.init = w.starts;
    }
    const long long ctas = (long long)w.d.nseq * d.heads * blocks;
    delta_walk_tc_kernel<kPanels, false><<<(unsigned)ctas, kWalkThreads, Lay::kBytes, stream>>>(q, k, v, w);
    return cudaGetLastError();
}

}  // namespace

namespace ssddelta {

// In how many parts a sequence is walked.  One walk a head leaves most SMs idle where there
// are few heads and sequences, and a part's end depends on its beginning by a map of N x N:
// the parts' own ends and their maps, side by side, then all parts again, which pays from
// three parts on, all at the same time on an SM each; a first part, which has no map, of half
// the others' length lets two of them have an SM after each other.  65536 tokens through 32
// heads of 128 x 128: 2200 us in one walk, 1580 in three parts, 1370 in four with the first of
// half the length.  Parts have 8 chunks at least (one head, 24 chunks: 70 us in one, 62 in
// three; 47 chunks: 123 in one, 76 in five), 12 where they fill more than half of the SMs (48
// heads, 24 chunks: 84 us in one, 94 in three; 47 chunks: 153 in one, 147 in three).  The walk
// back is split by the same rule (48 heads, 47 chunks: 423 us in one, 391 in three).
InParts segments_of(const SsdDelta &d, int sms) {
    const long long walks = (long long)d.nseq * d.heads, blocks = (d.p + 127) / 128;
    const long long chunks = d.tokens / kC / d.nseq;
    const int least = 6 * walks * blocks > sms ? 12 : 8;
    InParts best{1, 0};
    for (int s = 3; s <= 16 && s * least <= chunks && walks * blocks * s <= sms; ++s) {
        const long long others = walks * (blocks + 1) * (s - 2), firsts = walks * blocks;
        if (others + firsts <= sms) best = {s, 0};
        else if (others + (firsts + 1) / 2 <= sms) best = {s, 1};
    }
    return best;
}
Parts parts_of(const SsdDelta &d, int segments, uint8_t *at) {
    Parts p{};
    if (segments <= 1) return p;
    const size_t starts = (size_t)segments * d.nseq * d.heads * d.p * d.n * 4;
    const size_t maps = (size_t)(segments - 2) * d.nseq * d.heads * d.n * d.n * 4;
    p.bytes = starts + maps + (size_t)(segments * d.nseq + 1) * 4;
    p.starts = reinterpret_cast<float *>(at);
    p.maps = reinterpret_cast<float *>(at + starts);
    p.cu = reinterpret_cast<int *>(at + starts + maps);
    return p;
}
cudaError_t launch_join(const SsdDelta &d, const float *init, InParts parts, int half, const Parts &p, int sms,
                        unsigned *err, cudaStream_t stream) {
    const long long walks = (long long)d.nseq * d.heads;
    // (four rows a thread for as long as that is a CTA an SM: 8 heads in 16 parts 25 us, with eight
    // rows 34; 16 heads in 6 parts 23 and 17)
    const auto run = [&](auto kernel, int r) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, join_bytes(r));
        if (e != cudaSuccess) return e;
        const dim3 grid((unsigned)walks, (unsigned)((d.p + 2 * r - 1) / (2 * r)));
        kernel<<<grid, 256, join_bytes(r), stream>>>(d, init, parts.parts, half, p.cu, p.starts, p.maps, err);
        return cudaGetLastError();
    };
    return walks * ((d.p + 7) / 8) <= sms ? run(delta_join_kernel<4>, 4) : run(delta_join_kernel<8>, 8);
}

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

cudaError_t launch_chunks(const SsdDelta &d, uint8_t *records, bool least_beta, int sms, unsigned *err,
                          cudaStream_t stream) {
    return d.n <= 64 ? launch_chunks_of<1>(d, records, least_beta, sms, err, stream)
                     : launch_chunks_of<2>(d, records, least_beta, sms, err, stream);
}

}  // namespace ssddelta

// Types and sizes that these kernels take, and alignments: the copies' rows start on 16 bytes.
bool ssd_delta_tc_sizes(const SsdDelta &d) {
    return d.bf16 && d.n <= 128 && d.n % 8 == 0 && d.p % 8 == 0 && d.tokens > 0;
}
bool ssd_delta_tc_inputs(const SsdDelta &d) {
    const auto rows_ok = [](const void *p, long long stride) { return on_16(p) && stride % 8 == 0; };
    return ssd_delta_tc_sizes(d) && rows_ok(d.q, d.q_stride) && rows_ok(d.k, d.k_stride) && rows_ok(d.v, d.v_stride) &&
           ssd_tensor_map_encoder() != nullptr;
}
bool ssd_delta_tc_handles(const SsdDeltaFwd &a) {
    return ssd_delta_tc_inputs(a.in) && on_16(a.init) && on_16(a.final_state) && on_16(a.checkpoints);
}

size_t ssd_delta_tc_workspace(const SsdDelta &d, int sms) {
    if (!ssd_delta_tc_sizes(d)) return 0;
    return records_bytes(d) + parts_of(d, segments_of(d, sms).parts, nullptr).bytes;
}

cudaError_t ssd_launch_delta_fwd_tc(const SsdDeltaFwd &a, void *ws, int sms, unsigned *err, cudaStream_t stream) {
    return a.in.n <= 64 ? launch_fwd<1>(a, ws, sms, err, stream) : launch_fwd<2>(a, ws, sms, err, stream);
}
