// Embedding: rows of a table by tokens, and the table's gradient by sorted tokens.
//
//   y_t = table[token_t] scale               (zeros for a token outside the table)
//   dtable[v] = scale * sum over the t with token_t = v of dy_t
//
// Both are bound by memory.  The gradient is dense: rows that no token names are zeros.
// It is found without atomic additions, so equal calls give equal bits:
//   1. the tokens are sorted, stably, with their places (a radix sort of at most 9 bits a
//      pass, by one cluster whose CTAs exchange their digits' counts, and where they fit
//      their keys too, through distributed shared memory).  Beside the sort, which takes
//      eight SMs, others write zeros to all of the table, named rows or not: that takes
//      longer than the sort for most tables, where looking for the rows that no token names
//      would have to wait for it;
//   2. pieces of some sorted tokens each add up their rows of dy in order.  A token whose
//      rows lie in one piece is written at once; the sums of one that goes on beyond its
//      piece are kept as parts;
//   3. the parts of such tokens are added in the pieces' order.
// 65536 rows of 2560 bf16: 77 us (7.7 TB/s: repeated rows come from L2).  The gradient of
// 16376 tokens, 50000 x 1024 fp32: 54 us, 34 of them the zeros (6.0 TB/s), 18 the pieces, which
// write named rows again.  The sorted keys say which rows are unnamed (those between two
// neighbours), so zeros written behind the sort could leave the named rows out, up to 8 us of
// them; beside the sort, as here, they cannot.  Not built.
#include "launch.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace {

// A token's row of the table, or -1.
template <typename I>
__device__ __forceinline__ int row_of(const void *tokens, long long t, int vocab) {
    const I id = static_cast<const I *>(tokens)[t];
    return id >= 0 && id < (I)vocab ? (int)id : -1;
}
__device__ __forceinline__ int row_of(const void *tokens, bool wide, long long t, int vocab) {
    return wide ? row_of<long long>(tokens, t, vocab) : row_of<int>(tokens, t, vocab);
}

// ------------------------------------------------------------------- forward
// A warp takes a token's run of up to kU vectors a lane.
constexpr int kU = 4, kFwdThreads = 256;

template <typename TI, typename TO, int V>
__global__ void __launch_bounds__(kFwdThreads)
embedding_kernel(const SsdEmbedding a, const int parts, const int steps) {
    ssdptx::griddep_wait();
    const int nvec = a.width / V, lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (kFwdThreads / 32);
    for (long long unit = (long long)blockIdx.x * (kFwdThreads / 32) + (threadIdx.x >> 5);
         unit < a.count * parts; unit += warps) {
        const long long t = unit / parts;
        const int first = (int)(unit - t * parts) * steps * 32 + lane;
        const int row = row_of(a.tokens, a.wide, t, a.vocab);
        const TI *src = static_cast<const TI *>(a.table) + (size_t)(row < 0 ? 0 : row) * a.width;
        TO *dst = static_cast<TO *>(a.y) + (size_t)t * a.width;
        SsdRaw<TI, V> r[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = first + 32 * u;
            r[u].zero();
            if (row >= 0 && u < steps && i < nvec) r[u].load(src + (size_t)i * V);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = first + 32 * u;
            if (u >= steps || i >= nvec) continue;
            float v[V];
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = r[u].get(k) * a.scale;
            ssd_store_vec<V>(dst + (size_t)i * V, v);
        }
    }
}

template <typename TI, typename TO>
cudaError_t launch_fwd(const SsdEmbedding &a, int sms, cudaStream_t stream) {
    const bool v8 = a.width % 8 == 0 && (((uintptr_t)a.table | (uintptr_t)a.y) & 15u) == 0;
    const int nvec = v8 ? a.width / 8 : a.width;
    const int parts = (nvec + 32 * kU - 1) / (32 * kU);
    const int steps = (nvec + 32 * parts - 1) / (32 * parts);
    const long long units = a.count * parts, per = kFwdThreads / 32;
    const long long most = (long long)sms * 8;
    const long long want = (units + per - 1) / per;
    const dim3 grid((unsigned)(want < most ? want : most));
    return v8 ? ssd_launch_early(embedding_kernel<TI, TO, 8>, grid, dim3(kFwdThreads), stream, a, parts, steps)
              : ssd_launch_early(embedding_kernel<TI, TO, 1>, grid, dim3(kFwdThreads), stream, a, parts, steps);
}

// ------------------------------------------------------------------- sorting
constexpr int kSortCtas = 8, kSortWarps = 32, kMostBits = 9;
struct Sort {
    const void *tokens;
    bool wide;
    int count, vocab, passes, bits;
    int run;                    // a warp's keys, whole 32s
    int *key[2], *at[2];        // the last pass writes key[0], at[0]
    // beside the sort, by the clusters behind the first: zeros, from byte to byte (even)
    uint8_t *zero;
    size_t bytes;
};
// Shared memory: counts [warp][digit], their sums [digit], the warps' sums; then, where keys
// stay on chip, two buffers of the CTA's keys with their places.
constexpr int kSortWords = kSortWarps * (1 << kMostBits) + (1 << kMostBits) + kSortWarps;
constexpr int kSortMostBytes = 232448;
constexpr int kMostLocal = (kSortMostBytes - 4 * kSortWords) / (16 * 32 * kSortWarps) * 32;        // longest run that fits

// kLocal: between passes the keys lie in the CTAs' shared memory, else in the workspace.
template <bool kLocal>
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(32 * kSortWarps)
sort_tokens_kernel(const Sort a) {
    if (blockIdx.x >= kSortCtas) {
        const size_t head = (size_t)(-(intptr_t)a.zero & 15) < a.bytes ? (size_t)(-(intptr_t)a.zero & 15) : a.bytes;
        const size_t vectors = (a.bytes - head) / 16;
        uint4 *const to = reinterpret_cast<uint4 *>(a.zero + head);
        const size_t step = (size_t)(gridDim.x - kSortCtas) * 32 * kSortWarps;
        const size_t first = (size_t)(blockIdx.x - kSortCtas) * 32 * kSortWarps + threadIdx.x;
        for (size_t i = first; i < vectors; i += 4 * step) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + u * step < vectors) __stcs(to + i + u * step, make_uint4(0, 0, 0, 0));
        }
        if (first < head / 2) reinterpret_cast<uint16_t *>(a.zero)[first] = 0;
        const size_t tail = head + 16 * vectors + 2 * first;
        if (tail < a.bytes) *reinterpret_cast<uint16_t *>(a.zero + tail) = 0;
        return;
    }
    extern __shared__ int sort_smem[];
    constexpr int kMost = 1 << kMostBits;
    int *const counts = sort_smem;                          // [warp][digit]
    int *const total = sort_smem + kSortWarps * kMost;      // [digit], read by the other CTAs
    int *const scan = total + kMost;                        // [warp]
    uint2 *const local = reinterpret_cast<uint2 *>(sort_smem + kSortWords);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)ssdptx::cluster_rank();
    const int digits = 1 << a.bits, slice = a.run * kSortWarps;
    const long long begin = (long long)(rank * kSortWarps + warp) * a.run;
    const int end = (int)(begin + a.run < a.count ? begin + a.run : a.count);
    constexpr int kAhead = 4;
    const bool few = a.run <= 32 * kAhead;      // a lane's keys stay in its registers
    int key[kAhead], at[kAhead];
    // the keys of a pass (vocab: outside the table) and their places
    const auto load = [&](int pass, int from, long long i0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const long long i = i0 + 32 * u + lane;
            key[u] = -1;
            if (i >= end) continue;
            if (pass == 0) {
                const int row = row_of(a.tokens, a.wide, i, a.vocab);
                key[u] = row < 0 ? a.vocab : row;
                at[u] = (int)i;
            } else if constexpr (kLocal) {
                const uint2 x = local[from * slice + (int)(i - (long long)rank * slice)];
                key[u] = (int)x.x;
                at[u] = (int)x.y;
            } else {
                key[u] = __ldcg(a.key[from] + i);
                at[u] = __ldcg(a.at[from] + i);
            }
        }
    };
    for (int pass = 0; pass < a.passes; ++pass) {
        const int to = (a.passes - 1 - pass) & 1, from = to ^ 1, shift = pass * a.bits;
        const bool last = pass == a.passes - 1;
        int *const mine = counts + warp * kMost;
        for (int d = lane; d < digits; d += 32) mine[d] = 0;
        __syncwarp();
        for (long long i0 = begin; i0 < end; i0 += 32 * kAhead) {
            load(pass, from, i0);
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (key[u] >= 0) atomicAdd(mine + ((key[u] >> shift) & (digits - 1)), 1);
        }
        __syncthreads();
        // counts become, by digit, the number in the CTA's warps in front
        if (threadIdx.x < digits) {
            int all = 0;
#pragma unroll
            for (int w0 = 0; w0 < kSortWarps; w0 += 8) {
                int n[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) n[w] = counts[(w0 + w) * kMost + threadIdx.x];
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    counts[(w0 + w) * kMost + threadIdx.x] = all;
                    all += n[w];
                }
            }
            total[threadIdx.x] = all;
        }
        ssdptx::cluster_sync_all();
        // where the digit's keys of this CTA begin: behind the smaller digits and behind
        // the CTAs in front
        int front = 0, sum = 0;
        if (threadIdx.x < digits) {
            int n[kSortCtas];
#pragma unroll
            for (int c = 0; c < kSortCtas; ++c)
                n[c] = (int)ssdptx::cluster_ld_u32(ssdptx::cluster_map(ssdptx::smem_u32(total + threadIdx.x), (uint32_t)c));
#pragma unroll
            for (int c = 0; c < kSortCtas; ++c) {
                if (c < rank) front += n[c];
                sum += n[c];
            }
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += n;
        }
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
        int below = lane < warp ? scan[lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
        const int base = upto - sum + front + below;
        if (threadIdx.x < digits) {
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) counts[w * kMost + threadIdx.x] += base;
        }
        __syncthreads();
        for (long long i0 = begin; i0 < end; i0 += 32 * kAhead) {
            if (!few) load(pass, from, i0);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const bool on = key[u] >= 0;
                const int d = on ? (key[u] >> shift) & (digits - 1) : -1;
                const unsigned same = __match_any_sync(0xffffffffu, d);
                int place = 0;
                if (on) place = mine[d] + __popc(same & ((1u << lane) - 1u));
                __syncwarp();
                if (on && lane == __ffs(same) - 1) mine[d] += __popc(same);
                __syncwarp();
                if (!on) continue;
                if (kLocal && !last) {
                    const int cta = place / slice;
                    ssdptx::cluster_st_u32x2(
                        ssdptx::cluster_map(ssdptx::smem_u32(local + to * slice + place - cta * slice), (uint32_t)cta),
                        (uint32_t)key[u], (uint32_t)at[u]);
                } else {
                    a.key[to][place] = key[u];
                    a.at[to][place] = at[u];
                }
            }
        }
        ssdptx::cluster_sync_all();
    }
}

// ------------------------------------------------------------------ gradient
// Sorted tokens a CTA adds up: few enough for some hundred CTAs, many enough that parts are
// few.  us by (16, 32, 64): 2048 tokens 45 49 56, 16376 80 58 66, 65536 165 103 95.
constexpr int kMostPiece = 64;
int piece_of(long long count) { return count < 4096 ? 16 : count < 32768 ? 32 : kMostPiece; }
constexpr int kSumThreads = 512;

struct Gradient {
    const int *key, *at;            // sorted
    int count, vocab, width;
    const void *dy;
    long long dy_stride;
    float scale;
    void *dtable;
    float *parts;                   // [piece][2][width]: what its first and its last token's
                                    // run keep for the pieces beside it
    int piece, pieces, blocks;      // tokens a piece, pieces, column blocks
};

template <typename T, typename TO, int V>
__global__ void __launch_bounds__(kSumThreads) embedding_bwd_kernel(const Gradient a) {
    ssdptx::griddep_wait();
    const int nvec = a.width / V;
    __shared__ int key[kMostPiece + 2], at[kMostPiece];     // key[0], key[n + 1]: the neighbours'
    const int piece = (int)(blockIdx.x / a.blocks), block = (int)(blockIdx.x % a.blocks);
    const int first = piece * a.piece, n = min(a.piece, a.count - first);
    for (int t = threadIdx.x; t < n + 2; t += blockDim.x) {
        const int i = first + t - 1;
        key[t] = i >= 0 && i < a.count ? __ldcg(a.key + i) : -1;
        if (t >= 1 && t <= n) at[t - 1] = __ldcg(a.at + i);
    }
    __syncthreads();
    const int vec = block * (int)blockDim.x + (int)threadIdx.x;
    if (vec >= nvec) return;
    const T *dy = static_cast<const T *>(a.dy) + (size_t)vec * V;
    constexpr int kAhead = 16;
    float acc[V] = {};
    bool whole = key[0] != key[1];      // whether the token's run began in this piece
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        SsdRaw<T, V> r[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            r[u].zero();
            if (i0 + u < n && key[i0 + u + 1] < a.vocab) r[u].load_cs(dy + at[i0 + u] * a.dy_stride);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u;
            if (i >= n) break;
            const int v = key[i + 1];
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += r[u].get(k);
            const bool last = key[i + 2] != v;
            if (!last && i + 1 < n) continue;
            if (v < a.vocab) {
                if (whole && last) {
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[k] *= a.scale;
                    ssd_store_vec<V>(static_cast<TO *>(a.dtable) + (size_t)v * a.width + (size_t)vec * V, acc);
                } else {
                    ssd_store_vec<V>(a.parts + ((size_t)piece * 2 + (whole ? 1 : 0)) * a.width + (size_t)vec * V, acc);
                }
            }
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = 0.f;
            whole = true;
        }
    }
}

// Tokens whose rows lie in several pieces: the CTA of the piece that such a run begins in
// adds that piece's part and those of the pieces behind it, in order.
template <typename TO, int V>
__global__ void __launch_bounds__(kSumThreads) embedding_join_kernel(const Gradient a) {
    ssdptx::griddep_wait();
    const int piece = (int)(blockIdx.x / a.blocks), block = (int)(blockIdx.x % a.blocks);
    const long long first = (long long)piece * a.piece, last = first + a.piece - 1;
    if (last + 1 >= a.count) return;
    const int v = __ldcg(a.key + last);
    if (v >= a.vocab || __ldcg(a.key + last + 1) != v) return;
    // a run that fills the piece and began in front of it belongs to another CTA
    if (first > 0 && __ldcg(a.key + first) == v && __ldcg(a.key + first - 1) == v) return;
    // the run's last piece: those behind begin with its token too
    int behind = piece;
    for (const int lane = threadIdx.x & 31;;) {
        const long long next = (long long)(behind + 1 + lane) * a.piece;
        const unsigned goes_on = __ballot_sync(0xffffffffu, next < a.count && __ldcg(a.key + next) == v);
        const int n = goes_on == 0xffffffffu ? 32 : __ffs(~goes_on) - 1;
        behind += n;
        if (n < 32) break;
    }
    const int vec = block * (int)blockDim.x + (int)threadIdx.x;
    if (vec >= a.width / V) return;
    const float *parts = a.parts + (size_t)vec * V;
    SsdRaw<float, V> r;
    r.load(parts + ((size_t)piece * 2 + 1) * a.width);
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = r.get(k);
    constexpr int kAhead = 16;
    for (int p0 = piece + 1; p0 <= behind; p0 += kAhead) {
        SsdRaw<float, V> part[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            part[u].zero();
            if (p0 + u <= behind) part[u].load(parts + (size_t)(p0 + u) * 2 * a.width);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += part[u].get(k);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] *= a.scale;
    ssd_store_vec<V>(static_cast<TO *>(a.dtable) + (size_t)v * a.width + (size_t)vec * V, acc);
}

struct BwdPlan {
    size_t keys, parts, total;      // bytes of one array of keys, where the parts begin, all
    int piece, pieces;
};
BwdPlan bwd_plan(long long count, int width) {
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    BwdPlan p;
    p.piece = piece_of(count);
    p.pieces = (int)((count + p.piece - 1) / p.piece);
    p.keys = up((size_t)count * 4);
    p.parts = 4 * p.keys;
    p.total = p.parts + (p.pieces > 1 ? (size_t)p.pieces * 2 * width * 4 : 0);
    return p;
}

template <typename T, typename TO, int V>
cudaError_t launch_sums(Gradient g, cudaStream_t stream) {
    const int nvec = g.width / V;
    g.blocks = (nvec + kSumThreads - 1) / kSumThreads;
    const dim3 block((unsigned)(((nvec + g.blocks - 1) / g.blocks + 31) / 32 * 32));
    const long long sums = (long long)g.pieces * g.blocks;
    if (sums >= (1ll << 31)) return cudaErrorInvalidValue;
    cudaError_t e = ssd_launch_early(embedding_bwd_kernel<T, TO, V>, dim3((unsigned)sums), block, stream, g);
    if (e != cudaSuccess || g.pieces < 2) return e;
    return ssd_launch_early(embedding_join_kernel<TO, V>, dim3((unsigned)sums), block, stream, g);
}

template <typename T, typename TO>
cudaError_t launch_sums_of(const Gradient &g, cudaStream_t stream) {
    const bool v8 = g.width % 8 == 0 && (((uintptr_t)g.dy | (uintptr_t)g.dtable) & 15u) == 0 &&
                    (g.dy_stride * sizeof(T)) % 16 == 0;
    return v8 ? launch_sums<T, TO, 8>(g, stream) : launch_sums<T, TO, 1>(g, stream);
}

}  // namespace

cudaError_t ssd_launch_embedding(const SsdEmbedding &a, int sms, cudaStream_t stream) {
    if (a.table_type == SSD_ELT_F32)
        return a.out_type == SSD_ELT_F32 ? launch_fwd<float, float>(a, sms, stream)
                                         : launch_fwd<float, __nv_bfloat16>(a, sms, stream);
    return a.out_type == SSD_ELT_F32 ? launch_fwd<__nv_bfloat16, float>(a, sms, stream)
                                     : launch_fwd<__nv_bfloat16, __nv_bfloat16>(a, sms, stream);
}

size_t ssd_embedding_bwd_workspace(long long count, int vocab, int width) {
    (void)vocab;
    return bwd_plan(count, width).total;
}

cudaError_t ssd_launch_embedding_bwd(const SsdEmbeddingBwd &a, void *ws, int sms,
                                     cudaStream_t stream) {
    const BwdPlan plan = bwd_plan(a.count, a.width);
    char *at = static_cast<char *>(ws);
    Sort s{};
    s.tokens = a.tokens;
    s.wide = a.wide;
    s.count = (int)a.count;
    s.vocab = a.vocab;
    int bits = 1;
    while (a.vocab >> bits) ++bits;
    s.passes = (bits + kMostBits - 1) / kMostBits;
    s.bits = (bits + s.passes - 1) / s.passes;
    s.run = (int)((a.count + 32ll * kSortCtas * kSortWarps - 1) / (32ll * kSortCtas * kSortWarps)) * 32;
    for (int i = 0; i < 2; ++i) {
        s.key[i] = reinterpret_cast<int *>(at + 2 * i * plan.keys);
        s.at[i] = reinterpret_cast<int *>(at + (2 * i + 1) * plan.keys);
    }
    s.zero = static_cast<uint8_t *>(a.dtable);
    s.bytes = (size_t)a.vocab * a.width * (a.out_type == SSD_ELT_F32 ? 4 : 2);
    // As many clusters beside the sort's as the device holds at once with it: SMs come in
    // groups of no multiple of eight, so it is fewer than its SMs over eight, and one more
    // would wait for the sort's end (50 us for 205 MB with 18 of them, 35 with 14)
    const size_t per = (size_t)kSortCtas * 32 * kSortWarps * 64;        // bytes a cluster takes at once
    const size_t want = (s.bytes + per - 1) / per, most = sms / kSortCtas > 6 ? sms / kSortCtas - 5 : 1;
    const unsigned ctas = kSortCtas * (1 + (unsigned)(want < most ? want : most));
    const bool local = s.run <= kMostLocal;
    const auto kernel = local ? sort_tokens_kernel<true> : sort_tokens_kernel<false>;
    const int smem = 4 * kSortWords + (local && s.passes > 1 ? 16 * s.run * kSortWarps : 0);
    // (the most that any call takes: the attribute is the kernel's, and another thread may be
    // about to launch it with more than this call needs)
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortMostBytes);
    if (e != cudaSuccess) return e;
    kernel<<<ctas, 32 * kSortWarps, smem, stream>>>(s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const Gradient g{s.key[0], s.at[0], (int)a.count, a.vocab, a.width, a.dy, a.dy_stride, a.scale, a.dtable,
                     reinterpret_cast<float *>(at + plan.parts), plan.piece, plan.pieces, 0};
    if (a.in == SSD_ELT_F32)
        return a.out_type == SSD_ELT_F32 ? launch_sums_of<float, float>(g, stream)
                                         : launch_sums_of<float, __nv_bfloat16>(g, stream);
    return a.out_type == SSD_ELT_F32 ? launch_sums_of<__nv_bfloat16, float>(g, stream)
                                     : launch_sums_of<__nv_bfloat16, __nv_bfloat16>(g, stream);
}
