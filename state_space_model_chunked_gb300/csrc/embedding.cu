// Embedding: rows of a table by tokens, and the table's gradient by sorted tokens.
//
//   y_t = table[token_t] scale               (zeros for a token outside the table)
//   dtable[v] = scale * sum over the t with token_t = v of dy_t
//
// Both are bound by memory.  The gradient is dense: rows that no token names are zeros.
// It is found without atomic additions, so equal calls give equal bits:
//   1. the tokens are sorted, stably, with their places (a radix sort of at most 9 bits a
//      pass, by one cluster whose CTAs exchange their digits' counts through distributed
//      shared memory; keys and places go through the workspace, that is, L2);
//   2. pieces of kPiece sorted tokens each add up their rows of dy in order.  A token whose
//      rows lie in one piece is written at once; the sums of one that goes on beyond its
//      piece are kept as parts.  Beside that, other CTAs write the zeros of the rows
//      that no token names;
//   3. the parts of such tokens are added in the pieces' order.
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
    int *key[2], *at[2];        // the last pass writes key[0], at[0]
};

// What a lane reads of the pass's input: the key (vocab: outside the table) and its place.
__device__ __forceinline__ void sort_input(const Sort &a, int pass, int from, int i, int &key, int &at) {
    if (pass == 0) {
        const int row = row_of(a.tokens, a.wide, i, a.vocab);
        key = row < 0 ? a.vocab : row;
        at = i;
    } else {
        key = __ldcg(a.key[from] + i);
        at = __ldcg(a.at[from] + i);
    }
}

__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(32 * kSortWarps)
sort_tokens_kernel(const Sort a) {
    extern __shared__ int sort_smem[];
    constexpr int kMost = 1 << kMostBits;
    int *const counts = sort_smem;                          // [warp][digit]
    int *const total = sort_smem + kSortWarps * kMost;      // [digit], read by the other CTAs
    int *const scan = total + kMost;                        // [warp]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)ssdptx::cluster_rank();
    const int digits = 1 << a.bits;
    // a warp's keys: a run of whole 32s
    const int run = (int)(((long long)a.count + 32ll * kSortCtas * kSortWarps - 1) / (32ll * kSortCtas * kSortWarps)) * 32;
    const long long begin = (long long)(rank * kSortWarps + warp) * run;
    const int end = (int)(begin + run < a.count ? begin + run : a.count);
    constexpr int kAhead = 4;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int to = (a.passes - 1 - pass) & 1, from = to ^ 1, shift = pass * a.bits;
        int *const mine = counts + warp * kMost;
        for (int d = lane; d < digits; d += 32) mine[d] = 0;
        __syncwarp();
        for (long long i0 = begin; i0 < end; i0 += 32 * kAhead) {
            int key[kAhead], at;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const long long i = i0 + 32 * u + lane;
                key[u] = -1;
                if (i < end) sort_input(a, pass, from, (int)i, key[u], at);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (key[u] >= 0) atomicAdd(mine + ((key[u] >> shift) & (digits - 1)), 1);
        }
        __syncthreads();
        // counts become, by digit, the number in the CTA's warps in front
        int all = 0;
        if (threadIdx.x < digits) {
            for (int w = 0; w < kSortWarps; ++w) {
                const int n = counts[w * kMost + threadIdx.x];
                counts[w * kMost + threadIdx.x] = all;
                all += n;
            }
            total[threadIdx.x] = all;
        }
        ssdptx::cluster_sync_all();
        // where the digit's keys of this CTA begin: behind the smaller digits and behind
        // the CTAs in front
        int front = 0, sum = 0;
        if (threadIdx.x < digits) {
            for (int c = 0; c < kSortCtas; ++c) {
                const int n = (int)ssdptx::cluster_ld_u32(
                    ssdptx::cluster_map(ssdptx::smem_u32(total + threadIdx.x), (uint32_t)c));
                if (c < rank) front += n;
                sum += n;
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
        int base = upto - sum + front;
        for (int w = 0; w < warp; ++w) base += scan[w];
        if (threadIdx.x < digits)
            for (int w = 0; w < kSortWarps; ++w) counts[w * kMost + threadIdx.x] += base;
        __syncthreads();
        for (long long i0 = begin; i0 < end; i0 += 32 * kAhead) {
            int key[kAhead], at[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const long long i = i0 + 32 * u + lane;
                key[u] = -1;
                if (i < end) sort_input(a, pass, from, (int)i, key[u], at[u]);
            }
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
                if (on) {
                    a.key[to][place] = key[u];
                    a.at[to][place] = at[u];
                }
            }
        }
        ssdptx::cluster_sync_all();
    }
}

// ------------------------------------------------------------------ gradient
constexpr int kPiece = 32;          // sorted tokens a CTA adds up
constexpr int kZeroRows = 64;       // table rows a CTA looks through for those without tokens
constexpr int kSumThreads = 128;

struct Gradient {
    const int *key, *at;            // sorted
    int count, vocab, width;
    const void *dy;
    long long dy_stride;
    float scale;
    void *dtable;
    float *parts;                   // [piece][2][width]: what its first and its last token's
                                    // run keep for the pieces beside it
    int pieces, blocks;             // column blocks
};

// The number of sorted keys below `v`.
__device__ __forceinline__ int keys_below(const int *key, int count, int v) {
    int lo = 0, hi = count;
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (__ldcg(key + mid) < v) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

template <typename T, typename TO, int V>
__global__ void __launch_bounds__(kSumThreads) embedding_bwd_kernel(const Gradient a) {
    ssdptx::griddep_wait();
    const int nvec = a.width / V;
    if ((long long)blockIdx.x >= (long long)a.pieces * a.blocks) {
        // the zeros of rows without tokens
        __shared__ unsigned char named[kZeroRows];
        __shared__ int ends[2];
        const long long r0 = ((long long)blockIdx.x - (long long)a.pieces * a.blocks) * kZeroRows;
        const int rows = (int)(a.vocab - r0 < kZeroRows ? a.vocab - r0 : kZeroRows);
        if (threadIdx.x < kZeroRows) named[threadIdx.x] = 0;
        if (threadIdx.x < 2) ends[threadIdx.x] = keys_below(a.key, a.count, (int)(threadIdx.x ? r0 + rows : r0));
        __syncthreads();
        for (int i = ends[0] + threadIdx.x; i < ends[1]; i += kSumThreads) named[__ldcg(a.key + i) - r0] = 1;
        __syncthreads();
        TO *out = static_cast<TO *>(a.dtable);
        const float zero[V] = {};
        for (int r = threadIdx.x >> 5; r < rows; r += kSumThreads / 32) {
            if (named[r]) continue;
            for (int i = threadIdx.x & 31; i < nvec; i += 32)
                ssd_store_vec<V>(out + (size_t)(r0 + r) * a.width + (size_t)i * V, zero);
        }
        return;
    }
    __shared__ int key[kPiece + 2], at[kPiece];     // key[0], key[n + 1]: the neighbours'
    const int piece = (int)(blockIdx.x / a.blocks), block = (int)(blockIdx.x % a.blocks);
    const int first = piece * kPiece, n = min(kPiece, a.count - first);
    if (threadIdx.x < n + 2) {
        const int i = first + (int)threadIdx.x - 1;
        key[threadIdx.x] = i >= 0 && i < a.count ? __ldcg(a.key + i) : -1;
        if (threadIdx.x >= 1 && threadIdx.x <= n) at[threadIdx.x - 1] = __ldcg(a.at + i);
    }
    __syncthreads();
    const int vec = block * kSumThreads + threadIdx.x;
    if (vec >= nvec) return;
    const T *dy = static_cast<const T *>(a.dy) + (size_t)vec * V;
    constexpr int kAhead = 8;
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
    const int first = piece * kPiece, last = first + kPiece - 1;
    if (last + 1 >= a.count) return;
    const int v = __ldcg(a.key + last);
    if (v >= a.vocab || __ldcg(a.key + last + 1) != v) return;
    // a run that fills the piece and began in front of it belongs to another CTA
    if (first > 0 && __ldcg(a.key + first) == v && __ldcg(a.key + first - 1) == v) return;
    const int vec = block * kSumThreads + threadIdx.x;
    if (vec >= a.width / V) return;
    const int behind = (keys_below(a.key, a.count, v + 1) - 1) / kPiece;    // the run's last piece
    const float *parts = a.parts + (size_t)vec * V;
    SsdRaw<float, V> r;
    r.load(parts + ((size_t)piece * 2 + 1) * a.width);
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = r.get(k);
    constexpr int kAhead = 8;
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
    int pieces;
};
BwdPlan bwd_plan(long long count, int width) {
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    BwdPlan p;
    p.pieces = (int)((count + kPiece - 1) / kPiece);
    p.keys = up((size_t)count * 4);
    p.parts = 4 * p.keys;
    p.total = p.parts + (p.pieces > 1 ? (size_t)p.pieces * 2 * width * 4 : 0);
    return p;
}

template <typename T, typename TO, int V>
cudaError_t launch_sums(Gradient g, cudaStream_t stream) {
    g.blocks = (g.width / V + kSumThreads - 1) / kSumThreads;
    const long long sums = (long long)g.pieces * g.blocks, zeros = ((long long)g.vocab + kZeroRows - 1) / kZeroRows;
    if (sums + zeros >= (1ll << 31)) return cudaErrorInvalidValue;
    cudaError_t e = ssd_launch_early(embedding_bwd_kernel<T, TO, V>, dim3((unsigned)(sums + zeros)),
                                     dim3(kSumThreads), stream, g);
    if (e != cudaSuccess || g.pieces < 2) return e;
    return ssd_launch_early(embedding_join_kernel<TO, V>, dim3((unsigned)sums), dim3(kSumThreads), stream, g);
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
    (void)sms;
    const BwdPlan plan = bwd_plan(a.count, a.width);
    char *at = static_cast<char *>(ws);
    Sort s{a.tokens, a.wide, (int)a.count, a.vocab, 1, 1, {}, {}};
    int bits = 1;
    while (a.vocab >> bits) ++bits;
    s.passes = (bits + kMostBits - 1) / kMostBits;
    s.bits = (bits + s.passes - 1) / s.passes;
    for (int i = 0; i < 2; ++i) {
        s.key[i] = reinterpret_cast<int *>(at + 2 * i * plan.keys);
        s.at[i] = reinterpret_cast<int *>(at + (2 * i + 1) * plan.keys);
    }
    constexpr int kSmem = (kSortWarps * (1 << kMostBits) + (1 << kMostBits) + kSortWarps) * 4;
    cudaError_t e = cudaFuncSetAttribute(sort_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    sort_tokens_kernel<<<kSortCtas, 32 * kSortWarps, kSmem, stream>>>(s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const Gradient g{s.key[0], s.at[0], (int)a.count, a.vocab, a.width, a.dy, a.dy_stride, a.scale, a.dtable,
                     reinterpret_cast<float *>(at + plan.parts), plan.pieces, 0};
    if (a.in == SSD_ELT_F32)
        return a.out_type == SSD_ELT_F32 ? launch_sums_of<float, float>(g, stream)
                                         : launch_sums_of<float, __nv_bfloat16>(g, stream);
    return a.out_type == SSD_ELT_F32 ? launch_sums_of<__nv_bfloat16, float>(g, stream)
                                     : launch_sums_of<__nv_bfloat16, __nv_bfloat16>(g, stream);
}
