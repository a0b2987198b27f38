// Gated delta rule in fp32 multiply-adds, token by token, for every size and type that the
// tensor-core kernels do not take, forward and backward.
//
//   S' = exp(g_t) S_{t-1},  u_t = beta_t (v_t - S' k_t),  S_t = S' + u_t k_t^T
//   o_t = scale S_t q_t                               S [P][N] a head
//
// The rows p of S do not meet but in the gradients of q and k, so a CTA takes a slab of
// rows of one head.  Eight lanes share a row: lane l of them holds the columns
// 32 j + 4 l + i (i < 4), which lie in shared memory as vectors of 16 bytes; a thread has
// kR rows.  o_t = scale (exp(g_t) S_{t-1} q_t + u_t (k_t q_t)), so both of a token's
// products with the state are taken of S_{t-1}, in one round of sums over the lanes.
//
// Backward, with L_t the gradient of S_t (from dfinal on, last token first):
//   L += scale do_t q_t^T;   w_t = L k_t (the gradient of u_t);   dv_t = beta_t w_t
//   dbeta_t = w_t (v_t - S' k_t);   L' = L - dv_t k_t^T;   L_{t-1} = exp(g_t) L'
//   dq_t = scale S_t^T do_t;   dk_t = L^T u_t - S'^T dv_t;   dg_t = <L', S'>
// The states are made again from those kept at every 64th token, all runs of 64 at once:
//   1. u_t of all tokens (runs of 64 side by side)
//   2. the walk back: w_t of all tokens, L^T u_t, and <L, S> before each run of 64
//   3. S again, with dq_t, S'^T dv_t, dbeta_t; and dg_t from
//      dg_{t+1} = dg_t - do_t o_t + dv_t v_t,  which starts anew at every 64th token
//   4. the sums over a group's heads and a head's slabs, rounded once.
// Bound by the fp32 pipe: about 4 P N multiply-adds a token forward, 12 backward, where one
// head's tokens follow each other at the latency of a token's two sums over eight lanes.
// 4 x 77 tokens, 8 heads of 64 x 64: 22 us, 0.29 a token.  8 x 2047 tokens, 16 heads of
// 128 x 128: 2.14 ms (16 TFLOP/s), in bf16 2.16, gradients 8.7 ms.  States and fp32 gradients
// are 1e-7 of their size off, those of g 5e-7.
#include "delta_tc.cuh"

namespace {

using ssddelta::chunk_at;
using ssddelta::ChunkAt;

constexpr int kC = kSsdDeltaChunk;
constexpr int kThreads = 256, kLanes = 8, kRowsPass = kThreads / kLanes;
constexpr int kTile = 16;           // tokens staged in shared memory at once

// Decays below this are zero in fp32 with room to spare; infinite ones would make 0 * inf.
__device__ __forceinline__ float decay_of(float g) { return expf(g < -200.f ? -200.f : g); }

__device__ __forceinline__ float load(const void *p, size_t i, bool bf16) {
    return bf16 ? ssd_ld(static_cast<const __nv_bfloat16 *>(p) + i) : ssd_ld(static_cast<const float *>(p) + i);
}
__device__ __forceinline__ void store(void *p, size_t i, bool bf16, float v) {
    if (bf16) ssd_st(static_cast<__nv_bfloat16 *>(p) + i, v);
    else ssd_st(static_cast<float *>(p) + i, v);
}

__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A sequence's tokens on the token axis.
__device__ __forceinline__ void range_of(const SsdDelta &d, int seq, long long &first, int &len) {
    if (d.cu) {
        first = d.cu[seq];
        len = d.cu[seq + 1] - d.cu[seq];
    } else {
        first = (long long)seq * d.length;
        len = d.length;
    }
}

// A CTA's head, slab of rows and, where it walks a sequence, that.
struct Place {
    int seq, head, slab, len, run;      // run: of 64 tokens, of a sequence's
    long long first;
};
__device__ __forceinline__ Place sequence_place(const SsdDelta &d, int slabs) {
    Place p{};
    p.slab = (int)(blockIdx.x % slabs);
    p.head = (int)(blockIdx.x / slabs % d.heads);
    p.seq = (int)(blockIdx.x / slabs / d.heads);
    range_of(d, p.seq, p.first, p.len);
    return p;
}
// Runs of 64 tokens side by side, numbered: sequences of one length have as many runs each;
// packed ones go by the kept states' slots, at most one more than runs a sequence, whatever the
// lengths.  (32 sequences of 500 by slots too: 2150 -> 2250 us.)
__host__ __device__ inline long long runs_of(const SsdDelta &d) {
    return d.cu ? ssd_delta_slots(d.tokens, d.nseq) : (long long)d.nseq * ((d.length + kC - 1) / kC);
}
__device__ __forceinline__ ChunkAt run_at(const SsdDelta &d, long long number) {
    if (d.cu) return chunk_at(d, number);
    ChunkAt at;
    at.seq = (int)(number % d.nseq);
    at.chunk = (int)(number / d.nseq);
    at.first = (long long)at.seq * d.length;
    at.len = d.length;
    at.live = true;
    return at;
}
// A CTA's run; false: none.
__device__ __forceinline__ bool run_place(const SsdDelta &d, int slabs, Place &p) {
    const ChunkAt at = run_at(d, blockIdx.x / slabs / d.heads);
    p.slab = (int)(blockIdx.x % slabs);
    p.head = (int)(blockIdx.x / slabs % d.heads);
    // (the same in every thread, which the compiler cannot see behind a search)
    const auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    p.seq = same(at.seq);
    p.first = same((int)at.first);      // (tokens are counted by ints)
    p.len = same(at.len);
    p.run = same(at.chunk);
    return same(at.live);
}

// One thread's part of the state: kR rows of kV columns.
template <int kV, int kR>
struct State {
    float s[kR][kV];
    int row[kR];        // of the head, or -1
    int lane;

    __device__ __forceinline__ void place(int slab, int p) {
        lane = threadIdx.x % kLanes;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int at = slab * kRowsPass * kR + r * kRowsPass + threadIdx.x / kLanes;
            row[r] = at < p ? at : -1;
        }
    }
    __device__ __forceinline__ static int column(int lane, int i) { return i / 4 * 32 + lane * 4 + i % 4; }
    // from / to [P][N] (null: zeros)
    __device__ __forceinline__ void load(const float *m, int n) {
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const int c = column(lane, i);
                s[r][i] = m && row[r] >= 0 && c < n ? m[(size_t)row[r] * n + c] : 0.f;
            }
    }
    __device__ __forceinline__ void store(float *m, int n) const {
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const int c = column(lane, i);
                if (row[r] >= 0 && c < n) m[(size_t)row[r] * n + c] = s[r][i];
            }
    }
};

// A lane's columns of a staged row of 8 kV values.
template <int kV>
__device__ __forceinline__ void columns(const float *row, int lane, float (&v)[kV]) {
#pragma unroll
    for (int i = 0; i < kV; i += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(row + i * 8 + lane * 4);
        v[i] = x.x;
        v[i + 1] = x.y;
        v[i + 2] = x.z;
        v[i + 3] = x.w;
    }
}
// (in four sums: one would be a chain of kV additions)
template <int kV>
__device__ __forceinline__ float dot(const float (&a)[kV], const float (&b)[kV]) {
    float v[4] = {};
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i & 3] += a[i] * b[i];
    return (v[0] + v[1]) + (v[2] + v[3]);
}

// kTile tokens' rows of `width` values at `offset` of each token, zeros behind them and in
// the columns up to `pad`.
__device__ __forceinline__ void stage(float *to, int pad, const void *from, bool bf16, long long token,
                                      long long stride, size_t offset, int width, int tokens) {
    for (int i = threadIdx.x; i < kTile * pad; i += kThreads) {
        const int t = i / pad, c = i - t * pad;
        to[i] = t < tokens && c < width ? load(from, (size_t)(token + t) * stride + offset + c, bf16) : 0.f;
    }
}

// ------------------------------------------------------------------- forward
// Whole sequences (kU false: o, the final state, the kept ones), or of every run of 64
// tokens from its kept state the u_t alone.
struct Walk {
    SsdDelta d;
    const float *init, *kept;
    void *o;
    long long o_stride;
    float *final_state, *checkpoints, *u;       // u [tokens][heads][P]
    int slabs;
};

template <int kV, int kR>
struct WalkTile {
    static constexpr int kN = kV * kLanes, kRows = kRowsPass * kR;
    float q[kTile][kN], k[kTile][kN], v[kTile][kRows];
    float decay[kTile], beta[kTile], kq[kTile];
};
// kTile tokens' rows of `pad` values, in the registers of kThreads threads on their way: as they
// lie in memory, since a conversion would wait for the load that it follows.
template <int kCount>
struct Ahead {
    static constexpr int kEach = (kCount + kThreads - 1) / kThreads;
    uint32_t x[kEach];
    __device__ __forceinline__ void fetch(int pad, const void *from, bool bf16, long long token, long long stride,
                                          size_t offset, int width, int tokens) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = threadIdx.x + j * kThreads, t = i / pad, c = i % pad;
            x[j] = 0;
            if (i >= kCount || t >= tokens || c >= width) continue;
            const size_t at = (size_t)(token + t) * stride + offset + c;
            x[j] = bf16 ? static_cast<const uint16_t *>(from)[at] : static_cast<const uint32_t *>(from)[at];
        }
    }
    __device__ __forceinline__ void put(float *to, bool bf16) const {
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            if (threadIdx.x + j * kThreads < kCount) to[threadIdx.x + j * kThreads] = __uint_as_float(bf16 ? x[j] << 16 : x[j]);
    }
};

template <int kV, int kR, bool kU>
__global__ void __launch_bounds__(kThreads) delta_walk_kernel(const Walk a) {
    extern __shared__ __align__(16) unsigned char delta_smem[];
    using Tile = WalkTile<kV, kR>;
    Tile *const tiles = reinterpret_cast<Tile *>(delta_smem);
    constexpr int kN = kV * kLanes, kRows = kRowsPass * kR;
    const SsdDelta &d = a.d;
    Place place;
    if constexpr (kU) {
        if (!run_place(d, a.slabs, place)) return;
    } else {
        place = sequence_place(d, a.slabs);
    }
    const int seq = place.seq, head = place.head, slab = place.slab, run = place.run, len = place.len;
    const long long first = place.first;
    const int group = head / (d.heads / d.groups);
    const size_t size = (size_t)d.p * d.n, state = ((size_t)seq * d.heads + head) * size;
    State<kV, kR> S;
    S.place(slab, d.p);
    int from = 0, to = len;
    if constexpr (kU) {
        from = run * kC;
        to = min(len, from + kC);
        S.load(a.kept + ((size_t)ssd_delta_slot(first, seq, run) * d.heads + head) * size, d.n);
    } else {
        S.load(a.init ? a.init + state : nullptr, d.n);
    }
    const int rows = min(kRows, d.p - slab * kRows), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the next tile is loaded while the present one is used
    Ahead<kTile * kN> qa, ka;
    Ahead<kTile * kRows> va;
    float ga = 0.f, ba = 0.f;
    const auto fetch = [&](int t0) {
        const int tokens = min(kTile, to - t0);
        ka.fetch(kN, d.k, d.bf16, first + t0, d.k_stride, (size_t)group * d.n, d.n, tokens);
        if constexpr (!kU) qa.fetch(kN, d.q, d.bf16, first + t0, d.q_stride, (size_t)group * d.n, d.n, tokens);
        va.fetch(kRows, d.v, d.bf16, first + t0, d.v_stride, (size_t)head * d.p + slab * kRows, rows, tokens);
        if (threadIdx.x < tokens) {
            const size_t i = (size_t)(first + t0 + threadIdx.x) * d.heads + head;
            ga = d.g[i];
            ba = d.beta[i];
        }
    };
    if (from < to) fetch(from);
    for (int t0 = from; t0 < to; t0 += kTile) {
        Tile &m = tiles[(t0 - from) / kTile & 1];
        ka.put(&m.k[0][0], d.bf16);
        if constexpr (!kU) qa.put(&m.q[0][0], d.bf16);
        va.put(&m.v[0][0], d.bf16);
        if (threadIdx.x < kTile) {
            m.decay[threadIdx.x] = decay_of(ga);
            m.beta[threadIdx.x] = ba;
        }
        // (one barrier a tile: the other buffer is written only behind the next one)
        __syncthreads();
        const int tokens = min(kTile, to - t0);
        if (t0 + kTile < to) fetch(t0 + kTile);
        if constexpr (!kU) {
            // k_t q_t, a token a warp
            for (int t = warp; t < tokens; t += kThreads / 32) {
                float v = 0.f;
                for (int c = lane; c < kN; c += 32) v += m.k[t][c] * m.q[t][c];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0) m.kq[t] = v;
            }
            __syncthreads();
            if (a.checkpoints && t0 % kC == 0)
                S.store(a.checkpoints + ((size_t)ssd_delta_slot(first, seq, t0 / kC) * d.heads + head) * size, d.n);
        }
        // Where a lane has many columns and one row, a token's keys and queries are read while the
        // one in front is in its sums (16384 tokens, 32 heads of 128 x 128: 6.8 -> 5.8 ms; with 8
        // columns, 77 tokens of 64 x 64, 22 -> 24 us; with two rows and all SMs full 2.8 -> 2.9 ms).
        constexpr bool kEarly = kV > 8 && kR == 1;
        float kc[kV], qc[kV], f, be, v[kR];
        const auto read = [&](int t, float (&kt)[kV], float (&qt)[kV], float &ft, float &bt, float (&vt)[kR]) {
            columns(m.k[t], S.lane, kt);
            if constexpr (!kU) columns(m.q[t], S.lane, qt);
            ft = m.decay[t];
            bt = m.beta[t];
#pragma unroll
            for (int r = 0; r < kR; ++r) vt[r] = m.v[t][r * kRowsPass + threadIdx.x / kLanes];
        };
        if constexpr (kEarly) read(0, kc, qc, f, be, v);
        for (int t = 0; t < tokens; ++t) {
            float sk[kR], sq[kR], kn[kV], qn[kV], fn, bn, vn[kR];
            if constexpr (!kEarly) read(t, kc, qc, f, be, v);
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                sk[r] = dot(S.s[r], kc);
                if constexpr (!kU) sq[r] = dot(S.s[r], qc);
            }
            if constexpr (kEarly) read(t + 1 < kTile ? t + 1 : t, kn, qn, fn, bn, vn);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    sk[r] += __shfl_xor_sync(0xffffffffu, sk[r], o);
                    if constexpr (!kU) sq[r] += __shfl_xor_sync(0xffffffffu, sq[r], o);
                }
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                const float u = be * (v[r] - f * sk[r]);
#pragma unroll
                for (int i = 0; i < kV; ++i) S.s[r][i] = f * S.s[r][i] + u * kc[i];
                if (S.lane == 0 && S.row[r] >= 0) {
                    const size_t at = (size_t)head * d.p + S.row[r];
                    if constexpr (kU) a.u[(size_t)(first + t0 + t) * d.heads * d.p + at] = u;
                    else store(a.o, (size_t)(first + t0 + t) * a.o_stride + at, d.bf16, d.scale * (f * sq[r] + u * m.kq[t]));
                }
                if constexpr (kEarly) v[r] = vn[r];
            }
            if constexpr (kEarly) {
#pragma unroll
                for (int i = 0; i < kV; ++i) {
                    kc[i] = kn[i];
                    if constexpr (!kU) qc[i] = qn[i];
                }
                f = fn;
                be = bn;
            }
        }
    }
    if constexpr (!kU) {
        if (a.final_state) S.store(a.final_state + state, d.n);
    }
}

// ------------------------------------------------------------------ backward
struct Back {
    SsdDelta d;
    const void *dout;
    const float *kept, *dfinal;
    long long do_stride, dv_stride;
    void *dv;
    float *dinit;
    float *u, *w;           // [tokens][heads][P]
    float *dq, *dk;         // [tokens][heads][slabs][N], sums over a slab's rows
    float *anchor;          // [slots][heads][slabs]: <L, S> before a run of 64 tokens
    float *ov, *rw;         // [tokens][heads][slabs]: do_t o_t - dv_t v_t and w_t (v_t - S' k_t)
    int slabs;
};

// The warp's sum over its rows (4 groups of lanes, kR rows each) of x_r s_r, into `part`'s
// row of this warp.
template <int kV, int kR>
__device__ __forceinline__ void rows_sum(const float (&s)[kR][kV], const float (&x)[kR], float *part) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < kR; ++r) v += s[r][i] * x[r];
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        if ((threadIdx.x & 31) < kLanes) part[State<kV, kR>::column(threadIdx.x % kLanes, i)] = v;
    }
}
// The CTA's sum of one value a thread, in thread 0.
__device__ __forceinline__ float cta_sum(float v, float *buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) v += buf[w];
    return v;
}

constexpr int kBackTile = 8;        // tokens whose sums over the warps wait in shared memory

template <int kV, int kR>
struct BackSmem {
    static constexpr int kN = kV * kLanes, kRows = kRowsPass * kR;
    float q[kTile][kN], k[kTile][kN];
    float part[kBackTile][kThreads / 32][kN];
    float x[kTile][kRows], y[kTile][kRows], z[kTile][kRows];
    float decay[kTile], beta[kTile];
    float sums[2][kBackTile][kThreads / 32];
    float buf[kThreads / 32];
};

// Step 2: the walk back.
template <int kV, int kR>
__global__ void __launch_bounds__(kThreads) delta_back_kernel(const Back a) {
    extern __shared__ __align__(16) unsigned char delta_smem[];
    auto &m = *reinterpret_cast<BackSmem<kV, kR> *>(delta_smem);
    constexpr int kN = kV * kLanes, kRows = kRowsPass * kR;
    const SsdDelta &d = a.d;
    const Place place = sequence_place(d, a.slabs);
    const int seq = place.seq, head = place.head, slab = place.slab, len = place.len;
    const long long first = place.first;
    const int group = head / (d.heads / d.groups);
    const size_t size = (size_t)d.p * d.n, state = ((size_t)seq * d.heads + head) * size;
    State<kV, kR> L;
    L.place(slab, d.p);
    L.load(a.dfinal ? a.dfinal + state : nullptr, d.n);
    const int rows = min(kRows, d.p - slab * kRows), warp = threadIdx.x >> 5;
    const size_t wide = (size_t)d.heads * a.slabs;
    for (int t0 = len ? (len - 1) / kTile * kTile : -1; t0 >= 0; t0 -= kTile) {
        const int tokens = min(kTile, len - t0);
        __syncthreads();
        stage(&m.q[0][0], kN, d.q, d.bf16, first + t0, d.q_stride, (size_t)group * d.n, d.n, tokens);
        stage(&m.k[0][0], kN, d.k, d.bf16, first + t0, d.k_stride, (size_t)group * d.n, d.n, tokens);
        const size_t at = (size_t)head * d.p + slab * kRows;
        stage(&m.x[0][0], kRows, a.dout, d.bf16, first + t0, a.do_stride, at, rows, tokens);
        stage(&m.y[0][0], kRows, a.u, false, first + t0, (long long)d.heads * d.p, at, rows, tokens);
        if (threadIdx.x < tokens) {
            const size_t i = (size_t)(first + t0 + threadIdx.x) * d.heads + head;
            m.decay[threadIdx.x] = decay_of(d.g[i]);
            m.beta[threadIdx.x] = d.beta[i];
        }
        __syncthreads();
        for (int b0 = (tokens - 1) / kBackTile * kBackTile; b0 >= 0; b0 -= kBackTile) {
            const int part = min(kBackTile, tokens - b0);
            for (int b = part - 1; b >= 0; --b) {
                const int t = b0 + b;
                float kc[kV], qc[kV], x[kR], w[kR];
                columns(m.k[t], L.lane, kc);
                columns(m.q[t], L.lane, qc);
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    x[r] = m.y[t][r * kRowsPass + threadIdx.x / kLanes];
                    const float dout = d.scale * m.x[t][r * kRowsPass + threadIdx.x / kLanes];
#pragma unroll
                    for (int i = 0; i < kV; ++i) L.s[r][i] += dout * qc[i];
                    w[r] = lanes_sum(dot(L.s[r], kc));
                }
                rows_sum<kV, kR>(L.s, x, m.part[b][warp]);
                const float f = m.decay[t];
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const float dv = m.beta[t] * w[r];
#pragma unroll
                    for (int i = 0; i < kV; ++i) L.s[r][i] = f * (L.s[r][i] - dv * kc[i]);
                    if (L.lane == 0 && L.row[r] >= 0) {
                        const size_t token = (size_t)(first + t0 + t), row = (size_t)head * d.p + L.row[r];
                        a.w[token * d.heads * d.p + row] = w[r];
                        store(a.dv, token * a.dv_stride + row, d.bf16, dv);
                    }
                }
            }
            __syncthreads();
            float *const out = a.dk + ((size_t)(first + t0 + b0) * wide + head * a.slabs + slab) * d.n;
            for (int i = threadIdx.x; i < part * kN; i += kThreads) {
                const int t = i / kN, c = i % kN;
                if (c >= d.n) continue;
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) v += m.part[t][w][c];
                out[(size_t)t * wide * d.n + c] = v;
            }
            __syncthreads();
        }
        if (t0 % kC == 0) {
            const size_t slot = (size_t)ssd_delta_slot(first, seq, t0 / kC);
            State<kV, kR> S;
            S.place(slab, d.p);
            S.load(a.kept + (slot * d.heads + head) * size, d.n);
            float v = 0.f;
#pragma unroll
            for (int r = 0; r < kR; ++r) v += dot(L.s[r], S.s[r]);
            v = cta_sum(v, m.buf);
            if (threadIdx.x == 0) a.anchor[slot * wide + head * a.slabs + slab] = v;
        }
    }
    if (a.dinit) L.store(a.dinit + state, d.n);
}

// Step 3: a run of 64 tokens forward again.
template <int kV, int kR>
__global__ void __launch_bounds__(kThreads) delta_again_kernel(const Back a) {
    extern __shared__ __align__(16) unsigned char delta_smem[];
    auto &m = *reinterpret_cast<BackSmem<kV, kR> *>(delta_smem);
    constexpr int kN = kV * kLanes, kRows = kRowsPass * kR;
    const SsdDelta &d = a.d;
    Place place;
    if (!run_place(d, a.slabs, place)) return;
    const int seq = place.seq, head = place.head, slab = place.slab, run = place.run, len = place.len;
    const long long first = place.first;
    const int group = head / (d.heads / d.groups);
    const int from = run * kC, to = min(len, from + kC);
    const size_t size = (size_t)d.p * d.n;
    State<kV, kR> S;
    S.place(slab, d.p);
    S.load(a.kept + ((size_t)ssd_delta_slot(first, seq, run) * d.heads + head) * size, d.n);
    const int rows = min(kRows, d.p - slab * kRows), warp = threadIdx.x >> 5;
    const size_t wide = (size_t)d.heads * a.slabs;
    for (int t0 = from; t0 < to; t0 += kBackTile) {
        const int tokens = min(kBackTile, to - t0);
        __syncthreads();
        stage(&m.q[0][0], kN, d.q, d.bf16, first + t0, d.q_stride, (size_t)group * d.n, d.n, tokens);
        stage(&m.k[0][0], kN, d.k, d.bf16, first + t0, d.k_stride, (size_t)group * d.n, d.n, tokens);
        const size_t at = (size_t)head * d.p + slab * kRows;
        stage(&m.x[0][0], kRows, a.dout, d.bf16, first + t0, a.do_stride, at, rows, tokens);
        stage(&m.y[0][0], kRows, a.w, false, first + t0, (long long)d.heads * d.p, at, rows, tokens);
        stage(&m.z[0][0], kRows, d.v, d.bf16, first + t0, d.v_stride, at, rows, tokens);
        if (threadIdx.x < tokens) {
            const size_t i = (size_t)(first + t0 + threadIdx.x) * d.heads + head;
            m.decay[threadIdx.x] = decay_of(d.g[i]);
            m.beta[threadIdx.x] = d.beta[i];
        }
        __syncthreads();
        const size_t out = ((size_t)(first + t0) * wide + head * a.slabs + slab) * d.n;
        // S' with S'^T dv, then S with S^T do: the sums over the warps of one token's two
        // rows go out in turn, kBackTile / 2 tokens at a time
        for (int b0 = 0; b0 < tokens; b0 += kBackTile / 2) {
            const int part = min(kBackTile / 2, tokens - b0);
            for (int b = 0; b < part; ++b) {
                const int t = b0 + b;
                float kc[kV], qc[kV], minus[kR], dout[kR], ov = 0.f, rw = 0.f;
                columns(m.k[t], S.lane, kc);
                columns(m.q[t], S.lane, qc);
                const float f = m.decay[t], be = m.beta[t];
                float u[kR];
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const int i0 = r * kRowsPass + threadIdx.x / kLanes;
                    const float w = m.y[t][i0], v = m.z[t][i0];
                    dout[r] = d.scale * m.x[t][i0];
                    minus[r] = -be * w;
#pragma unroll
                    for (int i = 0; i < kV; ++i) S.s[r][i] *= f;
                    const float miss = v - lanes_sum(dot(S.s[r], kc));
                    u[r] = be * miss;
                    rw += w * miss;
                    ov += minus[r] * v;
                }
                rows_sum<kV, kR>(S.s, minus, m.part[2 * b][warp]);
#pragma unroll
                for (int r = 0; r < kR; ++r) {
#pragma unroll
                    for (int i = 0; i < kV; ++i) S.s[r][i] += u[r] * kc[i];
                    ov += dout[r] * lanes_sum(dot(S.s[r], qc));
                }
                rows_sum<kV, kR>(S.s, dout, m.part[2 * b + 1][warp]);
                // eight lanes hold the same sums: one of them counts
                ov = S.lane == 0 ? ov : 0.f;
                rw = S.lane == 0 ? rw : 0.f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    ov += __shfl_xor_sync(0xffffffffu, ov, o);
                    rw += __shfl_xor_sync(0xffffffffu, rw, o);
                }
                if ((threadIdx.x & 31) == 0) {
                    m.sums[0][t][warp] = ov;
                    m.sums[1][t][warp] = rw;
                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * part * kN; i += kThreads) {
                const int t = i / kN / 2, which = i / kN % 2, c = i % kN;
                if (c >= d.n) continue;
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) v += m.part[2 * t + which][w][c];
                const size_t o = out + (size_t)(b0 + t) * wide * d.n + c;
                if (which) a.dq[o] = v;
                else a.dk[o] += v;
            }
            __syncthreads();
        }
        if (threadIdx.x < tokens) {
            float ov = 0.f, rw = 0.f;
            for (int w = 0; w < kThreads / 32; ++w) {
                ov += m.sums[0][threadIdx.x][w];
                rw += m.sums[1][threadIdx.x][w];
            }
            const size_t i = (size_t)(first + t0 + threadIdx.x) * wide + head * a.slabs + slab;
            a.ov[i] = ov;
            a.rw[i] = rw;
        }
    }
}

// Step 4: dq and dk, a group's sum over its heads and slabs.
struct Sums {
    const float *from;      // [tokens][groups][parts][N]
    void *to;
    long long tokens, stride;
    int groups, parts, n;
    bool bf16;
};
__global__ void __launch_bounds__(256) delta_group_sum_kernel(const Sums q, const Sums k) {
    const Sums &a = blockIdx.y ? k : q;
    const long long all = a.tokens * a.groups * a.n;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
        const long long row = i / a.n;
        const int c = (int)(i - row * a.n);
        float v = 0.f;
        for (int s = 0; s < a.parts; ++s) v += a.from[((size_t)row * a.parts + s) * a.n + c];
        const long long t = row / a.groups;
        store(a.to, (size_t)t * a.stride + (size_t)(row - t * a.groups) * a.n + c, a.bf16, v);
    }
}
// ... and dbeta and dg: a thread a head and run of 64 tokens.
__global__ void __launch_bounds__(128) delta_gates_kernel(const Back a, float *dg, float *dbeta) {
    const SsdDelta &d = a.d;
    const size_t wide = (size_t)d.heads * a.slabs;
    const long long all = runs_of(d) * d.heads;
    for (long long i = (long long)blockIdx.x * 128 + threadIdx.x; i < all; i += (long long)gridDim.x * 128) {
        const int head = (int)(i % d.heads);
        const ChunkAt run = run_at(d, i / d.heads);
        if (!run.live) continue;
        const long long first = run.first;
        const int len = run.len, chunk = run.chunk;
        const float *anchor = a.anchor + (size_t)ssd_delta_slot(first, run.seq, chunk) * wide + head * a.slabs;
        float at = 0.f;
        for (int s = 0; s < a.slabs; ++s) at += anchor[s];
        for (int t = chunk * kC; t < min(len, chunk * kC + kC); ++t) {
            const size_t token = (size_t)(first + t);
            float ov = 0.f, rw = 0.f;
            for (int s = 0; s < a.slabs; ++s) {
                ov += a.ov[token * wide + head * a.slabs + s];
                rw += a.rw[token * wide + head * a.slabs + s];
            }
            dg[token * d.heads + head] = at;
            dbeta[token * d.heads + head] = rw;
            at -= ov;
        }
    }
}

// Rows of the state a thread has: one for heads of few rows (and forward where there are few
// CTAs), else two: four leave an SM one CTA backward (8 x 2047 tokens, 16 heads of 128 x 128:
// 10.7 against 8.6 ms).
template <template <int, int> class Launch, typename... A>
cudaError_t by_shape(bool one, int n, A... args) {
    if (n <= 32) return one ? Launch<4, 1>::run(args...) : Launch<4, 2>::run(args...);
    if (n <= 64) return one ? Launch<8, 1>::run(args...) : Launch<8, 2>::run(args...);
    if (n <= 128) return one ? Launch<16, 1>::run(args...) : Launch<16, 2>::run(args...);
    return Launch<32, 1>::run(args...);
}
bool one_row(int p) { return p <= kRowsPass; }
int slab_rows(int p, int n) { return one_row(p) || n > 128 ? kRowsPass : 2 * kRowsPass; }

template <int kV, int kR>
struct LaunchFwd {
    static cudaError_t run(Walk a, cudaStream_t stream) {
        a.slabs = (a.d.p + kRowsPass * kR - 1) / (kRowsPass * kR);
        const long long ctas = (long long)a.d.nseq * a.d.heads * a.slabs;
        if (ctas >= (1ll << 31)) return cudaErrorInvalidValue;
        constexpr int kSmem = 2 * (int)sizeof(WalkTile<kV, kR>);
        const cudaError_t e = cudaFuncSetAttribute(delta_walk_kernel<kV, kR, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        delta_walk_kernel<kV, kR, false><<<(unsigned)ctas, kThreads, kSmem, stream>>>(a);
        return cudaGetLastError();
    }
};
template <int kV, int kR>
struct LaunchBack {
    static cudaError_t run(Walk u, Back a, cudaStream_t stream) {
        // (both below 2^31 for the sizes that the C entry lets pass)
        const long long ctas = (long long)a.d.nseq * a.d.heads * a.slabs;
        const long long runs = runs_of(a.d) * a.d.heads * a.slabs;
        if (runs >= (1ll << 31)) return cudaErrorInvalidValue;
        constexpr int kSmem = (int)sizeof(BackSmem<kV, kR>);
        cudaError_t e = cudaFuncSetAttribute(delta_back_kernel<kV, kR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(delta_again_kernel<kV, kR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        constexpr int kWalk = 2 * (int)sizeof(WalkTile<kV, kR>);
        e = cudaFuncSetAttribute(delta_walk_kernel<kV, kR, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kWalk);
        if (e != cudaSuccess) return e;
        delta_walk_kernel<kV, kR, true><<<(unsigned)runs, kThreads, kWalk, stream>>>(u);
        delta_back_kernel<kV, kR><<<(unsigned)ctas, kThreads, kSmem, stream>>>(a);
        delta_again_kernel<kV, kR><<<(unsigned)runs, kThreads, kSmem, stream>>>(a);
        return cudaGetLastError();
    }
};

// The workspace of the gradients, in bytes from its start.
struct BackPlan {
    size_t u, w, dq, dk, anchor, ov, rw, total;
    int slabs;
};
BackPlan back_plan(const SsdDelta &d) {
    const auto up = [](size_t n) { return (n * sizeof(float) + 255) / 256 * 256; };
    const int rows = slab_rows(d.p, d.n);
    BackPlan p;
    p.slabs = (d.p + rows - 1) / rows;
    const size_t wide = (size_t)d.heads * p.slabs, tokens = (size_t)d.tokens;
    p.u = 0;
    p.w = p.u + up(tokens * d.heads * d.p);
    p.dq = p.w + up(tokens * d.heads * d.p);
    p.dk = p.dq + up(tokens * wide * d.n);
    p.anchor = p.dk + up(tokens * wide * d.n);
    p.ov = p.anchor + up((size_t)ssd_delta_slots(d.tokens, d.nseq) * wide);
    p.rw = p.ov + up(tokens * wide);
    p.total = p.rw + up(tokens * wide);
    return p;
}

unsigned blocks_of(long long items, int per) {
    const long long n = (items + per - 1) / per;
    return (unsigned)(n < 8192 ? n : 8192);
}

}  // namespace

cudaError_t ssd_launch_delta_group_sums(const float *dq_parts, void *dq, long long dq_stride, const float *dk_parts,
                                        void *dk, long long dk_stride, const SsdDelta &d, int parts, cudaStream_t stream) {
    const Sums q{dq_parts, dq, d.tokens, dq_stride, d.groups, parts, d.n, d.bf16};
    const Sums k{dk_parts, dk, d.tokens, dk_stride, d.groups, parts, d.n, d.bf16};
    delta_group_sum_kernel<<<dim3(blocks_of(d.tokens * d.groups * d.n, 256), 2), 256, 0, stream>>>(q, k);
    return cudaGetLastError();
}

cudaError_t ssd_launch_delta_fwd_simt(const SsdDeltaFwd &a, int sms, cudaStream_t stream) {
    const Walk w{a.in, a.init, nullptr, a.o, a.o_stride, a.final_state, a.checkpoints, nullptr, 1};
    // few CTAs: slabs of one row a thread, which make a token shorter
    const long long most = (long long)a.in.nseq * a.in.heads * ((a.in.p + kRowsPass - 1) / kRowsPass);
    return by_shape<LaunchFwd>(one_row(a.in.p) || most <= 4ll * sms, a.in.n, w, stream);
}

size_t ssd_delta_bwd_simt_workspace(const SsdDelta &d) { return back_plan(d).total; }

cudaError_t ssd_launch_delta_bwd_simt(const SsdDeltaBwd &a, void *ws, cudaStream_t stream) {
    const SsdDelta &d = a.in;
    const BackPlan p = back_plan(d);
    const auto at = [&](size_t offset) { return reinterpret_cast<float *>(static_cast<char *>(ws) + offset); };
    const Walk u{d, nullptr, a.checkpoints, nullptr, 0, nullptr, nullptr, at(p.u), p.slabs};
    const Back b{d, a.dout, a.checkpoints, a.dfinal, a.do_stride, a.dv_stride, a.dv, a.dinit, at(p.u), at(p.w),
                 at(p.dq), at(p.dk), at(p.anchor), at(p.ov), at(p.rw), p.slabs};
    cudaError_t e = by_shape<LaunchBack>(one_row(d.p), d.n, u, b, stream);
    if (e != cudaSuccess) return e;
    e = ssd_launch_delta_group_sums(b.dq, a.dq, a.dq_stride, b.dk, a.dk, a.dk_stride, d, d.heads / d.groups * p.slabs, stream);
    if (e != cudaSuccess) return e;
    const long long runs = runs_of(d) * d.heads;
    delta_gates_kernel<<<blocks_of(runs, 128), 128, 0, stream>>>(b, a.dg, a.dbeta);
    return cudaGetLastError();
}
