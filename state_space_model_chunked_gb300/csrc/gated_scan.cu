// Gated linear recurrence, elementwise over the channels of each token:
//
//   f_t = sigmoid(g_t),  h_t = f_t h_{t-1} + (1 - f_t) x_t,  y_t = h_t silu(z_t)
//
// and its gradients: with dh_t = dy_t silu(z_t) (+ dfinal at a sequence's last
// token) and lam_t = dh_t + f_{t+1} lam_{t+1},
//
//   dx_t = (1 - f_t) lam_t,      dg_t = lam_t (h_{t-1} - x_t) f_t (1 - f_t),
//   dz_t = dy_t h_t silu'(z_t),  dinit = f_0 lam_0.
//
// f and 1 - f = sigmoid(-g) are each known to (1.25 |g| + 8) 2^-24 of themselves;
// states and gradients are carried in fp32.
//   Measured (time on the GPU): forward 65536 tokens of 5120 channels in bf16 with z
// 537 us (0.74 of the measured copy bandwidth), 47 sequences of 65518 tokens in all,
// 1536 channels, fp32 217 us (0.82); backward 8 x 2047 tokens of 2048 channels 131 us
// (0.53); a token of 256 rows of 5120 2.5 us, its arrays in L2.  Neither bytes nor
// instructions alone bound the two directions: a channel and token takes 41 and 77
// instructions, which fill 63 and 54 % of the issue slots, and 128 registers a thread
// leave an SM 16 warps, which most often wait at the CTA's barriers for the slowest
// warp's loads or for the tile in front.  That wait the walk's rule below keeps short:
// without the walk (wrong results) 521, 177 and 123 us.  The forward kernel's main form
// spills 48 bytes a thread under that bound (fp32 80).
#include "launch.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace {

constexpr int kEvery = kSsdCheckpointTokens;

// A lane's V channels: pairs go through the packed fp32 instructions.
template <int V>
struct Val {
    float v[V];
    __device__ __forceinline__ float &operator[](int k) { return v[k]; }
    __device__ __forceinline__ float operator[](int k) const { return v[k]; }
};
template <int V>
__device__ __forceinline__ Val<V> all(float a) {
    Val<V> r;
#pragma unroll
    for (int k = 0; k < V; ++k) r[k] = a;
    return r;
}
template <int V>
__device__ __forceinline__ Val<V> fma(const Val<V> &a, const Val<V> &b, const Val<V> &c) {
    Val<V> r;
    if constexpr (V == 2) {
        const float2 d = ssdptx::ffma2(make_float2(a[0], a[1]), make_float2(b[0], b[1]),
                                       make_float2(c[0], c[1]));
        r[0] = d.x, r[1] = d.y;
    } else {
        r[0] = fmaf(a[0], b[0], c[0]);
    }
    return r;
}
template <int V>
__device__ __forceinline__ Val<V> operator*(const Val<V> &a, const Val<V> &b) {
    Val<V> r;
    if constexpr (V == 2) {
        const float2 d = ssdptx::fmul2(make_float2(a[0], a[1]), make_float2(b[0], b[1]));
        r[0] = d.x, r[1] = d.y;
    } else {
        r[0] = a[0] * b[0];
    }
    return r;
}
template <int V>
__device__ __forceinline__ Val<V> operator+(const Val<V> &a, const Val<V> &b) {
    Val<V> r;
    if constexpr (V == 2) {
        const float2 d = ssdptx::fadd2(make_float2(a[0], a[1]), make_float2(b[0], b[1]));
        r[0] = d.x, r[1] = d.y;
    } else {
        r[0] = a[0] + b[0];
    }
    return r;
}
template <int V>
__device__ __forceinline__ Val<V> operator-(const Val<V> &a, const Val<V> &b) {
    return fma(b, all<V>(-1.f), a);
}
template <int V>
__device__ __forceinline__ Val<V> minus(Val<V> a) {
#pragma unroll
    for (int k = 0; k < V; ++k) a[k] = -a[k];
    return a;
}
template <typename T, int V>
__device__ __forceinline__ Val<V> value(const SsdRaw<T, V> &raw) {
    Val<V> r;
#pragma unroll
    for (int k = 0; k < V; ++k) r[k] = raw.get(k);
    return r;
}

constexpr float kLog2e = 1.44269504f;

// f = sigmoid(g) and 1 - f = sigmoid(-g).  With e = e^-|g| the smaller of the
// two is e / (1 + e), to (1.25 |g| + 8) 2^-24 of itself: the exponential's argument is
// one rounded product with a rounded log2 e, whose error grows with |g|, and the
// hardware's exponential, reciprocal and three roundings add 8.  The larger is 1
// minus it, rounded to nearest: its error has no sign, so it does not add up along
// a memory of thousands of tokens (1 / (1 + e) from the approximate reciprocal
// erred to one side and did).  Sharing one reciprocal between a lane's pair of
// channels takes more instructions than it saves (603 against 574 us forward,
// 65536 x 5120): the special-function unit is not what bounds this.
template <int V>
__device__ __forceinline__ void gate(const Val<V> &g, Val<V> &keep, Val<V> &drop) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const float e = ssdptx::ex2_approx(fabsf(g[k]) * -kLog2e);
        const float small = e * ssdptx::rcp_approx(1.f + e), big = 1.f - small;
        keep[k] = g[k] >= 0.f ? big : small;
        drop[k] = g[k] >= 0.f ? small : big;
    }
}
template <int V>
__device__ __forceinline__ Val<V> sigmoid(const Val<V> &z) {
    Val<V> s;
#pragma unroll
    for (int k = 0; k < V; ++k)
        s[k] = ssdptx::rcp_approx(1.f + ssdptx::ex2_approx(z[k] * -kLog2e));
    return s;
}

// n / d for 0 <= n < 2^31 by one multiplication: m = ceil(2^(31 + s) / d) with
// s = ceil(log2 d) errs by less than 2^s / d <= 1 of a quotient's last place.
struct Divisor {
    unsigned d, m, s;
    Divisor() = default;
    explicit Divisor(unsigned by) : d(by), m(0), s(0) {
        while ((1ull << s) < by) ++s;
        m = (unsigned)(((1ull << (31 + s)) + by - 1) / by);
    }
    __device__ __forceinline__ unsigned div(unsigned n) const {
        return (unsigned)(((unsigned long long)n * m) >> (31 + s));
    }
};

// What a launch hands its CTAs besides the arrays.
struct Walk {
    int blocks, tiles;
    int ahead;              // tiles to the one whose rows a CTA asks L2 for
    Divisor by_blocks, by_length;
};

// ------------------------------------------------------------- tiles and joins
// The token axis is cut into tiles, one CTA a tile and block of 32 V channels:
// each of its warps holds kTok consecutive tokens of it in registers, a lane V
// channels.  A run of tokens acts on the state that enters it as h -> A h + H,
// so the warps' (A, H) are joined through shared memory and the tiles' through
// global memory in one pass over the data:
//
//   a tile publishes its own (A, H) as soon as its loads have landed, then
//   walks back over its predecessors' until one has published the state that
//   leaves it, and replaces its (A, H) by its own leaving state.
//
// Tiles are handed out by a counter in the order of the walk, so a tile waits
// only for tiles that already run; every wait is bounded in time.
//
// A run that holds a sequence boundary is cut: what leaves it does not depend
// on what enters, and nothing is multiplied across the cut (0 times a NaN of
// the sequence before would reach the next one).  A cut tile publishes its
// leaving state at once.
constexpr int kFwdWarps = 4, kFwdTok = 16, kFwdCtas = 4;
constexpr int kBwdWarps = 8, kBwdTok = 8, kBwdCtas = 2;
constexpr int kFwdTile = kFwdWarps * kFwdTok, kBwdTile = kBwdWarps * kBwdTok;
static_assert(kBwdTile == kEvery, "a backward tile starts from a kept state");
static_assert(kEvery % kFwdTok == 0, "kept states are those that enter a warp's run");

// What a tile tells the tiles after it, per channel: one 64-bit word, written
// and read whole, so it needs no flag, no fence and no second trip to L2.  The
// low half is A of a run, or -1 for a state, or all ones: nothing yet (A of a
// run is in [0, 1] or the canonical NaN); the high half is H or the state.
// The words and the ticket are set to all ones before the kernel.
struct Joins {
    unsigned *ticket;
    uint2 *word;            // [tiles][width]
    unsigned *err;
    unsigned long long wait_ns;
    int withhold;           // test hook: the walk's first tile publishes nothing
};
constexpr unsigned kUnset = 0xffffffffu;

// One lane's V words.
template <int V>
struct Words {
    uint2 w[V];
    __device__ __forceinline__ void load(const uint2 *p) {
        if constexpr (V == 2) {
            unsigned long long a, b;
            asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];"
                         : "=l"(a), "=l"(b) : "l"(p) : "memory");
            w[0] = make_uint2((unsigned)a, (unsigned)(a >> 32));
            w[1] = make_uint2((unsigned)b, (unsigned)(b >> 32));
        } else {
            unsigned long long a;
            asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(a) : "l"(p) : "memory");
            w[0] = make_uint2((unsigned)a, (unsigned)(a >> 32));
        }
    }
    __device__ __forceinline__ void store(uint2 *p) const {
#pragma unroll
        for (int k = 0; k < V; ++k)
            asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p + k),
                         "l"((unsigned long long)w[k].x | ((unsigned long long)w[k].y << 32))
                         : "memory");
    }
    __device__ __forceinline__ bool set() const {
        bool all = true;
#pragma unroll
        for (int k = 0; k < V; ++k) all &= w[k].x != kUnset;
        return all;
    }
};

template <int V>
__device__ __forceinline__ void publish_run(uint2 *p, const Val<V> &A, const Val<V> &H) {
    Words<V> m;
#pragma unroll
    for (int k = 0; k < V; ++k)
        m.w[k] = make_uint2(A[k] == A[k] ? __float_as_uint(A[k]) : 0x7fffffffu,
                            __float_as_uint(H[k]));
    m.store(p);
}
template <int V>
__device__ __forceinline__ void publish_state(uint2 *p, const Val<V> &h) {
    Words<V> m;
#pragma unroll
    for (int k = 0; k < V; ++k) m.w[k] = make_uint2(__float_as_uint(-1.f), __float_as_uint(h[k]));
    m.store(p);
}

// The state that enters tile number `at` of the walk (at > 0) in a lane's V
// channels: back over the tiles at - 1, at - 2, ... to the nearest state, four
// words under way at a time.
template <int V>
__device__ __forceinline__ void walk_back(const Joins &j, int at, int width, int c, Val<V> &h) {
    constexpr int kAhead = 4;
    float A[V], H[V];
    bool done[V];
#pragma unroll
    for (int k = 0; k < V; ++k) A[k] = 1.f, H[k] = 0.f, done[k] = false;
    unsigned long long t0 = 0;
    bool open = true;
    for (int p = at - 1; open && p >= 0; p -= kAhead) {
        Words<V> m[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            m[q].load(j.word + (size_t)max(p - q, 0) * width + c);
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            if (!open || p - q < 0) continue;
            while (!m[q].set()) {
                unsigned long long now;
                asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
                if (t0 == 0) t0 = now;
                if (now - t0 > j.wait_ns) {
                    ssd_report(j.err, SSD_DEVERR_TIMEOUT);
                    open = false;
                    break;
                }
                m[q].load(j.word + (size_t)(p - q) * width + c);
            }
            if (!open) continue;
            open = false;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (done[k]) continue;
                const float a = __uint_as_float(m[q].w[k].x), v = __uint_as_float(m[q].w[k].y);
                H[k] += A[k] * v;
                done[k] = a < 0.f;
                A[k] *= a;
                open |= !done[k];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < V; ++k) h[k] = H[k];
}

// Which sequence each of a warp's tokens belongs to (lane i: token t0 + i, i < n)
// and which of them begin or end one.
struct Marks {
    int seq;
    unsigned starts, ends;
};
__device__ __forceinline__ Marks marks(const SsdGated &a, const Divisor &by_length, long long t0,
                                       int n) {
    const int lane = threadIdx.x & 31;
    const long long t = t0 + lane;
    const bool in = lane < n && t < a.tokens;
    Marks m;
    m.seq = 0;
    bool start = false, end = false;
    if (in) {
        if (a.cu) {
            int lo = 0, hi = a.nseq - 1;    // the last s with cu[s] <= t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (__ldg(a.cu + mid) <= t) lo = mid;
                else hi = mid - 1;
            }
            m.seq = lo;
            start = __ldg(a.cu + lo) == t;
            end = __ldg(a.cu + lo + 1) == t + 1;
        } else {
            m.seq = (int)by_length.div((unsigned)t);
            const int off = (int)t - m.seq * a.length;
            start = off == 0;
            end = off == a.length - 1;
        }
    }
    m.starts = __ballot_sync(0xffffffffu, start);
    m.ends = __ballot_sync(0xffffffffu, end);
    return m;
}

// Empty sequences hand `in` (zeros without one) on to `out`.  Each of the walk's tiles
// looks at its share of the sequences, a lane at one, behind all that others wait for:
// in front of the first tile's run, a million of them held the tiles behind it up for
// more than the limit of a wait.
template <int V>
__device__ __forceinline__ void pass_empty(const SsdGated &a, const float *in, float *out, int at,
                                           int tiles, int c) {
    if (!out || (!a.cu && a.length > 0)) return;
    const int lane = threadIdx.x & 31;
    const long long step = (long long)tiles * blockDim.x;
    for (long long s0 = (long long)at * blockDim.x + threadIdx.x - lane; s0 < a.nseq; s0 += step) {
        const long long mine = s0 + lane;
        const bool empty =
            mine < a.nseq && (!a.cu || __ldg(a.cu + mine) == __ldg(a.cu + mine + 1));
        for (unsigned left = __ballot_sync(0xffffffffu, empty); left; left &= left - 1) {
            const size_t s = (size_t)(s0 + __ffs((int)left) - 1);
            if (c >= a.width) continue;
#pragma unroll
            for (int k = 0; k < V; ++k)
                out[s * a.width + c + k] = in ? in[s * a.width + c + k] : 0.f;
        }
    }
}

template <int V>
__device__ __forceinline__ void load_f32(const float *p, bool on, float (&v)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = on ? p[k] : 0.f;
}

// The CTA's place: number in the walk, and block of channels.
template <bool kJoin>
__device__ __forceinline__ void place(const Joins &j, const Walk &walk, int &at, int &block) {
    if constexpr (kJoin) {
        __shared__ unsigned ticket;
        if (threadIdx.x == 0) ticket = atomicAdd(j.ticket, 1u) + 1u;    // from all ones: 0, 1, ...
        __syncthreads();
        const unsigned t = __shfl_sync(0xffffffffu, ticket, 0);     // one value in the warp
        at = (int)walk.by_blocks.div(t);
        block = (int)(t - (unsigned)at * walk.blocks);
    } else {
        at = 0;
        block = blockIdx.x;
    }
}

// The (A, H) of the CTA's warps in the order of the walk, and what enters the
// tile, in shared memory.
template <int V, int kWarps>
struct Runs {
    float A[kWarps][32 * V], H[kWarps][32 * V], in[32 * V];
    bool cut[kWarps];
};

// Joins the runs in three steps.  join_begin: the warps' runs through shared
// memory; with kJoin the last warp of the walk publishes the tile's.  Then every
// warp does what needs no entering state.  join_walk: the last warp walks back
// over the tiles.  join_end: what it found enters every warp's run.
template <int V>
struct Entering {
    Val<V> h;               // the state that enters the warp's run if nothing entered the tile
    Val<V> A;               // what the tile's entering state is multiplied by on the way
    bool cut;               // a boundary lies in between
    Val<V> tA, tH;          // the last warp: the tile's run
    bool tcut;
};
template <int V, int kWarps, bool kJoin>
__device__ __forceinline__ Entering<V> join_begin(Runs<V, kWarps> &r, const Joins &j, int at,
                                                  int width, int c, int place, bool cut,
                                                  const Val<V> &A, const Val<V> &H) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        r.A[place][lane * V + k] = A[k];
        r.H[place][lane * V + k] = H[k];
    }
    if (lane == 0) r.cut[place] = cut;
    __syncthreads();
    Entering<V> e{all<V>(0.f), all<V>(1.f), false, {}, {}, false};
    for (int w = 0; w < place; ++w) {
        const bool wcut = r.cut[w];
        e.cut |= wcut;
        Val<V> wa, wh;
#pragma unroll
        for (int k = 0; k < V; ++k) wa[k] = r.A[w][lane * V + k], wh[k] = r.H[w][lane * V + k];
        e.h = wcut ? wh : fma(wa, e.h, wh);
        e.A = e.A * wa;
    }
    if constexpr (kJoin) {
        if (place == kWarps - 1) {
            e.tcut = e.cut || cut;
            e.tA = A * e.A;
            e.tH = cut ? H : fma(A, e.h, H);
            if (c < width) {
                uint2 *word = j.word + (size_t)at * width + c;
                if (at == 0 || e.tcut) {
                    if (!(j.withhold && at == 0)) publish_state<V>(word, e.tH);
                } else {
                    publish_run<V>(word, e.tA, e.tH);
                }
            }
        }
    }
    return e;
}
template <int V, int kWarps, bool kJoin>
__device__ __forceinline__ void join_walk(Runs<V, kWarps> &r, const Joins &j, int at, int width,
                                          int c, int place, const Entering<V> &e) {
    if constexpr (kJoin) {
        if (place != kWarps - 1) return;
        Val<V> in = all<V>(0.f);
        if (at > 0 && c < width) {
            walk_back<V>(j, at, width, c, in);
            if (!e.tcut) publish_state<V>(j.word + (size_t)at * width + c, fma(e.tA, in, e.tH));
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < V; ++k) r.in[(threadIdx.x & 31) * V + k] = in[k];
    }
}
template <int V, int kWarps, bool kJoin>
__device__ __forceinline__ Val<V> join_end(const Runs<V, kWarps> &r, const Entering<V> &e) {
    if constexpr (kJoin) {
        __syncthreads();
        if (!e.cut) {
            Val<V> in;
#pragma unroll
            for (int k = 0; k < V; ++k) in[k] = r.in[(threadIdx.x & 31) * V + k];
            return fma(e.A, in, e.h);
        }
    }
    return e.h;
}

// kTok tokens of one array.  whole: all of them, in all of the warp's lanes.
template <typename T, int V, int kTok>
__device__ __forceinline__ void load_run(SsdRaw<T, V> (&raw)[kTok], const void *base,
                                         long long stride, long long t0, int n, int c, bool on,
                                         bool whole) {
    // a row's address is one value in the warp, a lane adds its channel to it
    const T *p = static_cast<const T *>(base) + t0 * stride;
    if (whole) {
#pragma unroll
        for (int i = 0; i < kTok; ++i) raw[i].load_cs(p + i * stride + (unsigned)c);
    } else {
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            raw[i].zero();
            if (on && i < n) raw[i].load_cs(p + i * stride + (unsigned)c);
        }
    }
}

// Asks L2 for the rows of the tile from t0 in kArrays arrays: a generation of CTAs
// ahead of their use, so their loads find them there.  A thread takes rows in turn.
template <typename T, int V, int kTile, int kArrays>
__device__ __forceinline__ void prefetch_tile(const void *const (&base)[kArrays],
                                              const long long (&stride)[kArrays], long long t0,
                                              long long tokens, int c0, int width) {
    static_assert((kTile & (kTile - 1)) == 0, "rows of an array");
    constexpr int kBytes = 32 * V * (int)sizeof(T);
    if (t0 < 0 || t0 + kTile > tokens) return;
    for (int i = threadIdx.x; i < kArrays * kTile; i += blockDim.x) {
        const void *b = base[0];
        long long s = stride[0];
#pragma unroll
        for (int k = 1; k < kArrays; ++k)
            if (i >= k * kTile) b = base[k], s = stride[k];
        const char *p = reinterpret_cast<const char *>(static_cast<const T *>(b) +
                                                       (t0 + (i & (kTile - 1))) * s + c0);
        // whole blocks of channels: the last of a ragged width may be asked for short
        if (c0 + 32 * V > width) {
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
            continue;
        }
#pragma unroll
        for (int o = 0; o < kBytes; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + o));
        if (((uintptr_t)p & 127u) != 0)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p + kBytes - 1));
    }
}

// Runs `body` as its plain form where a warp's tokens hold no sequence boundary
// and no end of the arrays, which leaves the tests for them out.
struct Plain {
    static constexpr bool kOn = true;
};
struct General {
    static constexpr bool kOn = false;
};
template <typename F>
__device__ __forceinline__ void by_form(bool plain, F &&body) {
    if (plain) body(Plain{});
    else body(General{});
}

template <typename T, int V, bool kGate, bool kJoin>
__global__ void __launch_bounds__(32 * kFwdWarps, kFwdCtas)
gated_fwd_kernel(const SsdGatedFwd a, const Joins joins, const Walk walk) {
    __shared__ Runs<V, kFwdWarps> runs;
    int at, block;
    place<kJoin>(joins, walk, at, block);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int width = a.in.width, c = (block * 32 + lane) * V;
    const bool on = c < width;
    const long long t0 = (long long)at * kFwdTile + warp * kFwdTok;
    const int n = (int)max(0ll, min((long long)kFwdTok, a.in.tokens - t0));
    const bool whole = n == kFwdTok && __all_sync(0xffffffffu, on);

    SsdRaw<T, V> graw[kFwdTok], xraw[kFwdTok], zraw[kGate ? kFwdTok : 1];
    load_run<T, V>(graw, a.in.g, a.in.g_stride, t0, n, c, on, whole);
    load_run<T, V>(xraw, a.in.x, a.in.x_stride, t0, n, c, on, whole);
    if constexpr (kGate) load_run<T, V>(zraw, a.in.z, a.in.z_stride, t0, n, c, on, whole);
    if constexpr (kJoin) {
        const long long tn = (long long)(at + walk.ahead) * kFwdTile;
        if constexpr (kGate) {
            const void *const base[3] = {a.in.g, a.in.x, a.in.z};
            const long long stride[3] = {a.in.g_stride, a.in.x_stride, a.in.z_stride};
            prefetch_tile<T, V, kFwdTile>(base, stride, tn, a.in.tokens, block * 32 * V, width);
        } else {
            const void *const base[2] = {a.in.g, a.in.x};
            const long long stride[2] = {a.in.g_stride, a.in.x_stride};
            prefetch_tile<T, V, kFwdTile>(base, stride, tn, a.in.tokens, block * 32 * V, width);
        }
    }
    const Marks m = marks(a.in, walk.by_length, t0, kFwdTok);
    const bool plain = whole && (m.starts | m.ends) == 0;

    Val<V> keep[kFwdTok], u[kFwdTok], A = all<V>(1.f), H = all<V>(0.f);
    by_form(plain, [&](auto form) {
        constexpr bool kPlain = decltype(form)::kOn;
#pragma unroll
        for (int i = 0; i < kFwdTok; ++i) {
            Val<V> drop;
            gate(value(graw[i]), keep[i], drop);
            u[i] = drop * value(xraw[i]);
            if (!kPlain && ((m.starts >> i) & 1u)) {
                const int seq = __shfl_sync(0xffffffffu, m.seq, i);
                Val<V> first;
                load_f32<V>(a.in.init + (size_t)seq * width + c, on && a.in.init != nullptr,
                            first.v);
                u[i] = fma(keep[i], first, u[i]);
                A = all<V>(0.f);
                H = u[i];
            } else if (kPlain || i < n) {
                A = A * keep[i];
                H = fma(keep[i], H, u[i]);
            }
        }
    });
    const Entering<V> e = join_begin<V, kFwdWarps, kJoin>(runs, joins, at, width, c, warp,
                                                          m.starts != 0, A, H);
    Val<V> silu[kGate ? kFwdTok : 1];
    if constexpr (kGate) {
#pragma unroll
        for (int i = 0; i < kFwdTok; ++i) {
            const Val<V> z = value(zraw[i]);
            silu[i] = z * sigmoid(z);
        }
    }
    join_walk<V, kFwdWarps, kJoin>(runs, joins, at, width, c, warp, e);
    Val<V> h = join_end<V, kFwdWarps, kJoin>(runs, e);

    if (a.checkpoints && n > 0 && t0 % kEvery == 0) {
        Val<V> before = h;
        const int seq = __shfl_sync(0xffffffffu, m.seq, 0);
        if (m.starts & 1u)
            load_f32<V>(a.in.init + (size_t)seq * width + c, on && a.in.init != nullptr, before.v);
        if (on) ssd_store_vec<V>(a.checkpoints + (size_t)(t0 / kEvery) * width + c, before.v);
    }
    by_form(plain, [&](auto form) {
        constexpr bool kPlain = decltype(form)::kOn;
        T *y = static_cast<T *>(a.y) + t0 * a.y_stride;
#pragma unroll
        for (int i = 0; i < kFwdTok; ++i) {
            if (!kPlain && i >= n) continue;
            h = !kPlain && ((m.starts >> i) & 1u) ? u[i] : fma(keep[i], h, u[i]);
            Val<V> o = h;
            if constexpr (kGate) o = h * silu[i];
            if (kPlain || on) ssd_store_vec<V>(y + i * a.y_stride + (unsigned)c, o.v);
            if (!kPlain && ((m.ends >> i) & 1u) && a.final_state) {
                const int seq = __shfl_sync(0xffffffffu, m.seq, i);
                if (on) ssd_store_vec<V>(a.final_state + (size_t)seq * width + c, h.v);
            }
        }
    });
    pass_empty<V>(a.in, a.in.init, a.final_state, at, walk.tiles, c);
}

// Backward: the same joins from the last tile to the first, on the gradient
// that a token hands to the one before it, mu_t = f_t lam_t: mu -> A mu + M
// over a run.  h is recomputed inside the tile from its kept state while the
// walk is under way; with s = sigmoid(z), dh = dy z s:
// dz = dy h s (1 + z (1 - s)) = h (s (dy - dh) + dh).
template <typename T, int V, bool kGate, bool kJoin>
__global__ void __launch_bounds__(32 * kBwdWarps, kBwdCtas)
gated_bwd_kernel(const SsdGatedBwd a, const Joins joins, const Walk walk) {
    __shared__ Runs<V, kBwdWarps> runs;
    __shared__ float fA[kBwdWarps][32 * V], fH[kBwdWarps][32 * V];
    __shared__ bool fcut[kBwdWarps];
    int at, block;
    place<kJoin>(joins, walk, at, block);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int width = a.in.width, c = (block * 32 + lane) * V;
    const bool on = c < width;
    const int tile = walk.tiles - 1 - at;
    const long long t0 = (long long)tile * kBwdTile + warp * kBwdTok;
    const int n = (int)max(0ll, min((long long)kBwdTok, a.in.tokens - t0));
    const bool whole = n == kBwdTok && __all_sync(0xffffffffu, on);

    SsdRaw<T, V> graw[kBwdTok], xraw[kBwdTok], yraw[kBwdTok], zraw[kGate ? kBwdTok : 1];
    load_run<T, V>(graw, a.in.g, a.in.g_stride, t0, n, c, on, whole);
    load_run<T, V>(yraw, a.dy, a.dy_stride, t0, n, c, on, whole);
    if constexpr (kGate) load_run<T, V>(zraw, a.in.z, a.in.z_stride, t0, n, c, on, whole);
    load_run<T, V>(xraw, a.in.x, a.in.x_stride, t0, n, c, on, whole);
    Val<V> h;           // the state that enters the tile
    load_f32<V>(a.checkpoints + (size_t)tile * width + c, on && a.in.tokens > 0, h.v);
    if constexpr (kJoin) {
        const long long tn = (long long)(tile - walk.ahead) * kBwdTile;
        if constexpr (kGate) {
            const void *const base[4] = {a.in.g, a.dy, a.in.z, a.in.x};
            const long long stride[4] = {a.in.g_stride, a.dy_stride, a.in.z_stride, a.in.x_stride};
            prefetch_tile<T, V, kBwdTile>(base, stride, tn, a.in.tokens, block * 32 * V, width);
        } else {
            const void *const base[3] = {a.in.g, a.dy, a.in.x};
            const long long stride[3] = {a.in.g_stride, a.dy_stride, a.in.x_stride};
            prefetch_tile<T, V, kBwdTile>(base, stride, tn, a.in.tokens, block * 32 * V, width);
        }
    }
    const Marks m = marks(a.in, walk.by_length, t0, kBwdTok);
    const bool plain = whole && (m.starts | m.ends) == 0;

    // the run forward (A, H) and backward (A, M)
    Val<V> keep[kBwdTok], drop[kBwdTok], dh[kBwdTok], sig[kGate ? kBwdTok : 1];
    Val<V> A = all<V>(1.f), H = all<V>(0.f), M = all<V>(0.f);
    by_form(plain, [&](auto form) {
        constexpr bool kPlain = decltype(form)::kOn;
#pragma unroll
        for (int i = 0; i < kBwdTok; ++i) {
            gate(value(graw[i]), keep[i], drop[i]);
            const Val<V> u = drop[i] * value(xraw[i]);
            if (!kPlain && ((m.starts >> i) & 1u)) {
                const int seq = __shfl_sync(0xffffffffu, m.seq, i);
                Val<V> first;
                load_f32<V>(a.in.init + (size_t)seq * width + c, on && a.in.init != nullptr,
                            first.v);
                A = all<V>(0.f);
                H = fma(keep[i], first, u);
            } else if (kPlain || i < n) {
                A = A * keep[i];
                H = fma(keep[i], H, u);
            }
        }
#pragma unroll
        for (int i = kBwdTok - 1; i >= 0; --i) {
            dh[i] = value(yraw[i]);
            if constexpr (kGate) {
                const Val<V> z = value(zraw[i]);
                sig[i] = sigmoid(z);
                dh[i] = dh[i] * (z * sig[i]);
            }
            if (!kPlain && i >= n) continue;
            Val<V> lam = dh[i] + M;
            if (!kPlain && ((m.ends >> i) & 1u)) {
                const int seq = __shfl_sync(0xffffffffu, m.seq, i);
                load_f32<V>(a.dfinal + (size_t)seq * width + c, on && a.dfinal != nullptr, lam.v);
                lam = dh[i] + lam;
            }
            M = !kPlain && ((m.starts >> i) & 1u) ? all<V>(0.f) : keep[i] * lam;
        }
    });
#pragma unroll
    for (int k = 0; k < V; ++k) {
        fA[warp][lane * V + k] = A[k];
        fH[warp][lane * V + k] = H[k];
    }
    if (lane == 0) fcut[warp] = m.starts != 0;
    const Entering<V> e = join_begin<V, kBwdWarps, kJoin>(
        runs, joins, at, width, c, kBwdWarps - 1 - warp, m.starts != 0, A, M);

    // forward: the states, f (1 - f) (x - h_{t-1}), and dz
    Val<V> q[kBwdTok];
    for (int w = 0; w < warp; ++w) {
        Val<V> wa, wh;
#pragma unroll
        for (int k = 0; k < V; ++k) wa[k] = fA[w][lane * V + k], wh[k] = fH[w][lane * V + k];
        h = fcut[w] ? wh : fma(wa, h, wh);
    }
    by_form(plain, [&](auto form) {
        constexpr bool kPlain = decltype(form)::kOn;
        [[maybe_unused]] T *dz = kGate ? static_cast<T *>(a.dz) + t0 * a.dz_stride : nullptr;
#pragma unroll
        for (int i = 0; i < kBwdTok; ++i) {
            if (!kPlain && i >= n) continue;
            if (!kPlain && ((m.starts >> i) & 1u)) {
                const int seq = __shfl_sync(0xffffffffu, m.seq, i);
                load_f32<V>(a.in.init + (size_t)seq * width + c, on && a.in.init != nullptr, h.v);
            }
            const Val<V> x = value(xraw[i]);
            q[i] = keep[i] * drop[i] * (x - h);
            h = fma(keep[i], h, drop[i] * x);   // as the forward pass has it
            if constexpr (kGate) {
                const Val<V> o = h * fma(sig[i], value(yraw[i]) - dh[i], dh[i]);
                if (kPlain || on) ssd_store_vec<V>(dz + i * a.dz_stride + (unsigned)c, o.v);
            }
        }
    });
    join_walk<V, kBwdWarps, kJoin>(runs, joins, at, width, c, kBwdWarps - 1 - warp, e);
    Val<V> mu = join_end<V, kBwdWarps, kJoin>(runs, e);
    // backward
    by_form(plain, [&](auto form) {
        constexpr bool kPlain = decltype(form)::kOn;
        T *dx = static_cast<T *>(a.dx) + t0 * a.dx_stride;
        T *dg = static_cast<T *>(a.dg) + t0 * a.dg_stride;
#pragma unroll
        for (int i = kBwdTok - 1; i >= 0; --i) {
            if (!kPlain && i >= n) continue;
            Val<V> lam = dh[i] + mu;
            if (!kPlain && ((m.ends >> i) & 1u)) {
                const int seq = __shfl_sync(0xffffffffu, m.seq, i);
                load_f32<V>(a.dfinal + (size_t)seq * width + c, on && a.dfinal != nullptr, lam.v);
                lam = dh[i] + lam;
            }
            // f lam by f, not as lam - (1 - f) lam: where dy is zero, f lam is all that the
            // tokens in front receive, and the difference has no digits of a small f
            const Val<V> ox = drop[i] * lam;
            mu = keep[i] * lam;
            const Val<V> og = minus(lam * q[i]);
            if (kPlain || on) {
                ssd_store_vec<V>(dx + i * a.dx_stride + (unsigned)c, ox.v);
                ssd_store_vec<V>(dg + i * a.dg_stride + (unsigned)c, og.v);
            }
            if (!kPlain && ((m.starts >> i) & 1u) && a.dinit) {
                const int seq = __shfl_sync(0xffffffffu, m.seq, i);
                if (on) ssd_store_vec<V>(a.dinit + (size_t)seq * width + c, mu.v);
            }
        }
    });
    pass_empty<V>(a.in, a.dfinal, a.dinit, at, walk.tiles, c);
}

// One token of every (row, channel): the state is read and written in place.
// Bound by memory (and, for few rows, by the launch): a thread takes V channels.
template <typename T, int V, bool kGate>
__global__ void __launch_bounds__(256) gated_step_kernel(const SsdGatedStep a) {
    const long long r = blockIdx.x;
    const int c = (blockIdx.y * 256 + threadIdx.x) * V;
    ssdptx::griddep_wait();
    if (c >= a.width) return;
    SsdRaw<T, V> gr, xr, zr;
    SsdRaw<float, V> sr;
    float *state = a.state + r * a.width + c;
    gr.load_cs(static_cast<const T *>(a.g) + r * a.g_stride + c);
    xr.load_cs(static_cast<const T *>(a.x) + r * a.x_stride + c);
    sr.load_cs(state);
    if constexpr (kGate) zr.load_cs(static_cast<const T *>(a.z) + r * a.z_stride + c);
    float h[V], y[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        Val<1> g, keep, drop;
        g[0] = gr.get(k);
        gate(g, keep, drop);
        h[k] = keep[0] * sr.get(k) + drop[0] * xr.get(k);
        y[k] = h[k];
        if constexpr (kGate) {
            Val<1> z;
            z[0] = zr.get(k);
            y[k] *= z[0] * sigmoid(z)[0];
        }
    }
    ssd_store_vec<V>(state, h);
    ssd_store_vec<V>(static_cast<T *>(a.y) + r * a.width + c, y);
}

}  // namespace

// Channels a lane: two when every row of every array starts on a boundary of
// two elements (4-byte loads in bf16: a warp reads whole 128-byte lines), else one.
static bool pairs(bool bf16, int width, const void *p, long long stride) {
    return p == nullptr || (width % 2 == 0 && stride % 2 == 0 &&
                            ((uintptr_t)p & (bf16 ? 3u : 7u)) == 0);
}
static bool pairs_in(const SsdGated &a) {
    return pairs(a.bf16, a.width, a.x, a.x_stride) && pairs(a.bf16, a.width, a.g, a.g_stride) &&
           pairs(a.bf16, a.width, a.z, a.z_stride) && pairs(false, a.width, a.init, 0);
}

// Tiles of a walk (at least one: it also hands on the empty sequences' states).
static int tiles_of(long long tokens, int tile) {
    return tokens > 0 ? (int)((tokens + tile - 1) / tile) : 1;
}

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The joins' memory, sized for the smaller tiles: a ticket, then a
// word for every (tile, channel).
constexpr size_t kTicketBytes = 256;
static size_t joins_bytes(int tiles, int width) {
    return kTicketBytes + sizeof(uint2) * (size_t)tiles * (size_t)width;
}
size_t ssd_gated_workspace(long long tokens, int width) {
    const int tiles = tiles_of(tokens, kBwdTile < kFwdTile ? kBwdTile : kFwdTile);
    return tiles == 1 ? 0 : up256(joins_bytes(tiles, width));
}

// Carves the joins out of the workspace and sets them to all ones.
static cudaError_t joins_of(void *workspace, int tiles, int width, unsigned *err,
                            cudaStream_t stream, Joins *j) {
    const SsdDebug dbg = ssd_debug_config();
    char *ws = static_cast<char *>(workspace);
    j->ticket = reinterpret_cast<unsigned *>(ws);
    j->word = reinterpret_cast<uint2 *>(ws + kTicketBytes);
    j->err = err;
    j->wait_ns = dbg.wait_ns;
    j->withhold = dbg.fault == kSsdFaultWithholdSignal;
    return cudaMemsetAsync(ws, 0xff, joins_bytes(tiles, width), stream);
}

// One launch: `one` for calls of a single tile, which has nothing to join.
template <int V, typename Args>
static cudaError_t launch(void (*one)(Args, Joins, Walk), void (*joined)(Args, Joins, Walk),
                          const Args &a, int tile, int threads, int ctas, int sms, void *ws,
                          unsigned *err, cudaStream_t stream) {
    Walk w;
    w.tiles = tiles_of(a.in.tokens, tile);
    w.blocks = (a.in.width + 32 * V - 1) / (32 * V);
    w.ahead = (sms * ctas + w.blocks - 1) / w.blocks;
    w.by_blocks = Divisor((unsigned)w.blocks);
    w.by_length = Divisor(a.in.length > 0 ? (unsigned)a.in.length : 1u);
    Joins j{};
    if (w.tiles > 1) {
        const cudaError_t e = joins_of(ws, w.tiles, a.in.width, err, stream, &j);
        if (e != cudaSuccess) return e;
    }
    (w.tiles > 1 ? joined : one)<<<(unsigned)((size_t)w.tiles * w.blocks), threads, 0, stream>>>(a, j, w);
    return cudaGetLastError();
}
template <typename T, int V, bool kGate>
static cudaError_t launch_fwd(const SsdGatedFwd &a, int sms, void *ws, unsigned *err,
                              cudaStream_t stream) {
    return launch<V>(gated_fwd_kernel<T, V, kGate, false>, gated_fwd_kernel<T, V, kGate, true>, a,
                     kFwdTile, 32 * kFwdWarps, kFwdCtas, sms, ws, err, stream);
}
template <typename T, int V, bool kGate>
static cudaError_t launch_bwd(const SsdGatedBwd &a, int sms, void *ws, unsigned *err,
                              cudaStream_t stream) {
    return launch<V>(gated_bwd_kernel<T, V, kGate, false>, gated_bwd_kernel<T, V, kGate, true>, a,
                     kBwdTile, 32 * kBwdWarps, kBwdCtas, sms, ws, err, stream);
}

cudaError_t ssd_launch_gated_fwd(const SsdGatedFwd &a, int sms, void *ws, unsigned *err,
                                 cudaStream_t stream) {
    const bool two = pairs_in(a.in) && pairs(a.in.bf16, a.in.width, a.y, a.y_stride) &&
                     pairs(false, a.in.width, a.final_state, 0) &&
                     pairs(false, a.in.width, a.checkpoints, 0);
    const bool gate = a.in.z != nullptr;
    if (a.in.bf16) {
        using T = __nv_bfloat16;
        if (two) return gate ? launch_fwd<T, 2, true>(a, sms, ws, err, stream)
                             : launch_fwd<T, 2, false>(a, sms, ws, err, stream);
        return gate ? launch_fwd<T, 1, true>(a, sms, ws, err, stream)
                    : launch_fwd<T, 1, false>(a, sms, ws, err, stream);
    }
    if (two) return gate ? launch_fwd<float, 2, true>(a, sms, ws, err, stream)
                         : launch_fwd<float, 2, false>(a, sms, ws, err, stream);
    return gate ? launch_fwd<float, 1, true>(a, sms, ws, err, stream)
                : launch_fwd<float, 1, false>(a, sms, ws, err, stream);
}

cudaError_t ssd_launch_gated_bwd(const SsdGatedBwd &a, int sms, void *ws, unsigned *err,
                                 cudaStream_t stream) {
    const bool bf16 = a.in.bf16, gate = a.in.z != nullptr;
    const int w = a.in.width;
    const bool two = pairs_in(a.in) && pairs(bf16, w, a.dy, a.dy_stride) &&
                     pairs(bf16, w, a.dx, a.dx_stride) && pairs(bf16, w, a.dg, a.dg_stride) &&
                     (!gate || pairs(bf16, w, a.dz, a.dz_stride)) && pairs(false, w, a.dinit, 0);
    if (bf16) {
        using T = __nv_bfloat16;
        if (two) return gate ? launch_bwd<T, 2, true>(a, sms, ws, err, stream)
                             : launch_bwd<T, 2, false>(a, sms, ws, err, stream);
        return gate ? launch_bwd<T, 1, true>(a, sms, ws, err, stream)
                    : launch_bwd<T, 1, false>(a, sms, ws, err, stream);
    }
    if (two) return gate ? launch_bwd<float, 2, true>(a, sms, ws, err, stream)
                         : launch_bwd<float, 2, false>(a, sms, ws, err, stream);
    return gate ? launch_bwd<float, 1, true>(a, sms, ws, err, stream)
                : launch_bwd<float, 1, false>(a, sms, ws, err, stream);
}

template <typename T, int V>
static cudaError_t launch_step(const SsdGatedStep &a, cudaStream_t stream) {
    const dim3 grid((unsigned)a.rows, (unsigned)((a.width + 256 * V - 1) / (256 * V)));
    return ssd_launch_early(a.z ? gated_step_kernel<T, V, true> : gated_step_kernel<T, V, false>, grid,
                            dim3(256), stream, a);
}

cudaError_t ssd_launch_gated_step(const SsdGatedStep &a, cudaStream_t stream) {
    const size_t size = a.bf16 ? 2 : 4;
    const auto four = [&](const void *p, long long stride, size_t bytes) {
        return !p || ((uintptr_t)p % (4 * bytes) == 0 && stride % 4 == 0);
    };
    const bool v4 = a.width % 4 == 0 && four(a.state, a.width, 4) && four(a.x, a.x_stride, size) &&
                    four(a.g, a.g_stride, size) && four(a.z, a.z_stride, size) &&
                    four(a.y, a.width, size);
    if (a.bf16)
        return v4 ? launch_step<__nv_bfloat16, 4>(a, stream) : launch_step<__nv_bfloat16, 1>(a, stream);
    return v4 ? launch_step<float, 4>(a, stream) : launch_step<float, 1>(a, stream);
}
