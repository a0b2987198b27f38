// What the tensor-core kernels of the gated delta rule share: the chunk's record in the
// workspace, its layout in shared memory, and small device helpers.
#pragma once

#include <stdint.h>

#include "launch.h"
#include "ptx.cuh"

namespace ssddelta {

using namespace ssdptx;

constexpr int kC = kSsdDeltaChunk;          // tokens a chunk
static_assert(kC == 64, "a chunk's matrices are one 128-byte-swizzled panel wide");
constexpr uint32_t kPanel = 64 * 128;       // 64 rows of 64 bf16 values

// A chunk's record, for every head: the matrices T diag(beta) without its diagonal (which is
// beta, and is multiplied in fp32) and P, each in two bf16 parts and each an image of a
// 128-byte-swizzled panel (row: the later token), then for every token the decay from the chunk's start up to it, from it to the chunk's end, beta,
// and log2(e) g summed from its half's first token on, in two floats.
constexpr uint32_t kRecT = 0, kRecP = 2 * kPanel, kRecGates = 4 * kPanel;
constexpr int kGateW = kC, kGateBeta = 2 * kC, kGateSums = 3 * kC, kGates = 5 * kC;
constexpr uint32_t kRecord = kRecGates + kGates * 4;
static_assert(kRecord % 128 == 0, "records are copied to 128-byte boundaries");
// Where beta is smaller than this the gradients' records have this: dbeta is Z U over its square.
// Elsewhere such a token's U counts by its beta's share of this (its value may be any size); its Z,
// which is a gradient times this, is below fp32's last bit of those for keys of some length.
constexpr float kLeastBeta = 9.094947017729282e-13f;

// Byte of element (row, col) in a panel.
__device__ __forceinline__ uint32_t panel_at(uint32_t row, uint32_t col) {
    return (row >> 3) * 1024u + (row & 7u) * 128u + ((((col >> 3) ^ row) & 7u) << 4) + (col & 7u) * 2u;
}

// One lane of the warp, chosen so that what it issues needs no reconvergence: a thread picked
// by its lane number issues a tcgen05.mma every 45 to 60 cycles, one elected so as often as
// the tensor core takes them (N = 64: 32 cycles).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Two values as bf16 pairs: the rounded ones and what rounding left.
struct Split {
    uint32_t hi, lo;
};
__device__ __forceinline__ uint32_t rest2(float a, float b, uint32_t hi) {
    const float2 l = ffma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)),
                           make_float2(-1.f, -1.f), make_float2(a, b));
    return pack_bf16x2(l.x, l.y);
}
__device__ __forceinline__ Split split2(float a, float b) {
    Split s;
    s.hi = pack_bf16x2(a, b);
    s.lo = rest2(a, b, s.hi);
    return s;
}

// A bounded wait.  After any wait of the CTA has run out, every later one that would have
// to wait returns false at once; the roles then leave their loops, and the CTA lets its
// copies and products in flight complete before it ends.  (Polls that sleep up to 20 us, or
// that never sleep, make the forward walk 14 and 22% slower: the waiting warps wake late, or
// take the working ones' issue slots.)
struct Waiter {
    volatile int *abort;
    unsigned *err;
    unsigned long long limit;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (mbar_wait(bar, parity, limit)) return true;
        *abort = 1;
        ssd_report(err, SSD_DEVERR_TIMEOUT);
        return false;
    }
    // of a whole warp
    __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, (*this)(bar, parity));
    }
};

// Which chunk a slot of the kept states (ssd_delta_slot) stands for.
struct ChunkAt {
    long long first;    // the sequence's first token
    int seq, len, chunk;
    bool live;
};
__device__ __forceinline__ ChunkAt chunk_at(const SsdDelta &d, long long slot) {
    int lo = 0, hi = d.nseq;        // the last sequence whose first slot is at or before it
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        const long long first = d.cu ? d.cu[mid] : (long long)mid * d.length;
        if (ssd_delta_slot(first, mid, 0) <= slot) lo = mid;
        else hi = mid;
    }
    ChunkAt c;
    c.seq = lo;
    c.first = d.cu ? d.cu[lo] : (long long)lo * d.length;
    c.len = d.cu ? d.cu[lo + 1] - d.cu[lo] : d.length;
    const long long chunk = slot - ssd_delta_slot(c.first, lo, 0);
    c.chunk = (int)chunk;
    c.live = chunk * kC < c.len;
    return c;
}

// Eight values of a row as the two parts' vectors in the images at `image`.
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

// The sequence that a walk's CTA takes as number `rank`: packed ones by falling length, so
// that the longest do not begin last (47 sequences of 4 to 5000 tokens: 580 -> 487 us).  All
// threads of the CTA; `place` in shared memory.
__device__ __forceinline__ int sequence_of(const SsdDelta &d, int rank, volatile int *place) {
    constexpr int kMost = 512;          // above this each CTA's count would take too long
    if (!d.cu || d.nseq > kMost) return rank;
    for (int s = threadIdx.x; s < d.nseq; s += blockDim.x) {
        const int len = d.cu[s + 1] - d.cu[s];
        int before = 0;
        for (int o = 0, at = d.cu[0]; o < d.nseq; ++o) {
            const int next = d.cu[o + 1];
            before += next - at > len || (next - at == len && o < s);
            at = next;
        }
        if (before == rank) *place = s;
    }
    __syncthreads();
    return *place;
}

// Zeros in the rows of 64-token panels behind a sequence's end: they are another sequence's,
// or nothing's, and a NaN there would not be stopped by a factor of zero.
__device__ __forceinline__ void clean_rows(uint8_t *panels, uint32_t stride, int count, int tokens, int thread,
                                           int threads) {
    if (tokens >= kC) return;
    const int each = (kC - tokens) * 8;
    for (int i = thread; i < count * each; i += threads)
        *reinterpret_cast<uint4 *>(panels + (i / each) * stride + tokens * 128 + (i % each) * 16) = make_uint4(0, 0, 0, 0);
}

// A warp's 32 rows of kMine fp32 values, a row a lane, to rows `n` apart (those below
// `rows`, columns below `cols`), by way of 2 KB of the warp's own: a lane that wrote its own
// row would touch a line for every 16 bytes (a state of 128 x 128 took 8000 cycles).
template <int kMine>
__device__ __forceinline__ void store_rows(float *stage, const float (&v)[kMine], float *to, int n, int rows, int cols) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < kMine / 16; ++h) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4 *>(stage + lane * 16 + ((i ^ (lane >> 1)) & 3) * 4) =
                make_float4(v[16 * h + 4 * i], v[16 * h + 4 * i + 1], v[16 * h + 4 * i + 2], v[16 * h + 4 * i + 3]);
        __syncwarp();
        const int c = (lane & 3) * 4 + 16 * h;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 8 * j + (lane >> 2);
            const float4 x = *reinterpret_cast<const float4 *>(stage + r * 16 + ((lane ^ (r >> 1)) & 3) * 4);
            if (r < rows && c < cols) *reinterpret_cast<float4 *>(to + (size_t)r * n + c) = x;
        }
    }
}
// And from there.
template <int kMine>
__device__ __forceinline__ void load_rows(float *stage, float (&v)[kMine], const float *from, int n, int rows, int cols) {
    const int lane = threadIdx.x & 31;
    float4 x[kMine / 4];
#pragma unroll
    for (int i = 0; i < kMine / 4; ++i) {
        const int r = 8 * (i & 3) + (lane >> 2), c = (lane & 3) * 4 + 16 * (i >> 2);
        x[i] = r < rows && c < cols ? *reinterpret_cast<const float4 *>(from + (size_t)r * n + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int h = 0; h < kMine / 16; ++h) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 8 * j + (lane >> 2);
            *reinterpret_cast<float4 *>(stage + r * 16 + ((lane ^ (r >> 1)) & 3) * 4) = x[4 * h + j];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 y = *reinterpret_cast<const float4 *>(stage + lane * 16 + ((i ^ (lane >> 1)) & 3) * 4);
            v[16 * h + 4 * i] = y.x;
            v[16 * h + 4 * i + 1] = y.y;
            v[16 * h + 4 * i + 2] = y.z;
            v[16 * h + 4 * i + 3] = y.w;
        }
    }
    __syncwarp();
}
constexpr uint32_t kStageRows = 2048;       // bytes a warp

// A part's first token within its sequence of `len`: parts are whole chunks, but for the end,
// and all as long, but for one of half that length: the first where `half` is 1, the last
// where it is -1.
__device__ __forceinline__ int part_start(int len, int part, int parts, int half) {
    if (part == 0) return 0;
    const int all = 2 * parts - (half ? 1 : 0);
    const long long at = (long long)((len + kC - 1) / kC) * (2 * part - (half > 0 ? 1 : 0)) / all * kC;
    return at < len ? (int)at : len;
}
// In how many parts a sequence is walked, whether one of them has half the others' length,
// and what lies in the workspace for them (delta_tc.cu).
struct InParts {
    int parts, half;
};
InParts segments_of(const SsdDelta &d, int sms);
struct Parts {
    float *starts, *maps;
    int *cu;
    size_t bytes;
};
Parts parts_of(const SsdDelta &d, int segments, uint8_t *at);
// The states that parts start from, by their ends and maps, in the order of the walk; `half`
// as for part_start.
cudaError_t launch_join(const SsdDelta &d, const float *init, InParts parts, int half, const Parts &p, int sms,
                        unsigned *err, cudaStream_t stream);

inline bool on_16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// The records of all chunks (delta_tc.cu); least_beta: see kLeastBeta.
cudaError_t launch_chunks(const SsdDelta &d, uint8_t *records, bool least_beta, int sms, unsigned *err,
                          cudaStream_t stream);
// [tokens][heads][width] bf16 by boxes of `cols` values of one head and 64 tokens.
bool make_map(CUtensorMap *m, const void *p, int width, int heads, long long tokens, long long stride, int cols,
              bool swizzle);

}  // namespace ssddelta
