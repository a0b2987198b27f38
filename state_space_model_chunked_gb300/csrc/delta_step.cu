// One token of the gated delta rule for every head's state [P][N]:
//
//   S' = exp(g) S,  u = beta (v - S' k),  S <- S' + u k^T,  o = scale S q
//
// Bound by memory: a state is read once and written once.  Both of its products are taken
// of the state as it is read, S k and S q, since o = scale (exp(g) S q + u (k q)): one round
// of sums over the lanes between the loads and the stores.  Eight lanes share a row, a
// thread has kR rows of kV columns in registers, all their loads under way together.  16
// sequences, 32 heads of 128 x 128 in fp32: 13.5 us, 0.74 of a copy's rate; 2 are the launch
// and the first loads' latency.
#include "launch.h"
#include "ptx.cuh"

namespace {

constexpr int kThreads = 256, kLanes = 8, kGroups = kThreads / kLanes;

template <int kO>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = kO / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Columns 32 j + 4 lane + i of a row of n values; kVec: vectors of four.
template <int kV, bool kVec, typename T>
__device__ __forceinline__ void load_row(const T *row, int n, int lane, bool on, float (&v)[kV]) {
#pragma unroll
    for (int i = 0; i < kV; i += 4) {
        const int c = i * kLanes + lane * 4;
        if constexpr (kVec) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on && c < n) x = ssd_ld4_cs(row + c);
            v[i] = x.x;
            v[i + 1] = x.y;
            v[i + 2] = x.z;
            v[i + 3] = x.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i + j] = on && c + j < n ? ssd_ld(row + c + j) : 0.f;
        }
    }
}

template <typename TS, typename T, int kV, int kR, bool kVec>
__global__ void __launch_bounds__(kThreads) delta_step_kernel(const SsdDeltaStep a, const int blocks) {
    ssdptx::griddep_wait();
    const int block = (int)(blockIdx.x % blocks), head = (int)(blockIdx.x / blocks) % a.heads;
    const long long batch = blockIdx.x / blocks / a.heads;
    const int lane = threadIdx.x % kLanes, at = threadIdx.x / kLanes;
    const size_t which = (size_t)batch * a.heads + head;
    const TS *state = static_cast<const TS *>(a.state) + which * a.p * a.n;
    TS *out = static_cast<TS *>(a.state_out) + which * a.p * a.n;
    int row[kR];
    float s[kR][kV], v[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        row[r] = (block * kR + r) * kGroups + at;
        const bool on = row[r] < a.p;
        load_row<kV, kVec>(state + (size_t)(on ? row[r] : 0) * a.n, a.n, lane, on, s[r]);
        v[r] = on ? ssd_ld(static_cast<const T *>(a.v) + batch * a.v_stride + (size_t)head * a.p + row[r]) : 0.f;
    }
    const size_t keys = (size_t)(head / (a.heads / a.groups)) * a.n;
    float k[kV], q[kV], kq = 0.f;
    load_row<kV, false>(static_cast<const T *>(a.k) + batch * a.k_stride + keys, a.n, lane, true, k);
    load_row<kV, false>(static_cast<const T *>(a.q) + batch * a.q_stride + keys, a.n, lane, true, q);
    const float g = a.g[which], beta = a.beta[which];
    const float f = expf(g < -200.f ? -200.f : g);
#pragma unroll
    for (int i = 0; i < kV; ++i) kq += k[i] * q[i];
    kq = lanes_sum<kLanes>(kq);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            sk += s[r][i] * k[i];
            sq += s[r][i] * q[i];
        }
        sk = lanes_sum<kLanes>(sk);
        sq = lanes_sum<kLanes>(sq);
        const float u = beta * (v[r] - f * sk);
        if (row[r] >= a.p) continue;
#pragma unroll
        for (int i = 0; i < kV; ++i) s[r][i] = f * s[r][i] + u * k[i];
        TS *to = out + (size_t)row[r] * a.n;
#pragma unroll
        for (int i = 0; i < kV; i += 4) {
            const int c = i * kLanes + lane * 4;
            if constexpr (kVec) {
                if (c < a.n) ssd_st4_cs(to + c, make_float4(s[r][i], s[r][i + 1], s[r][i + 2], s[r][i + 3]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + j < a.n) ssd_st(to + c + j, s[r][i + j]);
            }
        }
        if (lane == 0)
            ssd_st(static_cast<T *>(a.o) + which * a.p + row[r], a.scale * (f * sq + u * kq));
    }
}

template <typename TS, typename T, int kV, int kR>
cudaError_t launch(const SsdDeltaStep &a, cudaStream_t stream) {
    const int blocks = (a.p + kGroups * kR - 1) / (kGroups * kR);
    const long long ctas = (long long)a.batch * a.heads * blocks;
    if (ctas >= (1ll << 31)) return cudaErrorInvalidValue;
    const bool vec = a.n % 4 == 0 && (((uintptr_t)a.state | (uintptr_t)a.state_out) & (4 * sizeof(TS) - 1)) == 0;
    const dim3 grid((unsigned)ctas), block(kThreads);
    return vec ? ssd_launch_early(delta_step_kernel<TS, T, kV, kR, true>, grid, block, stream, a, blocks)
               : ssd_launch_early(delta_step_kernel<TS, T, kV, kR, false>, grid, block, stream, a, blocks);
}

template <typename TS, typename T>
cudaError_t launch_sizes(const SsdDeltaStep &a, cudaStream_t stream) {
    if (a.n <= 32) return launch<TS, T, 4, 2>(a, stream);
    if (a.n <= 64) return launch<TS, T, 8, 2>(a, stream);
    if (a.n <= 128) return launch<TS, T, 16, 2>(a, stream);
    return launch<TS, T, 32, 1>(a, stream);
}

}  // namespace

cudaError_t ssd_launch_delta_step(const SsdDeltaStep &a, int sms, cudaStream_t stream) {
    (void)sms;
    if (!a.bf16) return a.bf16_state ? cudaErrorInvalidValue : launch_sizes<float, float>(a, stream);
    return a.bf16_state ? launch_sizes<__nv_bfloat16, __nv_bfloat16>(a, stream)
                        : launch_sizes<float, __nv_bfloat16>(a, stream);
}
