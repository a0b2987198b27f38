// Runs of V consecutive values of an array as fp32 in registers: V = 16, 8, 4
// or 2 move as aligned vectors of at most 16 bytes each (the caller has checked
// the alignment), V = 1 as a scalar.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

template <int kBytes>
struct SsdWord;
template <>
struct SsdWord<1> { using type = uint8_t; };
template <>
struct SsdWord<2> { using type = uint16_t; };
template <>
struct SsdWord<4> { using type = uint32_t; };
template <>
struct SsdWord<8> { using type = uint2; };
template <>
struct SsdWord<16> { using type = uint4; };

// The raw bits of V values, loaded ahead of their use.
template <typename T, int V>
struct SsdRaw {
    static constexpr int kBytes = V * (int)sizeof(T);
    static constexpr int kWordBytes = kBytes > 16 ? 16 : kBytes;
    static constexpr int kWords = kBytes / kWordBytes;
    using Word = typename SsdWord<kWordBytes>::type;
    Word w[kWords];

    // read once, not kept in L1 or, beyond this use, in L2
    __device__ __forceinline__ void load_cs(const T *p) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __ldcs(reinterpret_cast<const Word *>(p) + i);
    }
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = *(reinterpret_cast<const Word *>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = Word{};
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) {
            return reinterpret_cast<const float *>(w)[i];
        } else {
            return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(w)[i]);
        }
    }
};

template <int V>
__device__ __forceinline__ void ssd_store_vec(float *p, const float (&v)[V]) {
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<float4 *>(p)[i] =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else if constexpr (V == 2) {
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
    } else {
        *p = v[0];
    }
}

template <int V>
__device__ __forceinline__ void ssd_store_vec(__nv_bfloat16 *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = __float2bfloat16_rn(v[0]);
    } else {
        uint32_t u[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        if constexpr (V == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        else if constexpr (V == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(u[0], u[1]);
        else *reinterpret_cast<uint32_t *>(p) = u[0];
    }
}

// E4M3, rounded to nearest even; magnitudes above 448 give 448, NaN gives NaN.
template <int V>
__device__ __forceinline__ void ssd_store_vec(__nv_fp8_e4m3 *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        reinterpret_cast<__nv_fp8_storage_t *>(p)[0] =
            __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint16_t u[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            u[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE,
                                            __NV_E4M3);
        if constexpr (V == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2((uint32_t)u[0] | ((uint32_t)u[1] << 16),
                                                       (uint32_t)u[2] | ((uint32_t)u[3] << 16));
        else if constexpr (V == 4)
            *reinterpret_cast<uint32_t *>(p) = (uint32_t)u[0] | ((uint32_t)u[1] << 16);
        else
            *reinterpret_cast<uint16_t *>(p) = u[0];
    }
}

__device__ __forceinline__ float ssd_warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float ssd_warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
