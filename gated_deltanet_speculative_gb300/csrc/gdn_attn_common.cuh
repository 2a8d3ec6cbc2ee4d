// gdn_attn_common.cuh -- element types and addresses shared by the kernels
// of the attention layers.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gdn_paths.cuh"

namespace gdn {

// Storage and conversions of an element type (GDN_BF16, GDN_FP16, GDN_E4M3).
template <int T>
struct Elem;
template <>
struct Elem<GDN_BF16> {
    using type = __nv_bfloat16;
    __device__ static float2 unpack2(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    __device__ static uint32_t pack2(float a, float b) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&x);
    }
};
template <>
struct Elem<GDN_FP16> {
    using type = __half;
    __device__ static float2 unpack2(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    }
    __device__ static uint32_t pack2(float a, float b) {
        const __half2 x = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&x);
    }
};
template <>
struct Elem<GDN_E4M3> {
    using type = uint8_t;
    __device__ static float2 unpack2(uint16_t u) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(u, __NV_E4M3);
        return __half22float2(__half2(h));
    }
    // nearest even, saturated at +-448; a NaN stays one
    __device__ static uint16_t pack2(float a, float b) {
        return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    }
};

// N consecutive elements at an address aligned to their size, as floats and back.
template <int T, int N>
__device__ __forceinline__ void load_floats(const void *src, float (&x)[N]) {
    if constexpr (T == GDN_E4M3) {
        uint16_t w[N / 2];
        if constexpr (N == 8) *reinterpret_cast<uint2 *>(w) = *static_cast<const uint2 *>(src);
        else if constexpr (N == 4) *reinterpret_cast<uint32_t *>(w) = *static_cast<const uint32_t *>(src);
        else w[0] = *static_cast<const uint16_t *>(src);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 f = Elem<T>::unpack2(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    } else {
        uint32_t w[N / 2];
        if constexpr (N == 8) *reinterpret_cast<uint4 *>(w) = *static_cast<const uint4 *>(src);
        else if constexpr (N == 4) *reinterpret_cast<uint2 *>(w) = *static_cast<const uint2 *>(src);
        else w[0] = *static_cast<const uint32_t *>(src);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 f = Elem<T>::unpack2(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

template <int T, int N>
__device__ __forceinline__ void store_floats(void *dst, const float (&x)[N]) {
    if constexpr (T == GDN_E4M3) {
        uint16_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = Elem<T>::pack2(x[2 * i], x[2 * i + 1]);
        if constexpr (N == 8) *static_cast<uint2 *>(dst) = *reinterpret_cast<uint2 *>(w);
        else if constexpr (N == 4) *static_cast<uint32_t *>(dst) = *reinterpret_cast<uint32_t *>(w);
        else *static_cast<uint16_t *>(dst) = w[0];
    } else {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = Elem<T>::pack2(x[2 * i], x[2 * i + 1]);
        if constexpr (N == 8) *static_cast<uint4 *>(dst) = *reinterpret_cast<uint4 *>(w);
        else if constexpr (N == 4) *static_cast<uint2 *>(dst) = *reinterpret_cast<uint2 *>(w);
        else *static_cast<uint32_t *>(dst) = w[0];
    }
}

// Two of the 8-bit type with more range (2^-16 to 57344) and 3 bits, nearest even, saturated.
__device__ __forceinline__ uint16_t pack2_e5m2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E5M2);
}

template <int T>
constexpr int elem_bytes = T == GDN_E4M3 ? 1 : 2;

}  // namespace gdn
