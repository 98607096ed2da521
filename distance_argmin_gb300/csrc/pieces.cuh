// 16-bit conversions, and 16-byte pieces of rows that need not start on 16
// bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "experts.cuh"

namespace km {

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ __half narrow(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow(float v) { return __float2bfloat16_rn(v); }

// Two values in one word, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t narrow2(float a, float b);
template <>
__device__ __forceinline__ uint32_t narrow2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t narrow2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t v);
template <>
__device__ __forceinline__ float2 widen2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
template <>
__device__ __forceinline__ float2 widen2<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// Bytes [s, s + 16) of a and b in a row; s is even and below 16.
__device__ __forceinline__ uint4 shifted(const uint4 &a, const uint4 &b, uint32_t s) {
    uint32_t w0 = a.x, w1 = a.y, w2 = a.z, w3 = a.w, w4 = b.x, w5 = b.y, w6 = b.z;
    if (s & 8u) {
        w0 = w2; w1 = w3; w2 = w4; w3 = w5; w4 = w6; w5 = b.w;
    }
    if (s & 4u) {
        w0 = w1; w1 = w2; w2 = w3; w3 = w4; w4 = w5;
    }
    const uint32_t r = (s & 3u) * 8u;
    return make_uint4(__funnelshift_r(w0, w1, r), __funnelshift_r(w1, w2, r), __funnelshift_r(w2, w3, r),
                      __funnelshift_r(w3, w4, r));
}

// Where a tensor's bytes lie.
struct Span {
    const uint8_t *lo, *hi;
};

// `bytes` of the piece at p exist (1 .. 16).
template <bool WHOLE>
__device__ __forceinline__ uint4 load_piece(const uint8_t *p, int bytes, const Span &in) {
    if constexpr (WHOLE) return *reinterpret_cast<const uint4 *>(p);
    const uint32_t s = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;
    const uint8_t *a = p - s;
    const bool two = s + bytes > 16;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (a >= in.lo && a + (two ? 32 : 16) <= in.hi) {
        const uint4 first = *reinterpret_cast<const uint4 *>(a);
        const uint4 second = two ? *reinterpret_cast<const uint4 *>(a + 16) : zero;
        uint4 v = shifted(first, second, s);
        if (bytes < 16) {  // nothing past the row
            uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int left = bytes - 4 * i;
                u[i] = left >= 4 ? u[i] : (left >= 2 ? u[i] & 0xffffu : 0u);
            }
            v = make_uint4(u[0], u[1], u[2], u[3]);
        }
        return v;
    }
    uint32_t u[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (2 * i < bytes) u[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(p + 2 * i) << ((i & 1) * 16);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// The sixteen bytes at p, an even address that may lie before or past the
// tensor: bytes outside it read as zero.
__device__ __forceinline__ uint4 load_word(const uint8_t *p, const Span &in) {
    const uint32_t s = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;
    const uint8_t *a = p - s;
    if (a >= in.lo && a + (s ? 32 : 16) <= in.hi) {
        const uint4 first = *reinterpret_cast<const uint4 *>(a);
        return s ? shifted(first, *reinterpret_cast<const uint4 *>(a + 16), s) : first;
    }
    uint32_t u[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (p + 2 * i >= in.lo && p + 2 * i + 2 <= in.hi)
            u[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(p + 2 * i) << ((i & 1) * 16);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Bytes [lo, hi) of the aligned word at p, both even.
__device__ __forceinline__ void store_word(uint8_t *p, const uint4 &v, int lo, int hi) {
    if (lo <= 0 && hi >= 16) {
        *reinterpret_cast<uint4 *>(p) = v;
        return;
    }
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool low = 4 * i >= lo && 4 * i + 2 <= hi, high = 4 * i + 2 >= lo && 4 * i + 4 <= hi;
        if (low && high)
            *reinterpret_cast<uint32_t *>(p + 4 * i) = u[i];
        else if (low)
            *reinterpret_cast<uint16_t *>(p + 4 * i) = (uint16_t)u[i];
        else if (high)
            *reinterpret_cast<uint16_t *>(p + 4 * i + 2) = (uint16_t)(u[i] >> 16);
    }
}

}  // namespace km
