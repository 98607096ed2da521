// What the kernels of the experts' products share: 16-bit conversions, the
// activations, and which rows belong to whom.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "experts.cuh"

namespace km {

// forward  y = act(x W^T + b) + residual
// rows     dx = dz W
// weights  dW = dz^T x
// All three are out(q, p) = sum_c A(p, c) B(q, c), with p the contiguous
// dimension of the output: output features, input features, input features.
enum class Product { kForward, kRows, kWeights };

struct Product16 {
    const void *a;            // w (forward, rows) or x (weights)
    int64_t lda;              // pitch of x (weights)
    int64_t pitch_w;          // pitch of w's rows (forward, rows)
    const void *b;            // x (forward) or dz
    int64_t ldb;
    const void *bias, *residual;
    int64_t ldr;
    int activation;
    void *out, *pre;
};

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

// f applied with the activation as a compile-time constant: one branch around
// a whole loop instead of one per value.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F &&f) {
    switch (act) {
        case KMEANS_ACT_RELU: f(std::integral_constant<int, KMEANS_ACT_RELU>{}); break;
        case KMEANS_ACT_GELU: f(std::integral_constant<int, KMEANS_ACT_GELU>{}); break;
        case KMEANS_ACT_GELU_TANH: f(std::integral_constant<int, KMEANS_ACT_GELU_TANH>{}); break;
        case KMEANS_ACT_SILU: f(std::integral_constant<int, KMEANS_ACT_SILU>{}); break;
        default: f(std::integral_constant<int, KMEANS_ACT_NONE>{}); break;
    }
}

// First row past expert e - 1's when the rows before `from` are taken: the
// offset, kept inside [from, m].
__device__ __forceinline__ int64_t first_row(const int32_t *offsets, int e, int64_t from, int64_t m) {
    const int64_t v = offsets[e];
    return v < from ? from : (v > m ? m : v);
}

// A matrix whose rows all start on 16 bytes.
inline bool rows16(const void *base, int64_t pitch_elems) {
    return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && pitch_elems % 8 == 0;
}

// The product on the tensor cores; w, x and dz must be rows16.  `clear`: the
// kernel is the call's first and clears the status word.
cudaError_t launch_linear_tc(Product mode, const LinearShape &sh, const Product16 &g, uint32_t *status, bool clear,
                             cudaStream_t s);

}  // namespace km
