// Expert routing (slots sorted by expert, rows moved there and back) and the
// experts' matrix products: layouts and launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace km {

// ------------------------------------------------------------------ routing
// One thread-block cluster sorts all slots; nothing but the status word needs
// device scratch.
inline int64_t route_ws_bytes() { return (int64_t)sizeof(WsHeader); }

cudaError_t launch_route(const void *experts, int id_bytes, int64_t slots, int n_experts, int32_t *offsets,
                         int32_t *order, int32_t *rows, uint32_t *status, cudaStream_t s);

// Rows between token order and expert order.  `dtype` is a KMEANS_F32 /
// KMEANS_F16 / KMEANS_BF16 code, ld* a row pitch in elements.
struct RouteRows {
    const int32_t *rows;     // (n, topk) row of every slot in expert order
    const int32_t *offsets;  // (n_experts + 1); rows at or past the last one are dropped slots
    int64_t n;
    int topk, n_experts;
    int64_t d;
};

cudaError_t launch_route_gather(const RouteRows &r, int dtype, const void *x, int64_t ldx, void *xs, cudaStream_t s);
cudaError_t launch_route_combine(const RouteRows &r, int dtype, const void *ys, const float *weights,
                                 const void *residual, int64_t ldr, void *y, cudaStream_t s);
cudaError_t launch_route_combine_grad(const RouteRows &r, int dtype, const void *dy, int64_t lddy, const void *ys,
                                      const float *weights, void *dys, float *dweights, cudaStream_t s);

// ----------------------------------------------------------------- products
// Rows [offsets[e], offsets[e + 1]) of x belong to expert e; without offsets
// there is one expert and every row is its own.
struct LinearShape {
    int64_t m, n, k;         // rows, output features, input features
    int n_experts;
    const int32_t *offsets;  // null: one expert
    bool bf16;               // else fp16
};

struct LinearLayout {
    int64_t off_x;   // x with its rows on 16 bytes, where the caller's are not
    int64_t off_w;   // w likewise (0: its rows are a multiple of 16 bytes)
    int64_t off_dz;  // dy after the activation's slope, rows on 16 bytes (gradient)
    int64_t bytes;
};

LinearLayout linear_layout(bool grad, int64_t m, int64_t n, int64_t k, int64_t n_experts);

cudaError_t launch_linear(const LinearShape &sh, const void *x, int64_t ldx, const void *w, const void *bias,
                          const void *residual, int64_t ldr, int activation, void *y, void *pre,
                          const LinearLayout &L, uint8_t *ws, cudaStream_t s);
cudaError_t launch_linear_grad(const LinearShape &sh, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                               const void *w, const void *pre, int activation, void *dx, void *dw, void *db,
                               const LinearLayout &L, uint8_t *ws, cudaStream_t s);

// --------------------------------------------------------- shared arithmetic
// The activations and their slopes, in float32.  exp is the accurate expf:
// the products' epilogues have time for it, and a value that is kept in 16
// bits should carry that rounding alone.
template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == KMEANS_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays
    if constexpr (ACT == KMEANS_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    if constexpr (ACT == KMEANS_ACT_GELU_TANH)
        return 0.5f * z * (1.f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
    if constexpr (ACT == KMEANS_ACT_SILU) return z / (1.f + expf(-z));
    return z;
}

template <int ACT>
__device__ __forceinline__ float slope(float z) {
    if constexpr (ACT == KMEANS_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if constexpr (ACT == KMEANS_ACT_GELU)
        return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
    if constexpr (ACT == KMEANS_ACT_GELU_TANH) {
        const float t = tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z));
        return 0.5f * (1.f + t) + 0.5f * z * (1.f - t * t) * 0.79788456080286536f * (1.f + 0.134145f * z * z);
    }
    if constexpr (ACT == KMEANS_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-z));
        return s * (1.f + z * (1.f - s));
    }
    return 1.f;
}

}  // namespace km
