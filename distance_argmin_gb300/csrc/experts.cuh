// Expert routing (slots sorted by expert, rows moved there and back) and the
// experts' matrix products: layouts and launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace km {

constexpr int kSMs = 152;  // of a GB300, which the rules on sizes are made for

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

// Starts with the header and the CTA pairs' status words.
struct LinearLayout {
    int64_t off_x;   // x with its rows on 16 bytes, where the caller's are not
    int64_t off_w;   // w likewise (0: its rows are a multiple of 16 bytes)
    int64_t off_dz;  // dy after the activation's slope, rows on 16 bytes (gradient)
    int64_t off_sums;     // sums of chunks of a contraction
    int64_t off_partial;  // the bias gradient's sums per row tile (gradient)
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
// The activations and their slopes in float32, on the hardware's exp2 and
// reciprocal (a few 2^-23 each): the products' epilogue has some twenty
// instructions per value before it, not the loads, sets the pace.
//   z Phi(z)        Phi through erf(x) = 1 - (a1 t + .. + a5 t^5) exp(-x^2),
//                   t = 1 / (1 + p x), x >= 0: Abramowitz and Stegun, formula
//                   7.1.26, within 1.5e-7; the slope's density shares the exp
//   its tanh form   (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
// Each is within 2^-19 (|z| + 1) of its formula.  Where the result goes to zero
// with z that says little of its own bits: there the logistic forms keep the
// exponential's relative error, and z Phi(z) takes the tail 1 - erf as it
// stands, not as a difference, so that its relative error is 7.1.26's own, 5e-4
// at z = -4 (two of float16's last bits there), 0.4% at -6 and 3% at -12.
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float reciprocal_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2E = 1.4426950408889634f;

// 1 / (1 + 2^-x)
__device__ __forceinline__ float logistic2(float x) { return reciprocal_approx(1.f + exp2_approx(-x)); }
__device__ __forceinline__ float logistic(float z) { return logistic2(z * kLog2E); }

template <int ACT>
__device__ __forceinline__ float2 activate2(float2 z);

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == KMEANS_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN stays
    if constexpr (ACT == KMEANS_ACT_GELU) return activate2<ACT>(make_float2(z, z)).x;
    if constexpr (ACT == KMEANS_ACT_GELU_TANH)
        return z * logistic2(z * fmaf(0.0713548162726f * kLog2E, z * z, 1.5957691216057308f * kLog2E));
    if constexpr (ACT == KMEANS_ACT_SILU) return z * logistic(z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float slope(float z) {
    static_assert(ACT != KMEANS_ACT_GELU, "by pairs: slope2");
    if constexpr (ACT == KMEANS_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if constexpr (ACT == KMEANS_ACT_GELU_TANH) {
        // u' = 2 sqrt(2 / pi) (1 + 3 a z^2); far out s (1 - s) is 0 while z u'
        // may be infinite, hence the cut
        const float zz = fminf(z * z, 1e4f);
        const float s = logistic2(z * fmaf(0.0713548162726f * kLog2E, z * z, 1.5957691216057308f * kLog2E));
        return fmaf(z * s * (1.f - s), fmaf(0.2140644488178f, zz, 1.5957691216057308f), s);
    }
    if constexpr (ACT == KMEANS_ACT_SILU) {
        const float s = logistic(z);
        return fmaf(z * s, 1.f - s, s);
    }
    return 1.f;
}

// Two values at a time: z Phi(z) takes some thirty instructions a value, and the
// multiplications and additions among them go by pairs.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Phi(z), and exp(-z^2 / 2) beside it
__device__ __forceinline__ float2 normal_cdf2(float2 z, float2 &e) {
    const float2 e2 = __fmul2_rn(__fmul2_rn(z, z), both(-0.5f * kLog2E));
    e = make_float2(exp2_approx(e2.x), exp2_approx(e2.y));
    constexpr float P = 0.3275911f * 0.70710678118654752f;
    const float2 t = make_float2(reciprocal_approx(fmaf(P, fabsf(z.x), 1.f)), reciprocal_approx(fmaf(P, fabsf(z.y), 1.f)));
    float2 poly = __ffma2_rn(t, both(0.5f * 1.061405429f), both(0.5f * -1.453152027f));
    poly = __ffma2_rn(t, poly, both(0.5f * 1.421413741f));
    poly = __ffma2_rn(t, poly, both(0.5f * -0.284496736f));
    poly = __ffma2_rn(t, poly, both(0.5f * 0.254829592f));
    const float2 tail = __fmul2_rn(__fmul2_rn(poly, t), e);  // 1 - Phi(|z|)
    const float2 rest = __fadd2_rn(both(1.f), make_float2(-tail.x, -tail.y));
    return make_float2(z.x < 0.f ? tail.x : rest.x, z.y < 0.f ? tail.y : rest.y);
}

// 1 / (1 + 2^x)
__device__ __forceinline__ float2 inverse_power2(float2 x) {
    const float2 d = __fadd2_rn(make_float2(exp2_approx(x.x), exp2_approx(x.y)), both(1.f));
    return make_float2(reciprocal_approx(d.x), reciprocal_approx(d.y));
}

template <int ACT>
__device__ __forceinline__ float2 activate2(float2 z) {
    if constexpr (ACT == KMEANS_ACT_GELU) {
        float2 e;
        return __fmul2_rn(z, normal_cdf2(z, e));
    } else if constexpr (ACT == KMEANS_ACT_GELU_TANH) {
        const float2 u = __ffma2_rn(both(-0.0713548162726f * kLog2E), __fmul2_rn(z, z), both(-1.5957691216057308f * kLog2E));
        return __fmul2_rn(z, inverse_power2(__fmul2_rn(z, u)));
    } else if constexpr (ACT == KMEANS_ACT_SILU) {
        return __fmul2_rn(z, inverse_power2(__fmul2_rn(z, both(-kLog2E))));
    } else {
        return make_float2(activate<ACT>(z.x), activate<ACT>(z.y));
    }
}

template <int ACT>
__device__ __forceinline__ float2 slope2(float2 z) {
    if constexpr (ACT == KMEANS_ACT_GELU) {
        float2 e;
        const float2 cdf = normal_cdf2(z, e);
        return __ffma2_rn(__fmul2_rn(z, both(0.39894228040143268f)), e, cdf);
    } else {
        return make_float2(slope<ACT>(z.x), slope<ACT>(z.y));
    }
}

}  // namespace km
