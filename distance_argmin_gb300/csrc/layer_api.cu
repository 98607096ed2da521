// C ABI of the gate, the layer norm and the cross entropy (declared in include/kmeans_gb300.h):
// argument validation and the launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "api_checks.cuh"
#include "layer.cuh"

using namespace km;

namespace {

// What the gate and its gradient share.
int check_gate(int dtype, int scores, int64_t n, int64_t n_experts, int64_t topk, int64_t groups, int64_t topk_groups,
               float scale, const void *logits, int64_t ldl) {
    if (!known_dtype(dtype) || (scores != KMEANS_GATE_SOFTMAX && scores != KMEANS_GATE_SIGMOID) || n < 0 ||
        n > kMaxIndex || n_experts < 1 || topk < 0 || topk > n_experts || !isfinite(scale))
        return KMEANS_ERR_INVALID_ARG;
    if (groups < 1 || n_experts % groups != 0 || topk_groups < 1 || topk_groups > groups) return KMEANS_ERR_INVALID_ARG;
    if (n > 0 && (!logits || ldl < n_experts || !elem_aligned(logits, dtype))) return KMEANS_ERR_INVALID_ARG;
    if (n_experts > KMEANS_ROUTE_MAX_EXPERTS || topk > KMEANS_ROUTE_MAX_TOPK || groups > KMEANS_GATE_MAX_GROUPS)
        return KMEANS_ERR_UNSUPPORTED;
    return KMEANS_OK;
}

GateShape gate_shape(int scores, int64_t n, int64_t n_experts, int64_t topk, int64_t groups, int64_t topk_groups,
                     int renormalize, float scale) {
    return {n, (int)n_experts, (int)topk, (int)groups, (int)topk_groups, scores == KMEANS_GATE_SIGMOID, renormalize != 0,
            scale};
}

bool norm_sizes_ok(int64_t n, int64_t d) { return n >= 0 && n <= kMaxIndex && d >= 1 && d <= kMaxIndex; }

// (The matrices' and the workspace's sizes in bytes then fit 64 bits.)
bool xent_sizes_ok(int64_t m, int64_t n, int64_t k) {
    constexpr int64_t most = KMEANS_LINEAR_MAX_SIZE, values = (int64_t)1 << 42;
    return m >= 0 && m <= most && n >= 1 && n <= most && k >= 1 && k <= most && m * n < values && m * k < values &&
           n * k < values;
}

int check_xent(int dtype, const void *x, int64_t ldx, const void *w, const void *labels, int id_bytes, float scale,
               int64_t m, int64_t n, int64_t k) {
    // (scale / ln 2, which the logits are multiplied with, has to be finite)
    if (!known_dtype(dtype) || (id_bytes != 4 && id_bytes != 8) || !xent_sizes_ok(m, n, k) || !(scale > 0.f) ||
        scale > 0x1p127f)
        return KMEANS_ERR_INVALID_ARG;
    if (m > 0 && (!x || !w || !labels || ldx < k)) return KMEANS_ERR_INVALID_ARG;
    if (!elem_aligned(x, dtype) || !elem_aligned(w, dtype) ||
        (reinterpret_cast<uintptr_t>(labels) & (uintptr_t)(id_bytes - 1)))
        return KMEANS_ERR_INVALID_ARG;
    if (dtype == KMEANS_F32 || k > KMEANS_CROSS_ENTROPY_MAX_WIDTH || !aligned16(w)) return KMEANS_ERR_UNSUPPORTED;
    return KMEANS_OK;
}

}  // namespace

extern "C" {

int kmeans_gate(const void *logits, int64_t ldl, int dtype, int scores, const float *bias, int64_t n, int64_t n_experts,
                int64_t topk, int64_t groups, int64_t topk_groups, int renormalize, float scale, int32_t *ids,
                float *weights, void *stream) {
    const int st = check_gate(dtype, scores, n, n_experts, topk, groups, topk_groups, scale, logits, ldl);
    if (st != KMEANS_OK) return st;
    if (!aligned4(bias) || !aligned4(ids) || !aligned4(weights)) return KMEANS_ERR_INVALID_ARG;
    if (n * topk == 0) return KMEANS_OK;
    if (!ids || !weights) return KMEANS_ERR_INVALID_ARG;
    return cuda_status(launch_gate(gate_shape(scores, n, n_experts, topk, groups, topk_groups, renormalize, scale), dtype,
                                   logits, ldl, bias, ids, weights, static_cast<cudaStream_t>(stream)));
}

int kmeans_gate_grad(const float *dweights, const void *logits, int64_t ldl, int dtype, int scores, const int32_t *ids,
                     int64_t n, int64_t n_experts, int64_t topk, int renormalize, float scale, void *dlogits,
                     void *stream) {
    const int st = check_gate(dtype, scores, n, n_experts, topk, 1, 1, scale, logits, ldl);
    if (st != KMEANS_OK) return st;
    if (!aligned4(dweights) || !aligned4(ids) || !elem_aligned(dlogits, dtype)) return KMEANS_ERR_INVALID_ARG;
    if (n == 0) return KMEANS_OK;
    if (!dlogits || (topk > 0 && (!dweights || !ids))) return KMEANS_ERR_INVALID_ARG;
    return cuda_status(launch_gate_grad(gate_shape(scores, n, n_experts, topk, 1, 1, renormalize, scale), dtype, dweights,
                                        logits, ldl, ids, dlogits, static_cast<cudaStream_t>(stream)));
}

size_t kmeans_layernorm_workspace_bytes(int64_t n, int64_t d) {
    if (!norm_sizes_ok(n, d) || d > KMEANS_ROUTE_MAX_WIDTH) return 0;
    return (size_t)norm_layout(n, d).bytes;
}

int kmeans_layernorm(const void *x, int64_t ldx, int dtype, const void *weight, const void *bias, float eps, int64_t n,
                     int64_t d, void *y, float *mean, float *rstd, void *stream) {
    if (!known_dtype(dtype) || !norm_sizes_ok(n, d) || !(eps >= 0.f) || !isfinite(eps)) return KMEANS_ERR_INVALID_ARG;
    const void *all[] = {x, weight, bias, y};
    for (const void *p : all)
        if (!elem_aligned(p, dtype)) return KMEANS_ERR_INVALID_ARG;
    if (!aligned4(mean) || !aligned4(rstd)) return KMEANS_ERR_INVALID_ARG;
    if (d > KMEANS_ROUTE_MAX_WIDTH) return KMEANS_ERR_UNSUPPORTED;
    if (n == 0) return KMEANS_OK;
    if (!x || !y || ldx < d) return KMEANS_ERR_INVALID_ARG;
    return cuda_status(launch_norm({n, d, dtype}, x, ldx, weight, bias, eps, y, mean, rstd,
                                   static_cast<cudaStream_t>(stream)));
}

int kmeans_layernorm_grad(const void *dy, int64_t lddy, const void *x, int64_t ldx, int dtype, const float *mean,
                          const float *rstd, const void *weight, const void *residual, int64_t ldr, int64_t n, int64_t d,
                          void *dx, void *dweight, void *dbias, void *ws, size_t ws_bytes, void *stream) {
    if (!known_dtype(dtype) || !norm_sizes_ok(n, d)) return KMEANS_ERR_INVALID_ARG;
    const void *all[] = {dy, x, weight, residual, dx, dweight, dbias};
    for (const void *p : all)
        if (!elem_aligned(p, dtype)) return KMEANS_ERR_INVALID_ARG;
    if (!aligned4(mean) || !aligned4(rstd)) return KMEANS_ERR_INVALID_ARG;
    if (d > KMEANS_ROUTE_MAX_WIDTH) return KMEANS_ERR_UNSUPPORTED;
    if (n > 0 && (!dy || !x || !mean || !rstd || lddy < d || ldx < d || (residual && ldr < d)))
        return KMEANS_ERR_INVALID_ARG;
    const NormLayout L = norm_layout(n, d);
    const int wst = check_ws(ws, ws_bytes, (size_t)L.bytes);
    if (wst != KMEANS_OK) return wst;
    return cuda_status(launch_norm_grad({n, d, dtype}, dy, lddy, x, ldx, mean, rstd, weight, residual, ldr, dx, dweight,
                                        dbias, L, static_cast<uint8_t *>(ws), static_cast<cudaStream_t>(stream)));
}

size_t kmeans_cross_entropy_workspace_bytes(int grad, int64_t m, int64_t n, int64_t k) {
    if ((grad != 0 && grad != 1) || !xent_sizes_ok(m, n, k) || k > KMEANS_CROSS_ENTROPY_MAX_WIDTH) return 0;
    return (size_t)xent_layout(grad != 0, m, n, k).bytes;
}

int kmeans_cross_entropy(const void *x, int64_t ldx, const void *w, int dtype, const void *labels, int id_bytes,
                         float scale, int64_t m, int64_t n, int64_t k, float *loss, float *lse, void *ws,
                         size_t ws_bytes, void *stream) {
    const int st = check_xent(dtype, x, ldx, w, labels, id_bytes, scale, m, n, k);
    if (st != KMEANS_OK) return st;
    if ((m > 0 && (!loss || !lse)) || !aligned4(loss) || !aligned4(lse)) return KMEANS_ERR_INVALID_ARG;
    const XentLayout L = xent_layout(false, m, n, k);
    const int wst = check_ws(ws, ws_bytes, (size_t)L.bytes);
    if (wst != KMEANS_OK) return wst;
    return cuda_status(launch_xent({m, n, k, labels, id_bytes, scale, dtype == KMEANS_BF16}, x, ldx, w, loss, lse, L,
                                   static_cast<uint8_t *>(ws), static_cast<cudaStream_t>(stream)));
}

int kmeans_cross_entropy_grad(const float *dloss, const void *x, int64_t ldx, const void *w, int dtype,
                              const void *labels, int id_bytes, const float *lse, float scale, int64_t m, int64_t n,
                              int64_t k, void *dx, void *dw, void *ws, size_t ws_bytes, void *stream) {
    const int st = check_xent(dtype, x, ldx, w, labels, id_bytes, scale, m, n, k);
    if (st != KMEANS_OK) return st;
    if ((m > 0 && (!dloss || !lse)) || !aligned4(dloss) || !aligned4(lse) || !elem_aligned(dx, dtype) ||
        !elem_aligned(dw, dtype))
        return KMEANS_ERR_INVALID_ARG;
    const XentLayout L = xent_layout(true, m, n, k);
    const int wst = check_ws(ws, ws_bytes, (size_t)L.bytes);
    if (wst != KMEANS_OK) return wst;
    return cuda_status(launch_xent_grad({m, n, k, labels, id_bytes, scale, dtype == KMEANS_BF16}, dloss, x, ldx, w, lse,
                                        dx, dw, L, static_cast<uint8_t *>(ws), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
