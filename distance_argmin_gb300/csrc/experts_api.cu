// C ABI of the expert routing and the experts' products (declared in
// include/kmeans_gb300.h): argument validation and the launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "api_checks.cuh"
#include "experts.cuh"

using namespace km;

namespace {

bool route_sizes_ok(int64_t n, int64_t topk, int64_t n_experts) {
    return n >= 0 && topk >= 0 && n <= kMaxIndex && topk <= kMaxIndex && n * topk <= kMaxIndex && n_experts >= 1 &&
           n_experts <= kMaxIndex;
}

int route_limits(int64_t topk, int64_t n_experts) {
    return (topk <= KMEANS_ROUTE_MAX_TOPK && n_experts <= KMEANS_ROUTE_MAX_EXPERTS) ? KMEANS_OK
                                                                                     : KMEANS_ERR_UNSUPPORTED;
}

// What the three row-moving calls share.  `rows` and `offsets` may be null
// only when there is no slot to look up.
int check_rows(const int32_t *rows, const int32_t *offsets, int dtype, int64_t n, int64_t topk, int64_t n_experts,
               int64_t d) {
    if (!known_dtype(dtype) || !route_sizes_ok(n, topk, n_experts) || d < 0 || d > kMaxIndex)
        return KMEANS_ERR_INVALID_ARG;
    if (n * topk > 0 && (!rows || !offsets)) return KMEANS_ERR_INVALID_ARG;
    if (!aligned4(rows) || !aligned4(offsets)) return KMEANS_ERR_INVALID_ARG;
    if (d > KMEANS_ROUTE_MAX_WIDTH) return KMEANS_ERR_UNSUPPORTED;
    return route_limits(topk, n_experts);
}

RouteRows route_rows(const int32_t *rows, const int32_t *offsets, int64_t n, int64_t topk, int64_t n_experts,
                     int64_t d) {
    RouteRows r{};
    r.rows = rows;
    r.offsets = offsets;
    r.n = n;
    r.topk = (int)topk;
    r.n_experts = (int)n_experts;
    r.d = d;
    return r;
}

// (The matrices' sizes in bytes, and the workspace's, then fit 64 bits.)
bool linear_sizes_ok(int64_t m, int64_t n, int64_t k, int64_t n_experts) {
    constexpr int64_t most = KMEANS_LINEAR_MAX_SIZE, values = (int64_t)1 << 42;
    return m >= 0 && m <= most && n >= 1 && n <= most && k >= 1 && k <= most && n_experts >= 1 &&
           n_experts <= KMEANS_LINEAR_MAX_EXPERTS && n_experts * n <= kMaxIndex && m * n < values && m * k < values &&
           n_experts * n * k < values;
}

int check_linear(int dtype, int activation, const int32_t *offsets, int64_t m, int64_t n, int64_t k,
                 int64_t n_experts) {
    if (!known_dtype(dtype) || activation < KMEANS_ACT_NONE || activation > KMEANS_ACT_SILU)
        return KMEANS_ERR_INVALID_ARG;
    if (n_experts > KMEANS_LINEAR_MAX_EXPERTS && n_experts <= kMaxIndex) return KMEANS_ERR_UNSUPPORTED;
    if (!linear_sizes_ok(m, n, k, n_experts)) return KMEANS_ERR_INVALID_ARG;
    if ((!offsets && n_experts != 1) || !aligned4(offsets)) return KMEANS_ERR_INVALID_ARG;
    return dtype == KMEANS_F32 ? KMEANS_ERR_UNSUPPORTED : KMEANS_OK;
}

LinearShape linear_shape(int dtype, const int32_t *offsets, int64_t m, int64_t n, int64_t k, int64_t n_experts) {
    LinearShape sh{};
    sh.m = m;
    sh.n = n;
    sh.k = k;
    sh.n_experts = (int)n_experts;
    sh.offsets = offsets;
    sh.bf16 = dtype == KMEANS_BF16;
    return sh;
}

}  // namespace

extern "C" {

size_t kmeans_route_workspace_bytes(int64_t n, int64_t topk, int64_t n_experts) {
    if (!route_sizes_ok(n, topk, n_experts) || route_limits(topk, n_experts) != KMEANS_OK) return 0;
    return (size_t)route_ws_bytes();
}

int kmeans_route(const void *experts, int id_bytes, int64_t n, int64_t topk, int64_t n_experts, int32_t *offsets,
                 int32_t *order, int32_t *rows, void *ws, size_t ws_bytes, void *stream) {
    if ((id_bytes != 4 && id_bytes != 8) || !route_sizes_ok(n, topk, n_experts) || !offsets)
        return KMEANS_ERR_INVALID_ARG;
    if (n * topk > 0 && (!experts || !order || !rows)) return KMEANS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(experts) & (uintptr_t)(id_bytes - 1)) || !aligned4(offsets) || !aligned4(order) ||
        !aligned4(rows))
        return KMEANS_ERR_INVALID_ARG;
    const int lim = route_limits(topk, n_experts);
    if (lim != KMEANS_OK) return lim;
    const int wst = check_ws(ws, ws_bytes, (size_t)route_ws_bytes());
    if (wst != KMEANS_OK) return wst;
    return cuda_status(launch_route(experts, id_bytes, n * topk, (int)n_experts, offsets, order, rows,
                                    &static_cast<WsHeader *>(ws)->status, static_cast<cudaStream_t>(stream)));
}

int kmeans_route_gather(const void *x, int64_t ldx, int dtype, const int32_t *rows, const int32_t *offsets, int64_t n,
                        int64_t topk, int64_t n_experts, int64_t d, void *xs, void *stream) {
    const int st = check_rows(rows, offsets, dtype, n, topk, n_experts, d);
    if (st != KMEANS_OK) return st;
    if (n * topk == 0 || d == 0) return KMEANS_OK;
    if (!x || !xs || ldx < d || !elem_aligned(x, dtype) || !elem_aligned(xs, dtype)) return KMEANS_ERR_INVALID_ARG;
    return cuda_status(launch_route_gather(route_rows(rows, offsets, n, topk, n_experts, d), dtype, x, ldx, xs,
                                           static_cast<cudaStream_t>(stream)));
}

int kmeans_route_combine(const void *ys, int dtype, const float *weights, const void *residual, int64_t ldr,
                         const int32_t *rows, const int32_t *offsets, int64_t n, int64_t topk, int64_t n_experts,
                         int64_t d, void *y, void *stream) {
    const int st = check_rows(rows, offsets, dtype, n, topk, n_experts, d);
    if (st != KMEANS_OK) return st;
    if (n == 0 || d == 0) return KMEANS_OK;
    if (!y || (topk > 0 && !ys) || (residual && ldr < d)) return KMEANS_ERR_INVALID_ARG;
    if (!elem_aligned(ys, dtype) || !elem_aligned(y, dtype) || !elem_aligned(residual, dtype) || !aligned4(weights))
        return KMEANS_ERR_INVALID_ARG;
    return cuda_status(launch_route_combine(route_rows(rows, offsets, n, topk, n_experts, d), dtype, ys, weights,
                                            residual, ldr, y, static_cast<cudaStream_t>(stream)));
}

int kmeans_route_combine_grad(const void *dy, int64_t lddy, const void *ys, int dtype, const float *weights,
                              const int32_t *rows, const int32_t *offsets, int64_t n, int64_t topk, int64_t n_experts,
                              int64_t d, void *dys, float *dweights, void *stream) {
    const int st = check_rows(rows, offsets, dtype, n, topk, n_experts, d);
    if (st != KMEANS_OK) return st;
    if (n * topk == 0) return KMEANS_OK;
    if (!weights || !dweights || !aligned4(weights) || !aligned4(dweights)) return KMEANS_ERR_INVALID_ARG;
    if (d > 0 && (!dy || !ys || !dys || lddy < d)) return KMEANS_ERR_INVALID_ARG;
    if (!elem_aligned(dy, dtype) || !elem_aligned(ys, dtype) || !elem_aligned(dys, dtype)) return KMEANS_ERR_INVALID_ARG;
    return cuda_status(launch_route_combine_grad(route_rows(rows, offsets, n, topk, n_experts, d), dtype, dy, lddy, ys,
                                                 weights, dys, dweights, static_cast<cudaStream_t>(stream)));
}

size_t kmeans_linear_workspace_bytes(int grad, int64_t m, int64_t n, int64_t k, int64_t n_experts) {
    if ((grad != 0 && grad != 1) || !linear_sizes_ok(m, n, k, n_experts)) return 0;
    return (size_t)linear_layout(grad != 0, m, n, k, n_experts).bytes;
}

int kmeans_linear(const void *x, int64_t ldx, const void *w, const void *bias, const void *residual, int64_t ldr,
                  int dtype, int activation, const int32_t *offsets, int64_t m, int64_t n, int64_t k,
                  int64_t n_experts, void *y, void *pre, void *ws, size_t ws_bytes, void *stream) {
    const int st = check_linear(dtype, activation, offsets, m, n, k, n_experts);
    if (st != KMEANS_OK) return st;
    if (!w || !elem_aligned(w, dtype) || !elem_aligned(bias, dtype)) return KMEANS_ERR_INVALID_ARG;
    if (m > 0 && (!x || !y || ldx < k || (residual && ldr < n))) return KMEANS_ERR_INVALID_ARG;
    if (!elem_aligned(x, dtype) || !elem_aligned(residual, dtype) || !elem_aligned(y, dtype) ||
        !elem_aligned(pre, dtype))
        return KMEANS_ERR_INVALID_ARG;
    if (!aligned16(w)) return KMEANS_ERR_UNSUPPORTED;
    const LinearLayout L = linear_layout(false, m, n, k, n_experts);
    const int wst = check_ws(ws, ws_bytes, (size_t)L.bytes);
    if (wst != KMEANS_OK) return wst;
    return cuda_status(launch_linear(linear_shape(dtype, offsets, m, n, k, n_experts), x, ldx, w, bias, residual, ldr,
                                     activation, y, pre, L, static_cast<uint8_t *>(ws),
                                     static_cast<cudaStream_t>(stream)));
}

int kmeans_linear_grad(const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *w, const void *pre,
                       int dtype, int activation, const int32_t *offsets, int64_t m, int64_t n, int64_t k,
                       int64_t n_experts, void *dx, void *dw, void *db, void *ws, size_t ws_bytes, void *stream) {
    const int st = check_linear(dtype, activation, offsets, m, n, k, n_experts);
    if (st != KMEANS_OK) return st;
    if (m > 0 && (!dy || lddy < n || (activation != KMEANS_ACT_NONE && !pre))) return KMEANS_ERR_INVALID_ARG;
    if ((m > 0 && dw && (!x || ldx < k)) || (dx && !w)) return KMEANS_ERR_INVALID_ARG;
    const void *all[] = {dy, x, w, pre, dx, dw, db};
    for (const void *p : all)
        if (!elem_aligned(p, dtype)) return KMEANS_ERR_INVALID_ARG;
    if (dx && !aligned16(w)) return KMEANS_ERR_UNSUPPORTED;
    const LinearLayout L = linear_layout(true, m, n, k, n_experts);
    const int wst = check_ws(ws, ws_bytes, (size_t)L.bytes);
    if (wst != KMEANS_OK) return wst;
    return cuda_status(launch_linear_grad(linear_shape(dtype, offsets, m, n, k, n_experts), dy, lddy, x, ldx, w, pre,
                                          activation, dx, dw, db, L, static_cast<uint8_t *>(ws),
                                          static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
