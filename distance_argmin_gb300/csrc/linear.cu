// The experts' matrix products with bias, activation and residual, and their
// gradients.
//
//   forward  y[r, :]  = act(x[r, :] W_e^T + b_e) + residual[r, :]
//   rows     dx[r, :] = dz[r, :] W_e              (r in expert e's rows)
//   weights  dW_e     = dz_e^T x_e
//
// All three are out(q, p) = sum_c A(p, c) B(q, c), with p the contiguous
// dimension of the output.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "experts.cuh"

namespace km {

namespace {

enum class Product { kForward, kRows, kWeights };

constexpr int kTile = 64;
constexpr int kStep = 16;
constexpr int kThreads = 256;

struct ProductParams {
    const void *a, *b, *bias, *residual;
    void *out, *pre;
    const int32_t *offsets;
    int64_t m, n, k, lda, ldb, ldr;
    int n_experts, activation;
};

__device__ __forceinline__ float wide(__half v) { return __half2float(v); }
__device__ __forceinline__ float wide(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ __half narrow(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float activate_as(int act, float z) {
    switch (act) {
        case KMEANS_ACT_RELU: return activate<KMEANS_ACT_RELU>(z);
        case KMEANS_ACT_GELU: return activate<KMEANS_ACT_GELU>(z);
        case KMEANS_ACT_GELU_TANH: return activate<KMEANS_ACT_GELU_TANH>(z);
        case KMEANS_ACT_SILU: return activate<KMEANS_ACT_SILU>(z);
        default: return z;
    }
}

__device__ __forceinline__ float slope_as(int act, float z) {
    switch (act) {
        case KMEANS_ACT_RELU: return slope<KMEANS_ACT_RELU>(z);
        case KMEANS_ACT_GELU: return slope<KMEANS_ACT_GELU>(z);
        case KMEANS_ACT_GELU_TANH: return slope<KMEANS_ACT_GELU_TANH>(z);
        case KMEANS_ACT_SILU: return slope<KMEANS_ACT_SILU>(z);
        default: return 1.f;
    }
}

// First row of expert e, kept inside [0, m] and not before `from`.
__device__ __forceinline__ int64_t first_row(const int32_t *offsets, int e, int64_t from, int64_t m) {
    const int64_t v = offsets[e];
    return v < from ? from : (v > m ? m : v);
}

// Rows of unit `u` of the row products: the tiles of expert 0, of expert 1, ...
// and last those of the rows that belong to no expert (expert = n_experts).
__device__ bool row_tile(const ProductParams &p, int64_t u, int &expert, int64_t &r0, int64_t &r1) {
    if (!p.offsets) {
        expert = 0;
        r0 = u * kTile;
        r1 = min(r0 + kTile, p.m);
        return r0 < p.m;
    }
    int64_t at = first_row(p.offsets, 0, 0, p.m);
    if (at > 0) at = 0;
    for (int e = 0; e <= p.n_experts; ++e) {
        const int64_t end = e < p.n_experts ? first_row(p.offsets, e + 1, at, p.m) : p.m;
        const int64_t tiles = (end - at + kTile - 1) / kTile;
        if (u < tiles) {
            expert = e;
            r0 = at + u * kTile;
            r1 = min(r0 + kTile, end);
            return true;
        }
        u -= tiles;
        at = end;
    }
    return false;
}

template <typename T, Product MODE>
__global__ void __launch_bounds__(kThreads) linear_tile_kernel(const ProductParams p) {
    __shared__ float as[kStep][kTile + 1], bs[kStep][kTile + 1];
    griddep_wait();
    const T *A = static_cast<const T *>(p.a), *B = static_cast<const T *>(p.b);
    int expert;
    int64_t q0, q1, c0, c1;  // output rows of this block, contraction range
    const int64_t cols = MODE == Product::kForward ? p.n : p.k;
    if (MODE == Product::kWeights) {
        expert = blockIdx.z;
        c0 = 0;
        c1 = p.m;
        if (p.offsets) {
            c0 = 0;
            c1 = 0;
            for (int e = 0; e <= expert; ++e) {
                c0 = c1;
                c1 = first_row(p.offsets, e + 1, c0, p.m);
            }
        }
        q0 = (int64_t)blockIdx.y * kTile;
        q1 = min(q0 + kTile, p.n);
    } else {
        if (!row_tile(p, blockIdx.y, expert, q0, q1)) return;
        c0 = 0;
        c1 = expert == p.n_experts ? 0 : (MODE == Product::kForward ? p.k : p.n);
    }
    const int64_t p0 = (int64_t)blockIdx.x * kTile;
    const int tp = threadIdx.x & 15, tq = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t c = c0; c < c1; c += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
            const bool by_c = MODE == Product::kForward;  // A's contiguous dimension is the contraction
            const int pi = by_c ? i / kStep : i % kTile, ci = by_c ? i % kStep : i / kTile;
            float v = 0.f;
            if (p0 + pi < cols && c + ci < c1) {
                if (MODE == Product::kForward) v = wide(A[((int64_t)expert * p.n + p0 + pi) * p.k + c + ci]);
                if (MODE == Product::kRows) v = wide(A[((int64_t)expert * p.n + c + ci) * p.k + p0 + pi]);
                if (MODE == Product::kWeights) v = wide(A[(c + ci) * p.lda + p0 + pi]);
            }
            as[ci][pi] = v;
            const bool rows_c = MODE != Product::kWeights;
            const int qi = rows_c ? i / kStep : i % kTile, cj = rows_c ? i % kStep : i / kTile;
            v = 0.f;
            if (q0 + qi < q1 && c + cj < c1)
                v = wide(rows_c ? B[(q0 + qi) * p.ldb + c + cj] : B[(c + cj) * p.ldb + q0 + qi]);
            bs[cj][qi] = v;
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kStep; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(bs[s][tq + 16 * i], as[s][tp + 16 * j], acc[i][j]);
        __syncthreads();
    }
    const bool real = MODE != Product::kForward || expert < p.n_experts;
    for (int i = 0; i < 4; ++i) {
        const int64_t q = q0 + tq + 16 * i;
        if (q >= q1) continue;
        for (int j = 0; j < 4; ++j) {
            const int64_t c = p0 + tp + 16 * j;
            if (c >= cols) continue;
            float v = acc[i][j];
            const int64_t at = (MODE == Product::kWeights ? (int64_t)expert * p.n + q : q) * cols + c;
            if (MODE == Product::kForward) {
                if (real && p.bias) v += wide(static_cast<const T *>(p.bias)[(int64_t)expert * p.n + c]);
                if (p.pre) static_cast<T *>(p.pre)[at] = narrow<T>(v);
                v = real ? activate_as(p.activation, v) : 0.f;
                if (real && p.residual) v += wide(static_cast<const T *>(p.residual)[q * p.ldr + c]);
            }
            static_cast<T *>(p.out)[at] = narrow<T>(v);
        }
    }
}

// dz = dy act'(pre), rounded to the matrices' type.
template <typename T>
__global__ void linear_slope_kernel(const T *dy, int64_t lddy, const T *pre, int64_t m, int64_t n, int act, T *dz) {
    griddep_wait();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < m * n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / n, c = i - r * n;
        const float g = wide(dy[r * lddy + c]);
        dz[i] = narrow<T>(act == KMEANS_ACT_NONE ? g : g * slope_as(act, wide(pre[i])));
    }
}

template <typename T>
__global__ void linear_bias_grad_kernel(const T *dy, int64_t lddy, const T *pre, const int32_t *offsets, int64_t m,
                                        int64_t n, int act, T *db) {
    griddep_wait();
    const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= n) return;
    const int expert = blockIdx.y;
    int64_t r0 = 0, r1 = m;
    if (offsets) {
        r1 = 0;
        for (int e = 0; e <= expert; ++e) {
            r0 = r1;
            r1 = first_row(offsets, e + 1, r0, m);
        }
    }
    float sum = 0.f, lost = 0.f;  // compensated: one thread adds a whole column
    for (int64_t r = r0; r < r1; ++r) {
        const float g = wide(dy[r * lddy + c]);
        const float v = (act == KMEANS_ACT_NONE ? g : g * slope_as(act, wide(pre[r * n + c]))) - lost;
        const float t = sum + v;
        lost = (t - sum) - v;
        sum = t;
    }
    db[(int64_t)expert * n + c] = narrow<T>(sum);
}

ProductParams product_params(const LinearShape &sh) {
    ProductParams p{};
    p.offsets = sh.offsets;
    p.m = sh.m;
    p.n = sh.n;
    p.k = sh.k;
    p.n_experts = sh.n_experts;
    return p;
}

unsigned tiles(int64_t v) { return (unsigned)((v + kTile - 1) / kTile); }

template <typename T, Product MODE>
cudaError_t launch_product(const LinearShape &sh, const ProductParams &p, cudaStream_t s) {
    const unsigned cols = tiles(MODE == Product::kForward ? sh.n : sh.k);
    const dim3 grid = MODE == Product::kWeights
                          ? dim3(cols, tiles(sh.n), (unsigned)sh.n_experts)
                          : dim3(cols, tiles(sh.m) + (sh.offsets ? (unsigned)sh.n_experts + 1 : 0));
    return launch_kernel(true, linear_tile_kernel<T, MODE>, grid, dim3(kThreads), 0, s, p);
}

template <typename T>
cudaError_t grad_typed(const LinearShape &sh, const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *w,
                       const void *pre, int activation, void *dx, void *dw, void *db, const LinearLayout &L,
                       uint8_t *ws, cudaStream_t s) {
    T *dz = reinterpret_cast<T *>(ws + L.off_dz);
    cudaError_t e = cudaSuccess;
    if (sh.m > 0)
        e = launch_kernel(true, linear_slope_kernel<T>, dim3(152 * 8), dim3(256), 0, s, static_cast<const T *>(dy),
                          lddy, static_cast<const T *>(pre), sh.m, sh.n, activation, dz);
    if (e == cudaSuccess && db)
        e = launch_kernel(true, linear_bias_grad_kernel<T>, dim3((unsigned)((sh.n + 127) / 128), (unsigned)sh.n_experts),
                          dim3(128), 0, s, static_cast<const T *>(dy), lddy, static_cast<const T *>(pre), sh.offsets,
                          sh.m, sh.n, activation, static_cast<T *>(db));
    ProductParams p = product_params(sh);
    p.b = dz;
    p.ldb = sh.n;
    if (e == cudaSuccess && dx && sh.m > 0) {
        p.a = w;
        p.out = dx;
        e = launch_product<T, Product::kRows>(sh, p, s);
    }
    if (e == cudaSuccess && dw) {
        p.a = x;
        p.lda = ldx;
        p.out = dw;
        e = launch_product<T, Product::kWeights>(sh, p, s);
    }
    return e;
}

}  // namespace

LinearLayout linear_layout(bool grad, int64_t m, int64_t n, int64_t k, int64_t n_experts) {
    (void)k;
    (void)n_experts;
    LinearLayout L{};
    int64_t o = align_up((int64_t)sizeof(WsHeader), 1024);
    if (grad) {
        L.off_dz = o;
        o = align_up(o + m * n * 2, 1024);
    }
    L.bytes = o;
    return L;
}

cudaError_t launch_linear(const LinearShape &sh, const void *x, int64_t ldx, const void *w, const void *bias,
                          const void *residual, int64_t ldr, int activation, void *y, void *pre,
                          const LinearLayout &L, uint8_t *ws, cudaStream_t s) {
    (void)L;
    cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(WsHeader), s);  // this call's status word
    if (e != cudaSuccess || sh.m == 0) return e;
    ProductParams p = product_params(sh);
    p.a = w;
    p.b = x;
    p.ldb = ldx;
    p.bias = bias;
    p.residual = residual;
    p.ldr = ldr;
    p.activation = activation;
    p.out = y;
    p.pre = pre;
    return sh.bf16 ? launch_product<__nv_bfloat16, Product::kForward>(sh, p, s)
                   : launch_product<__half, Product::kForward>(sh, p, s);
}

cudaError_t launch_linear_grad(const LinearShape &sh, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                               const void *w, const void *pre, int activation, void *dx, void *dw, void *db,
                               const LinearLayout &L, uint8_t *ws, cudaStream_t s) {
    const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(WsHeader), s);  // this call's status word
    if (e != cudaSuccess) return e;
    return sh.bf16 ? grad_typed<__nv_bfloat16>(sh, dy, lddy, x, ldx, w, pre, activation, dx, dw, db, L, ws, s)
                   : grad_typed<__half>(sh, dy, lddy, x, ldx, w, pre, activation, dx, dw, db, L, ws, s);
}

}  // namespace km
