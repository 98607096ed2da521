// The experts' matrix products and their gradients: which kernels a call runs,
// and what goes around the products (linear_tc.cu): rows brought to 16 bytes,
// dz = dy act'(pre), and the bias gradient.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "linear_common.cuh"

namespace km {

namespace {

__device__ __forceinline__ float slope_as(int act, float z) {
    switch (act) {
        case KMEANS_ACT_RELU: return slope<KMEANS_ACT_RELU>(z);
        case KMEANS_ACT_GELU: return slope<KMEANS_ACT_GELU>(z);
        case KMEANS_ACT_GELU_TANH: return slope<KMEANS_ACT_GELU_TANH>(z);
        case KMEANS_ACT_SILU: return slope<KMEANS_ACT_SILU>(z);
        default: return 1.f;
    }
}

// dst(r, c) = src(r, c) with the rows of dst on 16 bytes.
template <typename T>
__global__ void linear_align_kernel(const T *src, int64_t lds, int64_t rows, int64_t cols, T *dst, int64_t ldd,
                                    uint32_t *clear) {
    griddep_wait();
    if (clear && blockIdx.x == 0 && threadIdx.x == 0) *clear = 0u;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) dst[r * ldd + c] = src[r * lds + c];
}

// dz = dy act'(pre), rounded to the matrices' type.
template <typename T>
__global__ void linear_slope_kernel(const T *dy, int64_t lddy, const T *pre, int64_t m, int64_t n, int act, T *dz,
                                    int64_t ldz, uint32_t *clear) {
    griddep_wait();
    if (clear && blockIdx.x == 0 && threadIdx.x == 0) *clear = 0u;
    for (int64_t r = blockIdx.x; r < m; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < n; c += blockDim.x) {
            const float g = widen(dy[r * lddy + c]);
            dz[r * ldz + c] = narrow<T>(act == KMEANS_ACT_NONE ? g : g * slope_as(act, widen(pre[r * n + c])));
        }
}

template <typename T>
__global__ void linear_bias_grad_kernel(const T *dy, int64_t lddy, const T *pre, const int32_t *offsets, int64_t m,
                                        int64_t n, int act, T *db, uint32_t *clear) {
    griddep_wait();
    if (clear && (blockIdx.x | blockIdx.y | threadIdx.x) == 0u) *clear = 0u;
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
        const float g = widen(dy[r * lddy + c]);
        const float v = (act == KMEANS_ACT_NONE ? g : g * slope_as(act, widen(pre[r * n + c]))) - lost;
        const float t = sum + v;
        lost = (t - sum) - v;
        sum = t;
    }
    db[(int64_t)expert * n + c] = narrow<T>(sum);
}

// One call's kernels on the stream: the first of them clears the status word.
template <typename T>
struct Call {
    const LinearShape &sh;
    const LinearLayout &L;
    uint8_t *ws;
    cudaStream_t s;
    uint32_t *clear;

    Call(const LinearShape &sh_, const LinearLayout &L_, uint8_t *ws_, cudaStream_t s_)
        : sh(sh_), L(L_), ws(ws_), s(s_), clear(&reinterpret_cast<WsHeader *>(ws_)->status) {}
    uint32_t *first() {
        uint32_t *c = clear;
        clear = nullptr;
        return c;
    }

    cudaError_t align(const void *&src, int64_t &pitch, int64_t rows, int64_t cols, int64_t off) {
        if (rows16(src, pitch) || off == 0 || rows == 0) return cudaSuccess;
        T *dst = reinterpret_cast<T *>(ws + off);
        const int64_t ldd = align_up(cols, 8);
        const cudaError_t e = launch_kernel(true, linear_align_kernel<T>, dim3((unsigned)(rows < 8192 ? rows : 8192)),
                                            dim3(256), 0, s, static_cast<const T *>(src), pitch, rows, cols, dst, ldd,
                                            first());
        src = dst;
        pitch = ldd;
        return e;
    }
    cudaError_t align_w(Product16 &g) {
        return align(g.a, g.pitch_w, (int64_t)sh.n_experts * sh.n, sh.k, L.off_w);
    }
    template <Product MODE>
    cudaError_t product(const Product16 &g) {
        return launch_linear_tc(MODE, sh, g, &reinterpret_cast<WsHeader *>(ws)->status, first() != nullptr, s);
    }
};

template <typename T>
cudaError_t forward_typed(const LinearShape &sh, Product16 g, const LinearLayout &L, uint8_t *ws, cudaStream_t s) {
    Call<T> call(sh, L, ws, s);
    cudaError_t e = call.align_w(g);
    if (e == cudaSuccess) e = call.align(g.b, g.ldb, sh.m, sh.k, L.off_x);
    if (e == cudaSuccess) e = call.template product<Product::kForward>(g);
    return e;
}

template <typename T>
cudaError_t grad_typed(const LinearShape &sh, const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *w,
                       const void *pre, int activation, void *dx, void *dw, void *db, const LinearLayout &L,
                       uint8_t *ws, cudaStream_t s) {
    Call<T> call(sh, L, ws, s);
    cudaError_t e = cudaSuccess;
    Product16 g{};
    g.b = dy;
    g.ldb = lddy;
    if ((activation != KMEANS_ACT_NONE || !rows16(dy, lddy)) && sh.m > 0 && (dx || dw)) {
        T *dz = reinterpret_cast<T *>(ws + L.off_dz);
        g.b = dz;
        g.ldb = align_up(sh.n, 8);
        e = launch_kernel(true, linear_slope_kernel<T>, dim3((unsigned)(sh.m < 8192 ? sh.m : 8192)), dim3(256), 0, s,
                          static_cast<const T *>(dy), lddy, static_cast<const T *>(pre), sh.m, sh.n, activation, dz,
                          g.ldb, call.first());
    }
    if (e == cudaSuccess && db)
        e = launch_kernel(true, linear_bias_grad_kernel<T>, dim3((unsigned)((sh.n + 127) / 128), (unsigned)sh.n_experts),
                          dim3(128), 0, s, static_cast<const T *>(dy), lddy, static_cast<const T *>(pre), sh.offsets,
                          sh.m, sh.n, activation, static_cast<T *>(db), call.first());
    if (e == cudaSuccess && dx && sh.m > 0) {
        g.a = w;
        g.pitch_w = sh.k;
        g.out = dx;
        e = call.align_w(g);
        if (e == cudaSuccess) e = call.template product<Product::kRows>(g);
    }
    if (e == cudaSuccess && dw && sh.m == 0)
        return cudaMemsetAsync(dw, 0, (size_t)sh.n_experts * (size_t)sh.n * (size_t)sh.k * sizeof(T), s);
    if (e == cudaSuccess && dw) {
        g.a = x;
        g.lda = ldx;
        g.out = dw;
        e = call.align(g.a, g.lda, sh.m, sh.k, L.off_x);
        if (e == cudaSuccess) e = call.template product<Product::kWeights>(g);
    }
    return e;
}

}  // namespace

LinearLayout linear_layout(bool grad, int64_t m, int64_t n, int64_t k, int64_t n_experts) {
    LinearLayout L{};
    int64_t o = align_up((int64_t)sizeof(WsHeader), 1024);
    L.off_x = o;
    o = align_up(o + m * align_up(k, 8) * 2, 1024);
    if (k % 8 != 0) {
        L.off_w = o;
        o = align_up(o + n_experts * n * align_up(k, 8) * 2, 1024);
    }
    if (grad) {
        L.off_dz = o;
        o = align_up(o + m * align_up(n, 8) * 2, 1024);
    }
    L.bytes = o;
    return L;
}

cudaError_t launch_linear(const LinearShape &sh, const void *x, int64_t ldx, const void *w, const void *bias,
                          const void *residual, int64_t ldr, int activation, void *y, void *pre,
                          const LinearLayout &L, uint8_t *ws, cudaStream_t s) {
    if (sh.m == 0) return cudaMemsetAsync(ws, 0, sizeof(WsHeader), s);  // this call's status word
    Product16 g{};
    g.a = w;
    g.pitch_w = sh.k;
    g.b = x;
    g.ldb = ldx;
    g.bias = bias;
    g.residual = residual;
    g.ldr = ldr;
    g.activation = activation;
    g.out = y;
    g.pre = pre;
    return sh.bf16 ? forward_typed<__nv_bfloat16>(sh, g, L, ws, s) : forward_typed<__half>(sh, g, L, ws, s);
}

cudaError_t launch_linear_grad(const LinearShape &sh, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                               const void *w, const void *pre, int activation, void *dx, void *dw, void *db,
                               const LinearLayout &L, uint8_t *ws, cudaStream_t s) {
    if (sh.m == 0) {
        const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(WsHeader), s);  // this call's status word
        if (e != cudaSuccess) return e;
    }
    return sh.bf16 ? grad_typed<__nv_bfloat16>(sh, dy, lddy, x, ldx, w, pre, activation, dx, dw, db, L, ws, s)
                   : grad_typed<__half>(sh, dy, lddy, x, ldx, w, pre, activation, dx, dw, db, L, ws, s);
}

}  // namespace km
