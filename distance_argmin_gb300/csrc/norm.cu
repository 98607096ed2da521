// Layer norm over a row's features and its gradient.
//
//   mu = mean x   v = mean (x - mu)^2   r = 1 / sqrt(v + eps)
//   y = (x - mu) r w + b
//   g = dy w, h = (x - mu) r:  dx = r (g - mean g - h mean(g h)) + residual
//   dw = sum over rows of dy h, db = sum over rows of dy
//
// A group of TPR threads has a row and keeps it in registers as it lies in
// memory, 16-byte pieces of it per thread, so the row is read once: the mean,
// what the mean is off by (its sum rounds where the row lies far from zero) with
// the variance about it, and the result are three passes over registers.  Memory bounds it.  In the gradient a thread
// has the same columns in every row of its group, and adds up its share of dw
// and db in registers; the groups' sums meet in norm_join_kernel in a fixed
// order.  Rows too long for registers (or for the sums beside them) are read
// again for every pass, and dw and db get a kernel that goes down the columns.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "assign_common.cuh"
#include "layer.cuh"
#include "pieces.cuh"

namespace km {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

template <typename T>
struct Piece {  // 16 bytes of a row
    static constexpr int N = 16 / (int)sizeof(T);
    __device__ __forceinline__ static void open(const uint4 &u, float (&v)[N]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = widen2<T>(w[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
    __device__ __forceinline__ static uint4 close(const float (&v)[N]) {
        if constexpr (sizeof(T) == 4)
            return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        else
            return make_uint4(narrow2<T>(v[0], v[1]), narrow2<T>(v[2], v[3]), narrow2<T>(v[4], v[5]),
                              narrow2<T>(v[6], v[7]));
    }
};

// A matrix, or a vector as a matrix of one row, as bytes.
struct Rows {
    const uint8_t *base;  // null: not there
    int64_t pitch;
    Span in;
};

template <typename T>
Rows rows_of(const void *base, int64_t rows, int64_t ld, int64_t d) {
    const uint8_t *b = static_cast<const uint8_t *>(base);
    return {b, ld * (int64_t)sizeof(T), {b, b && rows > 0 ? b + ((rows - 1) * ld + d) * (int64_t)sizeof(T) : b}};
}

template <bool WHOLE>
__device__ __forceinline__ uint4 load_of(const Rows &m, int64_t r, int64_t at, int bytes) {
    return load_piece<WHOLE>(m.base + r * m.pitch + at, bytes, m.in);
}

// `count` values of a piece to p.
template <typename T, bool WHOLE>
__device__ __forceinline__ void store_piece(T *p, const float (&v)[Piece<T>::N], int count) {
    if constexpr (WHOLE) {
        *reinterpret_cast<uint4 *>(p) = Piece<T>::close(v);
    } else {
#pragma unroll
        for (int i = 0; i < Piece<T>::N; ++i)
            if (i < count) {
                if constexpr (sizeof(T) == 4)
                    p[i] = v[i];
                else
                    p[i] = narrow<T>(v[i]);
            }
    }
}

// Two sums over a group of TPR threads, in every one of them.  `turn` counts the
// calls: their shared memory alternates, so that one barrier is enough.
template <int TPR>
__device__ __forceinline__ float2 group_sum(float2 v, int &turn) {
    constexpr int WIDE = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = WIDE / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(kAll, v.x, o);
        v.y += __shfl_xor_sync(kAll, v.y, o);
    }
    if constexpr (TPR > 32) {
        constexpr int WARPS = TPR / 32;
        __shared__ float2 part[2][WARPS];
        float2 *mine = part[turn & 1];
        ++turn;
        if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
        __syncthreads();
        v = mine[0];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
            v.x += mine[w].x;
            v.y += mine[w].y;
        }
    }
    return v;
}

// (where all values are equal the difference may fall below zero by a rounding)
__device__ __forceinline__ float variance_of(float square, float off) {
    const float v = square - off * off;
    return v < 0.f ? 0.f : v;
}

__host__ __device__ constexpr int block_of(int tpr) { return tpr > 32 ? tpr : 128; }

template <typename T, int TPR, int PIECES, bool WHOLE>
__global__ void __launch_bounds__(block_of(TPR)) norm_kernel(const Rows x, const Rows w, const Rows b, float eps,
                                                             int64_t n, int d, T *y,
                                                             float *__restrict__ mean, float *__restrict__ rstd) {
    constexpr int N = Piece<T>::N, GROUPS = block_of(TPR) / TPR;
    griddep_wait();
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int pieces = (d + N - 1) / N;
    const float scale = 1.f / (float)d;
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < n; r0 += (int64_t)gridDim.x * GROUPS) {
        const int64_t r = r0 + group;
        const bool here = GROUPS == 1 || r < n;
        uint4 raw[PIECES];
        float2 sum = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int c = i * TPR + t, count = min(N, d - c * N);
            raw[i] = make_uint4(0, 0, 0, 0);
            if (here && c < pieces) raw[i] = load_of<WHOLE>(x, r, (int64_t)c * 16, count * (int)sizeof(T));
        }
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            float v[N];
            Piece<T>::open(raw[i], v);
#pragma unroll
            for (int j = 0; j < N; ++j) sum.x += v[j];
        }
        const float mu = group_sum<TPR>(sum, turn).x * scale;
        sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int count = d - (i * TPR + t) * N;
            float v[N];
            Piece<T>::open(raw[i], v);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (WHOLE ? count > 0 : j < count) {
                    sum.x += v[j] - mu;
                    sum.y += (v[j] - mu) * (v[j] - mu);
                }
        }
        sum = group_sum<TPR>(sum, turn);
        const float off = sum.x * scale, rs = rsqrtf(variance_of(sum.y * scale, off) + eps);
        if (!here) continue;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int c = i * TPR + t, count = min(N, d - c * N);
            if (c >= pieces) continue;
            float v[N], f[N];
            Piece<T>::open(raw[i], v);
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = ((v[j] - mu) - off) * rs;
            if (w.base) {
                Piece<T>::open(load_of<WHOLE>(w, 0, (int64_t)c * 16, count * (int)sizeof(T)), f);
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] *= f[j];
            }
            if (b.base) {
                Piece<T>::open(load_of<WHOLE>(b, 0, (int64_t)c * 16, count * (int)sizeof(T)), f);
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] += f[j];
            }
            store_piece<T, WHOLE>(y + r * d + (int64_t)c * N, v, count);
        }
        if (t == 0) {
            if (mean) mean[r] = mu + off;
            if (rstd) rstd[r] = rs;
        }
    }
}

// One row after the other, read again for every pass.
constexpr int kWideThreads = 1024;

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kWideThreads) norm_wide_kernel(const Rows x, const Rows w, const Rows b, float eps,
                                                                 int64_t n, int d, T *y,
                                                                 float *__restrict__ mean, float *__restrict__ rstd) {
    constexpr int N = Piece<T>::N;
    griddep_wait();
    const int pieces = (d + N - 1) / N;
    const float scale = 1.f / (float)d;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < n; r += gridDim.x) {
        float2 sum = {0.f, 0.f};
        float v[N], f[N];
        for (int c = threadIdx.x; c < pieces; c += kWideThreads) {
            Piece<T>::open(load_of<WHOLE>(x, r, (int64_t)c * 16, min(N, d - c * N) * (int)sizeof(T)), v);
#pragma unroll
            for (int j = 0; j < N; ++j) sum.x += v[j];
        }
        const float mu = group_sum<kWideThreads>(sum, turn).x * scale;
        sum = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < pieces; c += kWideThreads) {
            const int count = min(N, d - c * N);
            Piece<T>::open(load_of<WHOLE>(x, r, (int64_t)c * 16, count * (int)sizeof(T)), v);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (WHOLE || j < count) {
                    sum.x += v[j] - mu;
                    sum.y += (v[j] - mu) * (v[j] - mu);
                }
        }
        sum = group_sum<kWideThreads>(sum, turn);
        const float off = sum.x * scale, rs = rsqrtf(variance_of(sum.y * scale, off) + eps);
        for (int c = threadIdx.x; c < pieces; c += kWideThreads) {
            const int count = min(N, d - c * N);
            Piece<T>::open(load_of<WHOLE>(x, r, (int64_t)c * 16, count * (int)sizeof(T)), v);
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = ((v[j] - mu) - off) * rs;
            if (w.base) {
                Piece<T>::open(load_of<WHOLE>(w, 0, (int64_t)c * 16, count * (int)sizeof(T)), f);
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] *= f[j];
            }
            if (b.base) {
                Piece<T>::open(load_of<WHOLE>(b, 0, (int64_t)c * 16, count * (int)sizeof(T)), f);
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] += f[j];
            }
            store_piece<T, WHOLE>(y + r * d + (int64_t)c * N, v, count);
        }
        if (threadIdx.x == 0) {
            if (mean) mean[r] = mu + off;
            if (rstd) rstd[r] = rs;
        }
    }
}

struct GradRows {
    Rows dy, x, w, residual;
    const float *mean, *rstd;
    uint32_t *clear;  // the call's status word
    __device__ __forceinline__ void start() const {
        griddep_wait();
        if ((blockIdx.x | blockIdx.y | threadIdx.x) == 0u) *clear = 0u;
    }
};

// g and h of a piece.
template <typename T, bool WHOLE>
__device__ __forceinline__ void terms_of(const uint4 &dy, const uint4 &x, const Rows &w, int c, int count, float mu,
                                         float rs, float (&g)[Piece<T>::N], float (&h)[Piece<T>::N]) {
    constexpr int N = Piece<T>::N;
    Piece<T>::open(x, h);
    Piece<T>::open(dy, g);
#pragma unroll
    for (int j = 0; j < N; ++j) h[j] = (h[j] - mu) * rs;
    if (w.base) {
        float f[N];
        Piece<T>::open(load_of<WHOLE>(w, 0, (int64_t)c * 16, count * (int)sizeof(T)), f);
#pragma unroll
        for (int j = 0; j < N; ++j) g[j] *= f[j];
    }
}

template <typename T, bool WHOLE>
__device__ __forceinline__ void finish_piece(const Rows &residual, int64_t r, int c, int count, float rs, float mg,
                                             float mgh, const float (&g)[Piece<T>::N], const float (&h)[Piece<T>::N],
                                             T *out) {
    constexpr int N = Piece<T>::N;
    float v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = rs * (g[j] - mg - h[j] * mgh);
    if (residual.base) {
        float f[N];
        Piece<T>::open(load_of<WHOLE>(residual, r, (int64_t)c * 16, count * (int)sizeof(T)), f);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] += f[j];
    }
    store_piece<T, WHOLE>(out, v, count);
}

// SUMS: the group's part of dw and db to row `blockIdx.x` of `partial`, (blocks,
// 2, d).  dx may be null.
template <typename T, int TPR, int PIECES, bool WHOLE, bool SUMS>
__global__ void __launch_bounds__(block_of(TPR)) norm_grad_kernel(const GradRows in, int64_t n, int d,
                                                                  T *dx, float *__restrict__ partial) {
    constexpr int N = Piece<T>::N, GROUPS = block_of(TPR) / TPR;
    in.start();
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int pieces = (d + N - 1) / N;
    const float scale = 1.f / (float)d;
    float dw[SUMS ? PIECES : 1][N] = {}, db[SUMS ? PIECES : 1][N] = {};
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < n; r0 += (int64_t)gridDim.x * GROUPS) {
        const int64_t r = r0 + group;
        const bool here = GROUPS == 1 || r < n;
        const float mu = here ? in.mean[r] : 0.f, rs = here ? in.rstd[r] : 0.f;
        uint4 rx[PIECES], ry[PIECES];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int c = i * TPR + t, bytes = min(N, d - c * N) * (int)sizeof(T);
            rx[i] = ry[i] = make_uint4(0, 0, 0, 0);
            if (here && c < pieces) {
                rx[i] = load_of<WHOLE>(in.x, r, (int64_t)c * 16, bytes);
                ry[i] = load_of<WHOLE>(in.dy, r, (int64_t)c * 16, bytes);
            }
        }
        float2 sum = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int c = i * TPR + t, count = min(N, d - c * N);
            if (!here || c >= pieces) continue;
            float g[N], h[N];
            if (SUMS) {
                Piece<T>::open(rx[i], h);
                Piece<T>::open(ry[i], g);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (WHOLE || j < count) {
                        dw[i][j] += g[j] * ((h[j] - mu) * rs);
                        db[i][j] += g[j];
                    }
            }
            terms_of<T, WHOLE>(ry[i], rx[i], in.w, c, count, mu, rs, g, h);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (WHOLE || j < count) {
                    sum.x += g[j];
                    sum.y += g[j] * h[j];
                }
        }
        if (!dx) continue;
        sum = group_sum<TPR>(sum, turn);
        if (!here) continue;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int c = i * TPR + t, count = min(N, d - c * N);
            if (c >= pieces) continue;
            float g[N], h[N];
            terms_of<T, WHOLE>(ry[i], rx[i], in.w, c, count, mu, rs, g, h);
            finish_piece<T, WHOLE>(in.residual, r, c, count, rs, sum.x * scale, sum.y * scale, g, h,
                                   dx + r * d + (int64_t)c * N);
        }
    }
    if constexpr (SUMS) {
        float *out = partial + (int64_t)blockIdx.x * 2 * d;
        // the block's groups one after the other
        for (int k = 0; k < GROUPS; ++k) {
            if (k) __syncthreads();
            if (group != k) continue;
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int c = (i * TPR + t) * N + j;
                    if (c >= d) continue;
                    out[c] = (k ? out[c] : 0.f) + dw[i][j];
                    out[d + c] = (k ? out[d + c] : 0.f) + db[i][j];
                }
        }
    }
}

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kWideThreads) norm_grad_wide_kernel(const GradRows in, int64_t n, int d,
                                                                      T *dx) {
    constexpr int N = Piece<T>::N;
    in.start();
    const int pieces = (d + N - 1) / N;
    const float scale = 1.f / (float)d;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < n; r += gridDim.x) {
        const float mu = in.mean[r], rs = in.rstd[r];
        float2 sum = {0.f, 0.f};
        float g[N], h[N];
        for (int c = threadIdx.x; c < pieces; c += kWideThreads) {
            const int count = min(N, d - c * N), bytes = count * (int)sizeof(T);
            terms_of<T, WHOLE>(load_of<WHOLE>(in.dy, r, (int64_t)c * 16, bytes),
                               load_of<WHOLE>(in.x, r, (int64_t)c * 16, bytes), in.w, c, count, mu, rs, g, h);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (WHOLE || j < count) {
                    sum.x += g[j];
                    sum.y += g[j] * h[j];
                }
        }
        sum = group_sum<kWideThreads>(sum, turn);
        for (int c = threadIdx.x; c < pieces; c += kWideThreads) {
            const int count = min(N, d - c * N), bytes = count * (int)sizeof(T);
            terms_of<T, WHOLE>(load_of<WHOLE>(in.dy, r, (int64_t)c * 16, bytes),
                               load_of<WHOLE>(in.x, r, (int64_t)c * 16, bytes), in.w, c, count, mu, rs, g, h);
            finish_piece<T, WHOLE>(in.residual, r, c, count, rs, sum.x * scale, sum.y * scale, g, h,
                                   dx + r * d + (int64_t)c * N);
        }
    }
}

// dw and db of rows [blockIdx.y * rows, ..), a thread per piece of the columns.
constexpr int kColumnThreads = 128;

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kColumnThreads) norm_columns_kernel(const GradRows in, int64_t n, int d, int64_t rows,
                                                                      float *__restrict__ partial) {
    constexpr int N = Piece<T>::N;
    in.start();
    const int c = blockIdx.x * kColumnThreads + threadIdx.x;
    if (c >= (d + N - 1) / N) return;
    const int count = min(N, d - c * N), bytes = count * (int)sizeof(T);
    const int64_t r0 = blockIdx.y * rows, r1 = min(r0 + rows, n);
    float dw[N] = {}, db[N] = {};
    for (int64_t r = r0; r < r1; ++r) {
        float g[N], h[N];
        Piece<T>::open(load_of<WHOLE>(in.x, r, (int64_t)c * 16, bytes), h);
        Piece<T>::open(load_of<WHOLE>(in.dy, r, (int64_t)c * 16, bytes), g);
        const float mu = in.mean[r], rs = in.rstd[r];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            dw[j] += g[j] * ((h[j] - mu) * rs);
            db[j] += g[j];
        }
    }
    float *out = partial + (int64_t)blockIdx.y * 2 * d + (int64_t)c * N;
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < count) {
            out[j] = dw[j];
            out[d + j] = db[j];
        }
}

// The groups' sums in order: 32 columns to a block, its warps a part of the
// groups each.
constexpr int kJoinWarps = 32;

template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) norm_join_kernel(const float *__restrict__ partial, int count, int d,
                                                                    T *__restrict__ dweight, T *__restrict__ dbias) {
    __shared__ float sums[kJoinWarps][33];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T *out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    const int c = blockIdx.x * 32 + lane;
    const float *from = partial + (int64_t)blockIdx.y * d + c;
    float s = 0.f;
    if (c < d) {
#pragma unroll 4
        for (int k = warp; k < count; k += kJoinWarps) s += from[(int64_t)k * 2 * d];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) s += sums[w][lane];
    if (c < d) {
        if constexpr (sizeof(T) == 4)
            out[c] = s;
        else
            out[c] = narrow<T>(s);
    }
}

bool on16(const void *p, int64_t pitch_bytes) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && pitch_bytes % 16 == 0;
}

// Most rows of `partial`: one per block.
constexpr int64_t kMostBlocks = kSMs * 8;

template <typename F, typename... Args>
cudaError_t norm_launch(F kernel, int threads, int64_t rows_per_block, int64_t n, cudaStream_t s, Args... args) {
    const int64_t blocks = std::min((n + rows_per_block - 1) / rows_per_block, kMostBlocks);
    return launch_kernel(true, kernel, dim3((unsigned)blocks), dim3((unsigned)threads), 0, s, args...);
}

template <typename T, bool WHOLE>
cudaError_t norm_typed(const NormShape &sh, const Rows &x, const Rows &w, const Rows &b, float eps, T *y, float *mean,
                       float *rstd, cudaStream_t s) {
    const int64_t pieces = (sh.d + Piece<T>::N - 1) / Piece<T>::N;
    const int d = (int)sh.d;
#define KM_NORM(TPR, PIECES)                                                                                        \
    if (pieces <= TPR * PIECES)                                                                                     \
    return norm_launch(norm_kernel<T, TPR, PIECES, WHOLE>, block_of(TPR), block_of(TPR) / TPR, sh.n, s, x, w, b, eps, \
                       sh.n, d, y, mean, rstd)
    KM_NORM(8, 1);
    KM_NORM(32, 1);
    KM_NORM(32, 2);
    KM_NORM(32, 4);
    KM_NORM(64, 4);
    KM_NORM(128, 4);
    KM_NORM(256, 4);
    KM_NORM(512, 4);
    KM_NORM(1024, 4);
#undef KM_NORM
    return norm_launch(norm_wide_kernel<T, WHOLE>, kWideThreads, 1, sh.n, s, x, w, b, eps, sh.n, d, y, mean, rstd);
}

template <typename T, bool WHOLE>
cudaError_t norm_grad_typed(const NormShape &sh, const GradRows &in, T *dx, T *dweight, T *dbias, float *partial,
                            cudaStream_t s) {
    const int64_t pieces = (sh.d + Piece<T>::N - 1) / Piece<T>::N;
    const int d = (int)sh.d;
    const bool sums = dweight || dbias;
    cudaError_t e = cudaSuccess;
    int64_t count = 0;  // rows of partial
    bool done = false;
    if (sums) {
        const auto with = [&](auto kernel, int tpr, int per) {
            if (done || pieces > tpr * per) return;
            done = true;
            const int64_t rows = block_of(tpr) / tpr;
            count = std::min((sh.n + rows - 1) / rows, kMostBlocks);
            e = norm_launch(kernel, block_of(tpr), rows, sh.n, s, in, sh.n, d, dx, partial);
        };
        with(norm_grad_kernel<T, 8, 1, WHOLE, true>, 8, 1);
        with(norm_grad_kernel<T, 32, 1, WHOLE, true>, 32, 1);
        with(norm_grad_kernel<T, 32, 2, WHOLE, true>, 32, 2);
        with(norm_grad_kernel<T, 64, 2, WHOLE, true>, 64, 2);
        with(norm_grad_kernel<T, 128, 2, WHOLE, true>, 128, 2);
        with(norm_grad_kernel<T, 256, 2, WHOLE, true>, 256, 2);
        with(norm_grad_kernel<T, 512, 2, WHOLE, true>, 512, 2);
        with(norm_grad_kernel<T, 512, 4, WHOLE, true>, 512, 4);
    }
    if (sums && !done) {
        const int64_t strips = (pieces + kColumnThreads - 1) / kColumnThreads;
        int64_t parts = std::min(std::max(kMostBlocks / strips, (int64_t)1), sh.n);
        const int64_t rows = (sh.n + parts - 1) / parts;
        parts = (sh.n + rows - 1) / rows;
        count = parts;
        e = launch_kernel(true, norm_columns_kernel<T, WHOLE>, dim3((unsigned)strips, (unsigned)parts),
                          dim3(kColumnThreads), 0, s, in, sh.n, d, rows, partial);
    }
    // (dx may be dy itself, so what else reads dy goes first)
    if (e == cudaSuccess && dx && !done) {
        const auto with = [&](auto kernel, int tpr, int per) {
            if (done || pieces > tpr * per) return;
            done = true;
            e = norm_launch(kernel, block_of(tpr), block_of(tpr) / tpr, sh.n, s, in, sh.n, d, dx, (float *)nullptr);
        };
        with(norm_grad_kernel<T, 8, 1, WHOLE, false>, 8, 1);
        with(norm_grad_kernel<T, 32, 1, WHOLE, false>, 32, 1);
        with(norm_grad_kernel<T, 32, 2, WHOLE, false>, 32, 2);
        with(norm_grad_kernel<T, 64, 2, WHOLE, false>, 64, 2);
        with(norm_grad_kernel<T, 128, 2, WHOLE, false>, 128, 2);
        with(norm_grad_kernel<T, 256, 2, WHOLE, false>, 256, 2);
        with(norm_grad_kernel<T, 512, 2, WHOLE, false>, 512, 2);
        with(norm_grad_kernel<T, 1024, 2, WHOLE, false>, 1024, 2);
        if (!done) e = norm_launch(norm_grad_wide_kernel<T, WHOLE>, kWideThreads, 1, sh.n, s, in, sh.n, d, dx);
    }
    if (e == cudaSuccess && sums)
        e = launch_kernel(true, norm_join_kernel<T>, dim3((unsigned)((sh.d + 31) / 32), 2), dim3(32 * kJoinWarps), 0, s,
                          (const float *)partial, (int)count, d, dweight, dbias);
    return e;
}

template <typename T>
cudaError_t norm_any(const NormShape &sh, const void *x, int64_t ldx, const void *weight, const void *bias, float eps,
                     void *y, float *mean, float *rstd, cudaStream_t s) {
    const Rows rx = rows_of<T>(x, sh.n, ldx, sh.d), w = rows_of<T>(weight, 1, sh.d, sh.d),
               b = rows_of<T>(bias, 1, sh.d, sh.d);
    const int64_t row = sh.d * (int64_t)sizeof(T);
    const bool whole = on16(x, rx.pitch) && on16(y, row) && on16(weight, 0) && on16(bias, 0);
    return whole ? norm_typed<T, true>(sh, rx, w, b, eps, static_cast<T *>(y), mean, rstd, s)
                 : norm_typed<T, false>(sh, rx, w, b, eps, static_cast<T *>(y), mean, rstd, s);
}

template <typename T>
cudaError_t norm_grad_any(const NormShape &sh, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                          const float *mean, const float *rstd, const void *weight, const void *residual, int64_t ldr,
                          void *dx, void *dweight, void *dbias, uint32_t *status, float *partial, cudaStream_t s) {
    const GradRows in{rows_of<T>(dy, sh.n, lddy, sh.d), rows_of<T>(x, sh.n, ldx, sh.d),
                      rows_of<T>(weight, 1, sh.d, sh.d), rows_of<T>(residual, sh.n, ldr, sh.d), mean, rstd, status};
    const int64_t row = sh.d * (int64_t)sizeof(T);
    const bool whole = on16(dy, in.dy.pitch) && on16(x, in.x.pitch) && on16(weight, 0) &&
                       (!residual || on16(residual, in.residual.pitch)) && on16(dx, row);
    return whole ? norm_grad_typed<T, true>(sh, in, static_cast<T *>(dx), static_cast<T *>(dweight),
                                            static_cast<T *>(dbias), partial, s)
                 : norm_grad_typed<T, false>(sh, in, static_cast<T *>(dx), static_cast<T *>(dweight),
                                             static_cast<T *>(dbias), partial, s);
}

}  // namespace

NormLayout norm_layout(int64_t n, int64_t d) {
    NormLayout L{};
    L.off_partial = align_up((int64_t)sizeof(WsHeader), 1024);
    L.bytes = align_up(L.off_partial + std::min(n, kMostBlocks) * 2 * d * 4, 1024);
    return L;
}

cudaError_t launch_norm(const NormShape &sh, const void *x, int64_t ldx, const void *weight, const void *bias, float eps,
                        void *y, float *mean, float *rstd, cudaStream_t s) {
    if (sh.dtype == KMEANS_F32) return norm_any<float>(sh, x, ldx, weight, bias, eps, y, mean, rstd, s);
    return sh.dtype == KMEANS_F16 ? norm_any<__half>(sh, x, ldx, weight, bias, eps, y, mean, rstd, s)
                                  : norm_any<__nv_bfloat16>(sh, x, ldx, weight, bias, eps, y, mean, rstd, s);
}

cudaError_t launch_norm_grad(const NormShape &sh, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                             const float *mean, const float *rstd, const void *weight, const void *residual,
                             int64_t ldr, void *dx, void *dweight, void *dbias, const NormLayout &L, uint8_t *ws,
                             cudaStream_t s) {
    if (sh.n == 0 || !(dx || dweight || dbias)) {  // no kernel that clears it
        cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(WsHeader), s);  // this call's status word
        const size_t bytes = (size_t)sh.d * (sh.dtype == KMEANS_F32 ? 4 : 2);
        if (e == cudaSuccess && dweight) e = cudaMemsetAsync(dweight, 0, bytes, s);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, bytes, s);
        return e;
    }
    uint32_t *status = &reinterpret_cast<WsHeader *>(ws)->status;
    float *partial = reinterpret_cast<float *>(ws + L.off_partial);
    const auto run = [&](auto of_type) {
        return of_type(sh, dy, lddy, x, ldx, mean, rstd, weight, residual, ldr, dx, dweight, dbias, status, partial, s);
    };
    if (sh.dtype == KMEANS_F32) return run(norm_grad_any<float>);
    return sh.dtype == KMEANS_F16 ? run(norm_grad_any<__half>) : run(norm_grad_any<__nv_bfloat16>);
}

}  // namespace km
