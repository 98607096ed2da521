// Layer norm over a row's features and its gradient.
//
//   mu = mean x   v = mean (x - mu)^2   r = 1 / sqrt(v + eps)
//   y = (x - mu) r w + b
//   g = dy w, h = (x - mu) r:  dx = r (g - mean g - h mean(g h)) + residual
//   dw = sum over rows of dy h, db = sum over rows of dy
//
// A group of threads has a row and keeps it in registers as it lies in memory,
// 16-byte words of it per thread, so the row is read once: the mean, what the mean
// is off by (its sum rounds where the row lies far from zero) with the variance
// about it, and the result are three passes over registers.  Memory bounds it.
// In the gradient a thread has the same columns in every row of its group: it
// holds their weight, and adds up its share of dw and db; the groups' sums meet in
// norm_join_kernel in a fixed order.  The next row's words are asked for before
// this one's sums meet.
//
// Rows that do not all start on 16 bytes are still read and written by aligned
// words: a block takes rows that start alike (every eighth, or fewer, of a period
// of the pitch), so that its threads' words hold the same columns in every row;
// only the words at a row's ends are cut.  Tensors whose rows start differently
// from each other are read as shifted words.
//
// Rows too long for registers are read again for every pass, and dw and db get a
// kernel that goes down the columns.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "assign_common.cuh"
#include "layer.cuh"
#include "pieces.cuh"

namespace km {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// How the rows lie: all on 16 bytes; alike from tensor to tensor; anyhow.
enum class Rows16 { kWhole, kAlike, kAny };

template <typename T>
struct Word {  // 16 bytes of a row
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

// A block's rows: `first`, `first` + step, ..; their first value is value `off` of
// an aligned word.
struct Place {
    int off;
    int64_t first, step;
};

template <typename T, Rows16 ROWS>
__device__ __forceinline__ Place place_of(const Rows &x, int period) {
    if constexpr (ROWS != Rows16::kAlike) return {0, (int64_t)blockIdx.x, (int64_t)gridDim.x};
    // (the grid is a multiple of the period)
    const int cls = (int)(blockIdx.x % (unsigned)period);
    const int off = (int)((reinterpret_cast<uintptr_t>(x.base) + cls * x.pitch) & 15u) / (int)sizeof(T);
    return {off, (int64_t)blockIdx.x, (int64_t)gridDim.x};
}

// Word c of a row of d values: which of its values are the row's.
template <typename T, Rows16 ROWS>
struct Cut {
    static constexpr int N = Word<T>::N;
    int lo, hi;
    __device__ __forceinline__ Cut(int c, int off, int d) {
        lo = ROWS == Rows16::kAlike ? max(0, off - c * N) : 0;
        hi = min(N, d + off - c * N);  // 0 or less: no such word
    }
    __device__ __forceinline__ bool none() const { return hi <= 0; }
    __device__ __forceinline__ bool has(int j) const {
        return ROWS == Rows16::kWhole ? hi > 0 : (ROWS == Rows16::kAlike ? j >= lo && j < hi : j < hi);
    }
};

template <typename T, Rows16 ROWS>
__device__ __forceinline__ uint4 load_row(const Rows &m, int64_t r, int c, int off, const Cut<T, ROWS> &cut) {
    constexpr int N = Word<T>::N;
    const uint8_t *p = m.base + r * m.pitch + ((int64_t)c * N - off) * (int)sizeof(T);
    if constexpr (ROWS == Rows16::kWhole) return *reinterpret_cast<const uint4 *>(p);
    if constexpr (ROWS == Rows16::kAlike) {
        if (cut.lo == 0 && cut.hi == N) return *reinterpret_cast<const uint4 *>(p);
        return load_word(p, m.in);
    }
    return load_piece<false>(p, cut.hi * (int)sizeof(T), m.in);
}

// The same columns of a vector, 0 where there are none.
template <typename T, Rows16 ROWS>
__device__ __forceinline__ uint4 load_columns(const Rows &m, int c, int off, const Cut<T, ROWS> &cut) {
    constexpr int N = Word<T>::N;
    if constexpr (ROWS == Rows16::kWhole) return reinterpret_cast<const uint4 *>(m.base)[c];
    T v[N];
    const T *p = reinterpret_cast<const T *>(m.base) + (int64_t)c * N - off;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = cut.has(j) ? p[j] : T(0.f);
    uint4 u;
    memcpy(&u, v, 16);
    return u;
}

// p: the row's first value.
template <typename T, Rows16 ROWS>
__device__ __forceinline__ void store_row(T *p, const float (&v)[Word<T>::N], int c, int off, const Cut<T, ROWS> &cut) {
    constexpr int N = Word<T>::N;
    p += (int64_t)c * N - off;
    if constexpr (ROWS == Rows16::kAny) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < cut.hi) {
                if constexpr (sizeof(T) == 4)
                    p[j] = v[j];
                else
                    p[j] = narrow<T>(v[j]);
            }
    } else if constexpr (ROWS == Rows16::kWhole) {
        *reinterpret_cast<uint4 *>(p) = Word<T>::close(v);
    } else {
        store_word(reinterpret_cast<uint8_t *>(p), Word<T>::close(v), cut.lo * (int)sizeof(T), cut.hi * (int)sizeof(T));
    }
}

// Two sums over a group, in every thread of it: LANES lanes of a warp, or (0) the
// whole block.  `turn` counts the calls: their shared memory alternates, so that
// one barrier is enough.
template <int LANES>
__device__ __forceinline__ float2 group_sum(float2 v, int &turn) {
#pragma unroll
    for (int o = (LANES ? LANES : 32) / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(kAll, v.x, o);
        v.y += __shfl_xor_sync(kAll, v.y, o);
    }
    if constexpr (LANES == 0) {
        __shared__ float2 part[2][32];
        float2 *mine = part[turn & 1];
        ++turn;
        const int warps = blockDim.x >> 5;
        if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
        __syncthreads();
        v = mine[0];
        for (int w = 1; w < warps; ++w) {
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

// Rows of LANES lanes share blocks of 128 threads; longer rows have a block.
constexpr int kSharedBlock = 128;

// PIECES words per thread.
template <typename T, int LANES, int PIECES, Rows16 ROWS>
__global__ void __launch_bounds__(LANES ? kSharedBlock : 1024)
    norm_kernel(const Rows x, const Rows w, const Rows b, float eps, int64_t n, int d, int period, T *y, float *mean,
                float *rstd) {
    constexpr int N = Word<T>::N, GROUPS = LANES ? kSharedBlock / LANES : 1;
    griddep_wait();
    const int width = LANES ? LANES : (int)blockDim.x;
    const int t = LANES ? (int)threadIdx.x % LANES : (int)threadIdx.x, group = LANES ? (int)threadIdx.x / LANES : 0;
    const Place at = place_of<T, ROWS>(x, period);
    const float scale = 1.f / (float)d;
    // vectors off 16 bytes cost eight loads a word: once
    constexpr bool KEEP = ROWS != Rows16::kWhole;
    uint4 kw[KEEP ? PIECES : 1], kb[KEEP ? PIECES : 1];
    if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const Cut<T, ROWS> cut(i * width + t, at.off, d);
            if (cut.none()) continue;
            if (w.base) kw[i] = load_columns<T, ROWS>(w, i * width + t, at.off, cut);
            if (b.base) kb[i] = load_columns<T, ROWS>(b, i * width + t, at.off, cut);
        }
    }
    int turn = 0;
    for (int64_t q = at.first; q < n; q += at.step * GROUPS) {
        const int64_t r = q + at.step * group;
        const bool here = GROUPS == 1 || r < n;
        uint4 raw[PIECES];
        float2 sum = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const Cut<T, ROWS> cut(i * width + t, at.off, d);
            raw[i] = make_uint4(0, 0, 0, 0);
            if (here && !cut.none()) raw[i] = load_row<T, ROWS>(x, r, i * width + t, at.off, cut);
        }
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const Cut<T, ROWS> cut(i * width + t, at.off, d);
            float v[N];
            Word<T>::open(raw[i], v);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (cut.has(j)) sum.x += v[j];
        }
        const float mu = group_sum<LANES>(sum, turn).x * scale;
        sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const Cut<T, ROWS> cut(i * width + t, at.off, d);
            float v[N];
            Word<T>::open(raw[i], v);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (cut.has(j)) {
                    sum.x += v[j] - mu;
                    sum.y += (v[j] - mu) * (v[j] - mu);
                }
        }
        sum = group_sum<LANES>(sum, turn);
        const float off = sum.x * scale, rs = rsqrtf(variance_of(sum.y * scale, off) + eps);
        if (!here) continue;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int c = i * width + t;
            const Cut<T, ROWS> cut(c, at.off, d);
            if (cut.none()) continue;
            float v[N], f[N];
            Word<T>::open(raw[i], v);
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = ((v[j] - mu) - off) * rs;
            if (w.base) {
                Word<T>::open(KEEP ? kw[i] : load_columns<T, ROWS>(w, c, at.off, cut), f);
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] *= f[j];
            }
            if (b.base) {
                Word<T>::open(KEEP ? kb[i] : load_columns<T, ROWS>(b, c, at.off, cut), f);
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] += f[j];
            }
            store_row<T, ROWS>(y + r * d, v, c, at.off, cut);
        }
        if (t == 0) {
            if (mean) mean[r] = mu + off;
            if (rstd) rstd[r] = rs;
        }
    }
}

// One row after the other, read again for every pass.
constexpr int kWideThreads = 1024;

template <typename T, Rows16 ROWS>
__global__ void __launch_bounds__(kWideThreads) norm_wide_kernel(const Rows x, const Rows w, const Rows b, float eps,
                                                                 int64_t n, int d, int period, T *y, float *mean,
                                                                 float *rstd) {
    constexpr int N = Word<T>::N;
    griddep_wait();
    const Place at = place_of<T, ROWS>(x, period);
    const float scale = 1.f / (float)d;
    const int words = (d + at.off + N - 1) / N;
    int turn = 0;
    for (int64_t r = at.first; r < n; r += at.step) {
        float2 sum = {0.f, 0.f};
        float v[N], f[N];
        for (int c = threadIdx.x; c < words; c += kWideThreads) {
            const Cut<T, ROWS> cut(c, at.off, d);
            Word<T>::open(load_row<T, ROWS>(x, r, c, at.off, cut), v);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (cut.has(j)) sum.x += v[j];
        }
        const float mu = group_sum<0>(sum, turn).x * scale;
        sum = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < words; c += kWideThreads) {
            const Cut<T, ROWS> cut(c, at.off, d);
            Word<T>::open(load_row<T, ROWS>(x, r, c, at.off, cut), v);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (cut.has(j)) {
                    sum.x += v[j] - mu;
                    sum.y += (v[j] - mu) * (v[j] - mu);
                }
        }
        sum = group_sum<0>(sum, turn);
        const float off = sum.x * scale, rs = rsqrtf(variance_of(sum.y * scale, off) + eps);
        for (int c = threadIdx.x; c < words; c += kWideThreads) {
            const Cut<T, ROWS> cut(c, at.off, d);
            Word<T>::open(load_row<T, ROWS>(x, r, c, at.off, cut), v);
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = ((v[j] - mu) - off) * rs;
            if (w.base) {
                Word<T>::open(load_columns<T, ROWS>(w, c, at.off, cut), f);
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] *= f[j];
            }
            if (b.base) {
                Word<T>::open(load_columns<T, ROWS>(b, c, at.off, cut), f);
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] += f[j];
            }
            store_row<T, ROWS>(y + r * d, v, c, at.off, cut);
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

// dx of a word from its dy and x.
template <typename T>
__device__ __forceinline__ void finish_word(const uint4 &dy, const uint4 &x, const uint4 &w, bool weighted,
                                            const uint4 &residual, bool add, float mu, float rs, float mg, float mgh,
                                            float (&v)[Word<T>::N]) {
    constexpr int N = Word<T>::N;
    float h[N], f[N];
    Word<T>::open(dy, v);
    Word<T>::open(x, h);
    if (weighted) {
        Word<T>::open(w, f);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] *= f[j];
    }
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = rs * (v[j] - mg - (h[j] - mu) * rs * mgh);
    if (add) {
        Word<T>::open(residual, f);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] += f[j];
    }
}

// SUMS: the block's part of dw and db to row `blockIdx.x` of `partial`, (blocks, 2,
// d).  dx may be null.  With up to two words per thread the next row's are asked
// for ahead.
template <typename T, int LANES, int PIECES, Rows16 ROWS, bool SUMS>
__global__ void __launch_bounds__(LANES ? kSharedBlock : 512)
    norm_grad_kernel(const GradRows in, int64_t n, int d, int period, T *dx, float *__restrict__ partial) {
    constexpr int N = Word<T>::N, GROUPS = LANES ? kSharedBlock / LANES : 1;
    constexpr bool AHEAD = PIECES <= 2;
    in.start();
    const int width = LANES ? LANES : (int)blockDim.x;
    const int t = LANES ? (int)threadIdx.x % LANES : (int)threadIdx.x, group = LANES ? (int)threadIdx.x / LANES : 0;
    const Place at = place_of<T, ROWS>(in.x, period);
    const float scale = 1.f / (float)d;
    float dw[SUMS ? PIECES : 1][N] = {}, db[SUMS ? PIECES : 1][N] = {};
    uint4 kw[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const Cut<T, ROWS> cut(i * width + t, at.off, d);
        kw[i] = make_uint4(0, 0, 0, 0);
        if (in.w.base && !cut.none()) kw[i] = load_columns<T, ROWS>(in.w, i * width + t, at.off, cut);
    }
    struct Row {
        uint4 x[PIECES], dy[PIECES], residual[PIECES];
        float mu, rs;
    };
    const auto load = [&](int64_t r, Row &row) {
        const bool here = r < n;
        row.mu = here ? in.mean[r] : 0.f;
        row.rs = here ? in.rstd[r] : 0.f;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int c = i * width + t;
            const Cut<T, ROWS> cut(c, at.off, d);
            row.x[i] = row.dy[i] = row.residual[i] = make_uint4(0, 0, 0, 0);
            if (!here || cut.none()) continue;
            row.x[i] = load_row<T, ROWS>(in.x, r, c, at.off, cut);
            row.dy[i] = load_row<T, ROWS>(in.dy, r, c, at.off, cut);
            if (in.residual.base && dx) row.residual[i] = load_row<T, ROWS>(in.residual, r, c, at.off, cut);
        }
    };
    int turn = 0;
    Row row, next;
    if (AHEAD) load(at.first + at.step * group, next);
    for (int64_t q = at.first; q < n; q += at.step * GROUPS) {
        const int64_t r = q + at.step * group;
        if (AHEAD) {
            row = next;
            load(r + at.step * GROUPS, next);
        } else {
            load(r, row);
        }
        float2 sum = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const Cut<T, ROWS> cut(i * width + t, at.off, d);
            float g[N], h[N], f[N];
            Word<T>::open(row.x[i], h);
            Word<T>::open(row.dy[i], g);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                h[j] = (h[j] - row.mu) * row.rs;
                if (ROWS != Rows16::kWhole && !cut.has(j)) g[j] = h[j] = 0.f;
                if (SUMS) {  // (rows and words that do not exist have dy = 0 and rs = 0)
                    dw[i][j] += g[j] * h[j];
                    db[i][j] += g[j];
                }
            }
            if (in.w.base) {
                Word<T>::open(kw[i], f);
#pragma unroll
                for (int j = 0; j < N; ++j) g[j] *= f[j];
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                sum.x += g[j];
                sum.y += g[j] * h[j];
            }
        }
        if (!dx) continue;
        sum = group_sum<LANES>(sum, turn);
        if (r >= n) continue;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int c = i * width + t;
            const Cut<T, ROWS> cut(c, at.off, d);
            if (cut.none()) continue;
            float v[N];
            finish_word<T>(row.dy[i], row.x[i], kw[i], in.w.base, row.residual[i], in.residual.base, row.mu, row.rs,
                           sum.x * scale, sum.y * scale, v);
            store_row<T, ROWS>(dx + r * d, v, c, at.off, cut);
        }
    }
    if constexpr (SUMS) {
        float *out = partial + (int64_t)blockIdx.x * 2 * d;
        // the block's groups one after the other
        for (int k = 0; k < GROUPS; ++k) {
            if (k) __syncthreads();
            if (group != k) continue;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const Cut<T, ROWS> cut(i * width + t, at.off, d);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int c = (i * width + t) * N + j - at.off;
                    if (ROWS == Rows16::kWhole ? cut.none() : !cut.has(j)) continue;
                    out[c] = (k ? out[c] : 0.f) + dw[i][j];
                    out[d + c] = (k ? out[d + c] : 0.f) + db[i][j];
                }
            }
        }
    }
}

template <typename T, Rows16 ROWS>
__global__ void __launch_bounds__(kWideThreads) norm_grad_wide_kernel(const GradRows in, int64_t n, int d, int period,
                                                                      T *dx) {
    constexpr int N = Word<T>::N;
    in.start();
    const Place at = place_of<T, ROWS>(in.x, period);
    const float scale = 1.f / (float)d;
    const int words = (d + at.off + N - 1) / N;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    int turn = 0;
    for (int64_t r = at.first; r < n; r += at.step) {
        const float mu = in.mean[r], rs = in.rstd[r];
        float2 sum = {0.f, 0.f};
        for (int c = threadIdx.x; c < words; c += kWideThreads) {
            const Cut<T, ROWS> cut(c, at.off, d);
            float g[N], h[N], f[N];
            Word<T>::open(load_row<T, ROWS>(in.dy, r, c, at.off, cut), g);
            Word<T>::open(load_row<T, ROWS>(in.x, r, c, at.off, cut), h);
            if (in.w.base) {
                Word<T>::open(load_columns<T, ROWS>(in.w, c, at.off, cut), f);
#pragma unroll
                for (int j = 0; j < N; ++j) g[j] *= f[j];
            }
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (cut.has(j)) {
                    sum.x += g[j];
                    sum.y += g[j] * ((h[j] - mu) * rs);
                }
        }
        sum = group_sum<0>(sum, turn);
        for (int c = threadIdx.x; c < words; c += kWideThreads) {
            const Cut<T, ROWS> cut(c, at.off, d);
            float v[N];
            finish_word<T>(load_row<T, ROWS>(in.dy, r, c, at.off, cut), load_row<T, ROWS>(in.x, r, c, at.off, cut),
                           in.w.base ? load_columns<T, ROWS>(in.w, c, at.off, cut) : zero, in.w.base,
                           in.residual.base ? load_row<T, ROWS>(in.residual, r, c, at.off, cut) : zero, in.residual.base,
                           mu, rs, sum.x * scale, sum.y * scale, v);
            store_row<T, ROWS>(dx + r * d, v, c, at.off, cut);
        }
    }
}

// dw and db of a share of the rows, a thread per word of the columns.
constexpr int kColumnThreads = 128;

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kColumnThreads) norm_columns_kernel(const GradRows in, int64_t n, int d, int64_t rows,
                                                                      float *__restrict__ partial) {
    constexpr Rows16 ROWS = WHOLE ? Rows16::kWhole : Rows16::kAny;
    constexpr int N = Word<T>::N;
    in.start();
    const int c = blockIdx.x * kColumnThreads + threadIdx.x;
    const Cut<T, ROWS> cut(c, 0, d);
    if (cut.none()) return;
    const int64_t r0 = blockIdx.y * rows, r1 = min(r0 + rows, n);
    float dw[N] = {}, db[N] = {};
#pragma unroll 2
    for (int64_t r = r0; r < r1; ++r) {
        float g[N], h[N];
        Word<T>::open(load_row<T, ROWS>(in.x, r, c, 0, cut), h);
        Word<T>::open(load_row<T, ROWS>(in.dy, r, c, 0, cut), g);
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
        if (cut.has(j)) {
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
#pragma unroll 8
        for (int k = warp; k < count; k += kJoinWarps) s += from[(int64_t)k * 2 * d];
    }
    sums[warp][lane] = s;
    __syncthreads();
    // warp w: column w, whose sums its lanes add up
    s = sums[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    if (lane == 0 && blockIdx.x * 32 + warp < d) {
        if constexpr (sizeof(T) == 4)
            out[blockIdx.x * 32 + warp] = s;
        else
            out[blockIdx.x * 32 + warp] = narrow<T>(s);
    }
}

// Rows of `partial` there can be: one per block.
constexpr int64_t kMostBlocks = kSMs * 8;

// Rows that start alike: how many until one starts like the first.
int period_of(int64_t pitch_bytes) {
    int period = 1;
    while ((period * pitch_bytes) % 16 != 0) ++period;
    return period;
}

struct Alignment {
    Rows16 rows;
    int period;
};

// Of the rows of several tensors (null: not there), the pitch in bytes of each.
Alignment alignment_of(int64_t n, std::initializer_list<std::pair<const void *, int64_t>> all,
                       std::initializer_list<const void *> vectors) {
    bool whole = true, alike = true;
    const void *first = nullptr;
    int64_t pitch = 0;
    for (const auto &m : all) {
        if (!m.first) continue;
        const int64_t own = n > 1 ? m.second : 0;
        if (!first) {
            first = m.first;
            pitch = own;
        }
        const uintptr_t a = reinterpret_cast<uintptr_t>(m.first), b = reinterpret_cast<uintptr_t>(first);
        whole = whole && (a & 15u) == 0 && m.second % 16 == 0;
        alike = alike && ((a ^ b) & 15u) == 0 && (own - pitch) % 16 == 0;
    }
    for (const void *v : vectors) whole = whole && (reinterpret_cast<uintptr_t>(v) & 15u) == 0;
    if (whole) return {Rows16::kWhole, 1};
    return alike ? Alignment{Rows16::kAlike, period_of(pitch)} : Alignment{Rows16::kAny, 1};
}

// Blocks for so many, a multiple of the period (of at most 8) that is no more than
// `most` (a multiple of 8), and covers every class of rows there is.
unsigned blocks_of(int64_t wanted, int64_t most, int period) {
    return (unsigned)std::min(align_up(std::max(wanted, (int64_t)1), period), most);
}

// A thread block for rows of so many words.
int threads_of(int64_t words, int pieces) { return (int)align_up((words + pieces - 1) / pieces, 32); }

template <typename T, Rows16 ROWS>
cudaError_t norm_typed(const NormShape &sh, const Rows &x, const Rows &w, const Rows &b, float eps, int period, T *y,
                       float *mean, float *rstd, cudaStream_t s) {
    constexpr int N = Word<T>::N;
    const int64_t words = (sh.d + N - 1) / N + (ROWS == Rows16::kAlike ? 1 : 0);
    const int d = (int)sh.d;
    const auto run = [&](auto kernel, int threads, int64_t rows) {
        const int64_t most = kSMs * std::max(1, std::min(16, 2048 / threads));
        return launch_kernel(true, kernel, dim3(blocks_of((sh.n + rows - 1) / rows, align_up(most, 8), period)),
                             dim3((unsigned)threads), 0, s, x, w, b, eps, sh.n, d, period, y, mean, rstd);
    };
    if (words <= 8) return run(norm_kernel<T, 8, 1, ROWS>, kSharedBlock, kSharedBlock / 8);
    if (words <= 32) return run(norm_kernel<T, 32, 1, ROWS>, kSharedBlock, kSharedBlock / 32);
    if (words <= 64) return run(norm_kernel<T, 32, 2, ROWS>, kSharedBlock, kSharedBlock / 32);
    if (words <= 128) return run(norm_kernel<T, 32, 4, ROWS>, kSharedBlock, kSharedBlock / 32);
    if (words <= 4096) return run(norm_kernel<T, 0, 4, ROWS>, threads_of(words, 4), 1);
    return run(norm_wide_kernel<T, ROWS>, kWideThreads, 1);
}

template <typename T, Rows16 ROWS>
cudaError_t norm_grad_typed(const NormShape &sh, const GradRows &in, int period, T *dx, T *dweight, T *dbias,
                            float *partial, cudaStream_t s) {
    constexpr int N = Word<T>::N;
    const int64_t words = (sh.d + N - 1) / N + (ROWS == Rows16::kAlike ? 1 : 0);
    const int d = (int)sh.d;
    const bool sums = dweight || dbias;
    cudaError_t e = cudaSuccess;
    int64_t count = 0;  // rows of partial
    // about 512 threads per SM, which the words they ask for ahead keep busy
    const auto run = [&](auto kernel, int threads, int64_t rows) {
        const int64_t most = kSMs * std::max(1, std::min(8, 640 / threads));
        count = blocks_of((sh.n + rows - 1) / rows, most, period);
        return launch_kernel(true, kernel, dim3((unsigned)count), dim3((unsigned)threads), 0, s, in, sh.n, d, period, dx,
                             partial);
    };
    const auto rows = [&](auto with_sums) {
        constexpr bool SUMS = decltype(with_sums)::value;
        if (words <= 8) return run(norm_grad_kernel<T, 8, 1, ROWS, SUMS>, kSharedBlock, kSharedBlock / 8);
        if (words <= 32) return run(norm_grad_kernel<T, 32, 1, ROWS, SUMS>, kSharedBlock, kSharedBlock / 32);
        if (words <= 256) return run(norm_grad_kernel<T, 0, 1, ROWS, SUMS>, threads_of(words, 1), 1);
        if (words <= 1024) return run(norm_grad_kernel<T, 0, 2, ROWS, SUMS>, threads_of(words, 2), 1);
        return run(norm_grad_kernel<T, 0, 4, ROWS, SUMS>, threads_of(words, 4), 1);
    };
    const bool fits = words <= 2048;
    if (fits) {
        e = sums ? rows(std::true_type{}) : rows(std::false_type{});
    } else {
        if (sums) {
            const int64_t strips = ((sh.d + N - 1) / N + kColumnThreads - 1) / kColumnThreads;
            int64_t parts = std::min(std::max(kMostBlocks / strips, (int64_t)1), sh.n);
            const int64_t share = (sh.n + parts - 1) / parts;
            parts = (sh.n + share - 1) / share;
            e = launch_kernel(true, norm_columns_kernel<T, ROWS == Rows16::kWhole>, dim3((unsigned)strips, (unsigned)parts),
                              dim3(kColumnThreads), 0, s, in, sh.n, d, share, partial);
            count = parts;
        }
        // (dx may be dy itself, so what else reads dy goes first)
        if (e == cudaSuccess && dx)
            e = launch_kernel(true, norm_grad_wide_kernel<T, ROWS>, dim3(blocks_of(sh.n, kSMs * 2, period)),
                              dim3(kWideThreads), 0, s, in, sh.n, d, period, dx);
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
    const Alignment a = alignment_of(sh.n, {{x, rx.pitch}, {y, sh.d * (int64_t)sizeof(T)}}, {weight, bias});
    const auto run = [&](auto typed) { return typed(sh, rx, w, b, eps, a.period, static_cast<T *>(y), mean, rstd, s); };
    if (a.rows == Rows16::kWhole) return run(norm_typed<T, Rows16::kWhole>);
    return a.rows == Rows16::kAlike ? run(norm_typed<T, Rows16::kAlike>) : run(norm_typed<T, Rows16::kAny>);
}

template <typename T>
cudaError_t norm_grad_any(const NormShape &sh, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                          const float *mean, const float *rstd, const void *weight, const void *residual, int64_t ldr,
                          void *dx, void *dweight, void *dbias, uint32_t *status, float *partial, cudaStream_t s) {
    const GradRows in{rows_of<T>(dy, sh.n, lddy, sh.d), rows_of<T>(x, sh.n, ldx, sh.d),
                      rows_of<T>(weight, 1, sh.d, sh.d), rows_of<T>(residual, sh.n, ldr, sh.d), mean, rstd, status};
    const Alignment a = alignment_of(sh.n, {{x, in.x.pitch}, {dy, in.dy.pitch}, {residual, in.residual.pitch},
                                            {dx, sh.d * (int64_t)sizeof(T)}}, {weight});
    const auto run = [&](auto typed) {
        return typed(sh, in, a.period, static_cast<T *>(dx), static_cast<T *>(dweight), static_cast<T *>(dbias), partial, s);
    };
    if (a.rows == Rows16::kWhole && sh.d % Word<T>::N == 0) return run(norm_grad_typed<T, Rows16::kWhole>);
    return a.rows != Rows16::kAny ? run(norm_grad_typed<T, Rows16::kAlike>) : run(norm_grad_typed<T, Rows16::kAny>);
}

}  // namespace

NormLayout norm_layout(int64_t n, int64_t d) {
    NormLayout L{};
    L.off_partial = align_up((int64_t)sizeof(WsHeader), 1024);
    L.bytes = align_up(L.off_partial + std::min(align_up(n, 8), kMostBlocks) * 2 * d * 4, 1024);
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
