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
// kExact: all on 16 bytes, and every thread has all the words it has room for;
// nothing is then asked about a word (with such questions 16384 x 4096 bfloat16
// took 53 us forward instead of 45, and the gradient with dw and db 107: they
// became selections of every value and every sum).
enum class Rows16 { kExact, kWhole, kAlike, kAny };
__host__ __device__ constexpr bool whole_rows(Rows16 r) { return r == Rows16::kExact || r == Rows16::kWhole; }

// 16 bytes of a row, as pairs: the arithmetic goes by two values an instruction,
// since some twenty per value would keep the SMs busier than the memory.
template <typename T>
struct Word {
    static constexpr int N = 16 / (int)sizeof(T), PAIRS = N / 2;
    __device__ __forceinline__ static void open(const uint4 &u, float2 (&v)[PAIRS]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) v[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = widen2<T>(w[i]);
        }
    }
    __device__ __forceinline__ static uint4 close(const float2 (&v)[PAIRS]) {
        if constexpr (sizeof(T) == 4)
            return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                              __float_as_uint(v[1].y));
        else
            return make_uint4(narrow2<T>(v[0].x, v[0].y), narrow2<T>(v[1].x, v[1].y), narrow2<T>(v[2].x, v[2].y),
                              narrow2<T>(v[3].x, v[3].y));
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
    __device__ __forceinline__ bool whole() const { return whole_rows(ROWS) || (lo == 0 && hi == N); }
    __device__ __forceinline__ bool has(int j) const { return j >= lo && j < hi; }
};

// What is not the row's of a word, as zero.
template <typename T, Rows16 ROWS>
__device__ __forceinline__ uint4 masked(const uint4 &w, const Cut<T, ROWS> &cut) {
    const int lo = cut.lo * (int)sizeof(T), hi = cut.hi * (int)sizeof(T);
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (4 * i < lo || 4 * i + 2 > hi) u[i] &= 0xffff0000u;
        if (4 * i + 2 < lo || 4 * i + 4 > hi) u[i] &= 0xffffu;
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// (a row's end shares its aligned word with its neighbour, or with nothing)
__device__ __forceinline__ bool in_tensor(const uint8_t *p, const Span &in) { return p >= in.lo && p + 16 <= in.hi; }

// A word of row r; what is not the row's reads as zero.
template <typename T, Rows16 ROWS>
__device__ __forceinline__ uint4 load_row(const Rows &m, int64_t r, int c, int off, const Cut<T, ROWS> &cut) {
    constexpr int N = Word<T>::N;
    const uint8_t *p = m.base + r * m.pitch + ((int64_t)c * N - off) * (int)sizeof(T);
    if constexpr (ROWS == Rows16::kAny) return load_piece<false>(p, cut.hi * (int)sizeof(T), m.in);
    if (cut.whole()) return *reinterpret_cast<const uint4 *>(p);
    return masked<T, ROWS>(in_tensor(p, m.in) ? *reinterpret_cast<const uint4 *>(p) : load_word(p, m.in), cut);
}

// The same columns of a vector, 0 where there are none.
template <typename T, Rows16 ROWS>
__device__ __forceinline__ uint4 load_columns(const Rows &m, int c, int off, const Cut<T, ROWS> &cut) {
    constexpr int N = Word<T>::N;
    if constexpr (whole_rows(ROWS)) return reinterpret_cast<const uint4 *>(m.base)[c];
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
__device__ __forceinline__ void store_row(T *p, const float2 (&v)[Word<T>::PAIRS], int c, int off, const Cut<T, ROWS> &cut) {
    constexpr int N = Word<T>::N;
    p += (int64_t)c * N - off;
    if constexpr (ROWS == Rows16::kAny) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < cut.hi) {
                const float one = j & 1 ? v[j / 2].y : v[j / 2].x;
                if constexpr (sizeof(T) == 4)
                    p[j] = one;
                else
                    p[j] = narrow<T>(one);
            }
    } else if constexpr (whole_rows(ROWS)) {
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
        if (warps > 4 && threadIdx.x >= (unsigned)warps && threadIdx.x < 32u) mine[threadIdx.x] = make_float2(0.f, 0.f);
        __syncthreads();
        if (warps <= 4) {
            v = mine[0];
            for (int w = 1; w < warps; ++w) v = __fadd2_rn(v, mine[w]);
        } else {
            v = mine[threadIdx.x & 31];  // zeros past the last warp's
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                v.x += __shfl_xor_sync(kAll, v.x, o);
                v.y += __shfl_xor_sync(kAll, v.y, o);
            }
        }
    }
    return v;
}

// (where all values are equal the difference may fall below zero by a rounding)
__device__ __forceinline__ float variance_of(float square, float off) {
    const float v = square - off * off;
    return v < 0.f ? 0.f : v;
}

// The sum of a word's values.
template <typename T>
__device__ __forceinline__ float2 add_word(const uint4 &raw, float2 sum) {
    float2 v[Word<T>::PAIRS];
    Word<T>::open(raw, v);
#pragma unroll
    for (int j = 0; j < Word<T>::PAIRS; ++j) sum = __fadd2_rn(sum, v[j]);
    return sum;
}

// The words of a row that a thread has: c0, c0 + width, .., `count` of them; a bit
// in `cut` for each that the row does not fill (or that does not lie on 16 bytes).
template <typename T, int PIECES, Rows16 ROWS>
struct Mine {
    int c0, width, count = 0;
    uint32_t cut = 0;
    __device__ __forceinline__ Mine(int t, int width_, int off, int d) : c0(t), width(width_) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const Cut<T, ROWS> one(c0 + i * width, off, d);
            if (!one.none()) count = i + 1;  // (their words are in a row)
            if (ROWS == Rows16::kAny || !one.whole()) cut |= 1u << i;
        }
    }
    __device__ __forceinline__ bool has(int i) const { return ROWS == Rows16::kExact || i < count; }
    __device__ __forceinline__ bool whole(int i) const { return whole_rows(ROWS) || !(cut >> i & 1u); }
    // from one word to the next, in bytes
    __device__ __forceinline__ int stride() const { return width * 16; }
};

// v - mu in place, and the sums of it and of its square.
template <typename T, Rows16 ROWS>
__device__ __forceinline__ void spread(float2 (&v)[Word<T>::PAIRS], bool whole, int c, int off, int d, float mu,
                                       float2 &first, float2 &second) {
#pragma unroll
    for (int j = 0; j < Word<T>::PAIRS; ++j) v[j] = __fadd2_rn(v[j], both(-mu));
    if (!whole) {
        const Cut<T, ROWS> cut(c, off, d);
#pragma unroll
        for (int j = 0; j < Word<T>::PAIRS; ++j) {
            if (!cut.has(2 * j)) v[j].x = 0.f;
            if (!cut.has(2 * j + 1)) v[j].y = 0.f;
        }
    }
#pragma unroll
    for (int j = 0; j < Word<T>::PAIRS; ++j) {
        first = __fadd2_rn(first, v[j]);
        second = __ffma2_rn(v[j], v[j], second);
    }
}

// (v - off) rs w + b of v, the values without their mean so far.
template <typename T>
__device__ __forceinline__ void normalise(float2 (&v)[Word<T>::PAIRS], float off, float rs, bool weighted, const uint4 &w,
                                          bool biased, const uint4 &b) {
    float2 f[Word<T>::PAIRS];
#pragma unroll
    for (int j = 0; j < Word<T>::PAIRS; ++j) v[j] = __fmul2_rn(__fadd2_rn(v[j], both(-off)), both(rs));
    if (weighted) {
        Word<T>::open(w, f);
#pragma unroll
        for (int j = 0; j < Word<T>::PAIRS; ++j) v[j] = __fmul2_rn(v[j], f[j]);
    }
    if (biased) {
        Word<T>::open(b, f);
#pragma unroll
        for (int j = 0; j < Word<T>::PAIRS; ++j) v[j] = __fadd2_rn(v[j], f[j]);
    }
}

// Rows of LANES lanes share blocks of 128 threads; longer rows have a block.
constexpr int kSharedBlock = 128;

// Copies into shared memory that the thread does not wait for.
__device__ __forceinline__ void copy16(uint4 *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Rows on their way or worked on at a time.  (Four words a thread fill shared memory
// with two.)
__host__ __device__ constexpr int stages_of(int pieces) { return pieces == 4 ? 2 : 4; }

// What a thread has of a row: PIECES words of up to three tensors in shared memory,
// in places of its own, so that nobody waits for anybody else's copies.
template <typename T, int PIECES, Rows16 ROWS>
struct Fetch {
    const Mine<T, PIECES, ROWS> &mine;
    int off, d;
    int64_t start;  // of the thread's first word from the row's first value on, in bytes
    __device__ __forceinline__ void operator()(const Rows &m, int64_t r, uint4 *to) const {
        const uint8_t *p = m.base + r * m.pitch + start;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            if (!mine.has(i)) continue;
            uint4 *at = to + i * (int)blockDim.x;
            if (mine.whole(i) || (ROWS == Rows16::kAlike && in_tensor(p + i * mine.stride(), m.in)))
                copy16(at, p + i * mine.stride());
            else
                *at = load_row<T, ROWS>(m, r, mine.c0 + i * mine.width, off, Cut<T, ROWS>(mine.c0 + i * mine.width, off, d));
        }
    }
    __device__ __forceinline__ uint4 read(const uint4 *from, int i) const {
        const uint4 u = from[i * (int)blockDim.x];
        if (ROWS != Rows16::kAlike || mine.whole(i)) return u;
        return masked<T, ROWS>(u, Cut<T, ROWS>(mine.c0 + i * mine.width, off, d));
    }
};

// A vector's columns of a thread: opened for good up to sixteen values a thread,
// which takes a third off the instructions per value, and as they are above.
template <typename T, int PIECES, Rows16 ROWS>
struct Columns {
    static constexpr bool HOLD = PIECES * Word<T>::N <= 16;
    static constexpr int PAIRS = Word<T>::PAIRS;
    uint4 raw[HOLD ? 1 : PIECES];
    float2 open[HOLD ? PIECES : 1][PAIRS];
    bool there;
    __device__ __forceinline__ Columns(const Rows &v, const Mine<T, PIECES, ROWS> &mine, int off, int d) : there(v.base) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int c = mine.c0 + i * mine.width;
            const Cut<T, ROWS> cut(c, off, d);
            const uint4 u = there && !cut.none() ? load_columns<T, ROWS>(v, c, off, cut) : make_uint4(0, 0, 0, 0);
            if constexpr (HOLD)
                Word<T>::open(u, open[i]);
            else
                raw[i] = u;
        }
    }
    __device__ __forceinline__ void get(int i, float2 (&f)[PAIRS]) const {
        if constexpr (HOLD) {
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) f[j] = open[i][j];
        } else {
            Word<T>::open(raw[i], f);
        }
    }
    __device__ __forceinline__ void multiply(int i, float2 (&v)[PAIRS]) const {
        if (!there) return;
        float2 f[PAIRS];
        get(i, f);
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) v[j] = __fmul2_rn(v[j], f[j]);
    }
    __device__ __forceinline__ void add(int i, float2 (&v)[PAIRS]) const {
        if (!there) return;
        float2 f[PAIRS];
        get(i, f);
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) v[j] = __fadd2_rn(v[j], f[j]);
    }
};

template <typename T, int LANES, int PIECES, Rows16 ROWS>
__global__ void __launch_bounds__(LANES ? kSharedBlock : PIECES == 2 ? 256 : 512, LANES ? 5 : PIECES == 2 ? 2 : 1)
    norm_kernel(const Rows x, const Rows w, const Rows b, float eps, int64_t n, int d, int period, T *y, float *mean,
                float *rstd) {
    extern __shared__ uint4 ring[];
    constexpr int GROUPS = LANES ? kSharedBlock / LANES : 1, PAIRS = Word<T>::PAIRS, N = Word<T>::N;
    constexpr int STAGES = stages_of(PIECES);
    griddep_wait();
    const int width = LANES ? LANES : (int)blockDim.x;
    const int t = LANES ? (int)threadIdx.x % LANES : (int)threadIdx.x, group = LANES ? (int)threadIdx.x / LANES : 0;
    const Place at = place_of<T, ROWS>(x, period);
    const Mine<T, PIECES, ROWS> mine(t, width, at.off, d);
    const float scale = 1.f / (float)d;
    const Fetch<T, PIECES, ROWS> fetch{mine, at.off, d, ((int64_t)t * N - at.off) * (int)sizeof(T)};
    const int stage_words = PIECES * (int)blockDim.x;
    uint4 *own = ring + threadIdx.x;
    const int64_t step = at.step * GROUPS, first = at.first + at.step * group;
    const auto issue = [&](int64_t r, int stage) {
        if (r < n) fetch(x, r, own + stage * stage_words);
        copy_commit();
    };
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) issue(first + k * step, k);
    const Columns<T, PIECES, ROWS> weight(w, mine, at.off, d), bias(b, mine, at.off, d);
    int turn = 0, stage = 0;
    for (int64_t q = at.first; q < n; q += step) {
        const int64_t r = q + at.step * group;
        const bool here = GROUPS == 1 || r < n;
        // (into the stage that the last row has left)
        issue(r + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
        copy_wait<STAGES - 1>();
        const uint4 *from = own + stage * stage_words;
        float2 v[PIECES][PAIRS], sum = {0.f, 0.f}, second = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const uint4 u = here && mine.has(i) ? fetch.read(from, i) : make_uint4(0, 0, 0, 0);
            Word<T>::open(u, v[i]);
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) sum = __fadd2_rn(sum, v[i][j]);
        }
        const float mu = group_sum<LANES>(make_float2(sum.x + sum.y, 0.f), turn).x * scale;
        sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            if (mine.has(i)) spread<T, ROWS>(v[i], mine.whole(i), i * width + t, at.off, d, mu, sum, second);
        sum = group_sum<LANES>(make_float2(sum.x + sum.y, second.x + second.y), turn);
        const float off = sum.x * scale, rs = rsqrtf(variance_of(sum.y * scale, off) + eps);
        if (here) {
            uint8_t *out = reinterpret_cast<uint8_t *>(y + r * d) + fetch.start;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                if (!mine.has(i)) continue;
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) v[i][j] = __fmul2_rn(__fadd2_rn(v[i][j], both(-off)), both(rs));
                weight.multiply(i, v[i]);
                bias.add(i, v[i]);
                if (mine.whole(i))
                    *reinterpret_cast<uint4 *>(out + i * mine.stride()) = Word<T>::close(v[i]);
                else
                    store_row<T, ROWS>(y + r * d, v[i], i * width + t, at.off, Cut<T, ROWS>(i * width + t, at.off, d));
            }
            if (t == 0) {
                if (mean) mean[r] = mu + off;
                if (rstd) rstd[r] = rs;
            }
        }
        stage = stage == STAGES - 1 ? 0 : stage + 1;
    }
    copy_wait<0>();
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
    const uint4 zero = make_uint4(0, 0, 0, 0);
    int turn = 0;
    for (int64_t r = at.first; r < n; r += at.step) {
        float2 sum = {0.f, 0.f}, second = {0.f, 0.f};
#pragma unroll 4
        for (int c = threadIdx.x; c < words; c += kWideThreads) {
            const Cut<T, ROWS> cut(c, at.off, d);
            sum = add_word<T>(load_row<T, ROWS>(x, r, c, at.off, cut), sum);
        }
        const float mu = group_sum<0>(make_float2(sum.x + sum.y, 0.f), turn).x * scale;
        sum = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int c = threadIdx.x; c < words; c += kWideThreads) {
            const Cut<T, ROWS> cut(c, at.off, d);
            float2 v[Word<T>::PAIRS];
            Word<T>::open(load_row<T, ROWS>(x, r, c, at.off, cut), v);
            spread<T, ROWS>(v, cut.whole(), c, at.off, d, mu, sum, second);
        }
        sum = group_sum<0>(make_float2(sum.x + sum.y, second.x + second.y), turn);
        const float off = sum.x * scale, rs = rsqrtf(variance_of(sum.y * scale, off) + eps);
#pragma unroll 2
        for (int c = threadIdx.x; c < words; c += kWideThreads) {
            const Cut<T, ROWS> cut(c, at.off, d);
            float2 v[Word<T>::PAIRS];
            Word<T>::open(load_row<T, ROWS>(x, r, c, at.off, cut), v);
#pragma unroll
            for (int j = 0; j < Word<T>::PAIRS; ++j) v[j] = __fadd2_rn(v[j], both(-mu));
            normalise<T>(v, off, rs, w.base, w.base ? load_columns<T, ROWS>(w, c, at.off, cut) : zero, b.base,
                         b.base ? load_columns<T, ROWS>(b, c, at.off, cut) : zero);
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

// g = dy w and h = (x - mu) rs of a word.
template <typename T>
__device__ __forceinline__ void terms_of(const uint4 &dy, const uint4 &x, float mu, float rs, float2 (&g)[Word<T>::PAIRS],
                                         float2 (&h)[Word<T>::PAIRS]) {
    Word<T>::open(dy, g);
    Word<T>::open(x, h);
#pragma unroll
    for (int j = 0; j < Word<T>::PAIRS; ++j) h[j] = __fmul2_rn(__fadd2_rn(h[j], both(-mu)), both(rs));
}

template <typename T>
__device__ __forceinline__ void weight_word(bool weighted, const uint4 &w, float2 (&g)[Word<T>::PAIRS]) {
    if (!weighted) return;
    float2 f[Word<T>::PAIRS];
    Word<T>::open(w, f);
#pragma unroll
    for (int j = 0; j < Word<T>::PAIRS; ++j) g[j] = __fmul2_rn(g[j], f[j]);
}

// The sums of g and g h.
template <typename T>
__device__ __forceinline__ void add_terms(const float2 (&g)[Word<T>::PAIRS], const float2 (&h)[Word<T>::PAIRS],
                                          float2 &first, float2 &second) {
#pragma unroll
    for (int j = 0; j < Word<T>::PAIRS; ++j) {
        first = __fadd2_rn(first, g[j]);
        second = __ffma2_rn(g[j], h[j], second);
    }
}

// A word's share of dw and db.
template <int PAIRS>
__device__ __forceinline__ void add_columns(const float2 (&dy)[PAIRS], const float2 (&h)[PAIRS], float2 (&dw)[PAIRS],
                                            float2 (&db)[PAIRS]) {
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
        dw[j] = __ffma2_rn(dy[j], h[j], dw[j]);
        db[j] = __fadd2_rn(db[j], dy[j]);
    }
}

// dx of a word: g becomes rs (g - mg - h mgh) + residual.
template <typename T>
__device__ __forceinline__ void finish_word(float2 (&g)[Word<T>::PAIRS], const float2 (&h)[Word<T>::PAIRS], float rs,
                                            float mg, float mgh, bool add, const uint4 &residual) {
    float2 f[Word<T>::PAIRS];
#pragma unroll
    for (int j = 0; j < Word<T>::PAIRS; ++j)
        g[j] = __fmul2_rn(__ffma2_rn(h[j], both(-mgh), __fadd2_rn(g[j], both(-mg))), both(rs));
    if (add) {
        Word<T>::open(residual, f);
#pragma unroll
        for (int j = 0; j < Word<T>::PAIRS; ++j) g[j] = __fadd2_rn(g[j], f[j]);
    }
}

// SUMS: the block's part of dw and db to row `blockIdx.x` of `partial`, (blocks, 2,
// d).  dx may be null.  The words of the next STAGES - 1 rows are on their way to
// shared memory while a row is worked on, each thread's to places of its own, so
// that nobody waits for anybody else's: in registers there is room for one row
// ahead, which kept 55% of the copy rate (16384 x 4096 bfloat16 with the residual's
// gradient: 126 us).
template <typename T, int LANES, int PIECES, Rows16 ROWS, bool SUMS>
__global__ void __launch_bounds__(LANES ? kSharedBlock : PIECES == 2 ? 256 : 512, LANES ? 4 : PIECES == 2 ? 2 : 1)
    norm_grad_kernel(const GradRows in, int64_t n, int d, int period, T *dx, float *__restrict__ partial) {
    extern __shared__ uint4 ring[];
    constexpr int N = Word<T>::N, GROUPS = LANES ? kSharedBlock / LANES : 1, PAIRS = Word<T>::PAIRS;
    constexpr int STAGES = stages_of(PIECES);
    in.start();
    const int width = LANES ? LANES : (int)blockDim.x;
    const int t = LANES ? (int)threadIdx.x % LANES : (int)threadIdx.x, group = LANES ? (int)threadIdx.x / LANES : 0;
    const Place at = place_of<T, ROWS>(in.x, period);
    const Mine<T, PIECES, ROWS> mine(t, width, at.off, d);
    const float scale = 1.f / (float)d;
    const bool add = in.residual.base && dx;
    float2 dw[SUMS ? PIECES : 1][PAIRS] = {}, db[SUMS ? PIECES : 1][PAIRS] = {};
    // (up to sixteen values a thread keeps its terms of the row, too)
    constexpr bool HOLD = Columns<T, PIECES, ROWS>::HOLD;
    const Columns<T, PIECES, ROWS> weight(in.w, mine, at.off, d);
    // this thread's places in a stage: x's words, dy's, the residual's
    const int tensor = PIECES * (int)blockDim.x, stage_words = (add ? 3 : 2) * tensor;
    uint4 *own = ring + threadIdx.x;
    const Fetch<T, PIECES, ROWS> fetch{mine, at.off, d, ((int64_t)t * N - at.off) * (int)sizeof(T)};
    const auto issue = [&](int64_t r, int stage) {
        if (r < n) {
            uint4 *to = own + stage * stage_words;
            fetch(in.x, r, to);
            fetch(in.dy, r, to + tensor);
            if (add) fetch(in.residual, r, to + 2 * tensor);
        }
        copy_commit();
    };
    const int64_t step = at.step * GROUPS, first = at.first + at.step * group;
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) issue(first + k * step, k);
    float next_mu = first < n ? in.mean[first] : 0.f, next_rs = first < n ? in.rstd[first] : 0.f;
    int turn = 0, stage = 0;
    for (int64_t q = at.first; q < n; q += step) {
        const int64_t r = q + at.step * group;
        const float mu = next_mu, rs = next_rs;
        // (into the stage that the last row has left)
        issue(r + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
        copy_wait<STAGES - 1>();
        next_mu = r + step < n ? in.mean[r + step] : 0.f;
        next_rs = r + step < n ? in.rstd[r + step] : 0.f;
        const uint4 *here = own + stage * stage_words;
        float2 sum = {0.f, 0.f}, second = {0.f, 0.f}, terms[HOLD ? PIECES : 1][2][PAIRS];
        if (GROUPS == 1 || r < n) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                if (!mine.has(i)) continue;
                float2(&g)[PAIRS] = terms[HOLD ? i : 0][0], (&h)[PAIRS] = terms[HOLD ? i : 0][1];
                const uint4 uy = fetch.read(here + tensor, i), ux = fetch.read(here, i);  // (what is not there: dy = 0)
                terms_of<T>(uy, ux, mu, rs, g, h);
                if (SUMS) add_columns<PAIRS>(g, h, dw[SUMS ? i : 0], db[SUMS ? i : 0]);
                weight.multiply(i, g);
                add_terms<T>(g, h, sum, second);
            }
        }
        if (dx) {
            sum = group_sum<LANES>(make_float2(sum.x + sum.y, second.x + second.y), turn);
            const float mg = sum.x * scale, mgh = sum.y * scale;
            uint8_t *out = reinterpret_cast<uint8_t *>(dx + r * d) + fetch.start;
            if (GROUPS == 1 || r < n) {
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    if (!mine.has(i)) continue;
                    float2(&g)[PAIRS] = terms[HOLD ? i : 0][0], (&h)[PAIRS] = terms[HOLD ? i : 0][1];
                    if (!HOLD) {
                        terms_of<T>(here[tensor + i * (int)blockDim.x], here[i * (int)blockDim.x], mu, rs, g, h);
                        weight.multiply(i, g);
                    }
                    finish_word<T>(g, h, rs, mg, mgh, add, add ? here[2 * tensor + i * (int)blockDim.x] : uint4{});
                    if (mine.whole(i))
                        *reinterpret_cast<uint4 *>(out + i * mine.stride()) = Word<T>::close(g);
                    else
                        store_row<T, ROWS>(dx + r * d, g, i * width + t, at.off, Cut<T, ROWS>(i * width + t, at.off, d));
                }
            }
        }
        stage = stage == STAGES - 1 ? 0 : stage + 1;
    }
    copy_wait<0>();
    if constexpr (SUMS) {
        float *out = partial + (int64_t)blockIdx.x * 2 * d;
        // the block's groups one after the other
        for (int k = 0; k < GROUPS; ++k) {
            if (k) __syncthreads();
            if (group != k) continue;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int c0 = (i * width + t) * N - at.off;
                if (whole_rows(ROWS)) {  // d and c0 are multiples of 4
                    if (!mine.has(i)) continue;
#pragma unroll
                    for (int j = 0; j < PAIRS; j += 2) {
                        float4 *to = reinterpret_cast<float4 *>(out + c0 + 2 * j);
                        float4 *too = reinterpret_cast<float4 *>(out + d + c0 + 2 * j);
                        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f), a = k ? *to : none, b = k ? *too : none;
                        *to = make_float4(a.x + dw[i][j].x, a.y + dw[i][j].y, a.z + dw[i][j + 1].x, a.w + dw[i][j + 1].y);
                        *too = make_float4(b.x + db[i][j].x, b.y + db[i][j].y, b.z + db[i][j + 1].x, b.w + db[i][j + 1].y);
                    }
                    continue;
                }
                const Cut<T, ROWS> cut(i * width + t, at.off, d);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int c = c0 + j;
                    if (!cut.has(j)) continue;
                    const float2 w2 = dw[i][j / 2], b2 = db[i][j / 2];
                    out[c] = (k ? out[c] : 0.f) + (j & 1 ? w2.y : w2.x);
                    out[d + c] = (k ? out[d + c] : 0.f) + (j & 1 ? b2.y : b2.x);
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
        const auto load = [&](int c, const Cut<T, ROWS> &cut, float2 (&g)[Word<T>::PAIRS], float2 (&h)[Word<T>::PAIRS]) {
            terms_of<T>(load_row<T, ROWS>(in.dy, r, c, at.off, cut), load_row<T, ROWS>(in.x, r, c, at.off, cut), mu, rs, g, h);
            weight_word<T>(in.w.base, in.w.base ? load_columns<T, ROWS>(in.w, c, at.off, cut) : zero, g);
        };
        float2 sum = {0.f, 0.f}, second = {0.f, 0.f}, g[Word<T>::PAIRS], h[Word<T>::PAIRS];
#pragma unroll 2
        for (int c = threadIdx.x; c < words; c += kWideThreads) {
            load(c, Cut<T, ROWS>(c, at.off, d), g, h);
            add_terms<T>(g, h, sum, second);
        }
        sum = group_sum<0>(make_float2(sum.x + sum.y, second.x + second.y), turn);
#pragma unroll 2
        for (int c = threadIdx.x; c < words; c += kWideThreads) {
            const Cut<T, ROWS> cut(c, at.off, d);
            load(c, cut, g, h);
            finish_word<T>(g, h, rs, sum.x * scale, sum.y * scale, in.residual.base,
                           in.residual.base ? load_row<T, ROWS>(in.residual, r, c, at.off, cut) : zero);
            store_row<T, ROWS>(dx + r * d, g, c, at.off, cut);
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
    constexpr int PAIRS = Word<T>::PAIRS;
    float2 dw[PAIRS] = {}, db[PAIRS] = {};
#pragma unroll 4
    for (int64_t r = r0; r < r1; ++r) {
        float2 g[PAIRS], h[PAIRS];
        terms_of<T>(load_row<T, ROWS>(in.dy, r, c, 0, cut), load_row<T, ROWS>(in.x, r, c, 0, cut), in.mean[r], in.rstd[r],
                    g, h);
        add_columns<PAIRS>(g, h, dw, db);
    }
    float *out = partial + (int64_t)blockIdx.y * 2 * d + (int64_t)c * N;
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (cut.has(j)) {
            out[j] = j & 1 ? dw[j / 2].y : dw[j / 2].x;
            out[d + j] = j & 1 ? db[j / 2].y : db[j / 2].x;
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

constexpr int kMostShared = 220 * 1024;

// Shared memory of so much may be asked for; once per kernel and device.
template <auto KERNEL>
cudaError_t allow_shared() {
    static std::once_flag once[kMaxDevices];
    static std::atomic<int> err[kMaxDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    const int slot = dev >= 0 && dev < kMaxDevices ? dev : 0;
    once_per_device(once, [&] {
        err[slot].store((int)cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared));
    });
    return (cudaError_t)err[slot].load();
}

template <typename T, int LANES, int PIECES, Rows16 ROWS>
cudaError_t launch_norm(const Rows &x, const Rows &w, const Rows &b, float eps, int64_t n, int d, int period, T *y,
                        float *mean, float *rstd, int threads, cudaStream_t s) {
    constexpr auto kernel = norm_kernel<T, LANES, PIECES, ROWS>;
    const cudaError_t e = allow_shared<kernel>();
    if (e != cudaSuccess) return e;
    const int64_t rows = LANES ? kSharedBlock / LANES : 1;
    const int shared = stages_of(PIECES) * PIECES * threads * 16;
    // as many blocks as run at once: by registers (see the launch bounds) and shared memory
    const int resident = std::min(std::max(1, (LANES ? 640 : 512) / threads), kMostShared / shared);
    return launch_kernel(true, kernel, dim3(blocks_of((n + rows - 1) / rows, align_up(kSMs * resident, 8), period)),
                         dim3((unsigned)threads), (size_t)shared, s, x, w, b, eps, n, d, period, y, mean, rstd);
}

template <typename T, Rows16 ROWS>
cudaError_t norm_typed(const NormShape &sh, const Rows &x, const Rows &w, const Rows &b, float eps, int period, T *y,
                       float *mean, float *rstd, cudaStream_t s) {
    constexpr int N = Word<T>::N;
    const int64_t words = (sh.d + N - 1) / N + (ROWS == Rows16::kAlike ? 1 : 0);
    const int d = (int)sh.d;
    constexpr Rows16 FULL = ROWS == Rows16::kWhole ? Rows16::kExact : ROWS;
    const auto run = [&](auto launch, int threads) { return launch(x, w, b, eps, sh.n, d, period, y, mean, rstd, threads, s); };
    if (words <= 8) return run(words == 8 ? launch_norm<T, 8, 1, FULL> : launch_norm<T, 8, 1, ROWS>, kSharedBlock);
    if (words <= 32) return run(words == 32 ? launch_norm<T, 32, 1, FULL> : launch_norm<T, 32, 1, ROWS>, kSharedBlock);
    if (words <= 64) return run(words == 64 ? launch_norm<T, 32, 2, FULL> : launch_norm<T, 32, 2, ROWS>, kSharedBlock);
    if (words <= 128) return run(words == 128 ? launch_norm<T, 32, 4, FULL> : launch_norm<T, 32, 4, ROWS>, kSharedBlock);
    if (words <= 2048)
        return run(words % 128 == 0 ? launch_norm<T, 0, 4, FULL> : launch_norm<T, 0, 4, ROWS>, threads_of(words, 4));
    return launch_kernel(true, norm_wide_kernel<T, ROWS>, dim3(blocks_of(sh.n, kSMs * 2, period)), dim3(kWideThreads), 0, s, x,
                         w, b, eps, sh.n, d, period, y, mean, rstd);
}

// The gradient's rows in registers' reach; `count`: its blocks.
template <typename T, int LANES, int PIECES, Rows16 ROWS, bool SUMS>
cudaError_t launch_grad(const GradRows &in, int64_t n, int d, int period, T *dx, float *partial, int threads,
                        int64_t &count, cudaStream_t s) {
    constexpr auto kernel = norm_grad_kernel<T, LANES, PIECES, ROWS, SUMS>;
    const cudaError_t e = allow_shared<kernel>();
    if (e != cudaSuccess) return e;
    const int64_t rows = LANES ? kSharedBlock / LANES : 1;
    const int shared = stages_of(PIECES) * (in.residual.base && dx ? 3 : 2) * PIECES * threads * 16;
    // as many blocks as run at once: by registers (see its launch bounds) and shared memory
    const int resident = std::min(std::max(1, 512 / threads), kMostShared / shared);
    count = blocks_of((n + rows - 1) / rows, kSMs * std::max(1, std::min(8, resident)), period);
    return launch_kernel(true, kernel, dim3((unsigned)count), dim3((unsigned)threads), (size_t)shared, s, in, n, d, period,
                         dx, partial);
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
    const auto rows = [&](auto with_sums) {
        constexpr bool SUMS = decltype(with_sums)::value;
        constexpr Rows16 FULL = ROWS == Rows16::kWhole ? Rows16::kExact : ROWS;
        const auto run = [&](auto launch, int threads) {
            return launch(in, sh.n, d, period, dx, partial, threads, count, s);
        };
        if (words <= 8)
            return run(words == 8 ? launch_grad<T, 8, 1, FULL, SUMS> : launch_grad<T, 8, 1, ROWS, SUMS>, kSharedBlock);
        if (words <= 32)
            return run(words == 32 ? launch_grad<T, 32, 1, FULL, SUMS> : launch_grad<T, 32, 1, ROWS, SUMS>, kSharedBlock);
        // sixteen values a thread (16-bit types: 16384 x 4096 73 us so, 91 with 32;
        // float32 x 2048: 130 so, 167 with eight)
        constexpr int FEW = 16 / N;
        if (words <= 32 * FEW)
            return run(words == 32 * FEW ? launch_grad<T, 32, FEW, FULL, SUMS> : launch_grad<T, 32, FEW, ROWS, SUMS>,
                       kSharedBlock);
        if (words <= 256 * FEW)
            return run(words % (32 * FEW) == 0 ? launch_grad<T, 0, FEW, FULL, SUMS> : launch_grad<T, 0, FEW, ROWS, SUMS>,
                       threads_of(words, FEW));
        return run(words % 128 == 0 ? launch_grad<T, 0, 4, FULL, SUMS> : launch_grad<T, 0, 4, ROWS, SUMS>,
                   threads_of(words, 4));
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
            e = launch_kernel(true, norm_columns_kernel<T, whole_rows(ROWS)>, dim3((unsigned)strips, (unsigned)parts),
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
