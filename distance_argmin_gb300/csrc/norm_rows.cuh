// What the layer norm and its gradient share: rows as 16-byte words, however they
// lie in memory, and their way through shared memory.
//
// A group of threads has a row: LANES lanes of a warp, or (0) a block.  A thread has
// PIECES of its words, and the same columns in every row of its group.
//
// Rows that do not all start on 16 bytes are still read and written by aligned
// words: a block takes rows that start alike (every eighth, or fewer, of a period
// of the pitch), so that its threads' words hold the same columns in every row;
// only the words at a row's ends are cut.  Tensors whose rows start differently
// from each other are read as shifted words.
//
// The words of the next rows are on their way to shared memory while a row is
// worked on (16384 x 4096 bfloat16, gradient with the residual's: 84 us so, 95% of
// the copy rate; with one row ahead in registers, for which there is room, 126).
#pragma once

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

// Rows that are read again for every pass have a block of so many threads.
constexpr int kWideThreads = 1024;

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

}  // namespace

}  // namespace km
