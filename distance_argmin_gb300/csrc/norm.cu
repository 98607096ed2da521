// Layer norm over a row's features.
//
//   mu = mean x   v = mean (x - mu)^2   r = 1 / sqrt(v + eps)   y = (x - mu) r w + b
//
// The row is read once: its mean, what the mean is off by (its sum rounds where the
// row lies far from zero) with the variance about it, and the result are three
// passes over registers.  Memory bounds it: 16384 x 4096 bfloat16 44 us, 92% of the
// copy rate, float32 84 us (96%); below that the sums' way through the block, twice
// a row, is what short rows wait for (262144 x 256 bfloat16: 55 us, 73%).  Four words
// a thread, so that what goes with a row is paid by few threads (16384 x 4096
// bfloat16 with two words 58 us, as 16 words of a warp 62).  Rows of more than 2048
// words are read again for every pass.
#include "norm_rows.cuh"

namespace km {

namespace {

// The sum of a word's values.
template <typename T>
__device__ __forceinline__ float2 add_word(const uint4 &raw, float2 sum) {
    float2 v[Word<T>::PAIRS];
    Word<T>::open(raw, v);
#pragma unroll
    for (int j = 0; j < Word<T>::PAIRS; ++j) sum = __fadd2_rn(sum, v[j]);
    return sum;
}

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

}  // namespace

cudaError_t launch_norm(const NormShape &sh, const void *x, int64_t ldx, const void *weight, const void *bias, float eps,
                        void *y, float *mean, float *rstd, cudaStream_t s) {
    if (sh.dtype == KMEANS_F32) return norm_any<float>(sh, x, ldx, weight, bias, eps, y, mean, rstd, s);
    return sh.dtype == KMEANS_F16 ? norm_any<__half>(sh, x, ldx, weight, bias, eps, y, mean, rstd, s)
                                  : norm_any<__nv_bfloat16>(sh, x, ldx, weight, bias, eps, y, mean, rstd, s);
}

}  // namespace km
