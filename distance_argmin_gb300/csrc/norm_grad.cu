// Layer norm's gradient.
//
//   g = dy w, h = (x - mu) r:  dx = r (g - mean g - h mean(g h)) + residual
//   dw = sum over rows of dy h, db = sum over rows of dy
//
// Memory bounds it: three tensors, four with the residual's gradient, each moved
// once (16384 x 4096 bfloat16 73 and 84 us, 83% and 95% of the copy rate; float32
// 133, 91%).  A thread holds its columns' weights and adds up its share of dw and
// db in registers; the blocks' sums meet in norm_join_kernel in a fixed order.
// For rows of more than 2048 words those sums have no room: dw and db get a kernel
// that goes down the columns, and dx reads its rows twice.
#include "norm_rows.cuh"

namespace km {

namespace {

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
// d).  dx may be null.
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
