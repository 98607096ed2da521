// The experts' matrix products and their gradients: which kernels a call runs,
// and what goes around the products (linear_tc.cu): rows brought to 16 bytes,
// dz = dy act'(pre), and the bias gradient.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "linear_common.cuh"

namespace km {

namespace {

// dst(r, c) = src(r, c) with the rows of dst on 16 bytes: a thread moves 16-byte
// pieces, read as shifted words.  One launch copies the experts' W, of which only
// those of experts that may have rows are taken, and x, where they need it: both
// have k columns (a launch each: 1 us more on the device, 3 us on the host).
constexpr int kAlignThreads = 256;

struct AlignJob {
    const uint8_t *src;
    uint8_t *dst;
    int64_t pitch, rows;  // bytes from row to row; rows of a matrix
    Span in;
    int blocks;  // of a matrix; 0: nothing to do
};

__global__ void __launch_bounds__(kAlignThreads) linear_align_kernel(const AlignJob w, int groups, const AlignJob x,
                                                                     int64_t row_bytes, int64_t pitch_out,
                                                                     const int32_t *offsets, uint32_t *clear) {
    griddep_wait();
    if (clear && (blockIdx.x | threadIdx.x) == 0u) *clear = 0u;
    const int w_blocks = w.blocks * groups;
    const bool of_w = (int)blockIdx.x < w_blocks;
    const AlignJob &job = of_w ? w : x;
    const int block = of_w ? (int)blockIdx.x % w.blocks : (int)blockIdx.x - w_blocks;
    const int group = of_w ? (int)blockIdx.x / w.blocks : 0;
    if (of_w && offsets && offsets[group + 1] <= offsets[group]) return;
    const int pieces = (int)((row_bytes + 15) / 16);
    // a row's pieces go to neighbouring threads
    for (int64_t i = (int64_t)block * kAlignThreads + threadIdx.x; i < job.rows * pieces;
         i += (int64_t)job.blocks * kAlignThreads) {
        const int64_t r = i / pieces;
        const int64_t at = (i - r * pieces) * 16;
        const int64_t row = group * job.rows + r;
        // (dst's rows are padded to whole pieces)
        *reinterpret_cast<uint4 *>(job.dst + row * pitch_out + at) =
            load_piece<false>(job.src + row * job.pitch + at, (int)min((int64_t)16, row_bytes - at), job.in);
    }
}

// dz = dy act'(pre), rounded to the matrices' type, and the bias gradient's
// partial sums from the same read.  The rounding is the products' operand type:
// float32 or a pair of 16-bit parts would double their tensor time and dz's
// traffic, for outputs that are rounded as much themselves (bf16 dx and dW 2.3e-3
// off, 1.7e-3 with dz in float32; 32 experts 4096 x 2048, 16384 rows).  A block takes up to 128 rows of one expert
// by 256 columns: a lane 8 columns (16 bytes where the rows allow), a warp every
// eighth row.  Its column sums of the unrounded values go to one row of
// `partial` per row tile; linear_bias_join_kernel adds an expert's in order, so
// the result does not depend on the schedule.
constexpr int kSlopeMaxRows = 128, kSlopeMinRows = 16;
constexpr int kSlopeCols = 256;
constexpr int kSlopeThreads = 256;

// Row tile `u` counted over the experts (whole warp): its expert, its rows, and
// the tiles before the expert's first.
struct RowTile {
    int expert, before;
    int64_t r0, r1;
};

__device__ bool find_row_tile(const int32_t *offsets, int n_experts, int64_t m, int rows, int u, RowTile &t) {
    const int lane = threadIdx.x & 31;
    int last = 0, count = 0;
    for (int e0 = 0; e0 < n_experts; e0 += 32) {
        const int e = e0 + lane;
        int end = 0;
        if (e < n_experts) end = offsets ? max(0, (int)min((int64_t)offsets[e + 1], m)) : (int)m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) end = max(end, __shfl_up_sync(0xffffffffu, end, o));
        end = max(end, last);
        int start = __shfl_up_sync(0xffffffffu, end, 1);
        if (lane == 0) start = last;
        const int own = (int)(((int64_t)end - start + rows - 1) / rows);
        int upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        upto += count;
        const uint32_t past = __ballot_sync(0xffffffffu, u < upto);
        if (past) {
            const int who = __ffs(past) - 1;
            t.expert = e0 + who;
            t.before = __shfl_sync(0xffffffffu, upto - own, who);
            t.r0 = __shfl_sync(0xffffffffu, start, who) + (int64_t)(u - t.before) * rows;
            t.r1 = min(t.r0 + rows, (int64_t)__shfl_sync(0xffffffffu, end, who));
            return true;
        }
        last = __shfl_sync(0xffffffffu, end, 31);
        count = __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

constexpr int kSlopeBatch = 2;  // rows whose loads are in flight together

template <bool WIDE, typename T>
__global__ void __launch_bounds__(kSlopeThreads, 4) linear_slope_kernel(const T *__restrict__ dy, int64_t lddy,
                                                                        Span dy_in, const T *__restrict__ pre,
                                                                        Span pre_in,
                                                                        const int32_t *__restrict__ offsets,
                                                                        int n_experts, int64_t m, int64_t n, int rows,
                                                                        int act, T *__restrict__ dz, int64_t ldz,
                                                                        float *__restrict__ partial, uint32_t *clear) {
    __shared__ float sums[kSlopeThreads / 32][kSlopeCols];
    griddep_wait();
    if (clear && (blockIdx.x | threadIdx.x) == 0u) *clear = 0u;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int WARPS = kSlopeThreads / 32;
    const int strips = (int)((n + kSlopeCols - 1) / kSlopeCols);
    const int tile = (int)(blockIdx.x / strips), strip = (int)(blockIdx.x % strips);
    RowTile t;
    if (!find_row_tile(offsets, n_experts, m, rows, tile, t)) return;
    const int64_t c0 = (int64_t)strip * kSlopeCols + lane * 8;
    const int left = (int)min((int64_t)8, n - c0);
    float sum[8] = {};
    if (left > 0)
        with_activation(act, [&](auto a) {
            constexpr int ACT = decltype(a)::value;
            for (int64_t r = t.r0 + warp; r < t.r1; r += WARPS * kSlopeBatch) {
                uint4 g[kSlopeBatch], z[kSlopeBatch];
#pragma unroll
                for (int b = 0; b < kSlopeBatch; ++b) {
                    const int64_t row = r + b * WARPS;
                    if (row >= t.r1) continue;
                    g[b] = load_piece<WIDE>(reinterpret_cast<const uint8_t *>(dy + row * lddy + c0), 2 * left, dy_in);
                    if constexpr (ACT != KMEANS_ACT_NONE)
                        z[b] = load_piece<WIDE>(reinterpret_cast<const uint8_t *>(pre + row * n + c0), 2 * left, pre_in);
                }
#pragma unroll
                for (int b = 0; b < kSlopeBatch; ++b) {
                    const int64_t row = r + b * WARPS;
                    if (row >= t.r1) continue;
                    const uint32_t gw[4] = {g[b].x, g[b].y, g[b].z, g[b].w}, zw[4] = {z[b].x, z[b].y, z[b].z, z[b].w};
                    uint32_t ow[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float2 v = widen2<T>(gw[c]);
                        if constexpr (ACT != KMEANS_ACT_NONE) {
                            v = __fmul2_rn(v, slope2<ACT>(widen2<T>(zw[c])));
                        }
                        sum[2 * c] += v.x;
                        sum[2 * c + 1] += v.y;
                        ow[c] = narrow2<T>(v.x, v.y);
                    }
                    if (dz) {
                        T *out = dz + row * ldz + c0;  // dz's rows always start on 16 bytes
                        if (left == 8) {
                            *reinterpret_cast<uint4 *>(out) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
                        } else {
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                if (c < left)
                                    reinterpret_cast<uint16_t *>(out)[c] = (uint16_t)(ow[c / 2] >> ((c & 1) * 16));
                        }
                    }
                }
            }
        });
    if (!partial) return;
#pragma unroll
    for (int c = 0; c < 8; ++c) sums[warp][lane * 8 + c] = sum[c];
    __syncthreads();
    const int64_t col = (int64_t)strip * kSlopeCols + threadIdx.x;
    if (col >= n) return;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) s += sums[w][threadIdx.x];
    partial[(int64_t)tile * n + col] = s;
}

template <typename T>
__global__ void __launch_bounds__(kSlopeThreads) linear_bias_join_kernel(const float *partial, const int32_t *offsets,
                                                                         int64_t m, int64_t n, int rows, T *db) {
    __shared__ int range[2];
    griddep_wait();
    const int expert = blockIdx.y;
    if (threadIdx.x < 32) {
        // the tiles before this expert's first and its own
        int first = 0, last = 0;
        if (!offsets) {
            last = (int)((m + rows - 1) / rows);
        } else {
            const int lane = threadIdx.x;
            int top = 0, sum = 0;
            for (int e0 = 0; e0 <= expert; e0 += 32) {
                const int e = e0 + lane;
                int end = e <= expert ? max(0, (int)min((int64_t)offsets[e + 1], m)) : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) end = max(end, __shfl_up_sync(0xffffffffu, end, o));
                end = max(end, top);
                int start = __shfl_up_sync(0xffffffffu, end, 1);
                if (lane == 0) start = top;
                const int own = (int)(((int64_t)end - start + rows - 1) / rows);
                const int before = e < expert ? own : 0;
                sum += __reduce_add_sync(0xffffffffu, before);
                if (expert - e0 < 32) last = __shfl_sync(0xffffffffu, own, expert - e0);
                top = __shfl_sync(0xffffffffu, end, 31);
            }
            first = sum;
            last += first;
        }
        if (threadIdx.x == 0) {
            range[0] = first;
            range[1] = last;
        }
    }
    __syncthreads();
    const int64_t col = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (col >= n) return;
    LongSum s;
#pragma unroll 8
    for (int u = range[0]; u < range[1]; ++u) s.add(partial[(int64_t)u * n + col]);
    db[(int64_t)expert * n + col] = narrow<T>(s.value());
}

// dw[e] = the sums of expert e's chunks of rows, in order, where it has several.
template <typename T>
__global__ void __launch_bounds__(kSlopeThreads) linear_weights_join_kernel(const float *__restrict__ partial,
                                                                            const int32_t *offsets, int n_experts,
                                                                            int64_t m, int chunk, int64_t size, T *dw) {
    extern __shared__ int join_smem[];
    int *edges = join_smem, *tiles = edges + n_experts + 2, *slots = tiles + n_experts + 2;
    griddep_wait();
    if (threadIdx.x < 32) fill_tables(offsets, n_experts, m, chunk, edges, tiles, slots, threadIdx.x);
    __syncthreads();
    for (int e = 0; e < n_experts; ++e) {
        const int chunks = slots[e + 1] - slots[e];
        if (chunks == 0) continue;
        const float *from = partial + (int64_t)slots[e] * size;
        for (int64_t i = (int64_t)blockIdx.x * kSlopeThreads + threadIdx.x; i < size;
             i += (int64_t)gridDim.x * kSlopeThreads) {
            LongSum s;
#pragma unroll 8
            for (int c = 0; c < chunks; ++c) s.add(from[(int64_t)c * size + i]);
            dw[(int64_t)e * size + i] = narrow<T>(s.value());
        }
    }
}

// Rows of a block: fewer where that gives every SM a block or two (257 rows of
// 1000 columns: 16 blocks of 128 rows, or 68 of 16).
int slope_rows(int64_t m, int64_t n) {
    int rows = kSlopeMaxRows;
    while (rows > kSlopeMinRows && (m + rows - 1) / rows * ((n + kSlopeCols - 1) / kSlopeCols) < 2 * kSMs) rows /= 2;
    return rows;
}

// Most row tiles that m rows of so many experts make.
int64_t slope_tiles(int64_t m, int64_t n, int64_t n_experts) {
    const int rows = slope_rows(m, n);
    return (m + rows - 1) / rows + n_experts;
}

// Bytes of `rows` rows of 16-bit values.
Span span16(const void *base, int64_t rows, int64_t pitch, int64_t cols) {
    const uint8_t *b = static_cast<const uint8_t *>(base);
    return {b, base && rows > 0 ? b + ((rows - 1) * pitch + cols) * 2 : b};
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

    AlignJob job(const void *src, int64_t pitch, int64_t groups, int64_t rows, int64_t off) const {
        const int64_t blocks = (rows * ((sh.k + 7) / 8) + kAlignThreads - 1) / kAlignThreads;
        return {static_cast<const uint8_t *>(src), ws + off, pitch * 2, rows, span16(src, groups * rows, pitch, sh.k),
                (int)(blocks < 4096 ? blocks : 4096)};
    }
    // x (null: not needed) and w (likewise) with their rows on 16 bytes
    cudaError_t align(const void **x, int64_t *ldx, const void **w, int64_t *ldw) {
        const bool do_x = x && !rows16(*x, *ldx) && sh.m > 0, do_w = w && !rows16(*w, *ldw);
        if (!do_x && !do_w) return cudaSuccess;
        const AlignJob jw = do_w ? job(*w, *ldw, sh.n_experts, sh.n, L.off_w) : AlignJob{};
        const AlignJob jx = do_x ? job(*x, *ldx, 1, sh.m, L.off_x) : AlignJob{};
        const int64_t ldd = align_up(sh.k, 8);
        const cudaError_t e = launch_kernel(true, linear_align_kernel, dim3((unsigned)(jw.blocks * sh.n_experts + jx.blocks)),
                                            dim3(kAlignThreads), 0, s, jw, sh.n_experts, jx, sh.k * 2, ldd * 2,
                                            sh.offsets, first());
        if (do_w) {
            *w = jw.dst;
            *ldw = ldd;
        }
        if (do_x) {
            *x = jx.dst;
            *ldx = ldd;
        }
        return e;
    }
    template <Product MODE>
    cudaError_t product(const Product16 &g) {
        return launch_linear_tc(MODE, sh, g, &reinterpret_cast<WsHeader *>(ws)->status, first() != nullptr, s);
    }
};

template <typename T>
cudaError_t forward_typed(const LinearShape &sh, Product16 g, const LinearLayout &L, uint8_t *ws, cudaStream_t s) {
    if (few_rows(sh)) return launch_linear_few(sh, g, &reinterpret_cast<WsHeader *>(ws)->status, s);
    Call<T> call(sh, L, ws, s);
    cudaError_t e = call.align(&g.b, &g.ldb, &g.a, &g.pitch_w);
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
    const bool keep = (activation != KMEANS_ACT_NONE || !rows16(dy, lddy)) && (dx || dw);
    if (sh.m > 0 && (keep || db)) {
        T *dz = keep ? reinterpret_cast<T *>(ws + L.off_dz) : nullptr;
        const int64_t ldz = align_up(sh.n, 8);
        if (keep) {
            g.b = dz;
            g.ldb = ldz;
        }
        const dim3 grid((unsigned)((sh.n + kSlopeCols - 1) / kSlopeCols * slope_tiles(sh.m, sh.n, sh.offsets ? sh.n_experts : 0)));
        const bool wide = sh.n % 8 == 0 && rows16(dy, lddy) && (activation == KMEANS_ACT_NONE || rows16(pre, sh.n));
        float *partial = db ? reinterpret_cast<float *>(ws + L.off_partial) : nullptr;
        e = launch_kernel(true, wide ? linear_slope_kernel<true, T> : linear_slope_kernel<false, T>, grid,
                          dim3(kSlopeThreads), 0, s, static_cast<const T *>(dy), lddy,
                          span16(dy, sh.m, lddy, sh.n), static_cast<const T *>(pre), span16(pre, sh.m, sh.n, sh.n),
                          sh.offsets, sh.n_experts, sh.m, sh.n, slope_rows(sh.m, sh.n), activation, dz, ldz, partial,
                          call.first());
        // The row tiles' sums are joined by the weight gradient's epilogue warps,
        // which have nothing to do yet when it starts (a launch of its own: 6.5 us
        // of the ragged gradient, 12 of 32768 rows of 512 x 512); a kernel with a
        // thread for each does it where there is no weight gradient, and where an
        // expert has more tiles than those warps can add up on the way.
        const int rows = slope_rows(sh.m, sh.n);
        const bool on_the_side = dw && db && sh.m / rows <= 512 * (int64_t)sh.n_experts;
        if (on_the_side) {
            g.db = db;
            g.bias_sums = partial;
            g.bias_rows = rows;
        }
        if (e == cudaSuccess && db && !on_the_side)
            e = launch_kernel(true, linear_bias_join_kernel<T>,
                              dim3((unsigned)((sh.n + kSlopeThreads - 1) / kSlopeThreads), (unsigned)sh.n_experts),
                              dim3(kSlopeThreads), 0, s, static_cast<const float *>(partial), sh.offsets, sh.m, sh.n,
                              slope_rows(sh.m, sh.n), static_cast<T *>(db));
    }
    if (e == cudaSuccess && db && sh.m == 0)
        e = cudaMemsetAsync(db, 0, (size_t)sh.n_experts * (size_t)sh.n * sizeof(T), s);
    int64_t ldw = sh.k;
    if (e == cudaSuccess && sh.m > 0) e = call.align(dw ? &x : nullptr, &ldx, dx ? &w : nullptr, &ldw);
    if (e == cudaSuccess && dx && sh.m > 0) {
        g.a = w;
        g.pitch_w = ldw;
        g.out = dx;
        g.partial = reinterpret_cast<float *>(ws + L.off_sums);
        e = call.template product<Product::kRows>(g);
    }
    if (e == cudaSuccess && dw && sh.m == 0)
        return cudaMemsetAsync(dw, 0, (size_t)sh.n_experts * (size_t)sh.n * (size_t)sh.k * sizeof(T), s);
    if (e == cudaSuccess && dw) {
        g.a = x;
        g.lda = ldx;
        g.out = dw;
        const WeightsSplit split = weights_split(sh.m, sh.n, sh.k, sh.n_experts);
        g.partial = reinterpret_cast<float *>(ws + L.off_sums);
        e = call.template product<Product::kWeights>(g);
        if (e == cudaSuccess && split.slots > 0) {
            const int64_t size = sh.n * sh.k, blocks = (size + kSlopeThreads - 1) / kSlopeThreads;
            e = launch_kernel(true, linear_weights_join_kernel<T>, dim3((unsigned)std::min(blocks, (int64_t)kSMs * 8)),
                              dim3(kSlopeThreads), 3 * (size_t)(sh.n_experts + 2) * 4, s,
                              static_cast<const float *>(g.partial), sh.offsets, sh.n_experts, sh.m, split.chunk, size,
                              static_cast<T *>(dw));
        }
    }
    return e;
}

}  // namespace

LinearLayout linear_layout(bool grad, int64_t m, int64_t n, int64_t k, int64_t n_experts) {
    LinearLayout L{};
    int64_t o = align_up((int64_t)(kPairWordsOffset + kMaxPairWords * sizeof(uint32_t)), 1024);
    L.off_x = o;
    o = align_up(o + m * align_up(k, 8) * 2, 1024);
    if (k % 8 != 0) {
        L.off_w = o;
        o = align_up(o + n_experts * n * align_up(k, 8) * 2, 1024);
    }
    // (the gradient's two products take turns with it)
    L.off_sums = o;
    o = align_up(o + std::max(chunk_sums_bytes(grad ? n : k),
                              grad ? weights_split(m, n, k, n_experts).slots * n * k * 4 : 0), 1024);
    if (grad) {
        L.off_dz = o;
        o = align_up(o + m * align_up(n, 8) * 2, 1024);
        L.off_partial = o;
        o = align_up(o + slope_tiles(m, n, n_experts) * n * 4, 1024);
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
    g.partial = reinterpret_cast<float *>(ws + L.off_sums);
    return sh.bf16 ? forward_typed<__nv_bfloat16>(sh, g, L, ws, s) : forward_typed<__half>(sh, g, L, ws, s);
}

cudaError_t launch_linear_grad(const LinearShape &sh, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                               const void *w, const void *pre, int activation, void *dx, void *dw, void *db,
                               const LinearLayout &L, uint8_t *ws, cudaStream_t s) {
    if (sh.m == 0 || !(dx || dw || db)) {  // no kernel that clears it
        const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(WsHeader), s);  // this call's status word
        if (e != cudaSuccess) return e;
    }
    return sh.bf16 ? grad_typed<__nv_bfloat16>(sh, dy, lddy, x, ldx, w, pre, activation, dx, dw, db, L, ws, s)
                   : grad_typed<__half>(sh, dy, lddy, x, ldx, w, pre, activation, dx, dw, db, L, ws, s);
}

}  // namespace km
