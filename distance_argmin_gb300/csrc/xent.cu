// Softmax cross entropy of rows against a matrix of classes, whose logits are
// never kept: z = scale x W^T, lse = log sum exp z, loss = lse - z_label, and
// the gradient dz = dloss scale (exp(z - lse) - 1[label]), dx = dz W, dW = dz^T x.
//
// The rows that count (label >= 0) are first brought together, on 16 bytes, so
// that the products see only them: ignored rows cost nothing, and whatever they
// hold reaches no result.
// Forward: the product (log sum, see linear_tc.cuh) leaves each row's largest
// logit and sum of exponentials per 16 to 64 classes (a quarter of a unit's; few
// rows: 32), which the join kernels bring together.  Gradient: piece by piece of the classes dz is formed from
// the logits once more, in 16 bits, and goes into both products while it is near;
// dx is added up in float32 from piece to piece.
//
// The tensor pipe bounds both, 2 and 6 operations per row, class and feature: 8192
// rows of 32768 classes, k = 2048, bfloat16, forward 568 to 577 us (1905 to 1935
// TFLOP/s; a library product that writes the logits 552 to 581 over the same runs),
// gradient 1710 to 1789 us (1844 to 1929 TFLOP/s).  Few rows are bound by the
// classes' matrix: 24 rows of 131072 classes, k = 4096, 173 us, 6.2 TB/s (the
// library's product 169).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <cstdlib>

#include "layer.cuh"
#include "linear_tc.cuh"

namespace km {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------- the rows that count
constexpr int kShareRows = 64;      // rows counted together
constexpr int kBringRows = 8;       // rows of a block, a warp each
constexpr int kBringThreads = 32 * kBringRows;
// Up to so many rows a block counts the ones before its own itself (16 labels to
// a thread); more are counted by two kernels in front.  (2048 rows of 32768 classes,
// k = 512: 46 us, 49 with them; 8192 of 4096: 35 us, 38 without, gradient 110 and
// 117; 4096 of 4096 25 and 27.)
constexpr int64_t kCountHere = 4096;

// A class matrix of up to so many values that has to be brought to 16 bytes is so by
// the rows' kernel, which saves a launch; larger ones by launch_align, whose warps
// keep more in flight.  (1031 rows of 10007 classes, k = 515: forward 28.8 and
// gradient 75 us, 32.3 and 80 apart; 2000 of 32768, k = 1023 the same; 24 of 32768,
// k = 2047 forward 86 and 83; 100 of 100000, k = 2047 248 and 230.)
constexpr int64_t kAlignHere = (int64_t)1 << 25;

// Of kShareRows rows: how many count (and then: before them), whether a label is
// past the classes, and the largest finite gradient's magnitude, dloss * scale.
struct alignas(16) Tally {
    int32_t count, bad;
    float top;
    int32_t pad;
};

struct Bring {
    const void *labels;
    int id_bytes;
    int64_t m, classes, k;
    const uint8_t *x;
    int64_t ldx;  // bytes
    Span x_in;
    uint8_t *xs;
    int64_t ldxs;  // bytes
    EntropyRow *rows;
    const Tally *tally;  // of all shares, then of everything (null: counted here)
    int32_t *offsets;    // (2): 0 and the rows that count
    uint32_t *header, *word;  // status, see common.cuh: the products' waits use the word
    float scale;
    // forward: the ignored rows' results
    float *loss, *lse;
    // gradient
    const float *dloss, *lse_in;
    const uint8_t *w;  // (classes, k)
    Span w_in;
    uint8_t *wt;          // w's rows on 16 bytes, pitch ldxs, where they are not
    unsigned row_blocks;  // blocks of rows; the ones behind them bring w's
    float *factors;    // dz's scale, and what undoes it
    float *share;      // per row, see below
    uint8_t *xw;       // share * x, where dW is wanted
    bool narrow;       // float16
    uint16_t *dx;      // ignored rows get zeros
};

__device__ __forceinline__ int64_t label_of(const Bring &b, int64_t r) {
    return b.id_bytes == 8 ? static_cast<const int64_t *>(b.labels)[r] : (int64_t)static_cast<const int32_t *>(b.labels)[r];
}

// (A row whose gradient is not finite has no say in what float16 keeps of the others.)
__device__ __forceinline__ float larger_gradient(const Bring &b, float top, int64_t r) {
    const float g = fabsf(b.dloss[r] * b.scale);
    return isfinite(g) ? fmaxf(top, g) : top;
}

__device__ __forceinline__ float warp_max(float v) {  // of what is not negative, and never NaN
    return __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(v)));
}

__global__ void __launch_bounds__(kBringThreads) xent_tally_kernel(const Bring b, Tally *tally, int64_t shares) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t share = (int64_t)blockIdx.x * (kBringThreads / 32) + (threadIdx.x >> 5);
    if (share >= shares) return;
    Tally t{0, 0, 0.f, 0};
#pragma unroll
    for (int i = 0; i < kShareRows / 32; ++i) {
        const int64_t r = share * kShareRows + i * 32 + lane;
        const int64_t l = r < b.m ? label_of(b, r) : -1;
        const bool real = l >= 0 && l < b.classes;
        t.count += __popc(__ballot_sync(kAll, real));
        t.bad |= __any_sync(kAll, l >= b.classes);
        if (b.dloss && real) t.top = larger_gradient(b, t.top, r);
    }
    t.top = warp_max(t.top);
    if (lane == 0) tally[share] = t;
}

// Each share's count becomes that of the rows before it; behind the shares, all.
constexpr int kScanThreads = 1024;

__global__ void __launch_bounds__(kScanThreads) xent_scan_kernel(Tally *tally, int64_t shares) {
    __shared__ int sums[kScanThreads / 32];
    __shared__ int any[kScanThreads / 32];
    __shared__ float tops[kScanThreads / 32];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int before = 0, bad = 0;
    float top = 0.f;
    for (int64_t i0 = 0; i0 < shares; i0 += kScanThreads) {
        const int64_t i = i0 + threadIdx.x;
        const Tally t = i < shares ? tally[i] : Tally{0, 0, 0.f, 0};
        bad |= t.bad;
        top = fmaxf(top, t.top);
        int upto = t.count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAll, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        int own = 0, all = 0;
        for (int w = 0; w < kScanThreads / 32; ++w) {
            if (w < warp) own += sums[w];
            all += sums[w];
        }
        if (i < shares) tally[i].count = before + own + upto - t.count;
        before += all;
        __syncthreads();
    }
    bad = __any_sync(kAll, bad);
    top = warp_max(top);
    if (lane == 0) {
        any[warp] = bad;
        tops[warp] = top;
    }
    __syncthreads();
    if (threadIdx.x) return;
    for (int w = 1; w < kScanThreads / 32; ++w) {
        bad |= any[w];
        top = fmaxf(top, tops[w]);
    }
    tally[shares] = {before, bad, top, 0};
}

// Sums and maxima over the block, in every thread.
struct Totals {
    int before, all, bad;
    float top;
};

__device__ __forceinline__ Totals block_totals(Totals t) {
    __shared__ Totals part[kBringThreads / 32];
    t.before = __reduce_add_sync(kAll, t.before);
    t.all = __reduce_add_sync(kAll, t.all);
    t.bad = __reduce_or_sync(kAll, t.bad);
    t.top = warp_max(t.top);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = t;
    __syncthreads();
    t = part[0];
#pragma unroll
    for (int w = 1; w < kBringThreads / 32; ++w) {
        t.before += part[w].before;
        t.all += part[w].all;
        t.bad |= part[w].bad;
        t.top = fmaxf(t.top, part[w].top);
    }
    return t;
}

// The power of two that takes gradients of at most `top` to [2^13, 2^14): dz has
// twice their magnitude at most, and float16 then keeps probabilities down to
// 2^-28 of it in full.  (bfloat16 has float32's range.)
__device__ __forceinline__ int scale_exponent(float top) {
    if (!(top > 0.f)) return 0;
    return max(-126, min(126, 13 - ilogbf(top)));
}

// dz is rounded to 16 bits, and where a row's dz has one large term, the label's
// -(1 - p), its rounding would be that of all of dx (up to 2^-8 where rows are
// few).  So a row's gradient is split into a share in [1/2, 1) and the rest, such
// that the label's term is a power of two: dz is formed with the rest, dx is
// multiplied with the share in float32, and dW takes share * x, whose roundings
// are each value's own.  The label's probability need not be exact for that.
__device__ __forceinline__ float share_of(float gradient, float z, float lse) {
    const float rest = fminf(fmaxf(-expm1f(z - lse), 0x1p-20f), 1.f);
    int e;
    const float share = fabsf(frexpf(gradient * rest, &e));
    return share >= 0.5f && share < 1.f ? share : 1.f;  // (0, infinite, NaN)
}

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kBringThreads) xent_bring_kernel(const Bring b) {
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!WHOLE && blockIdx.x >= b.row_blocks) {
        const int64_t r = (int64_t)(blockIdx.x - b.row_blocks) * kBringRows + warp, row_bytes = b.k * 2;
        if (r >= b.classes) return;
        const uint8_t *from = b.w + r * row_bytes;
        uint8_t *to = b.wt + r * b.ldxs;
#pragma unroll 4
        for (int64_t c = lane * 16; c < row_bytes; c += 32 * 16)
            *reinterpret_cast<uint4 *>(to + c) = load_piece<false>(from + c, (int)min((int64_t)16, row_bytes - c), b.w_in);
        return;
    }
    const int64_t r0 = (int64_t)blockIdx.x * kBringRows, share0 = r0 / kShareRows * kShareRows;
    Totals t{0, 0, 0, 0.f};
    if (b.tally) {
        const Tally before = b.tally[r0 / kShareRows], all = b.tally[(b.m + kShareRows - 1) / kShareRows];
        t = {before.count, all.count, all.bad, all.top};
    } else {
        for (int64_t r = threadIdx.x; r < b.m; r += kBringThreads) {
            const int64_t l = label_of(b, r);
            const bool real = l >= 0 && l < b.classes;
            t.all += real;
            if (r < share0) t.before += real;
            t.bad |= l >= b.classes;
            if (b.dloss && real) t.top = larger_gradient(b, t.top, r);
        }
        t = block_totals(t);
    }
    const int exponent = b.narrow ? scale_exponent(t.top) : 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        b.offsets[0] = 0;
        b.offsets[1] = t.all;
        *b.word = 0u;
        *b.header = kPairWordsMark | 1u << kPairCountShift | (t.bad ? kFlagBadLabel : 0u);
        if (b.factors) {
            b.factors[0] = ldexpf(1.f, exponent);
            b.factors[1] = ldexpf(1.f, -exponent);
        }
    }
    const int64_t r = r0 + warp;
    if (r >= b.m) return;
    // this row among the ones of its share that count
    int place = t.before;
    int64_t label = -1;
#pragma unroll
    for (int i = 0; i < kShareRows / 32; ++i) {
        const int64_t s = share0 + i * 32 + lane;
        const int64_t l = s <= r ? label_of(b, s) : -1;
        const uint32_t which = __ballot_sync(kAll, s < r && l >= 0 && l < b.classes);
        place += __popc(which);
        const uint32_t own = __ballot_sync(kAll, s == r);
        if (own) label = __shfl_sync(kAll, l, __ffs(own) - 1);
    }
    const int64_t row_bytes = b.k * 2;
    const int pieces = (int)((row_bytes + 15) / 16);
    if (label < 0 || label >= b.classes) {
        if (lane == 0 && b.loss) {
            b.loss[r] = 0.f;
            b.lse[r] = 0.f;
        }
        if (b.dx)
            for (int64_t c = lane; c < b.k; c += 32) b.dx[r * b.k + c] = 0;
        return;
    }
    const uint8_t *from = b.x + r * b.ldx;
    uint8_t *to = b.xs + place * b.ldxs;
    const auto piece = [&](const uint8_t *p, int c, const Span &in) {
        return load_piece<WHOLE>(p + (int64_t)c * 16, (int)min((int64_t)16, row_bytes - (int64_t)c * 16), in);
    };
    EntropyRow row{0.f, 0.f, (int32_t)label, (int32_t)r};
    if (!b.dloss) {
#pragma unroll 4
        for (int c = lane; c < pieces; c += 32)  // (xs's rows are padded to whole pieces)
            *reinterpret_cast<uint4 *>(to + (int64_t)c * 16) = piece(from, c, b.x_in);
    } else {
        const uint8_t *wl = b.w + label * row_bytes;
        float2 z = {0.f, 0.f};
#pragma unroll 4
        for (int c = lane; c < pieces; c += 32) {
            const uint4 ux = piece(from, c, b.x_in), uw = piece(wl, c, b.w_in);
            *reinterpret_cast<uint4 *>(to + (int64_t)c * 16) = ux;
            z = __ffma2_rn(widen2<T>(ux.x), widen2<T>(uw.x), z);
            z = __ffma2_rn(widen2<T>(ux.y), widen2<T>(uw.y), z);
            z = __ffma2_rn(widen2<T>(ux.z), widen2<T>(uw.z), z);
            z = __ffma2_rn(widen2<T>(ux.w), widen2<T>(uw.w), z);
        }
        float sum = z.x + z.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        const float lse = b.lse_in[r], gradient = b.dloss[r] * b.scale;
        const float share = share_of(gradient, sum * b.scale, lse);
        row.lse2 = lse * kLog2E;
        row.gradient = ldexpf(gradient / share, exponent);
        if (lane == 0) b.share[place] = share;
        if (b.xw) {
            uint8_t *out = b.xw + place * b.ldxs;
#pragma unroll 4
            for (int c = lane; c < pieces; c += 32) {
                const uint4 u = piece(from, c, b.x_in);
                uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = __fmul2_rn(widen2<T>(v[i]), both(share));
                    v[i] = narrow2<T>(f.x, f.y);
                }
                *reinterpret_cast<uint4 *>(out + (int64_t)c * 16) = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
    }
    if (lane == 0) b.rows[place] = row;
}

// ------------------------------------------------------------------- forward
constexpr int kJoinWarps = 32;

// Two parts' (reference, sum); nothing stands for itself as (-inf, 0), and an
// infinite sum stays one.
__device__ __forceinline__ float2 join_parts(float2 a, float2 b) {
    const float top = fmaxf(a.x, b.x);
    const float u = isinf(a.y) || a.x == top ? a.y : a.y * exp2f(a.x - top);
    const float v = isinf(b.y) || b.x == top ? b.y : b.y * exp2f(b.x - top);
    return make_float2(top, u + v);
}

__device__ __forceinline__ float2 join_lanes(float2 s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s = join_parts(s, make_float2(__shfl_xor_sync(kAll, s.x, o), __shfl_xor_sync(kAll, s.y, o)));
    return s;
}

__device__ __forceinline__ void write_loss(float2 s, const EntropyRow *rows, int64_t row, const float *target, float factor,
                                           float *loss, float *lse) {
    const float log = log2f(s.y);
    const int64_t at = rows[row].source;
    // The label's distance from the reference with one rounding, as in the sum's
    // exponentials: where the label is all there is the two cancel, however large
    // the logits.
    const float l = kLn2 * (log - fmaf(target[row], factor, -s.x));
    loss[at] = l < 0.f ? 0.f : l;
    lse[at] = kLn2 * (s.x + log);
}

// 32 rows to a block; its warps take a share of the class parts each.
__global__ void __launch_bounds__(32 * kJoinWarps) xent_join_kernel(const EntropyRow *__restrict__ rows,
                                                                    const int32_t *count, const float2 *__restrict__ stats,
                                                                    int64_t pitch, int parts,
                                                                    const float *__restrict__ target, float factor,
                                                                    float *__restrict__ loss, float *__restrict__ lse) {
    __shared__ float2 sums[kJoinWarps][33];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r = (int64_t)blockIdx.x * 32 + lane;
    float2 s = {-INFINITY, 0.f};
    if (r < *count) {
#pragma unroll 8
        for (int i = warp; i < parts; i += kJoinWarps) s = join_parts(s, stats[i * pitch + r]);
    }
    sums[warp][lane] = s;
    __syncthreads();
    // warp w: row w, whose shares its lanes bring together
    s = join_lanes(sums[lane][warp]);
    const int64_t row = (int64_t)blockIdx.x * 32 + warp;
    if (lane == 0 && row < *count) write_loss(s, rows, row, target, factor, loss, lse);
}

// Few rows: a block has one, whose parts are neighbours (24 rows of 1024 parts in
// the layout above: 5 us in one block).
constexpr int kJoinFewThreads = 256;

__global__ void __launch_bounds__(kJoinFewThreads) xent_join_few_kernel(const EntropyRow *__restrict__ rows,
                                                                        const int32_t *count,
                                                                        const float2 *__restrict__ stats, int64_t pitch,
                                                                        int parts, const float *__restrict__ target,
                                                                        float factor, float *__restrict__ loss,
                                                                        float *__restrict__ lse) {
    __shared__ float2 sums[kJoinFewThreads / 32];
    griddep_wait();
    const int64_t row = blockIdx.x;
    if (row >= *count) return;
    float2 s = {-INFINITY, 0.f};
#pragma unroll 4
    for (int i = threadIdx.x; i < parts; i += kJoinFewThreads) s = join_parts(s, stats[row * pitch + i]);
    s = join_lanes(s);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x) return;
    for (int w = 1; w < kJoinFewThreads / 32; ++w) s = join_parts(s, sums[w]);
    write_loss(s, rows, row, target, factor, loss, lse);
}

// ------------------------------------------------------------------ gradient
// dW of one piece = the chunks' sums, where its rows made several.
template <typename T>
__global__ void __launch_bounds__(256) xent_weights_join_kernel(const float *__restrict__ partial, const int32_t *offsets,
                                                                int chunk, int64_t size, const float *inverse, T *dw) {
    griddep_wait();
    const int chunks = (int)(((int64_t)offsets[1] + chunk - 1) / chunk);
    if (chunks <= 1) return;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < size; i += (int64_t)gridDim.x * 256) {
        LongSum s;
#pragma unroll 8
        for (int c = 0; c < chunks; ++c) s.add(partial[(int64_t)c * size + i]);
        dw[i] = narrow<T>(s.value() * *inverse);
    }
}

// dx = the sums of the parts of a split contraction, in order.
template <typename T>
__global__ void __launch_bounds__(256) xent_rows_join_kernel(const float *__restrict__ sums, int splits, int64_t stride,
                                                             const EntropyRow *__restrict__ rows,
                                                             const float *__restrict__ share, const int32_t *count,
                                                             int64_t k, const float *inverse, T *dx) {
    griddep_wait();
    const int64_t size = *count * k;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < size; i += (int64_t)gridDim.x * 256) {
        float s = 0.f;
#pragma unroll 4
        for (int c = 0; c < splits; ++c) s += sums[c * stride + i];
        const int64_t r = i / k;
        dx[rows[r].source * k + (i - r * k)] = narrow<T>(s * (*inverse * share[r]));
    }
}

int64_t pairs_here() { return std::min(device_sm_count() / 2, kPairs); }

int test_starve() {
    // test-only fault injection (no trap, no fault), as in the assignment
    const char *starve = getenv("KMEANS_GB300_TEST_STARVE_PIPELINE");
    return (starve != nullptr && starve[0] == '1') ? 1 : 0;
}

LinearTcParams params(const LinearShape &sh, int64_t cols, int64_t contraction, uint32_t *word, const EntropyArgs &e) {
    LinearTcParams p{};
    p.offsets = sh.offsets;
    p.m = sh.m;
    p.n_experts = 1;
    p.cols = (int)cols;
    p.num_p = (p.cols + lt::BP - 1) / lt::BP;
    p.out_rows = (int)sh.n;
    p.chunk = kChunk;
    p.contraction = (int)contraction;
    p.status = word;
    p.test_starve = test_starve();
    p.entropy = e;
    return p;
}

// Rows of a unit of a product with `rows` rows and num_p feature tiles.  A stage of
// t rows takes the tensor pipe 2 t cycles and shared memory 256 + t (an operand of
// 256 features goes in and out beside the rows), so large units are best; but all
// pairs wait for the last round of units.  (1031 rows of 10007 classes, 928 that
// count: three rounds of 256 or of 192.)
int rows_per_unit(int64_t rows, int64_t num_p) {
    int best = 256;
    int64_t least = INT64_MAX;
    for (int t = 256; t >= 64; t -= 32) {
        const int64_t units = (rows + t - 1) / t * num_p, rounds = (units + kPairs - 1) / kPairs;
        if (rounds * (256 + t) < least) {
            least = rounds * (256 + t);
            best = t;
        }
    }
    return best;
}

template <Product MODE>
cudaError_t product(const LinearShape &sh, const Product16 &g, LinearTcParams &p, int64_t rows, cudaStream_t s) {
    p.entropy.tile = rows_per_unit(rows, p.num_p * (MODE == Product::kRowsSum ? p.entropy.splits : 1));
    return p.entropy.tile <= 128 ? launch_typed<MODE, 128>(sh, g, p, s) : launch_typed<MODE, 256>(sh, g, p, s);
}

cudaError_t weights_product(const LinearShape &sh, const Product16 &g, const LinearTcParams &p, cudaStream_t s) {
    constexpr Product MODE = Product::kWeightsScaled;
    return (sh.n + 127) / 128 * p.num_p <= pairs_here() ? launch_typed<MODE, 128>(sh, g, p, s)
                                                        : launch_typed<MODE, 256>(sh, g, p, s);
}

// Parts of dx's contraction (the classes of a piece), where dx has few tiles: three
// at least, since the sums go through memory and a kernel of their own.  (Gradient
// of 24 rows of 32768 classes, k = 2048: 98 us, 175 in one part; 512 rows 161 and
// 212; 1031 of 10007, k = 520 70 and 89.  In two parts 4096 rows of 4096, k = 512
// take 73 us, in one 66; 1024 of 32768, k = 2048 256 and 257.)
int rows_splits(int64_t m, int64_t piece, int64_t k) {
    const int64_t units = (m + 255) / 256 * ((k + lt::BP - 1) / lt::BP);
    if (units == 0 || 3 * units > kPairs) return 1;  // (no rows: nothing to split)
    return (int)std::max((int64_t)1, std::min(kPairs / units, piece / 512));
}

// Few rows: the classes go on the tensor-memory lanes.  (24 and 64 rows of 131072
// classes, k = 4096: 172 and 175 us, with the rows on the lanes 195 and 196; of
// 32768, k = 2048: 37 and 37, 49 and 41.)
constexpr int64_t kFewRows = 64;

// Class parts that the forward product leaves sums of.
int64_t class_parts(int64_t m, int64_t n) {
    if (m <= kFewRows) return (n + 31) / 32;
    const int tile = rows_per_unit(n, (m + lt::BP - 1) / lt::BP);
    return (n + tile - 1) / tile * lt::PARTS;
}

}  // namespace

// Classes of a piece: about 2^28 values of dz (half a gigabyte), at least 2048
// (more than 2^28 values from 2^17 rows on) so that dx's sums are read and written
// rarely, at most one accumulator's terms; all pieces about equal.  (Gradient of 8192 rows of 32768 classes, k = 2048: 1.78 to
// 1.86 ms in one piece, 2.00 in four, 2.11 in eight; 24 of 131072, k = 4096: 629 us
// in four, 896 in sixteen.)
int64_t xent_piece(int64_t m, int64_t n) {
    int64_t most = ((int64_t)1 << 28) / std::max(m, (int64_t)1);
    most = std::min((int64_t)kChunk, std::max((int64_t)2048, most / 256 * 256));
    const int64_t pieces = (n + most - 1) / most;
    return std::min(align_up((n + pieces - 1) / pieces, 256), align_up(n, 8));
}

XentLayout xent_layout(bool grad, int64_t m, int64_t n, int64_t k) {
    XentLayout L{};
    int64_t o = align_up((int64_t)(kPairWordsOffset + kMaxPairWords * sizeof(uint32_t)), 1024);
    const auto take = [&](int64_t bytes) {
        const int64_t at = o;
        o = align_up(o + bytes, 1024);
        return at;
    };
    L.off_info = take(64);
    L.off_rows = take(m * (int64_t)sizeof(EntropyRow));
    L.off_tally = take(((m + kShareRows - 1) / kShareRows + 1) * (int64_t)sizeof(Tally));
    L.off_x = take(m * align_up(k, 8) * 2);
    if (k % 8 != 0) L.off_w = take(n * align_up(k, 8) * 2);
    if (!grad) {
        L.off_target = take(m * 4);
        L.off_stats = take(align_up(m, 32) * class_parts(m, n) * 8);
    } else {
        const int64_t piece = xent_piece(m, n);
        const int splits = rows_splits(m, piece, k);
        L.off_share = take(m * 4);
        L.off_xw = take(m * align_up(k, 8) * 2);
        L.off_dz = take(m * piece * 2);
        if (piece < n || splits > 1) L.off_sums = take(splits * m * k * 4);
        L.off_partial = take((m > kChunk ? (m + kChunk - 1) / kChunk : 0) * piece * k * 4);
    }
    L.bytes = grad ? std::max(o, xent_layout(false, m, n, k).bytes) : o;  // (the gradient's serves both)
    return L;
}

namespace {

// What both directions begin with.
struct Start {
    const void *w;
    int64_t ldw;
    const void *xs;
    int64_t ldxs;
    EntropyArgs entropy;
    int32_t *offsets;
    uint32_t *word;
    float *factors;
};

cudaError_t start(const XentShape &sh, const void *x, int64_t ldx, const void *w, Bring b, const XentLayout &L,
                  uint8_t *ws, Start &out, cudaStream_t s) {
    const int64_t ldxs = align_up(sh.k, 8);
    uint8_t *info = ws + L.off_info;
    b.labels = sh.labels;
    b.id_bytes = sh.id_bytes;
    b.m = sh.m;
    b.classes = sh.n;
    b.k = sh.k;
    b.x = static_cast<const uint8_t *>(x);
    b.ldx = ldx * 2;
    b.x_in = {b.x, b.x + ((sh.m - 1) * ldx + sh.k) * 2};
    b.xs = ws + L.off_x;
    b.ldxs = ldxs * 2;
    b.rows = reinterpret_cast<EntropyRow *>(ws + L.off_rows);
    b.offsets = reinterpret_cast<int32_t *>(info);
    b.header = &reinterpret_cast<WsHeader *>(ws)->status;
    b.word = reinterpret_cast<uint32_t *>(ws + kPairWordsOffset);
    b.scale = sh.scale;
    b.narrow = !sh.bf16;
    out.factors = b.factors = b.dloss ? reinterpret_cast<float *>(info + 16) : nullptr;
    b.w = static_cast<const uint8_t *>(w);
    b.w_in = {b.w, b.w + sh.n * sh.k * 2};
    cudaError_t e = cudaSuccess;
    if (sh.m > kCountHere) {
        Tally *tally = reinterpret_cast<Tally *>(ws + L.off_tally);
        const int64_t shares = (sh.m + kShareRows - 1) / kShareRows;
        constexpr int per = kBringThreads / 32;
        e = launch_kernel(true, xent_tally_kernel, dim3((unsigned)((shares + per - 1) / per)), dim3(kBringThreads), 0, s, b,
                          tally, shares);
        if (e == cudaSuccess) e = launch_kernel(true, xent_scan_kernel, dim3(1), dim3(kScanThreads), 0, s, tally, shares);
        b.tally = tally;
    }
    const bool whole = rows16(x, ldx) && sh.k % 8 == 0;
    const auto bring = sh.bf16 ? (whole ? xent_bring_kernel<__nv_bfloat16, true> : xent_bring_kernel<__nv_bfloat16, false>)
                               : (whole ? xent_bring_kernel<__half, true> : xent_bring_kernel<__half, false>);
    out.w = w;
    out.ldw = sh.k;
    b.row_blocks = (unsigned)((sh.m + kBringRows - 1) / kBringRows);
    unsigned blocks = b.row_blocks;
    if (sh.k % 8 != 0) {
        out.w = b.wt = ws + L.off_w;
        out.ldw = ldxs;
        if (sh.n * sh.k <= kAlignHere)
            blocks += (unsigned)((sh.n + kBringRows - 1) / kBringRows);
        else if (e == cudaSuccess)
            e = launch_align(w, sh.k, sh.n, sh.k, ws + L.off_w, s);
    }
    if (e == cudaSuccess) e = launch_kernel(true, bring, dim3(blocks), dim3(kBringThreads), 0, s, b);
    out.xs = b.xs;
    out.ldxs = ldxs;
    out.offsets = b.offsets;
    out.word = b.word;
    out.entropy = EntropyArgs{};
    out.entropy.rows = b.rows;
    out.entropy.count = b.offsets + 1;
    out.entropy.factor = sh.scale * kLog2E;
    out.entropy.splits = 1;
    return e;
}

}  // namespace

cudaError_t launch_xent(const XentShape &sh, const void *x, int64_t ldx, const void *w, float *loss, float *lse,
                        const XentLayout &L, uint8_t *ws, cudaStream_t s) {
    if (sh.m == 0) return cudaMemsetAsync(ws, 0, sizeof(WsHeader), s);  // this call's status word
    Bring b{};
    b.loss = loss;
    b.lse = lse;
    Start st;
    cudaError_t e = start(sh, x, ldx, w, b, L, ws, st, s);
    if (e != cudaSuccess) return e;
    EntropyArgs en = st.entropy;
    en.stats = reinterpret_cast<float2 *>(ws + L.off_stats);
    en.target = reinterpret_cast<float *>(ws + L.off_target);
    const int64_t parts = class_parts(sh.m, sh.n);
    en.pitch = sh.m <= kFewRows ? parts : align_up(sh.m, 32);
    Product16 g{};
    if (sh.m <= kFewRows) {
        const LinearShape ps{sh.m, sh.n, sh.k, 1, st.offsets, sh.bf16};
        g.a = st.w;
        g.pitch_w = st.ldw;
        g.b = st.xs;
        g.ldb = st.ldxs;
        const LinearTcParams p = params(ps, sh.n, sh.k, st.word, en);
        e = launch_typed<Product::kLogSumFew, 64>(ps, g, p, s);
    } else {
        // the classes are the product's rows, the rows its features
        const LinearShape ps{sh.n, sh.m, sh.k, 1, nullptr, sh.bf16};
        g.a = st.xs;
        g.pitch_w = st.ldxs;
        g.b = st.w;
        g.ldb = st.ldw;
        LinearTcParams p = params(ps, sh.m, sh.k, st.word, en);
        e = product<Product::kLogSum>(ps, g, p, sh.n, s);
    }
    if (e != cudaSuccess) return e;
    const auto join = [&](auto kernel, int64_t blocks, int threads) {
        return launch_kernel(true, kernel, dim3((unsigned)blocks), dim3((unsigned)threads), 0, s, en.rows, en.count,
                             (const float2 *)en.stats, en.pitch, (int)parts, (const float *)en.target, en.factor, loss, lse);
    };
    return sh.m <= kFewRows ? join(xent_join_few_kernel, sh.m, kJoinFewThreads)
                            : join(xent_join_kernel, (sh.m + 31) / 32, 32 * kJoinWarps);
}

cudaError_t launch_xent_grad(const XentShape &sh, const float *dloss, const void *x, int64_t ldx, const void *w,
                             const float *lse, void *dx, void *dw, const XentLayout &L, uint8_t *ws, cudaStream_t s) {
    if (sh.m == 0 || !(dx || dw)) {  // no kernel that clears it
        cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(WsHeader), s);  // this call's status word
        if (e == cudaSuccess && dw) e = cudaMemsetAsync(dw, 0, (size_t)sh.n * (size_t)sh.k * 2, s);
        return e;
    }
    Bring b{};
    b.dloss = dloss;
    b.lse_in = lse;
    b.dx = static_cast<uint16_t *>(dx);
    b.share = reinterpret_cast<float *>(ws + L.off_share);
    b.xw = dw ? ws + L.off_xw : nullptr;
    Start st;
    cudaError_t e = start(sh, x, ldx, w, b, L, ws, st, s);
    const int64_t piece = xent_piece(sh.m, sh.n);
    EntropyArgs en = st.entropy;
    en.pitch = piece;
    en.inverse = st.factors + 1;
    en.sums = reinterpret_cast<float *>(ws + L.off_sums);
    en.splits = rows_splits(sh.m, piece, sh.k);
    en.split_stride = sh.m * sh.k;
    en.share = b.share;
    void *dz = ws + L.off_dz;
    for (int64_t c = 0; c < sh.n && e == cudaSuccess; c += piece) {
        const int64_t here = std::min(piece, sh.n - c);
        const LinearShape ps{sh.m, here, sh.k, 1, st.offsets, sh.bf16};
        en.first = (int)c;
        en.begin = c == 0;
        en.last = c + here == sh.n;
        Product16 g{};
        g.a = static_cast<const uint16_t *>(st.w) + c * st.ldw;
        g.pitch_w = st.ldw;
        g.b = st.xs;
        g.ldb = st.ldxs;
        LinearTcParams p = params(ps, here, sh.k, st.word, en);
        p.out = dz;
        e = product<Product::kSoftmax>(ps, g, p, sh.m, s);
        g.b = dz;
        g.ldb = piece;
        if (e == cudaSuccess && dx) {
            p = params(ps, sh.k, here, st.word, en);
            p.out = dx;
            e = product<Product::kRowsSum>(ps, g, p, sh.m, s);
        }
        if (e == cudaSuccess && dw) {
            uint16_t *out = static_cast<uint16_t *>(dw) + c * sh.k;
            g.a = b.xw;
            g.lda = st.ldxs;
            g.out = out;
            p = params(ps, sh.k, here, st.word, en);
            p.out = out;
            p.wide = rows16(out, sh.k);
            p.partial = reinterpret_cast<float *>(ws + L.off_partial);
            e = weights_product(ps, g, p, s);
            if (e == cudaSuccess && sh.m > kChunk) {
                const int64_t size = here * sh.k, blocks = (size + 255) / 256;
                const dim3 grid((unsigned)std::min(blocks, (int64_t)kSMs * 8));
                const float *partial = p.partial;
                const int32_t *offsets = st.offsets;
                e = sh.bf16 ? launch_kernel(true, xent_weights_join_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, partial,
                                            offsets, kChunk, size, en.inverse, reinterpret_cast<__nv_bfloat16 *>(out))
                            : launch_kernel(true, xent_weights_join_kernel<__half>, grid, dim3(256), 0, s, partial, offsets,
                                            kChunk, size, en.inverse, reinterpret_cast<__half *>(out));
            }
        }
    }
    if (e == cudaSuccess && dx && en.splits > 1) {
        const int64_t blocks = (sh.m * sh.k + 255) / 256;
        const dim3 grid((unsigned)std::min(blocks, (int64_t)kSMs * 8));
        const float *sums = en.sums;
        const auto join = [&](auto kernel, auto *out) {
            return launch_kernel(true, kernel, grid, dim3(256), 0, s, sums, en.splits, en.split_stride, en.rows, en.share,
                                 en.count, sh.k, en.inverse, out);
        };
        e = sh.bf16 ? join(xent_rows_join_kernel<__nv_bfloat16>, static_cast<__nv_bfloat16 *>(dx))
                    : join(xent_rows_join_kernel<__half>, static_cast<__half *>(dx));
    }
    return e;
}

}  // namespace km
