// What the kernels of the experts' products share: 16-bit conversions, the
// activations, and which rows belong to whom.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "pieces.cuh"

namespace km {

// forward  y = act(x W^T + b) + residual
// rows     dx = dz W
// weights  dW = dz^T x
// All three are out(q, p) = sum_c A(p, c) B(q, c), with p the contiguous
// dimension of the output: output features, input features, input features.
//
// The cross entropy (xent.cu) takes three of them with other ends, and the
// weights product with a factor:
// log sum  z = x W^T with a row of x on each tensor-memory lane (p the rows, q the
//          classes): only each row's largest z and sum of exponentials leave
// few      the same of few rows, a class on each lane
// softmax  z once more as in the forward product, dz = g (exp(z - lse) - 1[label])
// sum      dx over a piece of the classes, added up in float32
// scaled   dW of such a dz, which is kept times a power of two
enum class Product { kForward, kRows, kWeights, kLogSum, kLogSumFew, kSoftmax, kRowsSum, kWeightsScaled };

__host__ __device__ constexpr bool is_weights(Product m) { return m == Product::kWeights || m == Product::kWeightsScaled; }
// A's contiguous dimension is the contraction.
__host__ __device__ constexpr bool is_forward(Product m) {
    return m == Product::kForward || m == Product::kLogSum || m == Product::kLogSumFew || m == Product::kSoftmax;
}

// A row that counts: its lse times log2(e), the factor of its gradient, its label,
// and which row of the caller's it is.
struct alignas(16) EntropyRow {
    float lse2, gradient;
    int32_t label, source;
};

struct EntropyArgs {
    const EntropyRow *rows;
    const int32_t *count;  // rows that count
    float factor;          // of z: the logits' scale, times log2(e)
    int tile;              // rows of a unit, a multiple of 32
    float2 *stats;         // log sum: (reference, sum of 2^(factor z - reference)) per class part and row
    float *target;         // log sum: z at the label
    int first;             // class of the piece's first
    int splits;            // sum: parts of the contraction, each with sums of its own
    float *sums;           // sum: dx so far
    int64_t split_stride;  // values from one part's sums to the next's
    bool begin, last;      // sum: the first, the last piece
    const float *inverse;  // of dz's scale
    const float *share;    // sum: per row, what dx is to be multiplied with
    int64_t pitch;         // of dz (softmax), of stats' class parts (log sum) or rows (few)
};

struct Product16 {
    const void *a;            // w (forward, rows) or x (weights)
    int64_t lda;              // pitch of x (weights)
    int64_t pitch_w;          // pitch of w's rows (forward, rows)
    const void *b;            // x (forward) or dz
    int64_t ldb;
    const void *bias, *residual;
    int64_t ldr;
    int activation;
    void *out, *pre;
    float *partial;           // the chunks' sums (see kChunk and WeightsSplit)
    void *db;                 // weights: the bias gradient, joined on the side from
    const float *bias_sums;   // the sums of `bias_rows` rows each (null: not here)
    int bias_rows;
};

// f applied with the activation as a compile-time constant: one branch around
// a whole loop instead of one per value.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F &&f) {
    switch (act) {
        case KMEANS_ACT_RELU: f(std::integral_constant<int, KMEANS_ACT_RELU>{}); break;
        case KMEANS_ACT_GELU: f(std::integral_constant<int, KMEANS_ACT_GELU>{}); break;
        case KMEANS_ACT_GELU_TANH: f(std::integral_constant<int, KMEANS_ACT_GELU_TANH>{}); break;
        case KMEANS_ACT_SILU: f(std::integral_constant<int, KMEANS_ACT_SILU>{}); break;
        default: f(std::integral_constant<int, KMEANS_ACT_NONE>{}); break;
    }
}

// A float32 sum with the error of each addition kept beside it, so that it does
// not drift with the number of terms (2^25 rows of one value in tiles of 128: a
// plain sum of the tiles' is off by 0.5%).  Infinite and NaN sums are the plain
// one's.
struct LongSum {
    float sum = 0.f, error = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float t = sum + v, of_v = t - sum;
        error += (sum - (t - of_v)) + (v - of_v);
        sum = t;
    }
    __device__ __forceinline__ float value() const { return isfinite(error) ? sum + error : sum; }
};

// First row past expert e - 1's when the rows before `from` are taken: the
// offset, kept inside [from, m].
__device__ __forceinline__ int64_t first_row(const int32_t *offsets, int e, int64_t from, int64_t m) {
    const int64_t v = offsets[e];
    return v < from ? from : (v > m ? m : v);
}

// The row tiles (of `rows` rows) of a call, expert by expert: edges[e] is expert
// e's first row (the offsets' running maximum, cut to m), tiles[e] the tiles
// before it; group n_experts holds the rows of no expert.  Filled by one warp;
// each table has n_experts + 2 entries.  With `slots` an expert has a tile also
// without rows, and slots[e] counts the tiles before it of experts that have
// more than one.
__device__ inline void fill_tables(const int32_t *offsets, int n_experts, int64_t m, int rows, int *edges, int *tiles,
                                   int *slots, int lane) {
    constexpr uint32_t all = 0xffffffffu;
    int last = 0, count = 0, taken = 0;
    if (lane == 0) {
        edges[0] = tiles[0] = 0;
        if (slots) slots[0] = 0;
    }
    for (int e0 = 0; e0 <= n_experts; e0 += 32) {
        const int e = e0 + lane;  // group e ends at edge e + 1
        int end = 0;
        if (e < n_experts) end = offsets ? max(0, (int)min((int64_t)offsets[e + 1], m)) : (int)m;
        if (e == n_experts) end = (int)m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) end = max(end, __shfl_up_sync(all, end, o));
        end = max(end, last);
        int start = __shfl_up_sync(all, end, 1);
        if (lane == 0) start = last;
        int t = (int)(((int64_t)end - start + rows - 1) / rows);
        if (slots) t = e < n_experts ? max(t, 1) : 0;
        int several = slots && t > 1 ? t : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(all, t, o), w = __shfl_up_sync(all, several, o);
            if (lane >= o) {
                t += v;
                several += w;
            }
        }
        t += count;
        several += taken;
        if (e <= n_experts) {
            edges[e + 1] = end;
            tiles[e + 1] = t;
            if (slots) slots[e + 1] = several;
        }
        last = __shfl_sync(all, end, 31);
        count = __shfl_sync(all, t, 31);
        taken = __shfl_sync(all, several, 31);
    }
}

// Most terms of a contraction in one accumulator.  The tensor cores cut off what
// a sum's last bit does not hold, some 6e-9 of it per term, so that 32768 terms
// lose up to 2e-4, half of float16's last bit, and 262144 would lose 1.7e-3.
// Longer contractions are sums of chunks that meet in float32.  In the forward
// and the rows product a pair goes through its unit's chunks one after the other
// and keeps their sum so far in the workspace, a tile per CTA.
constexpr int kChunk = 32768;
constexpr int kPairs = kSMs / 2;  // CTA pairs that run at once
constexpr int64_t kChunkTile = 128 * 256;  // values that a CTA has of a unit, at most
inline int64_t chunk_sums_bytes(int64_t contraction) {
    return contraction > kChunk ? 2 * kPairs * kChunkTile * 4 : 0;
}

// The weights product's contraction runs over an expert's rows, `chunk` of them
// (up to kChunk, fewer where few output tiles over many rows would leave most
// SMs idle) in one accumulator.  The chunks' sums of an expert with several meet
// in float32 in the workspace (`slots` matrices).
struct WeightsSplit {
    int chunk;
    int64_t slots;  // most partial matrices there can be; 0: every expert is one chunk
};
WeightsSplit weights_split(int64_t m, int64_t n, int64_t k, int64_t n_experts);

// A matrix whose rows all start on 16 bytes.
inline bool rows16(const void *base, int64_t pitch_elems) {
    return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && pitch_elems % 8 == 0;
}

// dst(r, c) = src(r, c) with the rows of dst on 16 bytes, pitch a multiple of 8.
cudaError_t launch_align(const void *src, int64_t pitch, int64_t rows, int64_t cols, void *dst, cudaStream_t s);

// The product on the tensor cores; w, x and dz must be rows16.  `clear`: the
// kernel is the call's first, so nothing has cleared the status word yet.
cudaError_t launch_linear_tc(Product mode, const LinearShape &sh, const Product16 &g, uint32_t *status, bool clear,
                             cudaStream_t s);

// The forward product of few rows per expert; x and w as they lie.
bool few_rows(const LinearShape &sh);
cudaError_t launch_linear_few(const LinearShape &sh, const Product16 &g, uint32_t *status, cudaStream_t s);

}  // namespace km
