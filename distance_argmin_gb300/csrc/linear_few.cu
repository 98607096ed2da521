// The forward product for few rows per expert: y = act(x W_e^T + b_e) + res
// where reading W is all that takes time.
//
// A unit is 16 features of one expert and up to 8 of its rows.  A block's 8
// warps share the contraction, 128 values (256 bytes of each feature) at a
// time: a lane loads 16 bytes of two features and of one row, which are operands
// of mma.m16n8k16 as they stand, because the order of the contraction inside an
// instruction is free as long as both operands use the same (words 0 and 1 of
// the lane's four make one instruction, words 2 and 3 the next).  The legacy
// MMA is enough here: one instruction per 512 bytes of W, far below its rate.
//
// W goes from memory to registers to the tensor cores, nothing is staged; what
// bounds it is how many bytes are on their way, 32 KB a block and four blocks
// an SM.  (A ring of cp.async slots per lane, filled across the ends of units,
// measured the same: 24 rows over 20 experts of 4096 x 2048 56 us against
// 55, 6.1 TB/s.)  Where there are few units for the SMs, a cluster of blocks splits each
// one's contraction, and the sums are joined through distributed shared memory
// (2048 features of 8192: 14.0 us without, 8.7 with).
//
// Rows that do not start on 16 bytes are read as shifted words (pieces.cuh)
// into registers, so W is never copied first.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "assign_common.cuh"
#include "linear_common.cuh"
#include "ptx.cuh"

namespace km {

namespace {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewFeatures = 16, kFewRows = 8;  // of one instruction
constexpr int kFewStep = 128;  // contraction of a warp's step
constexpr int kFewPieces = kFewStep / 32;
constexpr int kFewBlocks = 4;  // per SM
constexpr int kFewSplit = 8;   // most blocks of a cluster
static_assert(kFewRows * kFewFeatures == kFewThreads / 2, "half of the threads finish a unit");

struct FewParams {
    const int32_t *offsets;
    int64_t m;
    int n_experts, n, k, num_p;
    const uint8_t *w, *x;
    int64_t ldx;
    Span w_in, x_in;
    const void *bias, *residual;
    int64_t ldr;
    int activation;
    void *y, *pre;
    int split;  // blocks of a cluster that share a unit's contraction
    uint32_t *status;
};

template <typename T>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                  uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_cluster_f32(const float *p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_to_cta(smem_addr(p), rank)) : "memory");
    return v;
}

// The units in order: an expert's row tiles one after the other on the same
// features.
struct FewUnit {
    int e, f0, r0, rows;
};

__device__ __forceinline__ FewUnit few_unit(const FewParams &p, const int *edges, const int *tiles, int u, int &e) {
    while (u >= tiles[e + 1] * p.num_p) ++e;
    const int local = u - tiles[e] * p.num_p, per = tiles[e + 1] - tiles[e];
    const int feature = per == 1 ? local : local / per;
    FewUnit t;
    t.e = e;
    t.f0 = feature * kFewFeatures;
    t.r0 = edges[e] + (local - feature * per) * kFewRows;
    t.rows = min(kFewRows, edges[e + 1] - t.r0);
    return t;
}

template <bool WHOLE, typename T>
__global__ void __launch_bounds__(kFewThreads, WHOLE ? kFewBlocks : 2) linear_few_kernel(const FewParams p) {
    extern __shared__ int few_smem[];
    __shared__ float part[2][kFewWarps][kFewFeatures][kFewRows + 1];
    __shared__ float sums[2][kFewRows * kFewFeatures];  // of this block, for the cluster's first
    int *edges = few_smem, *tiles = edges + p.n_experts + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int split = p.split, crank = split > 1 ? (int)cluster_ctarank() : 0;
    griddep_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
    if (warp == 0) fill_tables(p.offsets, p.n_experts, p.m, kFewRows, edges, tiles, nullptr, lane);
    __syncthreads();
    const int total = tiles[p.n_experts + 1] * p.num_p;  // below 2^31: each is 16 rows of a matrix in memory
    const int first = blockIdx.x / split, stride = gridDim.x / split;
    const int kwarp = (crank * kFewWarps + warp) * kFewStep, kstride = split * kFewWarps * kFewStep;

    int e = 0, parity = 0;
    for (int u = first; u < total; u += stride, parity ^= 1) {
        const FewUnit t = few_unit(p, edges, tiles, u, e);
        const bool real = t.e < p.n_experts;
        float acc[4] = {};
        if (real) {
            const uint8_t *w0 = p.w + ((int64_t)t.e * p.n + t.f0 + g) * p.k * 2, *w1 = w0 + (int64_t)8 * p.k * 2;
            const bool on0 = t.f0 + g < p.n, on1 = t.f0 + g + 8 < p.n;
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 1
            for (int k0 = kwarp; k0 < p.k; k0 += kstride) {
                uint4 a[kFewPieces][2], b[kFewPieces];
#pragma unroll
                for (int i = 0; i < kFewPieces; ++i) {
                    const int k = k0 + 32 * i + t4 * 8, bytes = min(16, (p.k - k) * 2);
                    a[i][0] = on0 && bytes > 0 ? load_piece<WHOLE>(w0 + (int64_t)k * 2, bytes, p.w_in) : zero;
                    a[i][1] = on1 && bytes > 0 ? load_piece<WHOLE>(w1 + (int64_t)k * 2, bytes, p.w_in) : zero;
                    b[i] = g < t.rows && bytes > 0
                               ? load_piece<WHOLE>(p.x + (((int64_t)t.r0 + g) * p.ldx + k) * 2, bytes, p.x_in)
                               : zero;
                }
#pragma unroll
                for (int i = 0; i < kFewPieces; ++i) {
                    mma_16816<T>(acc, a[i][0].x, a[i][1].x, a[i][0].y, a[i][1].y, b[i].x, b[i].y);
                    mma_16816<T>(acc, a[i][0].z, a[i][1].z, a[i][0].w, a[i][1].w, b[i].z, b[i].w);
                }
            }
        }
        // The two copies of `part` alternate, and so do the half of the warps
        // that finishes a unit and the half that goes on with the next.
        part[parity][warp][g][2 * t4] = acc[0];
        part[parity][warp][g][2 * t4 + 1] = acc[1];
        part[parity][warp][g + 8][2 * t4] = acc[2];
        part[parity][warp][g + 8][2 * t4 + 1] = acc[3];
        __syncthreads();
        const int at_work = (int)threadIdx.x - parity * (kFewThreads / 2);
        const bool finishing = at_work >= 0 && at_work < kFewThreads / 2;
        if (split == 1 && !finishing) continue;
        const int f = at_work % kFewFeatures, r = at_work / kFewFeatures;
        const bool mine = finishing && r < t.rows && t.f0 + f < p.n;
        float z = 0.f, bias = 0.f;
        if (mine && crank == 0 && real && p.bias) bias = widen(static_cast<const T *>(p.bias)[(int64_t)t.e * p.n + t.f0 + f]);
        if (finishing) {
#pragma unroll
            for (int w = 0; w < kFewWarps; ++w) z += part[parity][w][f][r];
        }
        if (split > 1) {
            // the two halves of `sums` alternate: a unit's are read before the
            // next unit's barrier, and written again after it
            if (finishing) sums[parity][at_work] = z;
            cluster_sync();
            if (crank != 0 || !finishing) continue;
            z = 0.f;
            for (int c = 0; c < split; ++c) z += ld_cluster_f32(&sums[parity][at_work], (uint32_t)c);
        }
        if (mine) {
            const int64_t row = (int64_t)t.r0 + r, at = row * p.n + t.f0 + f;
            z += bias;
            if (p.pre) static_cast<T *>(p.pre)[at] = narrow<T>(z);
            float v = z;
            with_activation(p.activation, [&](auto a) { v = activate<decltype(a)::value>(z); });
            if (real && p.residual) v += widen(static_cast<const T *>(p.residual)[row * p.ldr + t.f0 + f]);
            static_cast<T *>(p.y)[at] = narrow<T>(v);
        }
    }
    if (split > 1) cluster_sync();  // no block leaves while its sums may still be read
}

template <bool WHOLE, typename T>
cudaError_t launch_few(const LinearShape &sh, FewParams p, cudaStream_t s) {
    const size_t smem = 2 * (size_t)(sh.n_experts + 2) * 4;
    // blocks that run at once
    const int64_t blocks = device_sm_count() * (int64_t)(WHOLE ? kFewBlocks : 2);
    // row tiles: at most, and about as many as rows that choose freely make
    const double n_e = (double)sh.n_experts, m = (double)sh.m;
    const int64_t most = sh.offsets ? (sh.m < sh.n_experts ? sh.m : sh.n_experts) + sh.m / kFewRows + 1 : 1;
    const double about = sh.offsets ? n_e * (1.0 - std::pow(1.0 - 1.0 / n_e, m)) + m / (2 * kFewRows * n_e) : 1.0;
    const int64_t units = (int64_t)(about * p.num_p + 0.5);
    // Split the contraction where that is sooner done: a block takes in some 11
    // bytes of W a nanosecond, a unit costs it 0.3 us besides and, split, 1.7 us
    // more for the cluster to meet.  Where a warp's accumulator would take more
    // than kChunk terms it is split in any case (few_rows ends at kFewSplit).
    p.split = 1;
    double best = INFINITY;
    for (int c = 1; c <= kFewSplit; c *= 2) {
        if (c > 1 && sh.k < (int64_t)c * kFewWarps * kFewStep) break;
        if (sh.k > (int64_t)c * kFewWarps * kChunk) continue;
        const int64_t clusters = blocks / c;
        const double each = (double)(kFewFeatures * 2 * sh.k) / c / 11.0 + (c > 1 ? 2000.0 : 300.0);
        const double cost = (double)((units + clusters - 1) / clusters) * each;
        if (cost < best) {
            best = cost;
            p.split = c;
        }
    }
    const int64_t clusters = blocks / p.split;
    const unsigned grid = (unsigned)((most * p.num_p < clusters ? most * p.num_p : clusters) * p.split);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2u : 1u;
    return cudaLaunchKernelEx(&cfg, linear_few_kernel<WHOLE, T>, p);
}

}  // namespace

// Where W is read once and little is done with it, up to 2^21 input features
// (kFewSplit blocks of kFewWarps accumulators of kChunk terms).  One expert: up to 8 rows
// (n = 8192, k = 2048: 8.1 us; the tensor-core units take 10.9 us for any
// number up to 24, 16 rows in two tiles of this kernel 11.2).  Several experts:
// their rows are not known here, so few of them on average; an expert with more
// reads its part of W again (from L2) every 8 rows (64 experts, n = 4096, k =
// 2048: 128 rows 159 us, 6.3 TB/s; 1024 rows 167 us in the tensor-core units).
bool few_rows(const LinearShape &sh) {
    return sh.k <= (int64_t)kFewSplit * kFewWarps * kChunk &&
           (sh.m <= kFewRows || (sh.offsets && sh.m <= 2 * (int64_t)sh.n_experts));
}

cudaError_t launch_linear_few(const LinearShape &sh, const Product16 &g, uint32_t *status, cudaStream_t s) {
    FewParams p{};
    p.offsets = sh.offsets;
    p.m = sh.m;
    p.n_experts = sh.n_experts;
    p.n = (int)sh.n;
    p.k = (int)sh.k;
    p.num_p = (int)((sh.n + kFewFeatures - 1) / kFewFeatures);
    p.w = static_cast<const uint8_t *>(g.a);
    p.x = static_cast<const uint8_t *>(g.b);
    p.ldx = g.ldb;
    p.w_in = {p.w, p.w + (int64_t)sh.n_experts * sh.n * sh.k * 2};
    p.x_in = {p.x, p.x + ((sh.m - 1) * g.ldb + sh.k) * 2};
    p.bias = g.bias;
    p.residual = g.residual;
    p.ldr = g.ldr;
    p.activation = g.activation;
    p.y = g.out;
    p.pre = g.pre;
    p.status = status;
    const bool whole = rows16(g.a, sh.k) && rows16(g.b, g.ldb);
    if (whole) return sh.bf16 ? launch_few<true, __nv_bfloat16>(sh, p, s) : launch_few<true, __half>(sh, p, s);
    return sh.bf16 ? launch_few<false, __nv_bfloat16>(sh, p, s) : launch_few<false, __half>(sh, p, s);
}

}  // namespace km
