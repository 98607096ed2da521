// The forward product for few rows per expert: y = act(x W_e^T + b_e) + res
// where reading W is all that takes time.
//
// A block takes 16 features of one expert and up to 8 NT of its rows.  Its 8
// warps share the contraction, 128 values (256 bytes of each feature) at a
// time: a lane loads 16 bytes of two features and of each row, which are
// operands of mma.m16n8k16 as they stand, because the order of the contraction
// inside an instruction is free as long as both operands use the same (words 0
// and 1 of the lane's four make one instruction, words 2 and 3 the next).  W
// goes from memory to registers to the tensor cores, nothing is staged; a
// block has 16 features of 128 x 8 values (32 KB) in flight at once.  The legacy MMA is enough here: one instruction per 32
// bytes of W loaded, far below its rate.  The warps' sums meet in shared
// memory, where bias, activation, residual and the rounding are applied.
//
// Rows that do not start on 16 bytes are read as shifted words (pieces.cuh), so
// W is never copied first.
#include <cuda_runtime.h>
#include <stdint.h>

#include "assign_common.cuh"
#include "linear_common.cuh"

namespace km {

namespace {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewFeatures = 16;
constexpr int kFewStep = 128;  // contraction of a warp's step
constexpr int kFewPieces = kFewStep / 32;

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

template <bool WHOLE, int NT, typename T>
__global__ void __launch_bounds__(kFewThreads, WHOLE && NT == 1 ? 4 : 2) linear_few_kernel(const FewParams p) {
    constexpr int ROWS = 8 * NT;
    extern __shared__ int few_smem[];
    __shared__ float part[kFewWarps][kFewFeatures][ROWS + 1];
    int *edges = few_smem, *tiles = edges + p.n_experts + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    griddep_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
    if (warp == 0) fill_tables<ROWS>(p.offsets, p.n_experts, p.m, edges, tiles, lane);
    __syncthreads();
    const int64_t total = (int64_t)tiles[p.n_experts + 1] * p.num_p;
    int e = 0;
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        while (u >= (int64_t)tiles[e + 1] * p.num_p) ++e;
        // an expert's row tiles one after the other on the same features
        const int64_t local = u - (int64_t)tiles[e] * p.num_p;
        const int per = tiles[e + 1] - tiles[e];
        const int f0 = (int)(local / per) * kFewFeatures;
        const int64_t r0 = edges[e] + (local % per) * ROWS;
        const int rows = (int)min((int64_t)ROWS, edges[e + 1] - r0);
        const bool real = e < p.n_experts;
        float acc[NT][4] = {};
        if (real) {
            const int64_t wrow = (int64_t)e * p.n + f0 + g;
            const uint8_t *w0 = p.w + wrow * p.k * 2, *w1 = w0 + (int64_t)8 * p.k * 2;
            const bool on0 = f0 + g < p.n, on1 = f0 + g + 8 < p.n;
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 1
            for (int k0 = warp * kFewStep; k0 < p.k; k0 += kFewWarps * kFewStep) {
                uint4 a[kFewPieces][2], b[kFewPieces][NT];
#pragma unroll
                for (int i = 0; i < kFewPieces; ++i) {
                    const int k = k0 + 32 * i + t4 * 8, bytes = min(16, (p.k - k) * 2);
                    a[i][0] = on0 && bytes > 0 ? load_piece<WHOLE>(w0 + (int64_t)k * 2, bytes, p.w_in) : zero;
                    a[i][1] = on1 && bytes > 0 ? load_piece<WHOLE>(w1 + (int64_t)k * 2, bytes, p.w_in) : zero;
#pragma unroll
                    for (int q = 0; q < NT; ++q)
                        b[i][q] = 8 * q + g < rows && bytes > 0
                                      ? load_piece<WHOLE>(p.x + ((r0 + 8 * q + g) * p.ldx + k) * 2, bytes, p.x_in)
                                      : zero;
                }
#pragma unroll
                for (int i = 0; i < kFewPieces; ++i)
#pragma unroll
                    for (int q = 0; q < NT; ++q) {
                        mma_16816<T>(acc[q], a[i][0].x, a[i][1].x, a[i][0].y, a[i][1].y, b[i][q].x, b[i][q].y);
                        mma_16816<T>(acc[q], a[i][0].z, a[i][1].z, a[i][0].w, a[i][1].w, b[i][q].z, b[i][q].w);
                    }
            }
        }
        __syncthreads();  // the previous unit's sums have been read
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            part[warp][g][8 * q + 2 * t4] = acc[q][0];
            part[warp][g][8 * q + 2 * t4 + 1] = acc[q][1];
            part[warp][g + 8][8 * q + 2 * t4] = acc[q][2];
            part[warp][g + 8][8 * q + 2 * t4 + 1] = acc[q][3];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kFewFeatures * rows; i += kFewThreads) {
            const int f = i % kFewFeatures, r = i / kFewFeatures;
            if (f0 + f >= p.n) continue;
            float z = 0.f;
#pragma unroll
            for (int w = 0; w < kFewWarps; ++w) z += part[w][f][r];
            const int64_t at = (r0 + r) * p.n + f0 + f;
            if (real && p.bias) z += widen(static_cast<const T *>(p.bias)[(int64_t)e * p.n + f0 + f]);
            if (p.pre) static_cast<T *>(p.pre)[at] = narrow<T>(z);
            float v = z;
            with_activation(p.activation, [&](auto a) { v = activate<decltype(a)::value>(z); });
            if (real && p.residual) v += widen(static_cast<const T *>(p.residual)[(r0 + r) * p.ldr + f0 + f]);
            static_cast<T *>(p.y)[at] = narrow<T>(v);
        }
    }
}

template <int NT, typename T>
cudaError_t launch_few(const LinearShape &sh, const FewParams &p, bool whole, cudaStream_t s) {
    const int64_t tiles = (sh.m + 8 * NT - 1) / (8 * NT) + (sh.offsets ? sh.n_experts : 0);
    const int64_t units = tiles * p.num_p, most = (int64_t)device_sm_count() * 4;
    const size_t smem = 2 * (size_t)(sh.n_experts + 2) * 4;
    return launch_kernel(true, whole ? linear_few_kernel<true, NT, T> : linear_few_kernel<false, NT, T>,
                         dim3((unsigned)(units < most ? units : most)), dim3(kFewThreads), smem, s, p);
}

}  // namespace

// Where W is read once and little is done with it.  One expert: up to 16 rows,
// two tiles of one instruction's 8 (n = 8192, k = 2048: 1 or 8 rows 8.1 us, 16
// rows 11.2, where the tensor-core units take 15.3 us for any number up to 64).
// Several experts: their rows are not known here, so few of them on average; an
// expert with more reads its part of W again (from L2) every 8 rows (64
// experts, n = 4096, k = 2048: 128 rows 159 us, 6.3 TB/s; 256 rows 207 us in
// tiles of 16, and 1024 rows 167 us in the tensor-core units).
bool few_rows(const LinearShape &sh) { return sh.offsets ? sh.m <= 2 * (int64_t)sh.n_experts : sh.m <= 16; }

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
    const bool one = sh.offsets || sh.m <= 8;
    if (sh.bf16) return one ? launch_few<1, __nv_bfloat16>(sh, p, whole, s) : launch_few<2, __nv_bfloat16>(sh, p, whole, s);
    return one ? launch_few<1, __half>(sh, p, whole, s) : launch_few<2, __half>(sh, p, whole, s);
}

}  // namespace km
