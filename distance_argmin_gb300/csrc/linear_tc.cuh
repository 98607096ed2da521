// The experts' products on the sm_103a tensor cores: the kernel, its variants for
// the cross entropy (see Product) among them, and its launch.
//
// All three products are out(q, p) = sum_c A(p, c) B(q, c) with p contiguous in
// the output (see linear_common.cuh).  The output's contiguous dimension is
// always the MMA's M: 256 wide per CTA pair, and the rows are its N, 32 to 256
// in steps of 32.  A group of few rows then costs an MMA of few columns, and
// each tensor-memory lane holds one output feature, so that a warp's 32 lanes
// are 32 neighbours in memory.
//
//              A (M = p)              B (N = q)            contraction
//   forward    W_e, K-major           x,  K-major          input features
//   rows       W_e, M contiguous      dz, K-major          output features
//   weights    x,   M contiguous      dz, N contiguous     the expert's rows
//
// Everything is loaded by TMA with the 128-byte swizzle; an operand whose
// contiguous dimension is not the contraction is fed to the MMA as it lies in
// memory (the descriptor's other major mode), so nothing is transposed.
// Ragged edges: the contraction's tail is the tensor maps' zero fill (W is a
// 3-D map, so an expert's last features never run into the next expert's);
// rows of the next expert that a tile of B covers are columns the epilogue does
// not store; and where the rows are the contraction (weights) the relay warp
// clears the rows past the expert's end in shared memory, in both operands
// (a zero times another expert's infinity would be NaN).
//
// Structure: CTA pairs (cta_group::2), persistent over the units (256 features
// x BN rows), a band of 8 feature tiles at a time so that the pairs running
// together share rows and features in L2.
//   warps 0-15  epilogue: tensor memory -> registers -> a padded shared-memory
//               tile per warp -> rows of 32 neighbouring features: bias,
//               activation, residual, one rounding, 16-byte stores
//   warp 16     TMA producer (each CTA: its half of A and of B)
//   warp 17     allocates tensor memory; in the even CTA issues the MMAs
//   warp 18     (weights) relay: sees this CTA's stage land, clears rows if
//               needed, and tells the even CTA; the row products' loads count
//               on the even CTA's barrier by themselves
// Two accumulators alternate, so a unit's epilogue overlaps the next one's
// MMAs.  Every wait is bounded as in the assignment.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "assign_common.cuh"
#include "linear_common.cuh"
#include "ptx.cuh"
#include "tensor_map.cuh"

namespace km {

namespace lt {
constexpr int BP = 256;            // features per unit (UMMA M of the pair)
constexpr int BP_CTA = BP / 2;
constexpr int BK = 64;             // contraction per stage: 128 bytes of 16-bit values
constexpr int CHUNK_BLOCKS = kChunk / BK;
constexpr int LOG_BLOCKS = 512 / BK;  // of an accumulator of the log sums
constexpr int EPI_WARPS = 16;       // four per tensor-memory lane quarter, a quarter of the columns each
constexpr int WARP_TMA = EPI_WARPS, WARP_MMA = WARP_TMA + 1, WARP_RELAY = WARP_TMA + 2;
constexpr int THREADS = (WARP_RELAY + 1) * 32;
constexpr int EPI_ROWS = 8;        // rows staged at a time per epilogue warp
constexpr int EPI_PITCH = 36;      // floats: 8 rows x 32 bytes then hit distinct banks
constexpr int STAGING = EPI_WARPS * EPI_ROWS * EPI_PITCH * 4;
constexpr int BAND = 8;            // feature tiles per raster band
constexpr int LIST_UNITS = 32;     // units a warp works out at a time
constexpr int LIST_BYTES = LIST_UNITS * 28;
constexpr int SMEM_LIMIT = 232448;
constexpr int BAR_BYTES = 512;

constexpr int PARTS = EPI_WARPS / 4;  // groups of four epilogue warps, one per lane quarter
constexpr int STORE_ROWS = 16;        // rows of a bulk store (weights): two buffers of 16 x 256 bytes per part
constexpr int STORE_BYTES = STORE_ROWS * BP_CTA * 2;

template <int BN, bool STORES = false>
struct Cfg {
    static constexpr int A_BYTES = BP_CTA * BK * 2;
    static constexpr int B_BYTES = BN / 2 * BK * 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = STORES ? (BN >= 256 ? 5 : 6) : BN >= 256 ? 6 : BN >= 128 ? 8 : 9;
    static constexpr int STAGING_BASE = STAGES * STAGE;
    static constexpr int BAR_BASE = STAGING_BASE + (STORES ? PARTS * 2 * STORE_BYTES : STAGING);
    static constexpr int LIST_BASE = BAR_BASE + BAR_BYTES;
    static constexpr int TABLE_BASE = LIST_BASE + 3 * LIST_BYTES;
    static constexpr int TMEM_COLS = 2 * BN;  // >= 64
    static constexpr int FULL = 0, READY = STAGES, EMPTY = 2 * STAGES, T_FULL = 3 * STAGES, T_EMPTY = T_FULL + 2,
                         DRAIN = T_EMPTY + 2, NUM_BARS = DRAIN + 1;
    static constexpr int TABLES = STORES ? 5 : 2;  // of the experts, see the kernel
    static constexpr int smem_bytes(int n_experts) { return TABLE_BASE + TABLES * (n_experts + 2) * 4 + 1024; }
    static_assert(NUM_BARS * 8 + 16 <= BAR_BYTES, "barriers fit");
    static_assert(STAGE % 1024 == 0 && STAGING % 1024 == 0, "stages stay 1 KiB aligned");
    static_assert(TABLE_BASE + TABLES * (KMEANS_LINEAR_MAX_EXPERTS + 2) * 4 + 1024 <= SMEM_LIMIT, "fits");
};
}  // namespace lt

struct LinearTcParams {
    const int32_t *offsets;
    int64_t m;
    int n_experts;
    int cols;         // size of the output's contiguous dimension
    int num_p;        // feature tiles
    int out_rows;     // weights: output features of an expert
    int chunk;        // weights: rows of a unit's contraction at most
    float *partial;
    void *db;         // weights: the bias gradient and the sums it is joined from
    const float *bias_sums;
    int bias_rows;
    int contraction;  // forward, rows
    const void *bias, *residual;
    int64_t ldr;
    int activation;
    void *out, *pre;
    int wide;  // the rows of the outputs and the residual start on 16 bytes
    uint32_t *status;
    int test_starve;  // test hook: the producer issues no loads, so the pipeline waits run out
    int clear;  // first kernel of the call: each pair has a status word of its own
    EntropyArgs entropy;
};

// Rows, features and their tiles are 32-bit: the sizes end KMEANS_LINEAR_MAX_SIZE,
// a tile below 2^31, so that no tile's end or box of rows passes it.
//
// The units: expert by expert, bands of BAND feature tiles, in a band the
// feature tiles of one row tile after the other (edges and tiles: see
// fill_tables).
struct Unit {
    int expert, p0, q0, qn;  // q0: first output row (row products: of the matrix, weights: of the expert)
    int c0, c1;              // contraction range (rows of x for weights)
    int slot;                // weights: the partial matrix this chunk of rows goes to (-1: the output);
                             // log sum: the row tile; sum: the contraction's part

    __device__ __forceinline__ Unit of_lane(int l) const {
        const auto from = [l](int v) { return __shfl_sync(0xffffffffu, v, l); };
        return {from(expert), from(p0), from(q0), from(qn), from(c0), from(c1), from(slot)};
    }
};

// (There are fewer than 2^31 units: each is 64 rows x 256 features or more of
// a matrix in memory.)
template <Product MODE, int BN>
struct Units {
    const LinearTcParams &p;
    const int *edges, *tiles, *slots;
    int total;
    int e = 0;
    int live = 0;  // log sum: feature tiles of the rows that count

    __device__ Units(const LinearTcParams &p_, const int *edges_, const int *tiles_, const int *slots_)
        : p(p_), edges(edges_), tiles(tiles_), slots(slots_) {
        if (MODE == Product::kLogSum) live = (*p.entropy.count + lt::BP - 1) / lt::BP;
        // (rows of no expert get zeros, but for the cross entropy, which has none of them)
        const bool rest = MODE == Product::kForward || MODE == Product::kRows || is_weights(MODE);
        total = tiles[p.n_experts + (rest ? 1 : 0)] * num_p() * (is_weights(MODE) ? row_tiles() : 1);
        if (MODE == Product::kRowsSum) total *= p.entropy.splits;
    }
    __device__ __forceinline__ int num_p() const {
        if constexpr (MODE == Product::kLogSum)
            return live;
        else
            return p.num_p;
    }
    __device__ int row_tiles() const { return (p.out_rows + BN - 1) / BN; }

    // `u` never decreases from call to call.
    __device__ Unit at(int u) {
        int per, chunk = 0;
        if (is_weights(MODE)) {
            per = row_tiles();
            const int g = u / (per * num_p());  // chunk of rows, over all experts
            while (g >= tiles[e + 1]) ++e;
            chunk = g - tiles[e];
            u -= g * per * num_p();
        } else {
            if (MODE == Product::kRowsSum) {  // part after part of the contraction
                chunk = u / (tiles[1] * num_p());
                u -= chunk * (tiles[1] * num_p());
            }
            while (u >= tiles[e + 1] * num_p()) ++e;
            u -= tiles[e] * num_p();
            per = tiles[e + 1] - tiles[e];
        }
        const int band = u / (lt::BAND * per), r = u - band * (lt::BAND * per);
        const int wide = min(lt::BAND, num_p() - band * lt::BAND);
        const int q = r / wide;
        Unit t;
        t.expert = e;
        t.p0 = (band * lt::BAND + r - q * wide) * lt::BP;
        if (is_weights(MODE)) {
            t.q0 = q * BN;
            t.qn = min(BN, p.out_rows - t.q0);
            t.c0 = edges[e] + chunk * p.chunk;
            t.c1 = t.c0 + min(edges[e + 1] - t.c0, p.chunk);  // (c0 + chunk may pass 2^31)
            t.slot = tiles[e + 1] - tiles[e] > 1 ? slots[e] + chunk : -1;
        } else {
            // an expert's rows in equal parts (multiples of 32) rather than full
            // ones and a rest: a stage of few rows takes more than its share,
            // and the pairs' turns come out more even (16384 ragged rows of 30
            // experts, dx of 4096 x 2048: 186 us with full ones, 174 so)
            const int rows = edges[e + 1] - edges[e];
            const int step = min(BN, ((rows - 1) / per + 32) & ~31);
            t.q0 = edges[e] + q * step;
            t.qn = min(step, edges[e + 1] - t.q0);
            if (MODE == Product::kLogSum) t.slot = q;
            t.c0 = 0;
            t.c1 = e < p.n_experts ? p.contraction : 0;
            if (MODE == Product::kRowsSum) {
                const int part = ((p.contraction - 1) / p.entropy.splits / lt::BK + 1) * lt::BK;
                t.slot = chunk;
                t.c0 = chunk * part;
                t.c1 = min(t.c0 + part, p.contraction);
            }
        }
        return t;
    }
};

// One warp's columns [c0, end) of a unit, 8 rows of 32 features at a time:
// accumulator -> staged rows -> memory.  In memory's order lane group l / 4 has
// a row, lane l % 4 eight of its features.  The residual of all the columns is
// asked for before the accumulator is waited for, so its latency passes behind
// the unit's MMAs, and the next chunk's accumulator is on its way while one is
// finished.  Rows that do not start on 16 bytes go straight from the
// accumulator's layout, 32 neighbouring features of a row at a time, with the
// residual asked for in the same layout as early (run_direct: 19456 x 4095 of 64
// products each 4.0 us a round of units, with a residual 13; it asked for late
// 34, and by 4-byte words out of staged rows 11 and 30.  For aligned rows it is
// slower: dense 8192 x 8192 x 2048 170 us against 164, and one bulk copy per row
// of 128 features 174).
// Up to some 600 products per output the epilogue sets the pace, not the tensor
// pipe.  Each SM then finishes 128 x 256 values, of a long matrix with 64 products
// each, say, in 2.8 us without an activation and 3.8 with GELU: shared memory 64%
// and issue 40 to 70% busy.  (Without the path for parts whose rows all exist, and with
// activations one value at a time, 3.0 and 4.8 us; 16 or 32 accumulator columns
// per load 3.1 and 3.5.)
template <Product MODE, int BN, typename T>
struct Finish {
    static constexpr int COLS = BN / (lt::EPI_WARPS / 4), CHUNKS = COLS / lt::EPI_ROWS;
    static constexpr bool FORWARD = MODE == Product::kForward;
    const LinearTcParams &p;
    float *staged;
    int lane;
    int c0, end, f;   // f: the warp's first feature
    int64_t out_row;  // of the unit's column 0
    bool add;
    uint4 res[FORWARD ? CHUNKS : 1];
    float factor = 1.f;  // scaled

    __device__ int f8() const { return f + (lane & 3) * 8; }

    __device__ void prefetch() {
        if constexpr (FORWARD) {
            if (!add) return;
            if (!p.wide) {  // a lane's feature of two rows to a word
                if (f + lane >= p.cols) return;
                const uint16_t *at = static_cast<const uint16_t *>(p.residual) + (out_row + c0) * p.ldr + f + lane;
#pragma unroll
                for (int i = 0; i < CHUNKS; ++i) {
                    uint32_t v[8];
#pragma unroll
                    for (int j = 0; j < lt::EPI_ROWS; ++j, at += p.ldr)
                        v[j] = c0 + i * lt::EPI_ROWS + j < end ? *at : 0;
                    res[i] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
                }
                return;
            }
            if (f8() >= p.cols) return;
            const T *at = static_cast<const T *>(p.residual) + (out_row + c0 + (lane >> 2)) * p.ldr + f8();
            const int64_t step = lt::EPI_ROWS * p.ldr;
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i, at += step)
                if (c0 + i * lt::EPI_ROWS + (lane >> 2) < end) res[i] = *reinterpret_cast<const uint4 *>(at);
        }
    }

    __device__ __forceinline__ static void store8(void *out, int64_t at, const float2 (&v)[4]) {
        *reinterpret_cast<uint4 *>(static_cast<T *>(out) + at) =
            make_uint4(narrow2<T>(v[0].x, v[0].y), narrow2<T>(v[1].x, v[1].y), narrow2<T>(v[2].x, v[2].y),
                       narrow2<T>(v[3].x, v[3].y));
    }

    template <int ACT>
    __device__ __forceinline__ void run(uint32_t acc, float bias, bool zero) {
        if (end - c0 == COLS && f + 32 <= p.cols && !zero)
            run_rows<ACT, true>(acc, bias, false);
        else
            run_rows<ACT, false>(acc, bias, zero);
    }

    // FULL: every row and feature of the warp's part exists.
    template <int ACT, bool FULL>
    __device__ void run_rows(uint32_t acc, float bias, bool zero) {
        const int row = c0 + (lane >> 2);
        const bool mine = FULL || f8() < p.cols;  // all eight: cols is a multiple of 8 here
        const int64_t step = (int64_t)lt::EPI_ROWS * p.cols;
        int64_t at = (out_row + row) * p.cols + f8();
        const float *src = staged + (lane >> 2) * lt::EPI_PITCH + (lane & 3) * 8;
        uint32_t r[8] = {};
        if (!zero) tmem_ld_8_issue(acc + (uint32_t)c0, r);
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i, at += step) {
            if (!FULL && c0 + i * lt::EPI_ROWS >= end) break;
            if (i) __syncwarp();  // the previous rows have been read; the warp is together again
            if (!zero) tmem_ld_8_wait(r);
#pragma unroll
            for (int j = 0; j < lt::EPI_ROWS; j += 2) {
                float2 v = __fadd2_rn(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), both(bias));
                if constexpr (MODE == Product::kWeightsScaled) v = __fmul2_rn(v, both(factor));
                staged[j * lt::EPI_PITCH + lane] = v.x;
                staged[(j + 1) * lt::EPI_PITCH + lane] = v.y;
            }
            __syncwarp();
            if (!zero && i + 1 < CHUNKS && (FULL || c0 + (i + 1) * lt::EPI_ROWS < end))
                tmem_ld_8_issue(acc + (uint32_t)(c0 + (i + 1) * lt::EPI_ROWS), r);
            if (!FULL && (row + i * lt::EPI_ROWS >= end || !mine)) continue;
            const float4 lo = *reinterpret_cast<const float4 *>(src), hi = *reinterpret_cast<const float4 *>(src + 4);
            float2 v[4] = {{lo.x, lo.y}, {lo.z, lo.w}, {hi.x, hi.y}, {hi.z, hi.w}};
            if constexpr (FORWARD) {
                if (p.pre) store8(p.pre, at, v);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = activate2<ACT>(v[k]);
                if (add) {
                    const uint32_t words[4] = {res[i].x, res[i].y, res[i].z, res[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = __fadd2_rn(v[k], widen2<T>(words[k]));
                }
            }
            store8(p.out, at, v);
        }
    }

    // A lane keeps its feature; any alignment.
    template <int ACT>
    __device__ __forceinline__ void run_direct(uint32_t acc, float bias, bool zero) {
        const bool mine = f + lane < p.cols;
        const int64_t at0 = (out_row + c0) * p.cols + f + lane;
        T *out = static_cast<T *>(p.out) + at0, *pre = FORWARD && p.pre ? static_cast<T *>(p.pre) + at0 : nullptr;
        uint32_t r[8] = {};
        if (!zero) tmem_ld_8_issue(acc + (uint32_t)c0, r);
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int c = c0 + i * lt::EPI_ROWS;
            if (c >= end) break;
            __syncwarp();
            if (!zero) tmem_ld_8_wait(r);
            float2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = __fadd2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), both(bias));
                if constexpr (MODE == Product::kWeightsScaled) v[j] = __fmul2_rn(v[j], both(factor));
            }
            if (!zero && i + 1 < CHUNKS && c + lt::EPI_ROWS < end) tmem_ld_8_issue(acc + (uint32_t)(c + lt::EPI_ROWS), r);
            if (FORWARD && pre) {
                store_rows(pre, v, c, mine);
                pre += (int64_t)lt::EPI_ROWS * p.cols;
            }
            if constexpr (FORWARD) {
                const uint32_t words[4] = {res[i].x, res[i].y, res[i].z, res[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = activate2<ACT>(v[j]);
                    if (add) v[j] = __fadd2_rn(v[j], widen2<T>(words[j]));
                }
            }
            store_rows(out, v, c, mine);
            out += (int64_t)lt::EPI_ROWS * p.cols;
        }
    }

    // A lane's feature of the rows c, c + 1, ..
    __device__ __forceinline__ void store_rows(T *at, const float2 (&v)[4], int c, bool mine) const {
#pragma unroll
        for (int j = 0; j < lt::EPI_ROWS; ++j, at += p.cols)
            if (mine && c + j < end) *at = narrow<T>(j & 1 ? v[j / 2].y : v[j / 2].x);
    }
};

// The weights product's output has no ragged rows and is the call's largest
// traffic, so here a part (four warps, one per lane quarter) rounds 16 rows of
// its 128 features into shared memory and one lane sends them off as two bulk
// tensor stores, whole lines that end at the matrix's edges by themselves.  The
// accumulator is read as MMA fragments, which stmatrix transposes into rows in
// the 128-byte swizzle.  (64 experts of 4096 x 2048 over 4096 rows, 1.07 GB
// written: 265 us with Finish, 236 with 2-byte stores into the same buffers,
// 211 as it stands; the same way out for the row products, whose last rows
// cannot leave by bulk stores, was no faster than Finish.)
template <typename T, bool SCALED>
__device__ __forceinline__ void store_part(const LinearTcParams &p, const CUtensorMap *tmOut, uint8_t *buffers, int &ring,
                                           uint32_t acc, int part, int quarter, int lane, int f, int q, int end,
                                           int expert, bool zero, float factor) {
    // stmatrix: lane l addresses row l % 8 of matrix l / 8; the matrices of half
    // h (16 of the warp's features) are rows 0-7 of features 0-7 and 8-15, then
    // rows 8-15 of both
    const int m = lane >> 3, row = (m >> 1) * 8 + (lane & 7);
    const uint32_t at = (uint32_t)((quarter >> 1) * (lt::STORE_ROWS * 128) + row * 128);
    const uint32_t chunk = (uint32_t)((quarter & 1) * 4 + (m & 1));
    for (int c = 0; c < end; c += lt::STORE_ROWS) {
        uint32_t r[2][8] = {};
        if (!zero) {
            tmem_ld_frag_issue(acc + (uint32_t)c, r[0]);
            tmem_ld_frag_issue(acc + (uint32_t)c + (16u << 16), r[1]);
            tmem_ld_8_wait(r[0]);
            tmem_ld_8_wait(r[1]);
        }
        const uint32_t buf = smem_addr(buffers + ring * lt::STORE_BYTES);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float2 v = make_float2(__uint_as_float(r[h][2 * k]), __uint_as_float(r[h][2 * k + 1]));
                if constexpr (SCALED) v = __fmul2_rn(v, both(factor));
                w[k] = narrow2<T>(v.x, v.y);
            }
            stmatrix_trans(buf + at + (((chunk + 2 * h) ^ (uint32_t)(row & 7)) << 4), w[0], w[1], w[2], w[3]);
        }
        // the stores out of the other buffer have read it: it may be written
        // once everyone has passed this barrier
        fence_proxy_async_smem();
        if (quarter == 0 && lane == 0) bulk_wait_read();
        named_barrier(1 + part, 128);
        if (quarter == 0 && lane == 0) {
            tma_store_3d(tmOut, buf, f, q + c, expert);
            if (f + 64 < p.cols) tma_store_3d(tmOut, buf + lt::STORE_ROWS * 128, f + 64, q + c, expert);
            bulk_commit();
        }
        __syncwarp();
        ring ^= 1;
    }
}

// The logits of the log sums are results in float32, whose last bits an
// accumulator of thousands of terms would cut off (see kChunk: 2048 terms left
// losses 1.5e-6 off, a float32 product 6e-7).  So their contraction goes through
// the two accumulators in chunks of 512 terms, which an epilogue warp adds up in
// registers: COLS columns from `acc` on.  The accumulators are free again before
// the exponentials begin.  Returns the count of accumulator uses, or -1 where a
// wait gave up.
template <int BN, int COLS, typename Status>
__device__ __forceinline__ int sum_logits(float (&v)[COLS], uint32_t acc, uint32_t full, uint32_t empty, int blocks, int use,
                                          const Status &status) {
    const auto chunk = [&](auto first) {
        const uint32_t buf = (uint32_t)use & 1u;
        if (!mbar_wait_warp(full + 8 * buf, (use >> 1) & 1, status)) return false;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < COLS; c += 8) {
            uint32_t r[8];
            tmem_ld_8_issue(acc + buf * BN + (uint32_t)c, r);
            tmem_ld_8_wait(r);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[c + j] = decltype(first)::value ? __uint_as_float(r[j]) : v[c + j] + __uint_as_float(r[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane_id() == 0) mbar_arrive_cluster(empty + 8 * buf);
        ++use;
        blocks -= lt::LOG_BLOCKS;
        return true;
    };
    if (!chunk(std::true_type{})) return -1;
#pragma unroll 1
    while (blocks > 0)
        if (!chunk(std::false_type{})) return -1;
    return use;
}

// Log sum: a lane has a row and `count` classes of it: the largest factor * z and
// the sum of the exponentials about it, in powers of two.  Where the largest is
// infinite they are taken about 0, so that the sum says what it is (0, infinite or
// NaN), and where it is minus infinity (closed classes, or none) that is the
// reference that leaves: (-inf, 0) counts for nothing beside other parts, however
// small their logits.  `label`: the row's, from the first class on.
template <int COLS>
__device__ __forceinline__ void log_sum(const EntropyArgs &g, float (&v)[COLS], int count, int64_t row, bool mine,
                                        int label, int part) {
    float high = -INFINITY;
    if (count < COLS) {
#pragma unroll
        for (int j = 0; j < COLS; ++j)
            if (j >= count) v[j] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < COLS; ++j) high = fmaxf(high, v[j]);
    if (__any_sync(0xffffffffu, (unsigned)label < (unsigned)COLS)) {
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < COLS; ++j)
            if (label == j) z = v[j];
        if (mine && (unsigned)label < (unsigned)COLS && label < count) g.target[row] = z;
    }
    const float top = high * g.factor, ref = isinf(top) ? 0.f : top;
    float2 sum = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < COLS; j += 2) {
        const float2 x = __ffma2_rn(make_float2(v[j], v[j + 1]), both(g.factor), both(-ref));
        sum = __fadd2_rn(sum, make_float2(exp2_approx(x.x), exp2_approx(x.y)));
    }
    if (mine) g.stats[part * g.pitch + row] = make_float2(top == -INFINITY ? top : ref, sum.x + sum.y);
}

// The same of few rows: a lane has a class, v[j] is row q0 + j (of `count`), and the
// warp's 32 classes from f on meet by shuffles; a row's parts are neighbours.
template <int COLS>
__device__ __forceinline__ void log_sum_few(const LinearTcParams &p, const float (&v)[COLS], int count, int f, int lane,
                                            int64_t q0) {
    const EntropyArgs &g = p.entropy;
    const bool real = f + lane < p.cols;
    const int label = lane < count ? g.rows[q0 + lane].label : -1;
    float2 mine = {-INFINITY, 0.f};  // lane j: row q0 + j
#pragma unroll
    for (int j = 0; j < COLS; ++j) {
        const float z = v[j];
        const int at = __shfl_sync(0xffffffffu, label, j);
        if (at == f + lane) g.target[q0 + j] = z;
        // (NaN is left out of the largest, and shows in the sum)
        const float x = real ? z * g.factor : -INFINITY;
        const float top = ord_to_float(__reduce_max_sync(0xffffffffu, x == x ? float_to_ord(x) : 0x007fffffu));
        const float ref = isinf(top) ? 0.f : top;
        float sum = real ? exp2_approx(fmaf(z, g.factor, -ref)) : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == j) mine = make_float2(top == -INFINITY ? top : ref, sum);
    }
    if (lane < count) g.stats[(q0 + lane) * g.pitch + (f >> 5)] = mine;
}

// Softmax: as Finish, a lane with eight classes of a row, whose record is asked for
// before the accumulator is waited for.  The matrix is rounded to the products'
// type, as dz is everywhere; times a power of two (in the records' gradient), so
// that float16 has room for small probabilities.
template <int BN, typename T>
struct FinishSoftmax {
    static constexpr int COLS = BN / (lt::EPI_WARPS / 4), CHUNKS = COLS / lt::EPI_ROWS;
    const LinearTcParams &p;
    float *staged;
    int lane;
    int c0, end, f;
    int64_t out_row;
    EntropyRow rows[CHUNKS];

    __device__ int f8() const { return f + (lane & 3) * 8; }

    __device__ void prefetch() {
        const EntropyRow *at = p.entropy.rows + out_row + c0 + (lane >> 2);
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i)
            if (c0 + i * lt::EPI_ROWS + (lane >> 2) < end) rows[i] = at[i * lt::EPI_ROWS];
    }

    __device__ __forceinline__ void run(uint32_t acc) {
        const int row = c0 + (lane >> 2);
        const bool mine = f8() < p.cols;
        // (the row is padded to whole pieces, and what the padding holds is not read)
        T *out = static_cast<T *>(p.out) + (out_row + row) * p.entropy.pitch + f8();
        const float *src = staged + (lane >> 2) * lt::EPI_PITCH + (lane & 3) * 8;
        const float factor = p.entropy.factor;
        uint32_t r[8];
        tmem_ld_8_issue(acc + (uint32_t)c0, r);
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i, out += lt::EPI_ROWS * p.entropy.pitch) {
            if (c0 + i * lt::EPI_ROWS >= end) break;
            if (i) __syncwarp();
            tmem_ld_8_wait(r);
#pragma unroll
            for (int j = 0; j < lt::EPI_ROWS; ++j) staged[j * lt::EPI_PITCH + lane] = __uint_as_float(r[j]);
            __syncwarp();
            if (i + 1 < CHUNKS && c0 + (i + 1) * lt::EPI_ROWS < end)
                tmem_ld_8_issue(acc + (uint32_t)(c0 + (i + 1) * lt::EPI_ROWS), r);
            if (row + i * lt::EPI_ROWS >= end || !mine) continue;
            const float4 lo = *reinterpret_cast<const float4 *>(src), hi = *reinterpret_cast<const float4 *>(src + 4);
            float2 v[4] = {{lo.x, lo.y}, {lo.z, lo.w}, {hi.x, hi.y}, {hi.z, hi.w}};
            const float ref = -rows[i].lse2;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = __ffma2_rn(v[k], both(factor), both(ref));
                v[k] = make_float2(exp2_approx(v[k].x), exp2_approx(v[k].y));
            }
            const int at = rows[i].label - p.entropy.first - f8();
            if ((unsigned)at < 8u) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (at == 2 * k) v[k].x -= 1.f;
                    if (at == 2 * k + 1) v[k].y -= 1.f;
                }
            }
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = __fmul2_rn(v[k], both(rows[i].gradient));
                w[k] = narrow2<T>(v[k].x, v[k].y);
            }
            *reinterpret_cast<uint4 *>(out) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// Sum: a warp's columns as rows of 32 neighbouring features, added to what the
// pieces before have left in float32; the last piece rounds once and goes to the
// rows' own places, unless the contraction is split: then the parts' sums meet
// after the last piece.  `none`: no term in this piece's part.
template <typename T>
__device__ __forceinline__ void add_sums(const LinearTcParams &p, uint32_t acc, int c0, int end, int f, int64_t row0,
                                         int lane, float factor, int part, bool none) {
    const EntropyArgs &g = p.entropy;
    const bool mine = f + lane < p.cols, last = g.last && g.splits == 1;
    float *sums = g.sums + part * g.split_stride + (row0 + c0) * p.cols + f + lane;
    T *out = static_cast<T *>(p.out) + f + lane;
#pragma unroll 1
    for (int c = c0; c < end; c += lt::EPI_ROWS, sums += (int64_t)lt::EPI_ROWS * p.cols) {
        uint32_t r[8] = {};
        float v[8];
        __syncwarp();
        if (!none) tmem_ld_8_issue(acc + (uint32_t)c, r);
#pragma unroll
        for (int j = 0; j < lt::EPI_ROWS; ++j) v[j] = !g.begin && mine && c + j < end ? sums[(int64_t)j * p.cols] : 0.f;
        if (!none) tmem_ld_8_wait(r);
#pragma unroll
        for (int j = 0; j < lt::EPI_ROWS; ++j) {
            if (!mine || c + j >= end) continue;
            v[j] += __uint_as_float(r[j]);
            if (last)
                out[(int64_t)g.rows[row0 + c + j].source * p.cols] = narrow<T>(v[j] * (factor * g.share[row0 + c + j]));
            else
                sums[(int64_t)j * p.cols] = v[j];
        }
    }
}

// One chunk's sums of a unit, as they are: a warp's columns as rows of 32
// neighbouring features.
template <int BN>
__device__ __forceinline__ void store_sums(float *out, int cols, uint32_t acc, int c0, int end, int f, int lane) {
    const bool mine = f + lane < cols;
    out += (int64_t)c0 * cols + f + lane;
#pragma unroll 1
    for (int c = c0; c < end; c += lt::EPI_ROWS) {
        uint32_t r[8];
        __syncwarp();
        tmem_ld_8_issue(acc + (uint32_t)c, r);
        tmem_ld_8_wait(r);
#pragma unroll
        for (int j = 0; j < lt::EPI_ROWS; ++j, out += cols)
            if (mine && c + j < end) *out = __uint_as_float(r[j]);
    }
}

// The word that this pair's waits raise errors in and look at.  Worked out again
// wherever a wait has to look (volatile): held in registers it costs the
// epilogue's (19456 x 4096 of 64 products each 47.4 us, 45.5 so).
struct PairStatus {
    const LinearTcParams &p;
    __device__ __forceinline__ uint32_t *word() const {
        uint32_t block;
        asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(block));
        return p.clear ? p.status + kPairWordsOffset / 4 + (block >> 1) : p.status;
    }
    __device__ __forceinline__ bool raised() const { return error_raised(word()); }
    __device__ __forceinline__ void flag(uint32_t f) const { flag_error(word(), f); }
};

// All but the last chunk of a row product's long contraction, for columns [c0,
// end) of a warp's 32 features: each accumulator (two alternate, BN columns from
// `acc` on) is added to the sum so far, which stays with the CTA, a lane reading
// what it wrote; the last chunk's accumulator takes the sum of the others and
// goes on as the unit's.  `at`: column 0 of the lane's feature.  Returns the last
// chunk's count of accumulator uses, or -1 where a wait gave up.
template <int BN>
__device__ int sum_chunks(float *at, int c0, int end, uint32_t acc, uint32_t full, uint32_t empty, int left, int use,
                          const PairStatus &status) {
    for (bool first = true;; first = false, ++use) {
        const uint32_t buf = (uint32_t)use & 1u;
        if (!mbar_wait_warp(full + 8 * buf, (use >> 1) & 1, status)) return -1;
        tc_fence_after();
        left -= kChunk;
#pragma unroll 1
        for (int c = c0; c < end; c += 8) {
            float *sum = at + c * lt::BP_CTA;
            uint32_t r[8];
            __syncwarp();
            tmem_ld_8_issue(acc + buf * BN + (uint32_t)c, r);
            tmem_ld_8_wait(r);
            if (!first) {
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + sum[j * lt::BP_CTA]);
            }
            if (left > 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j * lt::BP_CTA] = __uint_as_float(r[j]);
            } else {
                tmem_st_8(acc + buf * BN + (uint32_t)c, r);
            }
        }
        __syncwarp();
        if (left <= 0) return use;
        tc_fence_before();
        __syncwarp();
        if (lane_id() == 0) mbar_arrive_cluster(empty + 8 * buf);
    }
}

// A value that all lanes of a converged warp hold, in a uniform register.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

// LONG: the row products where the contraction is longer than kChunk (a variant of
// its own: the others' epilogue loses 8% to its registers where it sets the pace).
template <Product MODE, int BN, typename T, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(lt::THREADS, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmB32, const __grid_constant__ CUtensorMap tmOut,
                     const LinearTcParams p) {
    using C = lt::Cfg<BN, is_weights(MODE)>;
    constexpr bool A_MN = !is_forward(MODE), B_MN = is_weights(MODE);
    constexpr bool RELAY = is_weights(MODE);  // rows may have to be cleared before the MMA
    constexpr bool WEIGHTS = is_weights(MODE);
    constexpr bool LOG_SUM = MODE == Product::kLogSum || MODE == Product::kLogSumFew;
    constexpr int CHUNK = LONG ? lt::CHUNK_BLOCKS : LOG_SUM ? lt::LOG_BLOCKS : 0;  // k-blocks of an accumulator (0: all)
    static_assert(!B_MN || BN >= 128, "an N-contiguous operand comes in chunks of 64 per CTA");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const uint32_t sbase = smem_addr(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::BAR_BASE);
    auto bar = [&](int i) { return smem_addr(bars + i); };
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + C::NUM_BARS);
    int *edges = reinterpret_cast<int *>(smem + C::TABLE_BASE);
    int *tiles = edges + p.n_experts + 2, *slots = tiles + p.n_experts + 2, *bias_tiles = slots + p.n_experts + 2;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
    const PairStatus status{p};

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(bar(C::FULL + s), 1);
            mbar_init(bar(C::READY + s), 2);  // the relay of each CTA (even CTA's copy)
            mbar_init(bar(C::EMPTY + s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(C::T_FULL + b), 1);
            mbar_init(bar(C::T_EMPTY + b), 2 * lt::EPI_WARPS);  // both CTAs' epilogue warps (even CTA's copy)
        }
        mbar_init(bar(C::DRAIN), 1);
        fence_barrier_init();
    }
    if (warp == lt::WARP_TMA && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        if (!WEIGHTS) tma_prefetch_desc(&tmB32);
    }
    if (warp == lt::WARP_MMA) {
        tmem_alloc_pair(smem_addr(tmem_holder), C::TMEM_COLS);
        tmem_relinquish_pair();
        tc_fence_before();
    }
    griddep_wait();
    // cleared by the pair itself, ahead of the barrier below that its waits
    // come after; the other pairs have theirs, whatever the workspace held
    if (p.clear && rank == 0 && threadIdx.x == 0) {
        *status.word() = 0u;
        if (pair == 0) *p.status = kPairWordsMark | (uint32_t)num_pairs << kPairCountShift;
    }
    constexpr bool OWN_TILE = MODE == Product::kLogSum || MODE == Product::kSoftmax || MODE == Product::kRowsSum;
    if (warp == 0)
        fill_tables(p.offsets, p.n_experts, p.m, WEIGHTS ? p.chunk : OWN_TILE ? p.entropy.tile : BN, edges, tiles,
                    WEIGHTS ? slots : nullptr, lane);
    if (WEIGHTS && p.db && warp == 1)  // (the second table is a copy of the edges)
        fill_tables(p.offsets, p.n_experts, p.m, p.bias_rows, bias_tiles + p.n_experts + 2, bias_tiles, nullptr, lane);
    cluster_sync();  // barriers, tensor memory and tables exist in both CTAs
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    Units<MODE, BN> units(p, edges, tiles, slots);

    if (warp < lt::EPI_WARPS) {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3, part = warp >> 2;
        using F = std::conditional_t<MODE == Product::kSoftmax, FinishSoftmax<BN, T>, Finish<MODE, BN, T>>;
        F fin{p, reinterpret_cast<float *>(smem + C::STAGING_BASE) + warp * lt::EPI_ROWS * lt::EPI_PITCH, lane};
        if constexpr (MODE == Product::kRowsSum || MODE == Product::kWeightsScaled) fin.factor = *p.entropy.inverse;
        if (WEIGHTS && p.db) {
            // while the first units are on their way: the bias gradient, eight
            // columns to a warp, an expert's row tiles dealt to four lanes each
            // and their sums added in order
            const int groups = (p.out_rows + 7) / 8, sub = lane >> 3;
            for (int64_t i = (int64_t)blockIdx.x * lt::EPI_WARPS + warp; i < (int64_t)p.n_experts * groups;
                 i += (int64_t)gridDim.x * lt::EPI_WARPS) {
                const int e = (int)(i / groups), col = (int)(i - (int64_t)e * groups) * 8 + (lane & 7);
                LongSum part_sum;
                if (col < p.out_rows) {
#pragma unroll 8
                    for (int tile = bias_tiles[e] + sub; tile < bias_tiles[e + 1]; tile += 4)
                        part_sum.add(p.bias_sums[(int64_t)tile * p.out_rows + col]);
                }
                float s = part_sum.value();
                s += __shfl_xor_sync(0xffffffffu, s, 8);
                s += __shfl_xor_sync(0xffffffffu, s, 16);
                if (sub == 0 && col < p.out_rows) static_cast<T *>(p.db)[(int64_t)e * p.out_rows + col] = narrow<T>(s);
            }
            __syncwarp();
        }
        int use = 0, ring = 0;
        Unit mine{};  // 32 units ahead, one per lane
        for (int u = pair, i = 0; u < units.total; u += num_pairs, i = (i + 1) & 31) {
            if (i == 0) {
                const int ahead = u + lane * num_pairs;
                if (ahead < units.total) mine = units.at(ahead);
                __syncwarp();
            }
            const Unit t = mine.of_lane(i);
            const bool zero = t.c1 <= t.c0;  // nothing to multiply: rows of no expert, experts without rows
            const int f = t.p0 + rank * lt::BP_CTA + quarter * 32;  // this warp's first feature
            float bias = 0.f;
            if (MODE == Product::kForward && p.bias && !zero && f + lane < p.cols)
                bias = widen(static_cast<const T *>(p.bias)[(int64_t)t.expert * p.cols + f + lane]);
            fin.c0 = part * F::COLS;
            fin.end = min(t.qn, fin.c0 + F::COLS);
            fin.f = f;
            fin.out_row = WEIGHTS ? (int64_t)t.expert * p.out_rows + t.q0 : (int64_t)t.q0;
            if constexpr (MODE == Product::kForward) fin.add = p.residual && !zero;
            if constexpr (LOG_SUM) {
                float v[F::COLS];
                const int count = max(0, fin.end - fin.c0);
                use = sum_logits<BN>(v, tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)fin.c0, bar(C::T_FULL),
                                     map_to_cta(bar(C::T_EMPTY), 0), (t.c1 - t.c0 + lt::BK - 1) / lt::BK, use, status);
                if (use < 0) break;
                if constexpr (MODE == Product::kLogSumFew) {
                    if (count > 0 && f < p.cols) log_sum_few(p, v, count, f, lane, (int64_t)t.q0 + fin.c0);
                } else {
                    const bool mine = f + lane < *p.entropy.count;
                    const int label = mine ? p.entropy.rows[f + lane].label - t.q0 - fin.c0 : -1;
                    log_sum(p.entropy, v, count, f + lane, mine, label, t.slot * lt::PARTS + part);
                }
                continue;
            }
            bool ready = zero;
            if (LONG && t.c1 - t.c0 > kChunk) {
                use = sum_chunks<BN>(p.partial + (int64_t)blockIdx.x * kChunkTile + quarter * 32 + lane, fin.c0, fin.end,
                                     tmem_base + ((uint32_t)(quarter * 32) << 16), bar(C::T_FULL),
                                     map_to_cta(bar(C::T_EMPTY), 0), t.c1 - t.c0, use, status);
                if (use < 0) break;
                ready = true;
            }
            const int buf = use & 1;
            fin.prefetch();
            if (!ready) {
                bool ok = mbar_wait_warp(bar(C::T_FULL + buf), (use >> 1) & 1, status);
                // a part that meets at barriers goes on together or not at all
                if (WEIGHTS) ok = named_barrier_all(1 + part, 128, ok);
                if (!ok) break;
                tc_fence_after();
            }
            const uint32_t acc = tmem_base + (uint32_t)(buf * BN) + ((uint32_t)(quarter * 32) << 16);
            if constexpr (MODE == Product::kSoftmax) {
                if (fin.c0 < fin.end) fin.run(acc);
            } else if constexpr (MODE == Product::kRowsSum) {
                if (fin.c0 < fin.end) add_sums<T>(p, acc, fin.c0, fin.end, f, fin.out_row, lane, fin.factor, t.slot, zero);
            } else if (WEIGHTS && t.slot >= 0) {
                if (fin.c0 < fin.end)
                    store_sums<BN>(p.partial + ((int64_t)t.slot * p.out_rows + t.q0) * p.cols, p.cols, acc, fin.c0, fin.end,
                                   f, lane);
            } else if (WEIGHTS && p.wide) {
                const int fc = t.p0 + rank * lt::BP_CTA;
                if (fin.c0 < fin.end && fc < p.cols)
                    store_part<T, MODE == Product::kWeightsScaled>(p, &tmOut, smem + C::STAGING_BASE + part * 2 * lt::STORE_BYTES, ring,
                                  acc + (uint32_t)fin.c0, part, quarter, lane, fc, t.q0 + fin.c0, fin.end - fin.c0,
                                  t.expert, zero, fin.factor);
            } else if (fin.c0 < fin.end) {
                if constexpr (MODE == Product::kForward)
                    with_activation(p.activation, [&](auto a) {
                        if (p.wide)
                            fin.template run<decltype(a)::value>(acc, bias, zero);
                        else
                            fin.template run_direct<decltype(a)::value>(acc, bias, zero);
                    });
                else if (p.wide)
                    fin.template run<KMEANS_ACT_NONE>(acc, bias, zero);
                else
                    fin.template run_direct<KMEANS_ACT_NONE>(acc, bias, zero);
            }
            if (!zero) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_cta(bar(C::T_EMPTY + buf), 0));
                ++use;
            }
        }
        if (WEIGHTS && quarter == 0 && lane == 0) bulk_wait();  // this thread's stores out of shared memory
    } else {
        // These warps feed the pipeline, and an MMA or a load that they issue
        // late is lost time, also because the epilogue's warps take turns with
        // them.  So the whole warp walks the units (the addresses and
        // descriptors are then uniform and need no moves between register
        // files), one elected lane issues, and units are worked out 32 at a
        // time, one per lane (one after the other they cost some thousand
        // cycles each: 2200 cycles without an MMA between two units).
        Unit *list = reinterpret_cast<Unit *>(smem + C::LIST_BASE + (warp - lt::WARP_TMA) * lt::LIST_BYTES);
        const bool leader = elect_one();
        int s = 0, use = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = !(warp == lt::WARP_TMA && p.test_starve) && !(warp == lt::WARP_RELAY && !RELAY) &&
                  !(warp == lt::WARP_MMA && rank != 0);
        auto advance = [&] {
            if (++s == C::STAGES) {
                s = 0;
                phase ^= 1;
            }
        };
        for (int u0 = pair; u0 < units.total && ok; u0 += lt::LIST_UNITS * num_pairs) {
            __syncwarp();
            const int mine = u0 + lane * num_pairs;
            if (mine < units.total) list[lane] = units.at(mine);
            __syncwarp();
            const int here = min(lt::LIST_UNITS, (units.total - u0 + num_pairs - 1) / num_pairs);
            for (int i = 0; i < here && ok; ++i) {
                const Unit t = list[i];
                const int kblocks = uniform((t.c1 - t.c0 + lt::BK - 1) / lt::BK);
                if (warp == lt::WARP_TMA) {
                    // ------------------------------------------- TMA producer
                    const int pa = uniform(t.p0) + rank * lt::BP_CTA, e = uniform(t.expert);
                    // the MMA's N is cut to the rows that exist (a multiple of
                    // 32); each CTA holds half of it, and loads no more than
                    // that in boxes of 32 rows (all of it is one box)
                    const int half = WEIGHTS ? BN / 2 : uniform(min(BN, (t.qn + 31) & ~31) >> 1);
                    const int boxes = half == BN / 2 ? 0 : (half + 31) / 32;
                    const int qb = uniform(t.q0) + rank * half;
                    const uint32_t bytes = 2u * (boxes ? C::A_BYTES + boxes * (32 * lt::BK * 2) : C::STAGE);
                    int c = uniform(t.c0);
                    for (int left = kblocks; left > 0; --left, c += lt::BK) {
                        if (!mbar_wait_converged(bar(C::EMPTY + s), phase ^ 1, status)) {
                            ok = false;
                            break;
                        }
                        const uint32_t sa = sbase + s * C::STAGE, sb = sa + C::A_BYTES, full = bar(C::FULL + s);
                        if (leader) {
                            if constexpr (RELAY) {
                                mbar_arrive_expect_tx(full, C::STAGE);
#pragma unroll
                                for (int h = 0; h < lt::BP_CTA / 64; ++h)
                                    tma_load_2d(sa + h * (64 * lt::BK * 2), &tmA, full, pa + h * 64, c);
#pragma unroll
                                for (int h = 0; h < BN / 2 / 64; ++h)
                                    tma_load_2d(sb + h * (64 * lt::BK * 2), &tmB, full, qb + h * 64, c);
                            } else {
                                // both CTAs' bytes count on the even CTA's barrier
                                if (rank == 0) mbar_arrive_expect_tx(full, bytes);
                                const uint32_t pair_full = map_to_cta(full, 0);
                                if constexpr (!A_MN) {
                                    tma_load_3d_pair(sa, &tmA, pair_full, c, pa, e);
                                } else {
#pragma unroll
                                    for (int h = 0; h < lt::BP_CTA / 64; ++h)
                                        tma_load_3d_pair(sa + h * (64 * lt::BK * 2), &tmA, pair_full, pa + h * 64, c, e);
                                }
                                if (boxes == 0) tma_load_2d_pair(sb, &tmB, pair_full, c, qb);
                                for (int h = 0; h < boxes; ++h)
                                    tma_load_2d_pair(sb + h * (32 * lt::BK * 2), &tmB32, pair_full, c, qb + h * 32);
                            }
                        }
                        __syncwarp();
                        ++issued;
                        advance();
                    }
                } else if (warp == lt::WARP_RELAY) {
                    // -------------------------------------------------- relay
                    for (int c = t.c0; c < t.c1; c += lt::BK) {
                        if (!mbar_wait_converged(bar(C::FULL + s), phase, status)) {
                            ok = false;
                            break;
                        }
                        if (t.c1 - c < lt::BK) {
                            // rows past the expert's end: every 64-value chunk
                            // of both operands holds them as whole 128-byte
                            // lines
                            uint8_t *st = smem + s * C::STAGE;
                            constexpr int CHUNKS = C::STAGE / (64 * lt::BK * 2);
                            for (int k = (t.c1 - c) * 8 + lane; k < lt::BK * 8; k += 32)
#pragma unroll
                                for (int h = 0; h < CHUNKS; ++h)
                                    *reinterpret_cast<uint4 *>(st + h * (64 * lt::BK * 2) + k * 16) =
                                        make_uint4(0, 0, 0, 0);
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        if (leader) mbar_arrive_cluster(map_to_cta(bar(C::READY + s), 0));
                        __syncwarp();
                        advance();
                    }
                } else if (kblocks > 0) {
                    // ---------------------------------------------- MMA issue
                    const int n = WEIGHTS ? BN : uniform(min(BN, (t.qn + 31) & ~31));
                    const uint32_t idesc =
                        umma_idesc_16_f32(std::is_same<T, __nv_bfloat16>::value, A_MN, B_MN, lt::BP, n);
                    // 16 values of the contraction: 32 bytes along a K-major
                    // row, or 16 lines of 128 bytes
                    constexpr uint32_t A_STEP = (A_MN ? 2048 : 32) >> 4, B_STEP = (B_MN ? 2048 : 32) >> 4;
                    const uint64_t a0 = A_MN ? umma_smem_desc_mn(sbase, 64 * lt::BK * 2, 1024)
                                             : umma_smem_desc(sbase, 1024, kLayoutSW128);
                    const uint64_t b0 = B_MN ? umma_smem_desc_mn(sbase + C::A_BYTES, 64 * lt::BK * 2, 1024)
                                             : umma_smem_desc(sbase + C::A_BYTES, 1024, kLayoutSW128);
                    const uint32_t a_hi = (uint32_t)(a0 >> 32), b_hi = (uint32_t)(b0 >> 32);
                    // (a chunk of rows is a unit of its own in the weights product)
                    for (int blocks = kblocks; blocks > 0 && ok; blocks -= CHUNK ? CHUNK : blocks) {
                        const int buf = use & 1;
                        const uint32_t acc = tmem_base + (uint32_t)(buf * BN);
                        if (!mbar_wait_converged(bar(C::T_EMPTY + buf), ((use >> 1) & 1) ^ 1, status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        uint32_t more = 0;  // the first MMA of a chunk clears the accumulator
                        for (int left = CHUNK ? min(blocks, CHUNK) : blocks; left > 0; --left) {
                            const uint32_t off = (uint32_t)s * (C::STAGE >> 4);
                            const uint32_t a_lo = (uint32_t)a0 + off, b_lo = (uint32_t)b0 + off;
                            if (!mbar_wait_converged(bar((RELAY ? C::READY : C::FULL) + s), phase, status)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            if (leader) {
                                mma_16_ss_pair(acc, a_lo, a_hi, b_lo, b_hi, idesc, more);
                                mma_16_ss_pair(acc, a_lo + A_STEP, a_hi, b_lo + B_STEP, b_hi, idesc, 1u);
                                mma_16_ss_pair(acc, a_lo + 2 * A_STEP, a_hi, b_lo + 2 * B_STEP, b_hi, idesc, 1u);
                                mma_16_ss_pair(acc, a_lo + 3 * A_STEP, a_hi, b_lo + 3 * B_STEP, b_hi, idesc, 1u);
                                mma_commit_pair_multicast(bar(C::EMPTY + s), 0x3);
                            }
                            __syncwarp();
                            more = 1u;
                            advance();
                        }
                        if (!ok) break;
                        if (leader) mma_commit_pair_multicast(bar(C::T_FULL + buf), 0x3);
                        __syncwarp();
                        ++use;
                    }
                }
            }
        }
        if (warp == lt::WARP_TMA && leader && !ok && (RELAY || rank == 0)) {
            // let copies already in flight land before the CTAs exit (the odd
            // CTA's are on the even one's barriers, and it leaves last)
            for (int j = max(0, issued - C::STAGES); j < issued; ++j)
                mbar_wait_drain(bar(C::FULL + (j % C::STAGES)), (j / C::STAGES) & 1);
        }
        if (warp == lt::WARP_MMA && leader && rank == 0) {
            // no MMA may still be writing tensor memory when it is released
            mma_commit_pair(bar(C::DRAIN));
            mbar_wait_drain(bar(C::DRAIN), 0);
        }
    }

    __syncwarp();
    cluster_sync();  // no CTA leaves while its peer may still signal it
    if (warp == lt::WARP_MMA) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
inline bool encode(CUtensorMap *map, bool bf16, const void *base, int rank, const uint64_t *dims, const uint64_t *pitch_elems,
            const uint32_t *box) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t d[3], strides[2];
    cuuint32_t b[3], one[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i) strides[i - 1] = pitch_elems[i - 1] * 2;
    }
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
               const_cast<void *>(base), d, strides, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Product MODE, int BN, typename T, bool LONG>
cudaError_t launch_tc(const LinearShape &sh, const Product16 &g, const LinearTcParams &p, cudaStream_t s) {
    using C = lt::Cfg<BN, is_weights(MODE)>;
    static std::once_flag once[kMaxDevices];
    static std::atomic<int> err[kMaxDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    const int slot = dev >= 0 && dev < kMaxDevices ? dev : 0;
    once_per_device(once, [&] {
        err[slot].store((int)cudaFuncSetAttribute(linear_tc_kernel<MODE, BN, T, LONG>,
                                                  cudaFuncAttributeMaxDynamicSharedMemorySize, lt::SMEM_LIMIT));
    });
    if (err[slot].load() != cudaSuccess) return (cudaError_t)err[slot].load();

    CUtensorMap tmA, tmB, tmB32{}, tmOut{};
    bool ok;
    if (is_weights(MODE)) {
        const uint64_t da[2] = {(uint64_t)sh.k, (uint64_t)sh.m}, pa[1] = {(uint64_t)g.lda};
        const uint64_t db[2] = {(uint64_t)sh.n, (uint64_t)sh.m}, pb[1] = {(uint64_t)g.ldb};
        const uint32_t box[2] = {64, lt::BK};
        ok = encode(&tmA, sh.bf16, g.a, 2, da, pa, box) && encode(&tmB, sh.bf16, g.b, 2, db, pb, box);
        if (p.wide) {
            const uint64_t dd[3] = {(uint64_t)sh.k, (uint64_t)sh.n, (uint64_t)sh.n_experts};
            const uint64_t pd[2] = {(uint64_t)sh.k, (uint64_t)(sh.k * sh.n)};
            const uint32_t bd[3] = {64, lt::STORE_ROWS, 1};
            ok = ok && encode(&tmOut, sh.bf16, g.out, 3, dd, pd, bd);
        }
    } else {
        const uint64_t da[3] = {(uint64_t)sh.k, (uint64_t)sh.n, (uint64_t)sh.n_experts};
        const uint64_t pa[2] = {(uint64_t)g.pitch_w, (uint64_t)(g.pitch_w * sh.n)};
        const uint32_t ba[3] = {64, is_forward(MODE) ? (uint32_t)lt::BP_CTA : (uint32_t)lt::BK, 1};
        const uint64_t db[2] = {(uint64_t)p.contraction, (uint64_t)sh.m}, pb[1] = {(uint64_t)g.ldb};
        const uint32_t bb[2] = {lt::BK, BN / 2}, b32[2] = {lt::BK, 32};
        ok = encode(&tmA, sh.bf16, g.a, 3, da, pa, ba) && encode(&tmB, sh.bf16, g.b, 2, db, pb, bb) &&
             encode(&tmB32, sh.bf16, g.b, 2, db, pb, b32);
    }
    if (!ok) return cudaErrorInvalidValue;

    // at most one unit per row tile, expert and feature tile
    constexpr bool OWN_TILE = MODE == Product::kLogSum || MODE == Product::kSoftmax || MODE == Product::kRowsSum;
    const int64_t row_tiles = OWN_TILE           ? (sh.m + p.entropy.tile - 1) / p.entropy.tile *
                                             (MODE == Product::kRowsSum ? p.entropy.splits : 1)
                              : is_weights(MODE)
                                  ? (sh.n + BN - 1) / BN * (sh.n_experts + sh.m / p.chunk + 1)
                                                        : (sh.m + BN - 1) / BN + (sh.offsets ? sh.n_experts : 0);
    static_assert(kPairs <= kMaxPairWords, "a status word each");
    const int64_t most = std::min(device_sm_count() / 2, kPairs), units = row_tiles * p.num_p;
    const unsigned pairs = (unsigned)(units < most ? units : most);
    return launch_kernel(true, linear_tc_kernel<MODE, BN, T, LONG>, dim3(2 * (pairs ? pairs : 1)), dim3(lt::THREADS),
                         C::smem_bytes(sh.n_experts), s, tmA, tmB, tmB32, tmOut, p);
}

template <Product MODE, int BN, bool LONG = false>
cudaError_t launch_typed(const LinearShape &sh, const Product16 &g, const LinearTcParams &p, cudaStream_t s) {
    return sh.bf16 ? launch_tc<MODE, BN, __nv_bfloat16, LONG>(sh, g, p, s)
                   : launch_tc<MODE, BN, __half, LONG>(sh, g, p, s);
}

}  // namespace km
