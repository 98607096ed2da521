// Expert routing: the stable sort of slots by expert, and rows moved into that
// order, back with weights, and their gradients.
//
//   key(s)  = experts[s], or E (the bucket of dropped slots) when negative
//   row(s)  = #{s' : key(s') < key(s)} + #{s' < s : key(s') = key(s)}
//   xs[row(t, j)] = x[t]
//   y[t]    = residual[t] + sum_j w[t, j] ys[row(t, j)]
//   dys[row(t, j)] = w[t, j] dy[t],  dw[t, j] = <dy[t], ys[row(t, j)]>
//
// The sort is one thread-block cluster.  Every warp counts the keys of its own
// run of consecutive slots (a count per key and warp in shared memory); the
// counts become starting rows by a prefix over the warps, over the cluster's
// blocks (read through distributed shared memory) and over the keys; then each
// warp walks its run again and hands out rows in slot order, so equal keys keep
// their order and no atomic decides a place.
//
// The row movers are bound by memory: each token is read once and written (or
// its rows are read) topk times, 16 bytes a thread where the rows' alignment
// allows, several independent loads in flight per thread.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pieces.cuh"
#include "ptx.cuh"

namespace km {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ------------------------------------------------------------------ the sort
constexpr int kRouteThreads = 1024;
constexpr int kRouteSmemMax = 224 * 1024;
constexpr int kRouteMaxCluster = 16;
constexpr int kRouteSlotsPerBlock = 4096;  // below this many slots another block does not pay its exchange

struct RouteParams {
    const void *experts;
    int slots, n_experts;
    int warps;  // counting warps per block
    int32_t *offsets, *order, *rows;
    uint32_t *status;
};

__device__ __forceinline__ int ld_cluster_i32(const int *p, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(map_to_cta(smem_addr(p), rank)) : "memory");
    return v;
}

constexpr int kRouteBatch = 8;  // groups of 32 slots whose ids are in flight together

// The keys of slots s + 32 b + lane below `end` (-1 past it).
template <typename Id>
__device__ __forceinline__ void route_keys(const Id *experts, uint32_t s, uint32_t end, int n_experts, bool &bad,
                                           int (&key)[kRouteBatch]) {
    Id id[kRouteBatch];
#pragma unroll
    for (int b = 0; b < kRouteBatch; ++b) id[b] = s + 32u * b < end ? experts[s + 32u * b] : (Id)0;
#pragma unroll
    for (int b = 0; b < kRouteBatch; ++b) {
        const bool live = s + 32u * b < end;
        if (live && id[b] >= (Id)n_experts) bad = true;
        key[b] = !live ? -1 : (id[b] < 0 || id[b] >= (Id)n_experts) ? n_experts : (int)id[b];
    }
}

// Lanes of the warp whose key equals this lane's, by its bits: one vote per bit
// is far cheaper than a match instruction, which takes the warp's distinct keys
// one after the other (65536 slots over 1024 experts spent 19 of 38 thousand
// cycles in eight of them per warp).
__device__ __forceinline__ uint32_t same_key(int key, bool live, int bits) {
    uint32_t same = __ballot_sync(kFull, live);
    for (int b = 0; b < bits; ++b) {
        const bool one = (key >> b) & 1;
        const uint32_t ones = __ballot_sync(kFull, one);
        same &= one ? ones : ~ones;
    }
    return same;
}

// Shared memory: hist[warps][keys], tot[keys], base[keys], 32 words of scan
// scratch, with keys = n_experts + 1.
template <typename Id>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
    extern __shared__ __align__(16) int route_smem[];
    const int keys = p.n_experts + 1;
    int *hist = route_smem;
    int *tot = hist + p.warps * keys;
    int *base = tot + keys;
    int *scan = base + keys;
    const Id *experts = static_cast<const Id *>(p.experts);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int blocks = gridDim.x;
    const uint32_t below = (1u << lane) - 1u;

    griddep_wait();
    if (rank == 0 && tid == 0) *p.status = 0u;
    // this warp's run of consecutive slots, whole groups of 32
    const int total_warps = blocks * p.warps;
    const int groups = (int)(((uint32_t)p.slots + 31u) / 32u);
    const int per = (groups + total_warps - 1) / total_warps;
    const int64_t g0 = (int64_t)((int)rank * p.warps + warp) * per;
    const uint32_t s0 = (uint32_t)min(g0 * 32, (int64_t)p.slots);
    const uint32_t s1 = warp < p.warps ? (uint32_t)min((g0 + per) * 32, (int64_t)p.slots) : s0;
    int *mine = hist + warp * keys;

    bool bad = false;
    int key[kRouteBatch];
    if (s0 < s1) route_keys(experts, s0 + lane, s1, p.n_experts, bad, key);
    for (int i = tid * 4; i < p.warps * keys; i += blockDim.x * 4) {
        if (i + 4 <= p.warps * keys) {
            *reinterpret_cast<int4 *>(hist + i) = make_int4(0, 0, 0, 0);
        } else {
            for (int k = i; k < p.warps * keys; ++k) hist[k] = 0;
        }
    }
    __syncthreads();
    for (uint32_t s = s0; s < s1; s += 32 * kRouteBatch) {
        if (s != s0) route_keys(experts, s + lane, s1, p.n_experts, bad, key);
#pragma unroll
        for (int b = 0; b < kRouteBatch; ++b)
            if (key[b] >= 0) atomicAdd(mine + key[b], 1);
    }
    __syncthreads();
    // per key: each warp's first place among this block's, and the block's total
    for (int e = tid; e < keys; e += blockDim.x) {
        int sum = 0;
        for (int w0 = 0; w0 < p.warps; w0 += 8) {
            int c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = w0 + i < p.warps ? hist[(w0 + i) * keys + e] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (w0 + i < p.warps) hist[(w0 + i) * keys + e] = sum;
                sum += c[i];
            }
        }
        tot[e] = sum;
    }
    cluster_sync();  // every block's totals are readable; the status word is cleared
    if (__syncthreads_or(bad) && tid == 0) flag_error(p.status, kFlagBadLabel);

    // base[e] = all slots of smaller keys + the lower blocks' slots of key e;
    // a thread has two neighbouring keys, so that 1024 experts and their
    // dropped slots are one round
    int run = 0;
    for (int e0 = 0; e0 < keys; e0 += 2 * blockDim.x) {
        const int e = e0 + 2 * tid;
        int all[2] = {}, lower[2] = {};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (e + i >= keys) continue;
            if (blocks == 1) {
                all[i] = tot[e + i];
                continue;
            }
            int c[kRouteMaxCluster];
#pragma unroll
            for (int r = 0; r < kRouteMaxCluster; ++r) c[r] = r < blocks ? ld_cluster_i32(tot + e + i, (uint32_t)r) : 0;
#pragma unroll
            for (int r = 0; r < kRouteMaxCluster; ++r) {
                all[i] += c[r];
                if (r < (int)rank) lower[i] += c[r];
            }
        }
        const int own = all[0] + all[1];
        int inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        // each warp adds up the others' sums by itself
        const int warps = (int)(blockDim.x >> 5);
        const int sums = lane < warps ? scan[lane] : 0;
        const int before = __reduce_add_sync(kFull, lane < warp ? sums : 0), chunk = __reduce_add_sync(kFull, sums);
        int first = run + before + inc - own;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (e + i < keys) {
                base[e + i] = first + lower[i];
                if (rank == 0) p.offsets[e + i] = first;  // offsets[n_experts]: the kept slots
                first += all[i];
            }
        run += chunk;
        __syncthreads();
    }
    // hand out rows (one batch's keys are still in registers)
    const int bits = 32 - __clz(p.n_experts);
    for (uint32_t s = s0; s < s1; s += 32 * kRouteBatch) {
        if (s1 - s0 > 32 * kRouteBatch) route_keys(experts, s + lane, s1, p.n_experts, bad, key);
#pragma unroll
        for (int b = 0; b < kRouteBatch; ++b) {
            if (s + 32u * b >= s1) break;  // the same for the whole warp
            const bool live = key[b] >= 0;
            const uint32_t same = same_key(key[b], live, bits);
            int row = 0;
            if (live) row = base[key[b]] + mine[key[b]] + __popc(same & below);
            __syncwarp();
            if (live && (same & below) == 0u) mine[key[b]] += __popc(same);
            __syncwarp();
            if (live) {
                const uint32_t slot = s + 32u * b + lane;
                p.rows[slot] = row;
                p.order[row] = (int)slot;
            }
        }
    }
    cluster_sync();  // no block leaves while another may still read its totals
}

// -------------------------------------------------------------- row movement
// Rows move in words, neighbouring lanes at neighbouring words.  A word has as
// many bytes as every stored row is aligned to, VEC = 16, 8 or 4, and is one
// access (16384 tokens of 4 choices, d = 513 float32, 16-byte words put together
// by shifts: gather 49 us, combine 66, gradient 146; 4-byte words 33, 49, 78).
// Rows of an odd number of 16-bit values (VEC = 2) have words of 16 bytes: the
// aligned words of the stored row are written, only its two ends in part, and
// each is put together from the two aligned words of the source that hold it.
// Their latency and some 200 instructions a word then bound the kernels (16384
// tokens of 8 choices, d = 2047 bf16 against 2048: gather 141 us, 92; combine
// 224, 102; gradient 529, 178).  For 4097 tokens of three choices, d = 1031 in 16
// bits, the combine takes 12 us so; values one at a time took 31, 4-byte words
// 20, words shared between neighbouring lanes by shuffles 19.
template <int VEC>
constexpr int kWordBytes = VEC == 2 ? 16 : VEC;

template <typename T, int VEC>
struct Word {
    static constexpr int N = kWordBytes<VEC> / 4;          // 4-byte parts
    static constexpr int V = kWordBytes<VEC> / (int)sizeof(T);  // values
    uint32_t u[N];
    __device__ void to_floats(float (&f)[V]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(u[i]);
            } else {
                const float2 v = widen2<T>(u[i]);
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    }
    __device__ static Word from_floats(const float (&f)[V]) {
        Word w;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(T) == 4)
                w.u[i] = __float_as_uint(f[i]);
            else
                w.u[i] = narrow2<T>(f[2 * i], f[2 * i + 1]);
        }
        return w;
    }
    __device__ static Word zero() {
        Word w;
#pragma unroll
        for (int i = 0; i < N; ++i) w.u[i] = 0;
        return w;
    }
    __device__ static Word of(const uint4 &v) {
        static_assert(N == 4);
        return {v.x, v.y, v.z, v.w};
    }
    // One access of all its bytes, or pieces of `align` bytes.
    __device__ static Word load(const uint8_t *p, int align = kWordBytes<VEC>) {
        Word w;
        if (align >= 4 * N) {
            if constexpr (N == 4) w = of(*reinterpret_cast<const uint4 *>(p));
            if constexpr (N == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                w.u[0] = v.x;
                w.u[1] = v.y;
            }
            if constexpr (N == 1) w.u[0] = *reinterpret_cast<const uint32_t *>(p);
        } else if (align >= 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w.u[i] = reinterpret_cast<const uint32_t *>(p)[i];
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
            for (int i = 0; i < N; ++i) w.u[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
        }
        return w;
    }
    __device__ uint4 wide() const {
        static_assert(N == 4);
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

struct MoveParams {
    const int32_t *rows, *offsets;
    int64_t n, slots;
    int64_t row_bytes;
    int words;  // words that a row takes, at most
    int align;  // bytes, up to a word's, that the strided operand's rows are aligned to
    int topk, n_experts;
    int tpr_log2;  // threads per row
};

constexpr int kMoveThreads = 256;
template <int VEC>
constexpr int kGatherUnroll = VEC == 2 || VEC == 16 ? 4 : 8;

// What a word of a stored row takes of the row.
struct RowWord {
    int64_t at;  // the word's first byte within the row; negative in a shifted row's first word
    int lo, hi;  // the word's bytes that are in the row
};

template <int VEC>
__device__ __forceinline__ RowWord row_word(const uint8_t *row, int v, const MoveParams &p) {
    if (VEC > 2) return {(int64_t)v * VEC, 0, v < p.words ? VEC : 0};
    const int m = (int)(reinterpret_cast<uintptr_t>(row) & 15u);
    const int64_t at = (int64_t)v * 16 - m;
    return {at, v == 0 ? m : 0, (int)min((int64_t)16, p.row_bytes - at)};
}

template <typename T, int VEC>
__device__ __forceinline__ Word<T, VEC> load_row(const uint8_t *p, const Span &in) {
    if constexpr (VEC > 2)
        return Word<T, VEC>::load(p);
    else
        return Word<T, VEC>::of(load_word(p, in));
}

template <typename T, int VEC>
__device__ __forceinline__ Word<T, VEC> load_strided(const uint8_t *p, int align, const Span &in) {
    if constexpr (VEC > 2)
        return Word<T, VEC>::load(p, align);
    else
        return Word<T, VEC>::of(load_word(p, in));
}

template <typename T, int VEC>
__device__ __forceinline__ void store_row(uint8_t *p, const Word<T, VEC> &w, const RowWord &at) {
    if constexpr (VEC == 16) *reinterpret_cast<uint4 *>(p) = w.wide();
    if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w.u[0], w.u[1]);
    if constexpr (VEC == 4) *reinterpret_cast<uint32_t *>(p) = w.u[0];
    if constexpr (VEC == 2) store_word(p, w.wide(), at.lo, at.hi);
}

// xs[row(t, j)] = x[t]; a thread holds up to U words of its token and writes
// them to every choice's row.
template <int VEC>
__global__ void __launch_bounds__(kMoveThreads) route_gather_kernel(const MoveParams p, const uint8_t *x,
                                                                    int64_t pitch, Span in, uint8_t *xs) {
    using W = Word<float, VEC>;
    constexpr int U = kGatherUnroll<VEC>;
    griddep_wait();
    const int tpr = 1 << p.tpr_log2;
    const int sub = threadIdx.x & (tpr - 1);
    const int64_t t = (int64_t)blockIdx.x * (kMoveThreads >> p.tpr_log2) + (threadIdx.x >> p.tpr_log2);
    const int v0 = (int)blockIdx.y * (tpr * U) + sub;
    if (t >= p.n || v0 >= p.words) return;
    const int kept = p.offsets[p.n_experts];
    const uint8_t *src = x + t * pitch;
    W val[U];
    if (VEC > 2) {  // the same words for every choice
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + u * tpr < p.words) val[u] = load_strided<float, VEC>(src + (int64_t)(v0 + u * tpr) * VEC, p.align, in);
    }
    for (int j = 0; j < p.topk; ++j) {
        const int r = p.rows[t * p.topk + j];
        if (r < 0 || r >= p.slots) continue;
        const bool on = r < kept;
        uint8_t *dst = xs + (int64_t)r * p.row_bytes;
        RowWord at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            at[u] = row_word<VEC>(dst, v0 + u * tpr, p);
            if (VEC == 2 && at[u].hi > 0) val[u] = load_row<float, VEC>(src + at[u].at, in);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (at[u].hi > 0) store_row<float, VEC>(dst + at[u].at, on ? val[u] : W::zero(), at[u]);
    }
}

// A thread has U words of its token and the rows of CH choices in flight: few
// choices leave room for several words (one at a time, 65536 tokens of one
// choice, d = 2048 float32, took 398 us, 4.0 TB/s; four, 239).
template <int VEC, typename T, int CH, int U>
__global__ void __launch_bounds__(kMoveThreads) route_combine_kernel(const MoveParams p, const uint8_t *ys, Span in,
                                                                     const float *__restrict__ weights,
                                                                     const uint8_t *residual, int64_t pitch, Span res_in,
                                                                     uint8_t *y) {
    using P = Word<T, VEC>;
    griddep_wait();
    const int tpr = 1 << p.tpr_log2;
    const int sub = threadIdx.x & (tpr - 1);
    const int64_t t = (int64_t)blockIdx.x * (kMoveThreads >> p.tpr_log2) + (threadIdx.x >> p.tpr_log2);
    const int v0 = (int)blockIdx.y * (tpr * U) + sub;
    if (t >= p.n || v0 >= p.words) return;
    const int kept = p.topk > 0 ? p.offsets[p.n_experts] : 0;
    const int64_t limit = kept < p.slots ? kept : p.slots;
    uint8_t *dst = y + t * p.row_bytes;
    RowWord at[U];
    P res[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        at[u] = row_word<VEC>(dst, v0 + u * tpr, p);
        if (residual && at[u].hi > 0) res[u] = load_strided<T, VEC>(residual + t * pitch + at[u].at, p.align, res_in);
    }
    float acc[U][P::V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < P::V; ++i) acc[u][i] = 0.f;
    for (int j0 = 0; j0 < p.topk; j0 += CH) {
        P part[CH][U];
        float w[CH];
        bool on[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int j = j0 + c;
            const int r = j < p.topk ? p.rows[t * p.topk + j] : -1;
            on[c] = r >= 0 && r < limit;
            if (!on[c]) continue;
            w[c] = weights ? weights[t * p.topk + j] : 1.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (at[u].hi > 0) part[c][u] = load_row<T, VEC>(ys + r * p.row_bytes + at[u].at, in);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (on[c])
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float f[P::V];
                    part[c][u].to_floats(f);
#pragma unroll
                    for (int i = 0; i < P::V; ++i) acc[u][i] = fmaf(w[c], f[i], acc[u][i]);
                }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (at[u].hi <= 0) continue;
        if (residual) {
            float f[P::V];
            res[u].to_floats(f);
#pragma unroll
            for (int i = 0; i < P::V; ++i) acc[u][i] += f[i];
        }
        store_row<T, VEC>(dst + at[u].at, P::from_floats(acc[u]), at[u]);
    }
}

constexpr int64_t kManyTokens = kSMs * 16;

// A group of tpr threads per token walks the row, CH choices at a time and U
// words of each in flight; a block whose groups are wider than a warp joins
// the warps' sums in shared memory.  Shifted rows' sums run over dy's words from
// the row's start, wherever the row lies.
template <int VEC, typename T, int CH, int U>
__global__ void __launch_bounds__(kMoveThreads, 2) route_combine_grad_kernel(const MoveParams p, const uint8_t *dy,
                                                                          int64_t pitch, Span dy_in, const uint8_t *ys,
                                                                          Span in, const float *__restrict__ weights,
                                                                          uint8_t *dys, float *__restrict__ dweights) {
    using P = Word<T, VEC>;
    __shared__ float part[CH][kMoveThreads / 32];
    griddep_wait();
    const int tpr = 1 << p.tpr_log2;
    const int64_t t = (int64_t)blockIdx.x * (kMoveThreads >> p.tpr_log2) + (threadIdx.x >> p.tpr_log2);
    const int sub = threadIdx.x & (tpr - 1), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool live = t < p.n;
    const int kept = p.offsets[p.n_experts];
    const int64_t limit = kept < p.slots ? kept : p.slots;
    for (int j0 = 0; j0 < p.topk; j0 += CH) {
        float sum[CH], w[CH];
        int row[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int j = j0 + c;
            sum[c] = 0.f;
            row[c] = live && j < p.topk ? p.rows[t * p.topk + j] : -1;
            w[c] = row[c] >= 0 ? weights[t * p.topk + j] : 0.f;
            if (row[c] >= p.slots) row[c] = -1;
        }
        for (int v0 = sub; live && v0 < p.words; v0 += tpr * U) {
            P g[U], got[CH][U];
            bool here[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = (int64_t)(v0 + u * tpr) * kWordBytes<VEC>;
                const int bytes = (int)min((int64_t)kWordBytes<VEC>, p.row_bytes - at);
                here[u] = bytes > 0;
                if (!here[u]) continue;
                if constexpr (VEC > 2)
                    g[u] = load_strided<T, VEC>(dy + t * pitch + at, p.align, dy_in);
                else
                    g[u] = P::of(load_piece<false>(dy + t * pitch + at, bytes, dy_in));
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (row[c] < 0 || row[c] >= limit) continue;
                    if constexpr (VEC > 2)
                        got[c][u] = load_row<T, VEC>(ys + row[c] * p.row_bytes + at, in);
                    else
                        got[c][u] = P::of(load_piece<false>(ys + row[c] * p.row_bytes + at, bytes, in));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float gf[P::V], f[P::V];
                g[u].to_floats(gf);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const bool on = row[c] >= 0 && row[c] < limit;
                    if (here[u] && on) {
                        got[c][u].to_floats(f);
#pragma unroll
                        for (int i = 0; i < P::V; ++i) sum[c] = fmaf(gf[i], f[i], sum[c]);
                    }
                    if (row[c] < 0) continue;
                    uint8_t *dst = dys + row[c] * p.row_bytes;
                    const RowWord to = row_word<VEC>(dst, v0 + u * tpr, p);
                    if (to.hi <= 0) continue;
                    if constexpr (VEC > 2) {
#pragma unroll
                        for (int i = 0; i < P::V; ++i) f[i] = gf[i];
                    } else {
                        load_row<T, VEC>(dy + t * pitch + to.at, dy_in).to_floats(f);
                    }
#pragma unroll
                    for (int i = 0; i < P::V; ++i) f[i] = on ? w[c] * f[i] : 0.f;
                    store_row<T, VEC>(dst + to.at, P::from_floats(f), to);
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < CH; ++c)
            for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) sum[c] += __shfl_xor_sync(kFull, sum[c], o);
        if (tpr > 32) {
            __syncthreads();  // the previous choices' sums have been read
            if (lane == 0) {
#pragma unroll
                for (int c = 0; c < CH; ++c) part[c][warp] = sum[c];
            }
            __syncthreads();
            const int first = (threadIdx.x >> p.tpr_log2) * (tpr / 32);
            if (sub == 0) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    float s = 0.f;
                    for (int i = 0; i < tpr / 32; ++i) s += part[c][first + i];
                    sum[c] = s;
                }
            }
        }
        if (live && sub == 0) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (j0 + c < p.topk) dweights[t * p.topk + j0 + c] = sum[c];
        }
    }
}

int elem_bytes(int dtype) { return dtype == KMEANS_F32 ? 4 : 2; }

// The most bytes, 16, 8, 4 or 2, that every row starts on a multiple of.
int rows_align(int64_t pitch_bytes, std::initializer_list<const void *> ptrs) {
    uint64_t bits = (uint64_t)pitch_bytes | 16u;
    for (const void *q : ptrs) bits |= reinterpret_cast<uintptr_t>(q);
    return (int)(bits & (~bits + 1));
}

Span span(const void *base, int64_t rows, int64_t pitch_bytes, int64_t row_bytes) {
    const uint8_t *b = static_cast<const uint8_t *>(base);
    return {b, base && rows > 0 ? b + (rows - 1) * pitch_bytes + row_bytes : b};
}

int log2_at_least(int64_t v, int most) {
    int l = 0;
    while ((1 << l) < v && l < most) ++l;
    return l;
}

// The stored rows have words of vec bytes (2: shifted ones); the strided
// operand's rows are aligned to `align`.
MoveParams move_params(const RouteRows &r, int bytes_per, int vec, int align) {
    MoveParams p{};
    p.rows = r.rows;
    p.offsets = r.offsets;
    p.n = r.n;
    p.slots = r.n * r.topk;
    p.row_bytes = r.d * bytes_per;
    p.words = (int)(vec > 2 ? p.row_bytes / vec : (p.row_bytes + 29) / 16);  // a row may start 14 bytes into a word
    p.align = align;
    p.topk = r.topk;
    p.n_experts = r.n_experts;
    return p;
}

// Threads per row, 1 to 256 as a power of two, for rows of `units` of a
// thread's work: the count that leaves the fewest threads without any (129
// pieces take 160 threads by 32, 256 by 256).
int threads_per_row_log2(int64_t units) {
    int best = log2_at_least(units, 8);
    for (int l = best - 1; l >= 5; --l) {
        const auto used = [&](int k) { return ((units + (1 << k) - 1) >> k) << k; };
        if (used(l) < used(best) && (used(l) >> l) <= 65535) best = l;  // blocks of a grid's second dimension
    }
    return best;
}

unsigned row_blocks(const MoveParams &p) {
    const int64_t per = kMoveThreads >> p.tpr_log2;
    return (unsigned)((p.n + per - 1) / per);
}

// A grid over rows of p.words words, `each` to a thread.
dim3 word_grid(MoveParams &p, int each) {
    p.tpr_log2 = threads_per_row_log2((p.words + each - 1) / each);
    const int per = each << p.tpr_log2;
    return dim3(row_blocks(p), (unsigned)((p.words + per - 1) / per));
}

template <int VEC, typename T, int CH, int U>
cudaError_t combine_as(MoveParams p, const void *ys, const float *weights, const void *residual, int64_t pitch, void *y,
                       cudaStream_t s) {
    const dim3 grid = word_grid(p, U);
    return launch_kernel(true, route_combine_kernel<VEC, T, CH, U>, grid, dim3(kMoveThreads), 0, s, p,
                         static_cast<const uint8_t *>(ys), span(ys, p.slots, p.row_bytes, p.row_bytes), weights,
                         static_cast<const uint8_t *>(residual), pitch, span(residual, p.n, pitch, p.row_bytes),
                         static_cast<uint8_t *>(y));
}

template <typename T>
cudaError_t combine_typed(const RouteRows &r, const void *ys, const float *weights, const void *residual, int64_t ldr,
                          void *y, cudaStream_t s) {
    const int64_t pitch = ldr * (int64_t)sizeof(T);
    const int vec = rows_align(r.d * (int64_t)sizeof(T), {ys, y});
    const MoveParams p = move_params(r, (int)sizeof(T), vec, residual ? rows_align(pitch, {residual}) : 16);
    if constexpr (sizeof(T) == 2) {
        // 4097 tokens of 3 choices, d = 1031: four rows' words in flight 13.3 us,
        // two of two rows 12.1; 16384 of 8, d = 2047: 224 and 263
        if (vec == 2 && p.topk > 4) return combine_as<2, T, 4, 1>(p, ys, weights, residual, pitch, y, s);
        if (vec == 2) return combine_as<2, T, 2, 2>(p, ys, weights, residual, pitch, y, s);
    }
    // short words: more of one row rather than more rows (16384 tokens of 8
    // choices, d = 2046 bf16: one row's eight words 154 us, four rows' two 212,
    // eight rows' two 247; d = 2044: two rows' four words 127 us, one row's eight 134, eight
    // rows' one 291)
    if (vec == 4) return combine_as<4, T, 1, 8>(p, ys, weights, residual, pitch, y, s);
    if (vec == 8) return combine_as<8, T, 2, 4>(p, ys, weights, residual, pitch, y, s);
    // several words per thread only where the rows still fill the SMs
    const bool many = p.n * p.words >= kSMs * 2048 * 4;
    if (p.topk > 3 || !many) return combine_as<16, T, 4, 1>(p, ys, weights, residual, pitch, y, s);
    if (p.topk > 1) return combine_as<16, T, 2, 2>(p, ys, weights, residual, pitch, y, s);
    return combine_as<16, T, 1, 4>(p, ys, weights, residual, pitch, y, s);
}

template <int VEC, typename T, int CH, int U>
cudaError_t combine_grad_as(MoveParams p, const void *dy, int64_t pitch, const void *ys, const float *weights, void *dys,
                            float *dweights, cudaStream_t s) {
    // a warp per token where there are enough of them: no block-wide join, and
    // the rows of other tokens hide each other's latency (16384 tokens of 8
    // choices, d = 2048: a block per token 344 us, 178 so)
    p.tpr_log2 = log2_at_least((p.row_bytes + kWordBytes<VEC> - 1) / kWordBytes<VEC>, p.n >= kManyTokens ? 5 : 8);
    return launch_kernel(true, route_combine_grad_kernel<VEC, T, CH, U>, dim3(row_blocks(p)), dim3(kMoveThreads), 0, s,
                         p, static_cast<const uint8_t *>(dy), pitch, span(dy, p.n, pitch, p.row_bytes),
                         static_cast<const uint8_t *>(ys), span(ys, p.slots, p.row_bytes, p.row_bytes), weights,
                         static_cast<uint8_t *>(dys), dweights);
}

template <typename T>
cudaError_t combine_grad_typed(const RouteRows &r, const void *dy, int64_t lddy, const void *ys, const float *weights,
                               void *dys, float *dweights, cudaStream_t s) {
    const int64_t pitch = lddy * (int64_t)sizeof(T);
    const int vec = rows_align(r.d * (int64_t)sizeof(T), {ys, dys});
    const MoveParams p = move_params(r, (int)sizeof(T), vec, rows_align(pitch, {dy}));
    if constexpr (sizeof(T) == 2) {
        // a shifted word takes the registers of two
        if (vec == 2)
            return r.topk > 2 ? combine_grad_as<2, T, 4, 1>(p, dy, pitch, ys, weights, dys, dweights, s)
                              : combine_grad_as<2, T, 2, 2>(p, dy, pitch, ys, weights, dys, dweights, s);
    }
    // short words: two choices of eight words each, or as many rows as there are
    // choices (5233 tokens of 2 choices, d = 4554 bf16: four choices' four words
    // 102 us, two choices' eight 65; 13051 of 6, d = 1714 float32, words of 8 bytes:
    // four choices' four words 224 us, two choices' eight 208)
    if (vec == 4 && p.topk <= 2) return combine_grad_as<4, T, 2, 8>(p, dy, pitch, ys, weights, dys, dweights, s);
    if (vec == 4 && p.topk > 4) return combine_grad_as<4, T, 8, 4>(p, dy, pitch, ys, weights, dys, dweights, s);
    if (vec == 4) return combine_grad_as<4, T, 4, 4>(p, dy, pitch, ys, weights, dys, dweights, s);
    if (vec == 8) return combine_grad_as<8, T, 2, 8>(p, dy, pitch, ys, weights, dys, dweights, s);
    if (p.topk > 4) return combine_grad_as<16, T, 8, 1>(p, dy, pitch, ys, weights, dys, dweights, s);
    if (p.topk > 2) return combine_grad_as<16, T, 4, 2>(p, dy, pitch, ys, weights, dys, dweights, s);
    return combine_grad_as<16, T, 2, 4>(p, dy, pitch, ys, weights, dys, dweights, s);
}

// Most blocks of one cluster: 16 where the device can hold such a cluster (it
// needs that many free SMs next to each other), else the portable 8.
template <typename Id>
int route_max_cluster() {
    static std::atomic<int> cached[kMaxDevices];
    return cached_per_device(cached, [] {
        if (cudaFuncSetAttribute(route_kernel<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRouteSmemMax) !=
                cudaSuccess ||
            cudaFuncSetAttribute(route_kernel<Id>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            cudaGetLastError();  // clear; the launch reports what is wrong
            return 8;
        }
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(kRouteMaxCluster);
        cfg.blockDim = dim3(kRouteThreads);
        cfg.dynamicSmemBytes = kRouteSmemMax;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = kRouteMaxCluster;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, route_kernel<Id>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            clusters = 0;
        }
        return clusters > 0 ? kRouteMaxCluster : 8;
    });
}

template <typename Id>
cudaError_t route_as(const RouteParams &p, int blocks, int threads, size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, route_kernel<Id>, p);
}

}  // namespace

cudaError_t launch_route(const void *experts, int id_bytes, int64_t slots, int n_experts, int32_t *offsets,
                         int32_t *order, int32_t *rows, uint32_t *status, cudaStream_t s) {
    RouteParams p{};
    p.experts = experts;
    p.slots = (int)slots;
    p.n_experts = n_experts;
    p.offsets = offsets;
    p.order = order;
    p.rows = rows;
    p.status = status;
    const int keys = n_experts + 1;
    const int room = (kRouteSmemMax - 2 * keys * 4 - 128) / (keys * 4);
    const int most = id_bytes == 8 ? route_max_cluster<int64_t>() : route_max_cluster<int32_t>();
    int blocks = 1;
    while (blocks < most && (int64_t)blocks * kRouteSlotsPerBlock < slots) blocks *= 2;
    // no more counting warps than groups of 32 slots: their counts are cleared
    // and added up key by key
    const int64_t groups = (slots + 31) / 32, per_block = (groups + blocks - 1) / blocks;
    p.warps = room < kRouteThreads / 32 ? room : kRouteThreads / 32;
    if (per_block < p.warps) p.warps = per_block > 0 ? (int)per_block : 1;
    const int threads = p.warps > 8 || keys > 512 ? kRouteThreads : 256;
    const size_t smem = (size_t)((p.warps + 2) * keys + 32) * 4;
    return id_bytes == 8 ? route_as<int64_t>(p, blocks, threads, smem, s) : route_as<int32_t>(p, blocks, threads, smem, s);
}

cudaError_t launch_route_gather(const RouteRows &r, int dtype, const void *x, int64_t ldx, void *xs, cudaStream_t s) {
    const int bytes = elem_bytes(dtype);
    const int64_t pitch = ldx * bytes;
    const int vec = rows_align(r.d * bytes, {xs});
    MoveParams p = move_params(r, bytes, vec, rows_align(pitch, {x}));
    const auto as = [&](auto kernel, int unroll) {
        const dim3 grid = word_grid(p, unroll);
        return launch_kernel(true, kernel, grid, dim3(kMoveThreads), 0, s, p, static_cast<const uint8_t *>(x), pitch,
                             span(x, p.n, pitch, p.row_bytes), static_cast<uint8_t *>(xs));
    };
    if (vec == 16) return as(route_gather_kernel<16>, kGatherUnroll<16>);
    if (vec == 8) return as(route_gather_kernel<8>, kGatherUnroll<8>);
    if (vec == 4) return as(route_gather_kernel<4>, kGatherUnroll<4>);
    return as(route_gather_kernel<2>, kGatherUnroll<2>);
}

cudaError_t launch_route_combine(const RouteRows &r, int dtype, const void *ys, const float *weights,
                                 const void *residual, int64_t ldr, void *y, cudaStream_t s) {
    switch (dtype) {
        case KMEANS_F32: return combine_typed<float>(r, ys, weights, residual, ldr, y, s);
        case KMEANS_F16: return combine_typed<__half>(r, ys, weights, residual, ldr, y, s);
        default: return combine_typed<__nv_bfloat16>(r, ys, weights, residual, ldr, y, s);
    }
}

cudaError_t launch_route_combine_grad(const RouteRows &r, int dtype, const void *dy, int64_t lddy, const void *ys,
                                      const float *weights, void *dys, float *dweights, cudaStream_t s) {
    switch (dtype) {
        case KMEANS_F32: return combine_grad_typed<float>(r, dy, lddy, ys, weights, dys, dweights, s);
        case KMEANS_F16: return combine_grad_typed<__half>(r, dy, lddy, ys, weights, dys, dweights, s);
        default: return combine_grad_typed<__nv_bfloat16>(r, dy, lddy, ys, weights, dys, dweights, s);
    }
}

}  // namespace km
