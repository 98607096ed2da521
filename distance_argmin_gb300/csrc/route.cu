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

#include "experts.cuh"
#include "ptx.cuh"

namespace km {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ------------------------------------------------------------------ the sort
constexpr int kRouteThreads = 1024;
constexpr int kRouteSmemMax = 224 * 1024;
constexpr int kRouteMaxCluster = 8;
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

template <typename Id>
__device__ __forceinline__ int route_key(const Id *experts, uint32_t s, int n_experts, bool &bad) {
    const Id v = experts[s];
    if (v >= (Id)n_experts) bad = true;
    return (v < 0 || v >= (Id)n_experts) ? n_experts : (int)v;
}

// Shared memory: hist[warps][keys], tot[keys], base[keys], 32 words of scan
// scratch, with keys = n_experts + 1.
template <typename Id>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
    extern __shared__ int route_smem[];
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
    for (int i = tid; i < p.warps * keys; i += blockDim.x) hist[i] = 0;
    __syncthreads();

    // this warp's run of consecutive slots, whole groups of 32
    const int total_warps = blocks * p.warps;
    const int groups = (int)(((uint32_t)p.slots + 31u) / 32u);
    const int per = (groups + total_warps - 1) / total_warps;
    const int64_t g0 = (int64_t)((int)rank * p.warps + warp) * per;
    const uint32_t s0 = (uint32_t)min(g0 * 32, (int64_t)p.slots);
    const uint32_t s1 = warp < p.warps ? (uint32_t)min((g0 + per) * 32, (int64_t)p.slots) : s0;
    int *mine = hist + warp * keys;

    bool bad = false;
    for (uint32_t s = s0; s < s1; s += 32) {
        const bool live = s + lane < s1;
        const int key = live ? route_key(experts, s + lane, p.n_experts, bad) : -1;
        const uint32_t same = __match_any_sync(kFull, key);
        if (live && (same & below) == 0u) mine[key] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // per key: each warp's first place among this block's, and the block's total
    for (int e = tid; e < keys; e += blockDim.x) {
        int sum = 0;
        for (int w = 0; w < p.warps; ++w) {
            const int c = hist[w * keys + e];
            hist[w * keys + e] = sum;
            sum += c;
        }
        tot[e] = sum;
    }
    cluster_sync();  // every block's totals are readable; the status word is cleared
    if (__syncthreads_or(bad) && tid == 0) flag_error(p.status, kFlagBadLabel);

    // base[e] = all slots of smaller keys + the lower blocks' slots of key e
    int run = 0;  // keys are scanned blockDim.x at a time
    for (int e0 = 0; e0 < keys; e0 += blockDim.x) {
        const int e = e0 + tid;
        int all = 0, lower = 0;
        if (e < keys)
            for (int r = 0; r < blocks; ++r) {
                const int c = blocks == 1 ? tot[e] : ld_cluster_i32(tot + e, (uint32_t)r);
                all += c;
                if (r < (int)rank) lower += c;
            }
        int inc = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        int before = 0, chunk = 0;
        for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
            const int v = scan[w];
            if (w < warp) before += v;
            chunk += v;
        }
        if (e < keys) {
            const int first = run + before + inc - all;
            base[e] = first + lower;
            if (rank == 0) p.offsets[e] = first;  // offsets[n_experts]: the kept slots
        }
        run += chunk;
        __syncthreads();
    }
    // hand out rows
    for (uint32_t s = s0; s < s1; s += 32) {
        const bool live = s + lane < s1;
        const int key = live ? route_key(experts, s + lane, p.n_experts, bad) : -1;
        const uint32_t same = __match_any_sync(kFull, key);
        int row = 0;
        if (live) row = base[key] + mine[key] + __popc(same & below);
        __syncwarp();
        if (live && (same & below) == 0u) mine[key] += __popc(same);
        __syncwarp();
        if (live) {
            p.rows[s + lane] = row;
            p.order[row] = (int)(s + lane);
        }
    }
    cluster_sync();  // no block leaves while another may still read its totals
}

// -------------------------------------------------------------- row movement
template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }

// V consecutive elements moved as one access
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

// A piece of V elements at p, the first `left` of which exist, as one access
// (WHOLE: aligned, and every piece is complete) or element by element.
template <bool WHOLE, typename T, int V>
__device__ __forceinline__ Pack<T, V> load_piece(const T *p, int64_t left) {
    if constexpr (WHOLE) return *reinterpret_cast<const Pack<T, V> *>(p);
    Pack<T, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) v.v[i] = i < left ? p[i] : from_float<T>(0.f);
    return v;
}

template <bool WHOLE, typename T, int V>
__device__ __forceinline__ void store_piece(T *p, const Pack<T, V> &v, int64_t left) {
    if constexpr (WHOLE) {
        *reinterpret_cast<Pack<T, V> *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < left) p[i] = v.v[i];
    }
}

struct MoveParams {
    const int32_t *rows, *offsets;
    int64_t n, slots, vecs;  // vecs: pieces (accesses) per row
    int topk, n_experts;
    int tpr_log2;  // threads per row
};

constexpr int kMoveThreads = 256;
constexpr int kGatherUnroll = 4;

// xs[row(t, j)] = x[t]; a thread holds up to kGatherUnroll pieces of its token
// and writes them to every choice's row.
template <typename W>
__global__ void __launch_bounds__(kMoveThreads) route_gather_kernel(const MoveParams p, const W *__restrict__ x,
                                                                    int64_t ldx, W *__restrict__ xs) {
    griddep_wait();
    const int tpr = 1 << p.tpr_log2;
    const int64_t t = (int64_t)blockIdx.x * (kMoveThreads >> p.tpr_log2) + (threadIdx.x >> p.tpr_log2);
    if (t >= p.n) return;
    const int64_t v0 = (int64_t)blockIdx.y * (tpr * kGatherUnroll) + (threadIdx.x & (tpr - 1));
    const int kept = p.offsets[p.n_experts];
    W val[kGatherUnroll];
#pragma unroll
    for (int u = 0; u < kGatherUnroll; ++u)
        if (v0 + u * tpr < p.vecs) val[u] = x[t * ldx + v0 + u * tpr];
    for (int j = 0; j < p.topk; ++j) {
        const int r = p.rows[t * p.topk + j];
        if (r < 0 || r >= p.slots) continue;
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u)
            if (v0 + u * tpr < p.vecs) xs[(int64_t)r * p.vecs + v0 + u * tpr] = r < kept ? val[u] : W{};
    }
}

constexpr int kCombineUnroll = 4;  // choices whose rows are in flight together

template <typename T, int V>
__global__ void __launch_bounds__(kMoveThreads) route_combine_kernel(const MoveParams p, const T *__restrict__ ys,
                                                                     const float *__restrict__ weights,
                                                                     const T *residual, int64_t ldr, T *y) {
    using P = Pack<T, V>;
    griddep_wait();
    const int tpr = 1 << p.tpr_log2;
    const int64_t t = (int64_t)blockIdx.x * (kMoveThreads >> p.tpr_log2) + (threadIdx.x >> p.tpr_log2);
    const int64_t v = (int64_t)blockIdx.y * tpr + (threadIdx.x & (tpr - 1));
    if (t >= p.n || v >= p.vecs) return;
    const int kept = p.topk > 0 ? p.offsets[p.n_experts] : 0;
    const int64_t limit = kept < p.slots ? kept : p.slots;
    const int64_t d = p.vecs * V;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < p.topk; j0 += kCombineUnroll) {
        P part[kCombineUnroll];
        float w[kCombineUnroll];
        bool on[kCombineUnroll];
#pragma unroll
        for (int u = 0; u < kCombineUnroll; ++u) {
            const int j = j0 + u;
            const int r = j < p.topk ? p.rows[t * p.topk + j] : -1;
            on[u] = r >= 0 && r < limit;
            if (on[u]) {
                w[u] = weights ? weights[t * p.topk + j] : 1.f;
                part[u] = *reinterpret_cast<const P *>(ys + r * d + v * V);
            }
        }
#pragma unroll
        for (int u = 0; u < kCombineUnroll; ++u)
            if (on[u]) {
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(w[u], to_float(part[u].v[i]), acc[i]);
            }
    }
    P out;
    if (residual) {
        const P res = *reinterpret_cast<const P *>(residual + t * ldr + v * V);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += to_float(res.v[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) out.v[i] = from_float<T>(acc[i]);
    *reinterpret_cast<P *>(y + t * d + v * V) = out;
}

constexpr int kGradChoices = 8;  // choices whose products a thread sums in one walk along the row

// One group of tpr threads per token walks the row; a block whose groups are
// wider than a warp joins the warps' sums in shared memory.  A thread takes
// the same V elements at a time whatever the alignment, so the sums have one
// order.
template <bool WHOLE, typename T, int V>
__global__ void __launch_bounds__(kMoveThreads) route_combine_grad_kernel(const MoveParams p, int64_t d,
                                                                          const T *__restrict__ dy, int64_t lddy,
                                                                          const T *__restrict__ ys,
                                                                          const float *__restrict__ weights,
                                                                          T *__restrict__ dys,
                                                                          float *__restrict__ dweights) {
    using P = Pack<T, V>;
    __shared__ float part[kGradChoices][kMoveThreads / 32];
    griddep_wait();
    const int tpr = 1 << p.tpr_log2;
    const int64_t t = (int64_t)blockIdx.x * (kMoveThreads >> p.tpr_log2) + (threadIdx.x >> p.tpr_log2);
    const int sub = threadIdx.x & (tpr - 1), warp = threadIdx.x >> 5;
    const bool live = t < p.n;
    const int kept = p.offsets[p.n_experts];
    const int64_t limit = kept < p.slots ? kept : p.slots;
    for (int j0 = 0; j0 < p.topk; j0 += kGradChoices) {
        float sum[kGradChoices], w[kGradChoices];
        int row[kGradChoices];
#pragma unroll
        for (int u = 0; u < kGradChoices; ++u) {
            const int j = j0 + u;
            sum[u] = 0.f;
            row[u] = live && j < p.topk ? p.rows[t * p.topk + j] : -1;
            if (row[u] >= p.slots) row[u] = -1;
            w[u] = row[u] >= 0 && row[u] < limit ? weights[t * p.topk + j] : 0.f;
        }
        if (live)
            for (int64_t v = sub; v < p.vecs; v += tpr) {
                const int64_t left = d - v * V;
                const P g = load_piece<WHOLE, T, V>(dy + t * lddy + v * V, left);
                P in[kGradChoices];
#pragma unroll
                for (int u = 0; u < kGradChoices; ++u)
                    if (row[u] >= 0 && row[u] < limit) in[u] = load_piece<WHOLE, T, V>(ys + row[u] * d + v * V, left);
#pragma unroll
                for (int u = 0; u < kGradChoices; ++u) {
                    if (row[u] < 0) continue;
                    const bool on = row[u] < limit;
                    P out;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float gi = to_float(g.v[i]);
                        out.v[i] = from_float<T>(on ? w[u] * gi : 0.f);
                        if (on) sum[u] = fmaf(gi, to_float(in[u].v[i]), sum[u]);
                    }
                    store_piece<WHOLE, T, V>(dys + row[u] * d + v * V, out, left);
                }
            }
#pragma unroll
        for (int u = 0; u < kGradChoices; ++u)
            for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) sum[u] += __shfl_xor_sync(kFull, sum[u], o);
        if (tpr > 32) {
            __syncthreads();  // the previous choices' sums have been read
            if ((threadIdx.x & 31) == 0) {
#pragma unroll
                for (int u = 0; u < kGradChoices; ++u) part[u][warp] = sum[u];
            }
            __syncthreads();
            const int first = (threadIdx.x >> p.tpr_log2) * (tpr / 32);
            if (sub == 0) {
#pragma unroll
                for (int u = 0; u < kGradChoices; ++u) {
                    float s = 0.f;
                    for (int i = 0; i < tpr / 32; ++i) s += part[u][first + i];
                    sum[u] = s;
                }
            }
        }
        if (live && sub == 0) {
#pragma unroll
            for (int u = 0; u < kGradChoices; ++u)
                if (j0 + u < p.topk) dweights[t * p.topk + j0 + u] = sum[u];
        }
    }
}

int elem_bytes(int dtype) { return dtype == KMEANS_F32 ? 4 : 2; }

// Widest access (bytes, a power of two up to 16) that every row start allows.
int row_access(int64_t row_bytes, int64_t pitch_bytes, std::initializer_list<const void *> ptrs) {
    uint64_t bits = (uint64_t)row_bytes | (uint64_t)pitch_bytes | 16u;
    for (const void *q : ptrs) bits |= reinterpret_cast<uintptr_t>(q);
    return (int)(bits & (~bits + 1));
}

int log2_at_least(int64_t v, int most) {
    int l = 0;
    while ((1 << l) < v && l < most) ++l;
    return l;
}

MoveParams move_params(const RouteRows &r, int64_t vecs, int tpr_log2) {
    MoveParams p{};
    p.rows = r.rows;
    p.offsets = r.offsets;
    p.n = r.n;
    p.slots = r.n * r.topk;
    p.vecs = vecs;
    p.topk = r.topk;
    p.n_experts = r.n_experts;
    p.tpr_log2 = tpr_log2;
    return p;
}

template <typename W>
cudaError_t gather_as(const RouteRows &r, int64_t row_bytes, int64_t pitch_bytes, const void *x, void *xs,
                      cudaStream_t s) {
    const int64_t vecs = row_bytes / (int64_t)sizeof(W);
    const int l = log2_at_least((vecs + kGatherUnroll - 1) / kGatherUnroll, 8);
    const MoveParams p = move_params(r, vecs, l);
    const int64_t per_y = (int64_t)kGatherUnroll << l;
    const dim3 grid((unsigned)((r.n + (kMoveThreads >> l) - 1) / (kMoveThreads >> l)),
                    (unsigned)((vecs + per_y - 1) / per_y));
    return launch_kernel(true, route_gather_kernel<W>, grid, dim3(kMoveThreads), 0, s, p, static_cast<const W *>(x),
                         pitch_bytes / (int64_t)sizeof(W), static_cast<W *>(xs));
}

template <typename T, int V>
cudaError_t combine_as(const RouteRows &r, const void *ys, const float *weights, const void *residual, int64_t ldr,
                       void *y, cudaStream_t s) {
    const int64_t vecs = r.d / V;
    const int l = log2_at_least(vecs, 8);
    const dim3 grid((unsigned)((r.n + (kMoveThreads >> l) - 1) / (kMoveThreads >> l)),
                    (unsigned)((vecs + (1 << l) - 1) >> l));
    return launch_kernel(true, route_combine_kernel<T, V>, grid, dim3(kMoveThreads), 0, s, move_params(r, vecs, l),
                         static_cast<const T *>(ys), weights, static_cast<const T *>(residual), ldr,
                         static_cast<T *>(y));
}

template <bool WHOLE, typename T, int V>
cudaError_t combine_grad_as(const RouteRows &r, const void *dy, int64_t lddy, const void *ys, const float *weights,
                            void *dys, float *dweights, cudaStream_t s) {
    const int64_t vecs = (r.d + V - 1) / V;
    const int l = log2_at_least(vecs, 8);
    const dim3 grid((unsigned)((r.n + (kMoveThreads >> l) - 1) / (kMoveThreads >> l)));
    return launch_kernel(true, route_combine_grad_kernel<WHOLE, T, V>, grid, dim3(kMoveThreads), 0, s, move_params(r, vecs, l), r.d,
                         static_cast<const T *>(dy), lddy, static_cast<const T *>(ys), weights, static_cast<T *>(dys),
                         dweights);
}

template <typename T>
cudaError_t combine_typed(const RouteRows &r, const void *ys, const float *weights, const void *residual, int64_t ldr,
                          void *y, cudaStream_t s) {
    const int64_t b = sizeof(T);
    const int wide = row_access(r.d * b, residual ? ldr * b : 0, {ys, residual, y});
    return wide == 16 ? combine_as<T, 16 / (int)sizeof(T)>(r, ys, weights, residual, ldr, y, s)
                      : combine_as<T, 1>(r, ys, weights, residual, ldr, y, s);
}

template <typename T>
cudaError_t combine_grad_typed(const RouteRows &r, const void *dy, int64_t lddy, const void *ys, const float *weights,
                               void *dys, float *dweights, cudaStream_t s) {
    const int64_t b = sizeof(T);
    const int wide = row_access(r.d * b, lddy * b, {dy, ys, dys});
    constexpr int V = 16 / (int)sizeof(T);
    return wide == 16 ? combine_grad_as<true, T, V>(r, dy, lddy, ys, weights, dys, dweights, s)
                      : combine_grad_as<false, T, V>(r, dy, lddy, ys, weights, dys, dweights, s);
}

template <typename Id>
cudaError_t route_as(const RouteParams &p, int blocks, size_t smem, cudaStream_t s) {
    static std::once_flag once[kMaxDevices];
    static std::atomic<int> err[kMaxDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    const int slot = dev >= 0 && dev < kMaxDevices ? dev : 0;
    once_per_device(once, [&] {
        err[slot].store((int)cudaFuncSetAttribute(route_kernel<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                  kRouteSmemMax));
    });
    if (err[slot].load() != cudaSuccess) return (cudaError_t)err[slot].load();
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kRouteThreads);
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
    p.warps = room < kRouteThreads / 32 ? room : kRouteThreads / 32;
    int blocks = 1;
    while (blocks < kRouteMaxCluster && (int64_t)blocks * kRouteSlotsPerBlock < slots) blocks *= 2;
    const size_t smem = (size_t)((p.warps + 2) * keys + 32) * 4;
    return id_bytes == 8 ? route_as<int64_t>(p, blocks, smem, s) : route_as<int32_t>(p, blocks, smem, s);
}

cudaError_t launch_route_gather(const RouteRows &r, int dtype, const void *x, int64_t ldx, void *xs, cudaStream_t s) {
    const int64_t b = elem_bytes(dtype);
    switch (row_access(r.d * b, ldx * b, {x, xs})) {
        case 16: return gather_as<uint4>(r, r.d * b, ldx * b, x, xs, s);
        case 8: return gather_as<uint2>(r, r.d * b, ldx * b, x, xs, s);
        case 4: return gather_as<uint32_t>(r, r.d * b, ldx * b, x, xs, s);
        default: return gather_as<uint16_t>(r, r.d * b, ldx * b, x, xs, s);
    }
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
