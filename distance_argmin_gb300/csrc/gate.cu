// The gate: which experts a token goes to, and with what weights.
//
//   s = softmax(l) or 1 / (1 + exp(-l))      scores of the experts
//   c = s + b                                what the choice goes by
//
// With groups of neighbouring experts, those of the topk_groups groups whose two
// largest c have the largest sum stay; then the topk largest c are taken one
// after the other, equal ones by index.  A logit or a bias of minus infinity
// closes the expert: it is not chosen, and a token with too few open experts
// gets -1 with weight 0.  NaN counts as the largest value, so that a token that
// holds one shows it in its weights.
//
// The choice is that of exact arithmetic.  Without a bias the order is the
// logits' own.  Sums (c, and the groups' scores) are formed in float32; where two
// neighbours in the order, the last chosen and the first left out among them, are
// nearer than their errors (gap_of) and not equal in both logit and bias, the row
// is done again in float64.
//
// A warp has a token, a lane every 32nd expert.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "assign_common.cuh"
#include "layer.cuh"
#include "pieces.cuh"

namespace km {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kGateThreads = 128;

template <typename T>
__device__ __forceinline__ float load_logit(const T *p) {
    if constexpr (sizeof(T) == 4)
        return *p;
    else
        return widen<T>(*p);
}

template <typename T>
__device__ __forceinline__ void store_logit(T *p, float v) {
    if constexpr (sizeof(T) == 4)
        *p = v;
    else
        *p = narrow<T>(v);
}

// Order-preserving keys: 0 for what cannot be chosen, NaN the largest, the two
// zeros equal.
__device__ __forceinline__ uint32_t choice_key(float v) {
    if (v == -INFINITY) return 0u;
    if (v != v) return 0xffffffffu;
    return float_to_ord(v + 0.f);
}
__device__ __forceinline__ uint64_t choice_key(double v) {
    if (v == -(double)INFINITY) return 0ull;
    if (v != v) return ~0ull;
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ float key_value(uint32_t k) { return ord_to_float(k); }
__device__ __forceinline__ double key_value(uint64_t k) {
    return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float warp_fmax(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

// The largest key of the warp and the lowest expert that has it, which is taken
// out; -1 where nothing is left.
template <int PER>
__device__ __forceinline__ int take_best(uint32_t (&key)[PER], int lane, uint32_t &best) {
    uint32_t mine = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < PER; ++i)
        if (key[i] > mine) {
            mine = key[i];
            at = i;
        }
    best = warp_max(mine);
    if (best == 0) return -1;
    const int e = (int)__reduce_min_sync(kAll, mine == best ? (uint32_t)(at * 32 + lane) : 0x7fffffffu);
    if ((e & 31) == lane) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i == (e >> 5)) key[i] = 0;
    }
    return e;
}

// How near two values of the order may be in float32 without being looked at in
// float64: twice what they may be off by.  A score is off by less than 2^-18 (an
// exponential by |x| e^x 2^-23 + 2^-22 e^x, x <= 0; the sum of up to 4096 of
// them, 32 to an accumulator, by 39 2^-24 of itself; the quotient by 2^-22), the
// sum with the bias by half its last bit more, a group's two by twice that.
__device__ __forceinline__ float gap_of(float a, float b) { return 0x1p-17f + 0x1p-21f * (fabsf(a) + fabsf(b)); }

struct GateArgs {
    int64_t n, ldl;
    int n_experts, topk, groups, topk_groups, group_size;
    bool sigmoid, renormalize;
    float scale;
    const float *bias;
};

// The row's score parameters: softmax takes exp(l - top) / sum.
template <typename V>
struct Scores {
    bool sigmoid;
    V top, inverse;
};

__device__ __forceinline__ float score_of(const Scores<float> &s, float l) {
    if (s.sigmoid) return __fdividef(1.f, 1.f + __expf(-l));
    return __expf(l - s.top) * s.inverse;
}
__device__ __forceinline__ double score_of(const Scores<double> &s, float l) {
    if (s.sigmoid) return 1.0 / (1.0 + exp(-(double)l));
    return exp((double)l - s.top) * s.inverse;
}

template <typename V>
__device__ __forceinline__ V exp_of(V v) {
    if constexpr (sizeof(V) == 4)
        return __expf(v);
    else
        return exp(v);
}

// Chooses a row's experts: lane j receives the j-th (-1: none).  False: float32
// does not decide.
template <int PER, typename T>
__device__ __forceinline__ bool choose(const GateArgs &p, const T *row, int lane, const Scores<float> &sc, int &chosen) {
    using V = float;
    using K = uint32_t;
    K key[PER];
    const bool sums = p.bias || p.groups > 1;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        key[i] = 0;
        if (e < p.n_experts) {
            const float l = load_logit(row + e);
            if (l != -INFINITY) {
                V c = l;
                if (sums) c = score_of(sc, l);
                if (p.bias) c += (V)p.bias[e];
                key[i] = choice_key(c);
            }
        }
    }
    if (p.groups > 1) {
        K total[1] = {0};  // lane g: group g's score
        for (int g = 0; g < p.groups; ++g) {
            const int lo = g * p.group_size, hi = lo + p.group_size;
            K one = 0, two = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = i * 32 + lane;
                const K k = e >= lo && e < hi ? key[i] : 0;
                two = k > one ? one : (k > two ? k : two);
                one = k > one ? k : one;
            }
            const K first = warp_max(one);
            const uint32_t who = __ballot_sync(kAll, one == first);
            const K second = warp_max(lane == __ffs(who) - 1 ? two : one);
            if (lane == g && first) {
                V sum = key_value(first);
                if (second) sum += key_value(second);
                total[0] = choice_key(sum);
            }
        }
        uint32_t kept = 0;
        K last = 0, next;
        for (int j = 0; j < p.topk_groups; ++j) {
            const int g = take_best<1>(total, lane, next);
            if (g < 0) break;
            kept |= 1u << g;
            last = next;
        }
        // (equal sums are rarely sums of equal parts, so they are looked at too)
        if (take_best<1>(total, lane, next) >= 0 && last &&
            !(key_value(last) - key_value(next) > 2.f * gap_of(key_value(last), key_value(next))))
            return false;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 32 + lane;
            const bool in = e < p.n_experts && (kept >> (e / p.group_size) & 1u) && key[i];
            // without a bias the rest of the choice goes by the logits
            if (!in)
                key[i] = 0;
            else if (!p.bias)
                key[i] = choice_key((V)load_logit(row + e));
        }
    }
    chosen = -1;
    K value = 0, best;
    for (int j = 0; j < p.topk; ++j) {
        const int e = take_best(key, lane, best);
        if (e < 0) break;
        if (lane == j) {
            chosen = e;
            value = best;
        }
    }
    if (p.bias) {
        const int rest = take_best(key, lane, best);
        int after = __shfl_down_sync(kAll, chosen, 1);
        K after_value = __shfl_down_sync(kAll, value, 1);
        if (lane == p.topk - 1) {
            after = rest;
            after_value = best;
        }
        bool near = false;
        if (lane < p.topk && chosen >= 0 && after >= 0) {
            const V a = key_value(value), b = key_value(after_value);
            const bool same = load_logit(row + chosen) == load_logit(row + after) && p.bias[chosen] == p.bias[after];
            near = !(a - b > gap_of(a, b)) && !same;
        }
        if (__any_sync(kAll, near)) return false;
    }
    return true;
}

template <typename T, typename V>
__device__ __forceinline__ Scores<V> row_scores(const GateArgs &p, const T *row, int lane) {
    Scores<V> sc{p.sigmoid, 0, 0};
    if (p.sigmoid) return sc;
    float top = -INFINITY;
    for (int e = lane; e < p.n_experts; e += 32) top = fmaxf(top, load_logit(row + e));
    top = warp_fmax(top);
    sc.top = top == -INFINITY ? 0.f : top;  // no open expert: scores of 0
    V sum[4] = {};  // (a lane's 128 terms one after the other would lose up to 2^-17)
    for (int e0 = lane; e0 < p.n_experts; e0 += 128)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + i * 32;
            if (e < p.n_experts) sum[i] += exp_of((V)load_logit(row + e) - sc.top);
        }
    const V all = warp_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
    sc.inverse = all == (V)0 ? (V)0 : (V)1 / all;
    return sc;
}

// The same in float64, for the few rows that need it: as short as it can be, a
// lane's keys in local memory.
constexpr int kExactPer = KMEANS_ROUTE_MAX_EXPERTS / 32;

__device__ int take_best_exact(uint64_t *key, int per, int lane, uint64_t &best) {
    uint64_t mine = 0;
    int at = 0;
#pragma unroll 1
    for (int i = 0; i < per; ++i)
        if (key[i] > mine) {
            mine = key[i];
            at = i;
        }
    best = warp_max(mine);
    if (best == 0) return -1;
    const int e = (int)__reduce_min_sync(kAll, mine == best ? (uint32_t)(at * 32 + lane) : 0x7fffffffu);
    if ((e & 31) == lane) key[e >> 5] = 0;
    return e;
}

template <typename T>
__device__ __noinline__ int choose_exact(const GateArgs &p, const T *row, int lane) {
    uint64_t key[kExactPer];
    const Scores<double> sc = row_scores<T, double>(p, row, lane);
    const int per = (p.n_experts + 31) / 32;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        const int e = i * 32 + lane;
        const float l = e < p.n_experts ? load_logit(row + e) : -INFINITY;
        key[i] = 0;
        if (l != -INFINITY) key[i] = choice_key(score_of(sc, l) + (p.bias ? (double)p.bias[e] : 0.0));
    }
    uint64_t best;
    if (p.groups > 1) {
        uint64_t total = 0;
#pragma unroll 1
        for (int g = 0; g < p.groups; ++g) {
            const int lo = g * p.group_size, hi = lo + p.group_size;
            uint64_t one = 0, two = 0;
#pragma unroll 1
            for (int i = 0; i < per; ++i) {
                const int e = i * 32 + lane;
                const uint64_t k = e >= lo && e < hi ? key[i] : 0;
                two = k > one ? one : (k > two ? k : two);
                one = k > one ? k : one;
            }
            const uint64_t first = warp_max(one);
            const uint32_t who = __ballot_sync(kAll, one == first);
            const uint64_t second = warp_max(lane == __ffs(who) - 1 ? two : one);
            if (lane == g && first) total = choice_key(key_value(first) + (second ? key_value(second) : 0.0));
        }
        uint32_t kept = 0;
#pragma unroll 1
        for (int j = 0; j < p.topk_groups; ++j) {
            const int g = take_best_exact(&total, 1, lane, best);
            if (g < 0) break;
            kept |= 1u << g;
        }
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
            const int e = i * 32 + lane;
            if (key[i] && !(kept >> (e / p.group_size) & 1u))
                key[i] = 0;
            else if (key[i] && !p.bias)
                key[i] = choice_key((double)load_logit(row + e));
        }
    }
    int chosen = -1;
#pragma unroll 1
    for (int j = 0; j < p.topk; ++j) {
        const int e = take_best_exact(key, per, lane, best);
        if (e < 0) break;
        if (lane == j) chosen = e;
    }
    return chosen;
}

// The chosen experts' shares of their sum; lane j has expert j's logit.  Scaled
// by the largest of them where all are small, so that the quotient is defined.
__device__ __forceinline__ float share_of(bool sigmoid, float l, bool real) {
    float u;
    const float top = warp_fmax(real ? l : -INFINITY);
    if (sigmoid) {
        const float m = fminf(top, 0.f);
        u = l > 0.f ? __fdividef(1.f, 1.f + __expf(-l)) : __fdividef(__expf(l - m), 1.f + __expf(l));
    } else {
        u = __expf(l - top);
    }
    u = real ? u : 0.f;
    const float sum = warp_sum(u);
    return real ? u / sum : 0.f;
}

template <int PER, typename T>
__global__ void __launch_bounds__(kGateThreads) gate_kernel(const T *__restrict__ logits, const GateArgs p,
                                                            int32_t *__restrict__ ids, float *__restrict__ weights) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kGateThreads / 32);
    for (int64_t r = (int64_t)blockIdx.x * (kGateThreads / 32) + (threadIdx.x >> 5); r < p.n; r += step) {
        const T *row = logits + r * p.ldl;
        const Scores<float> sc = row_scores<T, float>(p, row, lane);
        int e;
        if (!choose<PER, T>(p, row, lane, sc, e)) e = choose_exact<T>(p, row, lane);
        const bool real = lane < p.topk && e >= 0;
        const float l = real ? load_logit(row + e) : 0.f;
        float w = p.renormalize ? share_of(p.sigmoid, l, real) : score_of(sc, l);
        if (lane < p.topk) {
            ids[r * p.topk + lane] = real ? e : -1;
            weights[r * p.topk + lane] = real ? w * p.scale : 0.f;
        }
    }
}

// Gradient.  With v the weights before the scale and g the scaled gradient of
// the weights, lane j's choice says about its expert's logit
//   softmax           p_e (g_j at the chosen - sum_j g_j p_j), every expert
//   softmax, renorm.  v_j (g_j - sum_m g_m v_m)
//   sigmoid           g_j s_j (1 - s_j)
//   sigmoid, renorm.  v_j (1 - s_j) (g_j - sum_m g_m v_m)
// It goes to a row in shared memory, and the whole row leaves from there.  An
// expert that is named twice gets the sum, in the choices' order.
template <typename T>
__global__ void __launch_bounds__(kGateThreads) gate_grad_kernel(const float *__restrict__ dweights,
                                                                 const T *__restrict__ logits, const GateArgs p,
                                                                 const int32_t *__restrict__ ids,
                                                                 T *__restrict__ dlogits) {
    extern __shared__ float gate_smem[];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *own = gate_smem + warp * p.n_experts;
    for (int e = lane; e < p.n_experts; e += 32) own[e] = 0.f;
    const bool dense = !p.sigmoid && !p.renormalize;
    const int64_t step = (int64_t)gridDim.x * (kGateThreads / 32);
    for (int64_t r = (int64_t)blockIdx.x * (kGateThreads / 32) + warp; r < p.n; r += step) {
        const T *row = logits + r * p.ldl;
        T *out = dlogits + r * p.n_experts;
        Scores<float> sc{p.sigmoid, 0.f, 0.f};
        if (dense) sc = row_scores<T, float>(p, row, lane);
        int e = lane < p.topk ? ids[r * p.topk + lane] : -1;
        if (e >= p.n_experts) e = -1;
        const float l = e >= 0 ? load_logit(row + e) : -INFINITY;
        const bool real = l != -INFINITY;  // an expert that is closed to the token has no weight
        const float g = real ? p.scale * dweights[r * p.topk + lane] : 0.f;
        float back = g, all = 0.f;
        if (p.renormalize) {
            const float v = share_of(p.sigmoid, l, real);
            back = v * (g - warp_sum(g * v));
        }
        if (p.sigmoid) {
            const float rest = __fdividef(1.f, 1.f + __expf(l));  // 1 - s
            back *= p.renormalize ? rest : rest * __fdividef(1.f, 1.f + __expf(-l));
        }
        if (dense) all = warp_sum(real ? g * score_of(sc, l) : 0.f);
        const uint32_t twins = __match_any_sync(kAll, real ? e : -1 - lane);
        const bool first = real && lane == __ffs(twins) - 1;
        if (__any_sync(kAll, (twins & (twins - 1)) != 0u)) {
            float sum = 0.f;
            for (int j = 0; j < p.topk; ++j) {
                const float other = __shfl_sync(kAll, back, j);
                if (twins >> j & 1u) sum += other;
            }
            back = sum;
        }
        __syncwarp();
        if (first) own[e] = back;
        __syncwarp();
        for (int i = lane; i < p.n_experts; i += 32) {
            float v = own[i];
            if (dense) v = score_of(sc, load_logit(row + i)) * (v - all);
            store_logit(out + i, v);
        }
        __syncwarp();
        if (first) own[e] = 0.f;
    }
}

unsigned gate_blocks(int64_t n) {
    const int64_t rows = kGateThreads / 32, blocks = (n + rows - 1) / rows, most = (int64_t)device_sm_count() * 16;
    return (unsigned)(blocks < most ? blocks : most);
}

GateArgs gate_args(const GateShape &g, int64_t ldl, const float *bias) {
    return {g.n,          ldl, g.n_experts, g.topk, g.groups, g.topk_groups, g.n_experts / g.groups, g.sigmoid,
            g.renormalize, g.scale, bias};
}

template <typename T>
cudaError_t gate_typed(const GateShape &g, const void *logits, int64_t ldl, const float *bias, int32_t *ids,
                       float *weights, cudaStream_t s) {
    const int per = (g.n_experts + 31) / 32;
    void (*kernel)(const T *, GateArgs, int32_t *, float *) =
        per <= 1    ? gate_kernel<1, T>
        : per <= 2  ? gate_kernel<2, T>
        : per <= 4  ? gate_kernel<4, T>
        : per <= 8  ? gate_kernel<8, T>
        : per <= 16 ? gate_kernel<16, T>
        : per <= 32 ? gate_kernel<32, T>
                    : gate_kernel<128, T>;
    return launch_kernel(true, kernel, dim3(gate_blocks(g.n)), dim3(kGateThreads), 0, s, static_cast<const T *>(logits),
                         gate_args(g, ldl, bias), ids, weights);
}

template <typename T>
cudaError_t gate_grad_typed(const GateShape &g, const float *dweights, const void *logits, int64_t ldl,
                            const int32_t *ids, void *dlogits, cudaStream_t s) {
    constexpr int most = KMEANS_ROUTE_MAX_EXPERTS * (kGateThreads / 32) * 4;
    static std::once_flag once[kMaxDevices];
    static std::atomic<int> err[kMaxDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    const int slot = dev >= 0 && dev < kMaxDevices ? dev : 0;
    once_per_device(once, [&] {
        err[slot].store((int)cudaFuncSetAttribute(gate_grad_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    });
    if (err[slot].load() != cudaSuccess) return (cudaError_t)err[slot].load();
    return launch_kernel(true, gate_grad_kernel<T>, dim3(gate_blocks(g.n)), dim3(kGateThreads),
                         (size_t)g.n_experts * (kGateThreads / 32) * 4, s, dweights, static_cast<const T *>(logits),
                         gate_args(g, ldl, nullptr), ids, static_cast<T *>(dlogits));
}

}  // namespace

cudaError_t launch_gate(const GateShape &g, int dtype, const void *logits, int64_t ldl, const float *bias, int32_t *ids,
                        float *weights, cudaStream_t s) {
    if (dtype == KMEANS_F32) return gate_typed<float>(g, logits, ldl, bias, ids, weights, s);
    return dtype == KMEANS_F16 ? gate_typed<__half>(g, logits, ldl, bias, ids, weights, s)
                               : gate_typed<__nv_bfloat16>(g, logits, ldl, bias, ids, weights, s);
}

cudaError_t launch_gate_grad(const GateShape &g, int dtype, const float *dweights, const void *logits, int64_t ldl,
                             const int32_t *ids, void *dlogits, cudaStream_t s) {
    if (dtype == KMEANS_F32) return gate_grad_typed<float>(g, dweights, logits, ldl, ids, dlogits, s);
    return dtype == KMEANS_F16 ? gate_grad_typed<__half>(g, dweights, logits, ldl, ids, dlogits, s)
                               : gate_grad_typed<__nv_bfloat16>(g, dweights, logits, ldl, ids, dlogits, s);
}

}  // namespace km
