// The gate: which experts a token goes to, and with what weights.
//
//   s = softmax(l) or 1 / (1 + exp(-l))      scores of the experts
//   c = s + b                                what the choice goes by
//
// With groups of neighbouring experts, those of the topk_groups groups whose two
// largest c have the largest sum stay; then the topk largest c are taken one
// after the other, equal ones by index.  A logit or a bias of minus infinity
// closes the expert: it is not chosen, and a token with too few open experts
// gets -1 with weight 0.  NaN counts as infinity, so that a token that holds one
// shows it in its weights.
//
// The choice is that of exact arithmetic.  Without a bias the order is the
// logits' own.  Sums (c, and the groups' scores) are formed in float32; where two
// neighbours in the order, the last chosen and the first left out among them, are
// nearer than their errors (Gap) and not equal in both logit and bias, what is near
// is formed again in pairs of floats, and what is near even so in float64.
//
// A warp has a token, a lane PER neighbouring experts in registers.  What is left
// out early costs least: no lane can hold one of the topk + 1 largest unless its
// own largest is among the lanes' topk + 1 largest, so the smallest of those
// bounds the values that are looked at further, a few more than topk.  They are
// brought together, one to a lane, and each counts the ones before it.
//
// Instructions bound it, 1239 of a warp per token: 16384 tokens, 8 of 256 float32
// experts in 4 of 8 groups, sigmoid and bias take 22 to 23 us a call, where reading
// the logits takes 2.6; 18.5 without the groups, 24 without the bias (the logits are
// loaded once more, for their order), 12.4 without both.  An argmax over all lanes
// and values for each choice took 68.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "assign_common.cuh"
#include "layer.cuh"
#include "pieces.cuh"

namespace km {

namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kGateThreads = 128;

// A token's logits.  Their type is looked at where they are loaded: the choice has
// hundreds of instructions to those few, and a kernel of its own for every type
// would be as much code again.
struct Logits {
    const uint8_t *p;
    int dtype;
    __device__ __forceinline__ float operator[](int e) const {
        if (dtype == KMEANS_F32) return reinterpret_cast<const float *>(p)[e];
        if (dtype == KMEANS_F16) return widen(reinterpret_cast<const __half *>(p)[e]);
        return widen(reinterpret_cast<const __nv_bfloat16 *>(p)[e]);
    }
};

// Order-preserving keys: 0 for what cannot be chosen, NaN as infinity, the two
// zeros equal.
__device__ __forceinline__ uint32_t choice_key(float v) {
    if (v == -INFINITY) return 0u;
    if (v != v) v = INFINITY;
    return float_to_ord(v + 0.f);
}
__device__ __forceinline__ uint64_t choice_key(double v) {
    if (v == -(double)INFINITY) return 0ull;
    if (v != v) v = INFINITY;
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

struct GateArgs {
    int64_t n, pitch;  // bytes
    int dtype;
    int n_experts, topk, groups, topk_groups, group_size;
    bool sigmoid, renormalize;
    float scale;
    const float *bias;
    bool whole, bias_whole;  // rows of the logits, the bias, start on 16 bytes
    int lanes_per_group;     // where a group is a power of two of whole lanes, else 0
    float gap;               // a score's error in float32, twice, over the largest score (see gate_args)
};

// The row's score parameters: softmax takes exp(l - top) / sum.
template <typename V>
struct Scores {
    bool sigmoid;
    V top, inverse;
};

// How near two values of the order may be in float32 without being looked at
// further: twice what they may be off by, which is a score's error, no more than
// the largest score's, and half a last bit of each sum with the bias.  A group's
// score is the sum of two such values, which may be far larger than it where their
// biases cancel: `of_group` is what it may be off by itself, half a last bit of each
// part and of the sum, and 2^-16 of them for what this is off by.  (Infinite ones are
// not off.)
struct Gap {
    float score;
    __device__ __forceinline__ Gap(const GateArgs &p, const Scores<float> &sc)
        : score(p.sigmoid ? p.gap : fminf(p.gap * sc.inverse, p.gap)) {}
    __device__ __forceinline__ float operator()(float a, float b) const {
        return score + 0x1p-23f * (fabsf(a) + fabsf(b));
    }
    __device__ __forceinline__ float of_group(float one, float two) const {
        constexpr float bit = 0x1.0001p-23f;
        const float parts = bit * fabsf(one) + (two == -INFINITY ? 0.f : bit * fabsf(two));
        return isfinite(parts) ? score + parts : 0.f;
    }
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

// PER values from p on, whose first is on 16 bytes or their own size.
template <int PER, typename T>
__device__ __forceinline__ void load_whole(const T *p, float (&f)[PER]) {
    constexpr int BYTES = PER * (int)sizeof(T), WORD = BYTES >= 16 ? 16 : BYTES, N = WORD / (int)sizeof(T);
    using W = std::conditional_t<WORD == 16, uint4, std::conditional_t<WORD == 8, uint2, std::conditional_t<WORD == 4, uint32_t, uint16_t>>>;
#pragma unroll
    for (int i = 0; i < PER; i += N) {
        const W w = reinterpret_cast<const W *>(p)[i / N];
        T v[N];
        memcpy(v, &w, sizeof w);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if constexpr (sizeof(T) == 4)
                f[i + j] = v[j];
            else
                f[i + j] = widen<T>(v[j]);
        }
    }
}

// A lane's PER neighbouring values of a row, absent ones minus infinity.
template <int PER>
__device__ __forceinline__ void load_run(const Logits &row, int e0, int n_experts, bool whole, float (&f)[PER]) {
    if (whole && e0 + PER <= n_experts) {
        if (row.dtype == KMEANS_F32)
            load_whole<PER>(reinterpret_cast<const float *>(row.p) + e0, f);
        else if (row.dtype == KMEANS_F16)
            load_whole<PER>(reinterpret_cast<const __half *>(row.p) + e0, f);
        else
            load_whole<PER>(reinterpret_cast<const __nv_bfloat16 *>(row.p) + e0, f);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) f[i] = e0 + i < n_experts ? row[e0 + i] : -INFINITY;
    }
}

template <int PER, typename T>
__device__ __forceinline__ void store_whole(T *p, const float (&f)[PER]) {
    constexpr int BYTES = PER * (int)sizeof(T), WORD = BYTES >= 16 ? 16 : BYTES, N = WORD / (int)sizeof(T);
    using W = std::conditional_t<WORD == 16, uint4, std::conditional_t<WORD == 8, uint2, std::conditional_t<WORD == 4, uint32_t, uint16_t>>>;
#pragma unroll
    for (int i = 0; i < PER; i += N) {
        T v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if constexpr (sizeof(T) == 4)
                v[j] = f[i + j];
            else
                v[j] = narrow<T>(f[i + j]);
        }
        W w;
        memcpy(&w, v, sizeof w);
        reinterpret_cast<W *>(p)[i / N] = w;
    }
}

template <int PER, typename T>
__device__ __forceinline__ void store_run(T *row, int e0, int n_experts, bool whole, const float (&f)[PER]) {
    if (whole && e0 + PER <= n_experts) {
        store_whole<PER>(row + e0, f);
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e0 + i < n_experts) {
                if constexpr (sizeof(T) == 4)
                    row[e0 + i] = f[i];
                else
                    row[e0 + i] = narrow<T>(f[i]);
            }
    }
}

// Values brought together: what the choice goes by, and the expert.
constexpr int kNear = 64;
struct alignas(8) Candidate {
    uint32_t key;
    int expert;
};
struct Candidates {
    Candidate found[kNear], sorted[33];
    double value[kNear];
};

// The largest of the lanes' values, each lane's taken out in turn (one lane a
// turn): the count-th largest, or 0 where there are fewer.
__device__ __forceinline__ uint32_t nth_largest(uint32_t key, int count, int lane) {
    uint32_t best = 0;
    for (int j = 0; j < count; ++j) {
        best = warp_max(key);
        if (best == 0) break;
        const uint32_t who = __ballot_sync(kAll, key == best);
        if (lane == __ffs(who) - 1) key = 0;
    }
    return best;
}

template <typename V>
__device__ __forceinline__ Scores<V> row_scores(const GateArgs &p, const Logits &row, int lane) {
    Scores<V> sc{p.sigmoid, 0, 0};
    if (p.sigmoid) return sc;
    float top = -INFINITY;
    for (int e = lane; e < p.n_experts; e += 32) top = fmaxf(top, row[e]);
    top = warp_fmax(top);
    sc.top = top == -INFINITY ? 0.f : top;  // no open expert: scores of 0
    V sum[4] = {};  // (a lane's 128 terms one after the other would lose up to 2^-17)
    for (int e0 = lane; e0 < p.n_experts; e0 += 128)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + i * 32;
            if (e < p.n_experts) sum[i] += exp_of((V)row[e] - sc.top);
        }
    const V all = warp_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
    sc.inverse = all == (V)0 ? (V)0 : (V)1 / all;
    return sc;
}

// The whole row in float64, where too much is near: as short as it can be, a
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

__device__ __noinline__ int choose_exact(const GateArgs &p, Logits row, int lane) {
    uint64_t key[kExactPer];
    const Scores<double> sc = row_scores<double>(p, row, lane);
    const int per = (p.n_experts + 31) / 32;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        const int e = i * 32 + lane;
        const float l = e < p.n_experts ? row[e] : -INFINITY, b = p.bias && e < p.n_experts ? p.bias[e] : 0.f;
        key[i] = 0;
        if (l != -INFINITY && b != -INFINITY)
            key[i] = p.bias || p.groups > 1 ? choice_key(score_of(sc, l) + (double)b) : choice_key((double)l);
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
                key[i] = choice_key((double)row[e]);
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

// A number as the sum of two floats, the second below half a last bit of the
// first, and the sums and products of Dekker (1971) and Knuth.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair short_sum(float a, float b) {  // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fadd_rn(b, -__fadd_rn(s, -a))};
}
__device__ __forceinline__ Pair sum_of(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
    return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t))};
}
__device__ __forceinline__ Pair product_of(float a, float b) {
    const float p = __fmul_rn(a, b);
    return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Pair add(const Pair &a, const Pair &b) {
    const Pair s = sum_of(a.hi, b.hi);
    return short_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Pair multiply(const Pair &a, const Pair &b) {
    const Pair p = product_of(a.hi, b.hi);
    return short_sum(p.hi, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, p.lo)));
}
__device__ __forceinline__ Pair inverse_of(const Pair &a) {
    const float q = __fdividef(1.f, a.hi);  // (what it is off by, twice 2^-24, goes out squared)
    return short_sum(q, __fmul_rn(q, __fmaf_rn(-q, a.lo, __fmaf_rn(-q, a.hi, 1.f))));
}

// 2^(j / 32).
__device__ const float2 kRoots[32] = {
    {0x1p+0f, 0.f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f}, {0x1.11301ep+0f, -0x1.fdb496p-25f},
    {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f}, {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.29e9ep+0f, -0x1.5c0424p-25f},
    {0x1.306fep+0f, 0x1.4636e2p-25f}, {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5342b6p+0f, -0x1.2c561p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f}, {0x1.6247ecp+0f, -0x1.f8b55p-25f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f}, {0x1.7a1148p+0f, -0x1.829fdp-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f},
    {0x1.8ace54p+0f, 0x1.15506ep-27f}, {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b7f77p+0f, -0x1.a09438p-25f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f}, {0x1.cb720ep+0f, -0x1.8837ccp-27f},
    {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f}, {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.f50766p+0f, -0x1.246ebp-26f}};

// exp of x in [-80, 80], 2^-43 of it for |x| <= 8, 2^-39 to the ends (below 2^-100
// its second float loses bits), by Tang's method (1989): x = n ln(2) / 32 + r, and
// exp(r) = 1 + r + r^2 / 2 + .. with |r| < 2^-6.5, whose terms from the cube on
// need one float.
__device__ __forceinline__ Pair exp_of(const Pair &x) {
    constexpr float STEP = 0x1.62e43p-6f, STEP_REST = -0x1.05c61p-34f;  // ln(2) / 32
    const float n = rintf(__fmul_rn(x.hi, 0x1.715476p+5f));
    const Pair p = product_of(n, STEP);
    const Pair r = sum_of(__fadd_rn(x.hi, -p.hi), __fmaf_rn(-n, STEP_REST, __fadd_rn(x.lo, -p.lo)));
    Pair q = product_of(r.hi, r.hi);
    q.lo = __fmaf_rn(2.f * r.hi, r.lo, q.lo);
    const float cube = __fmul_rn(__fmul_rn(r.hi, q.hi),
                                 __fmaf_rn(r.hi, __fmaf_rn(r.hi, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f));
    Pair u = sum_of(r.hi, 0.5f * q.hi);
    u.lo = __fadd_rn(u.lo, __fmaf_rn(0.5f, q.lo, __fadd_rn(r.lo, cube)));
    const int i = (int)n;
    const float2 root = kRoots[i & 31];
    Pair t = product_of(root.x, u.hi);
    t.lo = __fadd_rn(root.y, __fmaf_rn(root.x, u.lo, __fmaf_rn(root.y, u.hi, t.lo)));
    const Pair s = sum_of(root.x, t.hi);
    const Pair e = short_sum(s.hi, __fadd_rn(s.lo, t.lo));
    const float power = __int_as_float(((i >> 5) + 127) << 23);
    return {__fmul_rn(e.hi, power), __fmul_rn(e.lo, power)};
}

// exp(l - top), nothing where that is below e^-80.
__device__ __forceinline__ Pair exp_below(float l, float top) {
    const Pair x = sum_of(l, -top);
    if (!(x.hi > -80.f)) return {0.f, 0.f};
    return exp_of(x);
}

// What a row's scores as pairs need: nothing for the logistic function.
struct PairScores {
    float top;
    Pair inverse;
};

// False where the row holds what has no finite scores.
__device__ __forceinline__ bool pair_scores(const GateArgs &p, const Logits &row, int lane, PairScores &sc) {
    sc = {0.f, {1.f, 0.f}};
    if (p.sigmoid) return true;
    float top = -INFINITY;
    bool nan = false;
    for (int e = lane; e < p.n_experts; e += 32) {
        const float l = row[e];
        top = fmaxf(top, l);
        nan = nan || l != l;
    }
    top = warp_fmax(top);
    if (__any_sync(kAll, nan) || !isfinite(top)) return false;
    Pair sum = {0.f, 0.f};
#pragma unroll 4
    for (int e = lane; e < p.n_experts; e += 32) sum = add(sum, exp_below(row[e], top));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum = add(sum, Pair{__shfl_xor_sync(kAll, sum.hi, o), __shfl_xor_sync(kAll, sum.lo, o)});
    sc = {top, inverse_of(sum)};
    return true;
}

// What the choice goes by, the score within 2^-40.
__device__ __forceinline__ double pair_value(const GateArgs &p, const Logits &row, int e, const PairScores &sc) {
    const float l = row[e];
    const float b = p.bias ? p.bias[e] : 0.f;
    Pair s;
    if (p.sigmoid)  // (past the ends it is 0 or 1 to 2^-57)
        s = inverse_of(add({1.f, 0.f}, exp_of({fminf(fmaxf(-l, -40.f), 80.f), 0.f})));
    else
        s = multiply(exp_below(l, sc.top), sc.inverse);
    const double c = (double)s.hi + ((double)s.lo + (double)b);
    return l != l || c != c ? (double)INFINITY : c;
}

// The candidates' values so.
__device__ __noinline__ bool near_values(const GateArgs &p, Logits row, int lane, Candidates &list, int count) {
    PairScores sc;
    if (!pair_scores(p, row, lane, sc)) return false;
    for (int i = lane; i < count; i += 32) list.value[i] = pair_value(p, row, list.found[i].expert, sc);
    __syncwarp();
    return true;
}

// Whether the order of such values, or of sums of two of them, may be another one
// than that of the exact ones; `size`: the magnitude that their roundings go by.
__device__ __forceinline__ bool nearer(double a, double b, double size) {
    return !(fabs(a - b) > 0x1p-38 + 0x1p-50 * size);
}
__device__ __forceinline__ bool nearer(double a, double b) { return nearer(a, b, fabs(a)); }

// What the candidates' order goes by, in float64.
__device__ __noinline__ void exact_values(const GateArgs &p, Logits row, int lane, Candidates &list, int count) {
    Scores<double> sc{p.sigmoid, 0, 0};
    if (!p.sigmoid) sc = row_scores<double>(p, row, lane);
    for (int i = lane; i < count; i += 32) {
        const int e = list.found[i].expert;
        const double c = score_of(sc, row[e]) + (p.bias ? (double)p.bias[e] : 0.0);
        list.value[i] = c != c ? (double)INFINITY : c;
    }
    __syncwarp();
}

// The order where neighbours in it (lane j's expert and lane j + 1's) are near, each
// pair by itself: lane j's expert then, or -2 in every lane where that does not
// settle it.  A row that is looked at again keeps its SM waiting at the end, so this
// is short: without it, all candidates in float64 and ranked again, 16384 x 256 in 8
// groups took 26 us with sigmoid and 31 with softmax for a row in a thousand.
__device__ __noinline__ int settle_pairs(const GateArgs &p, Logits row, int lane, int expert, bool near) {
    PairScores sc;
    if (!pair_scores(p, row, lane, sc)) return -2;
    const double own = expert >= 0 ? pair_value(p, row, expert, sc) : 0.0, after = __shfl_down_sync(kAll, own, 1);
    if (__any_sync(kAll, near && nearer(own, after))) return -2;
    const uint32_t swap = __ballot_sync(kAll, near && after > own);
    const int down = __shfl_down_sync(kAll, expert, 1), up = __shfl_up_sync(kAll, expert, 1);
    return swap >> lane & 1u ? down : (swap << 1) >> lane & 1u ? up : expert;
}

// The groups that stay, of those (lane g: group g) with a bit in `near`, whose two
// largest values are among the candidates (their keys: the groups).  EXACT: in float64; else kAll where one
// that stays is near one that does not (which all 32 cannot: they are left out of).
template <bool EXACT>
__device__ __noinline__ uint32_t refine_groups(const GateArgs &p, int lane, const Candidates &list, int count,
                                               uint32_t near, int wanted) {
    double one = -INFINITY, two = -INFINITY;
    for (int i = 0; i < count; ++i) {
        if ((int)list.found[i].key != lane) continue;
        const double c = list.value[i];
        two = c > one ? one : (c > two ? c : two);
        one = c > one ? c : one;
    }
    const double score = two == -INFINITY ? one : one + two;
    const uint64_t total = choice_key(score);
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
        const uint64_t other = (uint64_t)__shfl_sync(kAll, (unsigned long long)total, g);
        rank += (near >> g & 1u) && (other > total || (other == total && g < lane));
    }
    __syncwarp();
    const uint32_t kept = __ballot_sync(kAll, (near >> lane & 1u) && rank < wanted);
    if constexpr (!EXACT) {
        // the last that stays and the first that does not
        const uint32_t last = __ballot_sync(kAll, (near >> lane & 1u) && rank == wanted - 1);
        const uint32_t next = __ballot_sync(kAll, (near >> lane & 1u) && rank == wanted);
        if (last && next) {
            const double a = __shfl_sync(kAll, score, __ffs(last) - 1), b = __shfl_sync(kAll, score, __ffs(next) - 1);
            // (the parts' magnitudes, not negative: their bits' order is the values')
            const float parts = (float)(fabs(one) + (two == -INFINITY ? 0.0 : fabs(two)));
            const float most = __uint_as_float(__reduce_max_sync(kAll, near >> lane & 1u ? __float_as_uint(parts) : 0u));
            if (nearer(a, b, most)) return kAll;
        }
    }
    return kept;
}

// The candidates' experts in order: lane j has the j-th (-1: none).  EXACT: in
// float64; else -2 in every lane where neighbours are near and not equal in both
// logit and bias.
template <bool EXACT>
__device__ __noinline__ int refine_order(const GateArgs &p, const Logits row, int lane, Candidates &list, int count) {
    for (int i = lane; i < count; i += 32) {
        const int e = list.found[i].expert;
        const uint64_t own = choice_key(list.value[i]);
        int rank = 0;
        for (int j = 0; j < count; ++j) {
            const uint64_t other = choice_key(list.value[j]);
            rank += other > own || (other == own && list.found[j].expert < e);
        }
        if (rank < 33) list.sorted[rank] = {(uint32_t)i, e};
    }
    __syncwarp();
    const int chosen = lane < p.topk && lane < count ? list.sorted[lane].expert : -1;
    if constexpr (!EXACT) {
        bool near = false;
        if (chosen >= 0 && lane + 1 < count) {
            const Candidate after = list.sorted[lane + 1];
            near = nearer(list.value[list.sorted[lane].key], list.value[after.key]) &&
                   !(row[chosen] == row[after.expert] && p.bias[chosen] == p.bias[after.expert]);
        }
        if (__any_sync(kAll, near)) return -2;
    }
    return chosen;
}

// (A sum past float32's range is not infinite; below it, it may still be wanted.)
__device__ __forceinline__ float group_total(float one, float two) {
    return two == -INFINITY || one == INFINITY ? one : fminf(fmaxf(one + two, -FLT_MAX), FLT_MAX);
}

// The two largest of two pairs.
__device__ __forceinline__ void merge_two(float &one, float &two, float other_one, float other_two) {
    two = fmaxf(fminf(one, other_one), fmaxf(two, other_two));
    one = fmaxf(one, other_one);
}

// The `wanted` largest in order, one after the other: where so many values are
// equal that they do not fit the list.  Returns how many there were.
template <int PER>
__device__ __forceinline__ int take_in_turn(float (&f)[PER], int wanted, int lane, Candidates &list) {
    int count = 0;
    for (; count < wanted; ++count) {
        float mine = f[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < PER; ++i)
            if (f[i] > mine) {
                mine = f[i];
                at = i;
            }
        const uint32_t key = choice_key(mine), best = warp_max(key);
        if (best == 0) break;
        // the lowest lane has the lowest experts
        if (lane == __ffs(__ballot_sync(kAll, key == best)) - 1) {
            list.sorted[count] = {best, lane * PER + at};
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i == at) f[i] = -INFINITY;
        }
    }
    return count;
}

// Chooses a row's experts: returns the j-th in lane j (-1: none).  SUMS: by sums with
// a bias or within groups; else by the logits alone.
template <int PER, bool SUMS>
__device__ __forceinline__ int choose(const GateArgs &p, const Logits &row, int lane, const Scores<float> &sc, float (&f)[PER],
                                      Candidates &list) {
    const int e0 = lane * PER;
    const Gap gap_of(p, sc);
    if constexpr (SUMS) {
        constexpr int RUN = PER < 4 ? PER : 4;
#pragma unroll
        for (int i = 0; i < PER; i += RUN) {
            float b[RUN] = {};
            if (p.bias)
                load_run<RUN>(Logits{reinterpret_cast<const uint8_t *>(p.bias), KMEANS_F32}, e0 + i, p.n_experts,
                              p.bias_whole, b);
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                const float c = score_of(sc, f[i + j]) + b[j];
                // (closed by the bias, too, where the score is NaN)
                f[i + j] = f[i + j] == -INFINITY || b[j] == -INFINITY ? -INFINITY : c;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) f[i] = f[i] != f[i] ? INFINITY : f[i];
    if (SUMS && p.groups > 1) {
        float total = -INFINITY, second = -INFINITY;  // lane g: group g's score, its second largest value
        float off = 0.f;                              // what a group's score may be off by: here the lane's own
        bool mine[PER];
        if (p.lanes_per_group > 0) {  // whole lanes, a power of two of them
            float one = -INFINITY, two = -INFINITY;
#pragma unroll
            for (int i = 0; i < PER; ++i) merge_two(one, two, f[i], -INFINITY);
            for (int o = 1; o < p.lanes_per_group; o <<= 1)
                merge_two(one, two, __shfl_xor_sync(kAll, one, o), __shfl_xor_sync(kAll, two, o));
            off = gap_of.of_group(one, two);
            const int from = (lane * p.lanes_per_group) & 31;
            total = __shfl_sync(kAll, group_total(one, two), from);
            second = __shfl_sync(kAll, two, from);
        } else {
            for (int g = 0; g < p.groups; ++g) {
                const int lo = g * p.group_size - e0, hi = lo + p.group_size;
                float one = -INFINITY, two = -INFINITY;
#pragma unroll
                for (int i = 0; i < PER; ++i) merge_two(one, two, i >= lo && i < hi ? f[i] : -INFINITY, -INFINITY);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
                    merge_two(one, two, __shfl_xor_sync(kAll, one, o), __shfl_xor_sync(kAll, two, o));
                if (lane == g) {
                    total = group_total(one, two);
                    second = two;
                    off = gap_of.of_group(one, two);
                }
            }
        }
        if (lane >= p.groups) total = -INFINITY;
        // the groups in order, and the first that is left out
        uint32_t kept = 0, key = choice_key(total), last = 0, next = 0;
        for (int j = 0; j <= p.topk_groups; ++j) {
            next = warp_max(key);
            if (next == 0 || j == p.topk_groups) break;
            const int g = __ffs(__ballot_sync(kAll, key == next)) - 1;
            kept |= 1u << g;
            last = next;
            if (lane == g) key = 0;
        }
        if (next != 0) {  // (some group is left out)
            // (not negative, so the bits' order is the values')
            const float worst = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(off)));
            if (!(key_value(last) - key_value(next) > 2.f * worst)) {
                // What the groups that stay are no less than, what the others are no more than.
                if (p.lanes_per_group > 0) off = __shfl_sync(kAll, off, (lane * p.lanes_per_group) & 31);
                const bool in = kept >> lane & 1u;
                off += isfinite(total) ? 0x1p-23f * fabsf(total) : 0.f;  // (these sums round, too)
                const float low = total > -FLT_MAX ? total - off : -INFINITY, high = total < FLT_MAX ? total + off : INFINITY;
                const float least = ord_to_float(__reduce_min_sync(kAll, float_to_ord(in ? low : INFINITY)));
                const float most = ord_to_float(__reduce_max_sync(kAll, float_to_ord(in ? -INFINITY : high)));
                if (!(least > most)) {
                    // Near (equal sums are rarely sums of equal parts, so they are looked
                    // at too): what is surely above all that are left out stays, what is
                    // surely below all that are kept goes, and the rest is compared in
                    // float64.
                    const uint32_t sure = __ballot_sync(kAll, in && low > most);
                    const uint32_t near = __ballot_sync(kAll, total != -INFINITY && (in ? !(low > most) : high >= least));
                    int count = 0, g = e0 / p.group_size, left = (g + 1) * p.group_size - e0;
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const float two = __shfl_sync(kAll, second, g & 31);
                        const bool take = f[i] != -INFINITY && (near >> (g & 31) & 1u) && !(two - f[i] > gap_of(two, f[i]));
                        const uint32_t who = __ballot_sync(kAll, take);
                        const int at = count + __popc(who & ((1u << lane) - 1u));
                        if (take && at < kNear) list.found[at] = {(uint32_t)g, e0 + i};
                        count += __popc(who);
                        if (--left == 0) {
                            ++g;
                            left = p.group_size;
                        }
                    }
                    // (infinite sums have no order in float32)
                    if (count > kNear || __any_sync(kAll, (near >> lane & 1u) && !isfinite(total)))
                        return choose_exact(p, row, lane);
                    __syncwarp();
                    const int wanted = p.topk_groups - __popc(sure);
                    uint32_t some = kAll;
                    if (near_values(p, row, lane, list, count))
                        some = refine_groups<false>(p, lane, list, count, near, wanted);
                    if (some == kAll) {
                        exact_values(p, row, lane, list, count);
                        some = refine_groups<true>(p, lane, list, count, near, wanted);
                    }
                    kept = sure | some;
                }
            }
        }
        if (p.lanes_per_group > 0) {
            const bool in = kept >> (lane / p.lanes_per_group) & 1u;
#pragma unroll
            for (int i = 0; i < PER; ++i) mine[i] = in && f[i] != -INFINITY;
        } else {
            int g = e0 / p.group_size, left = (g + 1) * p.group_size - e0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                mine[i] = g < 32 && (kept >> g & 1u) && f[i] != -INFINITY;
                if (--left == 0) {
                    ++g;
                    left = p.group_size;
                }
            }
        }
        if (!p.bias) {  // the rest of the choice goes by the logits
            load_run<PER>(row, e0, p.n_experts, p.whole, f);
#pragma unroll
            for (int i = 0; i < PER; ++i) f[i] = f[i] != f[i] ? INFINITY : f[i];
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) f[i] = mine[i] ? f[i] : -INFINITY;
    }
    float high = f[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) high = fmaxf(high, f[i]);
    const int wanted = min(p.topk + 1, 32);  // (32 lanes have no 33rd: then all are looked at)
    const uint32_t bound = p.topk < 32 ? nth_largest(choice_key(high), wanted, lane) : 0u;
    float least = bound ? key_value(bound) : -INFINITY;
    if (SUMS && p.bias && isfinite(least)) least -= gap_of(least, least);  // and what may be as large
    // a lane's candidates go behind those of the lanes before it: by expert
    using Mask = std::conditional_t<(PER > 32), unsigned long long, uint32_t>;
    constexpr int WORDS = (PER + 63) / 64, BITS = PER / WORDS;
    Mask in[WORDS] = {};
    int own_count = 0;
#pragma unroll
    for (int w = 0; w < WORDS; ++w) {
#pragma unroll
        for (int i = 0; i < BITS; ++i)
            if (f[w * BITS + i] >= least && f[w * BITS + i] != -INFINITY) in[w] |= (Mask)1 << i;
        own_count += sizeof(Mask) == 8 ? __popcll(in[w]) : __popc((uint32_t)in[w]);
    }
    int upto = own_count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, upto, o);
        if (lane >= o) upto += v;
    }
    int count = __shfl_sync(kAll, upto, 31);
    const bool listed = count <= kNear;
    if (listed) {
        int at = upto - own_count;
        if (own_count) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (in[i / BITS] >> (i % BITS) & 1) list.found[at++] = {choice_key(f[i]), e0 + i};
        }
        __syncwarp();
        for (int i = lane; i < count; i += 32) {
            const Candidate own = list.found[i];
            int rank = 0;
            for (int j = 0; j < count; ++j) {
                const uint32_t other = list.found[j].key;
                rank += other > own.key || (other == own.key && j < i);
            }
            if (rank < 33) list.sorted[rank] = own;
        }
    } else {
        __syncwarp();
        count = take_in_turn(f, p.topk + 1, lane, list);
    }
    __syncwarp();
    // (the first that is left out with them, to see what is near it)
    const int expert = lane <= p.topk && lane < count ? list.sorted[lane].expert : -1;
    const int chosen = lane < p.topk ? expert : -1;
    if (!SUMS || !p.bias) return chosen;
    bool near = false;
    if (expert >= 0 && lane + 1 < count) {
        const float a = key_value(list.sorted[lane].key), c = key_value(list.sorted[lane + 1].key);
        near = !(a - c > gap_of(a, c));
    }
    const uint32_t all = __ballot_sync(kAll, near);
    if (all == 0) return chosen;
    near = near && chosen >= 0;
    if (near) {  // equal in logit and bias: their order is the experts'
        const int after = list.sorted[lane + 1].expert;
        near = !(row[chosen] == row[after] && p.bias[chosen] == p.bias[after]);
    }
    const uint32_t some = __ballot_sync(kAll, near);
    if (some == 0) return chosen;
    if (!listed) return choose_exact(p, row, lane);
    int order = -2;
    if (!(some & (all << 1 | all >> 1)) && p.topk < 32) order = settle_pairs(p, row, lane, expert, near);
    if (order != -2) return lane < p.topk ? order : -1;
    if (near_values(p, row, lane, list, count)) order = refine_order<false>(p, row, lane, list, count);
    if (order == -2) {
        exact_values(p, row, lane, list, count);
        order = refine_order<true>(p, row, lane, list, count);
    }
    return order;
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
    return real ? __fdividef(u, sum) : 0.f;
}

// A softmax's parameters from the lanes' logits.
template <int PER>
__device__ __forceinline__ void softmax_scores(const float (&f)[PER], Scores<float> &sc) {
    float top = f[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) top = fmaxf(top, f[i]);
    top = warp_fmax(top);
    sc.top = top == -INFINITY ? 0.f : top;  // no open expert: scores of 0
    constexpr int SUMS = PER < 4 ? PER : 4;  // (see gate_args)
    float sum[SUMS] = {};
#pragma unroll
    for (int i = 0; i < PER; ++i) sum[i % SUMS] += __expf(f[i] - sc.top);
#pragma unroll
    for (int i = 1; i < SUMS; ++i) sum[0] += sum[i];
    const float all = warp_sum(sum[0]);
    sc.inverse = all == 0.f ? 0.f : 1.f / all;
}

// (A kernel of its own for the logits alone: what sums need would make 16384 x 256, 8
// choices, 15.0 us instead of 12.4, and 8192 x 1024 14.8 instead of 12.6.)
template <int PER, bool SUMS>
__global__ void __launch_bounds__(kGateThreads, PER <= 8 ? 8 : PER <= 32 ? 6 : 2)
    gate_kernel(const uint8_t *__restrict__ logits, const __grid_constant__ GateArgs p, int32_t *__restrict__ ids,
                float *__restrict__ weights) {
    __shared__ Candidates lists[kGateThreads / 32];
    griddep_wait();
    const int lane = threadIdx.x & 31;
    Candidates &list = lists[threadIdx.x >> 5];
    // (renormalised softmax weights that are chosen by the logits need no sum of all)
    const bool need_sum = !p.sigmoid && (SUMS || !p.renormalize);
    const int64_t step = (int64_t)gridDim.x * (kGateThreads / 32);
    for (int64_t r = (int64_t)blockIdx.x * (kGateThreads / 32) + (threadIdx.x >> 5); r < p.n; r += step) {
        const Logits row{logits + r * p.pitch, p.dtype};
        float f[PER];
        load_run<PER>(row, lane * PER, p.n_experts, p.whole, f);
        Scores<float> sc{p.sigmoid, 0.f, 0.f};
        if (need_sum) softmax_scores(f, sc);
        const int e = choose<PER, SUMS>(p, row, lane, sc, f, list);
        const bool real = lane < p.topk && e >= 0;
        const float l = real ? row[e] : 0.f;
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
// It goes to a row in shared memory, experts apart, from which the lanes take their
// PER neighbouring ones along.  (16384 x 128 bfloat16, 8 choices: 10.5 us; with one
// expert at a time, whose logit was read three times, 14.5.)  An expert that is
// named twice gets the sum, in the choices' order.
template <int PER, typename T>
__global__ void __launch_bounds__(kGateThreads) gate_grad_kernel(const float *__restrict__ dweights,
                                                                 const uint8_t *__restrict__ logits, const GateArgs p,
                                                                 const int32_t *__restrict__ ids, bool out_whole,
                                                                 T *__restrict__ dlogits) {
    extern __shared__ float4 gate_smem[];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * PER;
    float *own = reinterpret_cast<float *>(gate_smem) + warp * (32 * PER);
#pragma unroll
    for (int i = 0; i < PER; ++i) own[e0 + i] = 0.f;
    const bool dense = !p.sigmoid && !p.renormalize;
    const int64_t step = (int64_t)gridDim.x * (kGateThreads / 32);
    for (int64_t r = (int64_t)blockIdx.x * (kGateThreads / 32) + warp; r < p.n; r += step) {
        const Logits row{logits + r * p.pitch, p.dtype};
        int e = lane < p.topk ? ids[r * p.topk + lane] : -1;
        if (e >= p.n_experts) e = -1;
        const float l = e >= 0 ? row[e] : -INFINITY;
        const bool real = l != -INFINITY;  // an expert that is closed to the token has no weight
        const float g = real ? p.scale * dweights[r * p.topk + lane] : 0.f;
        Scores<float> sc{p.sigmoid, 0.f, 0.f};
        float f[PER];
        if (dense) {
            load_run<PER>(row, e0, p.n_experts, p.whole, f);
            softmax_scores(f, sc);
        }
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
        float v[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            v[i] = own[e0 + i];
            if (dense) v[i] = score_of(sc, f[i]) * (v[i] - all);
        }
        store_run<PER>(dlogits + r * p.n_experts, e0, p.n_experts, out_whole, v);
        __syncwarp();
        if (first) own[e] = 0.f;
    }
}

unsigned gate_blocks(int64_t n) {
    const int64_t rows = kGateThreads / 32, blocks = (n + rows - 1) / rows, most = (int64_t)device_sm_count() * 64;
    return (unsigned)(blocks < most ? blocks : most);
}

// Values of a lane: a power of two of them, or 128 for more than 1024 experts.
int gate_per(int n_experts) {
    int per = 1;
    while (per * 32 < n_experts) per *= per < 32 ? 2 : 4;
    return per;
}

bool on16(const void *p, int64_t pitch_bytes) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && pitch_bytes % 16 == 0;
}

GateArgs gate_args(const GateShape &g, int dtype, const void *logits, int64_t ldl, const float *bias) {
    const int size = g.n_experts / g.groups, per = gate_per(g.n_experts), lanes = size % per == 0 ? size / per : 0;
    // Twice a score's error in float32, in 2^-24: an exponential of x is off by (2
    // |x| + 4) of itself.  The logistic function damps that by s (1 - s), its sum
    // and quotient add 5: 7.  In softmax |x| e^x is at most 0.37, the sum of n
    // terms, four accumulators to a lane, adds n / 128 + 8, the rest 6, all of it
    // times the largest score, exp(0) over the sum.
    const float gap = (g.sigmoid ? 16.f : (float)g.n_experts / 64.f + 30.f) * 0x1p-24f;
    const int64_t pitch = ldl * (dtype == KMEANS_F32 ? 4 : 2);
    return {g.n, pitch, dtype, g.n_experts, g.topk, g.groups, g.topk_groups, size, g.sigmoid, g.renormalize, g.scale, bias,
            on16(logits, pitch), on16(bias, 0), (lanes & (lanes - 1)) == 0 ? lanes : 0, gap};
}

template <int PER, typename T>
cudaError_t launch_grad(const GateShape &g, int dtype, const float *dweights, const void *logits, int64_t ldl,
                        const int32_t *ids, void *dlogits, cudaStream_t s) {
    constexpr int shared = kGateThreads * PER * 4;  // a row per warp
    if (shared > 48 * 1024) {
        static std::once_flag once[kMaxDevices];
        static std::atomic<int> err[kMaxDevices];
        int dev = 0;
        cudaGetDevice(&dev);
        const int slot = dev >= 0 && dev < kMaxDevices ? dev : 0;
        once_per_device(once, [&] {
            err[slot].store((int)cudaFuncSetAttribute(gate_grad_kernel<PER, T>,
                                                      cudaFuncAttributeMaxDynamicSharedMemorySize, shared));
        });
        if (err[slot].load() != cudaSuccess) return (cudaError_t)err[slot].load();
    }
    return launch_kernel(true, gate_grad_kernel<PER, T>, dim3(gate_blocks(g.n)), dim3(kGateThreads), (size_t)shared, s,
                         dweights, static_cast<const uint8_t *>(logits), gate_args(g, dtype, logits, ldl, nullptr), ids,
                         on16(dlogits, (int64_t)g.n_experts * (int64_t)sizeof(T)), static_cast<T *>(dlogits));
}

template <typename T>
cudaError_t gate_grad_typed(const GateShape &g, int dtype, const float *dweights, const void *logits, int64_t ldl,
                            const int32_t *ids, void *dlogits, cudaStream_t s) {
    const int per = gate_per(g.n_experts);
    const auto run = [&](auto launch) { return launch(g, dtype, dweights, logits, ldl, ids, dlogits, s); };
    return per <= 1    ? run(launch_grad<1, T>)
           : per <= 2  ? run(launch_grad<2, T>)
           : per <= 4  ? run(launch_grad<4, T>)
           : per <= 8  ? run(launch_grad<8, T>)
           : per <= 16 ? run(launch_grad<16, T>)
           : per <= 32 ? run(launch_grad<32, T>)
                       : run(launch_grad<128, T>);
}

using GateKernel = void (*)(const uint8_t *, GateArgs, int32_t *, float *);

template <bool SUMS>
GateKernel gate_kernel_of(int n_experts) {
    const int per = gate_per(n_experts);
    return per <= 1    ? gate_kernel<1, SUMS>
           : per <= 2  ? gate_kernel<2, SUMS>
           : per <= 4  ? gate_kernel<4, SUMS>
           : per <= 8  ? gate_kernel<8, SUMS>
           : per <= 16 ? gate_kernel<16, SUMS>
           : per <= 32 ? gate_kernel<32, SUMS>
                       : gate_kernel<128, SUMS>;
}

}  // namespace

cudaError_t launch_gate(const GateShape &g, int dtype, const void *logits, int64_t ldl, const float *bias, int32_t *ids,
                        float *weights, cudaStream_t s) {
    const auto kernel = bias || g.groups > 1 ? gate_kernel_of<true>(g.n_experts) : gate_kernel_of<false>(g.n_experts);
    return launch_kernel(true, kernel, dim3(gate_blocks(g.n)), dim3(kGateThreads), 0, s,
                         static_cast<const uint8_t *>(logits), gate_args(g, dtype, logits, ldl, bias), ids, weights);
}

cudaError_t launch_gate_grad(const GateShape &g, int dtype, const float *dweights, const void *logits, int64_t ldl,
                             const int32_t *ids, void *dlogits, cudaStream_t s) {
    if (dtype == KMEANS_F32) return gate_grad_typed<float>(g, dtype, dweights, logits, ldl, ids, dlogits, s);
    return dtype == KMEANS_F16 ? gate_grad_typed<__half>(g, dtype, dweights, logits, ldl, ids, dlogits, s)
                               : gate_grad_typed<__nv_bfloat16>(g, dtype, dweights, logits, ldl, ids, dlogits, s);
}

}  // namespace km
