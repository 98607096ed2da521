// The experts' products: which variant of the kernel a call runs, and its
// parameters.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstdlib>

#include "linear_tc.cuh"

namespace km {

namespace {

// The row products in units of `bn` rows (long contractions: 64 or 256, which
// takes fewer rows as well).
template <Product MODE>
cudaError_t launch_rows(int bn, const LinearShape &sh, const Product16 &g, const LinearTcParams &p, cudaStream_t s) {
    if (p.contraction > kChunk)
        return bn == 64 ? launch_typed<MODE, 64, true>(sh, g, p, s) : launch_typed<MODE, 256, true>(sh, g, p, s);
    return bn == 256   ? launch_typed<MODE, 256>(sh, g, p, s)
           : bn == 128 ? launch_typed<MODE, 128>(sh, g, p, s)
                       : launch_typed<MODE, 64>(sh, g, p, s);
}

}  // namespace

WeightsSplit weights_split(int64_t m, int64_t n, int64_t k, int64_t n_experts) {
    constexpr int64_t longest = kChunk, shortest = 512;
    // output tiles of all experts, and how many chunks of an expert's average
    // rows would give every pair of SMs a unit
    const int64_t tiles = (n + 127) / 128 * ((k + lt::BP - 1) / lt::BP) * n_experts;
    int64_t chunk = longest;
    if (2 * tiles <= kPairs) {
        const int64_t parts = kPairs / tiles, average = m / n_experts;
        chunk = align_up((average + parts - 1) / parts, lt::BK);
        chunk = chunk < shortest ? shortest : chunk > longest ? longest : chunk;
    }
    // an expert of several chunks has at most twice as many as its rows fill
    return {(int)chunk, m > chunk ? (n_experts == 1 ? (m + chunk - 1) / chunk : 2 * m / chunk) : 0};
}

cudaError_t launch_linear_tc(Product mode, const LinearShape &sh, const Product16 &g, uint32_t *status, bool clear,
                             cudaStream_t s) {
    LinearTcParams p{};
    p.offsets = sh.offsets;
    p.m = sh.m;
    p.n_experts = sh.n_experts;
    p.cols = (int)(mode == Product::kForward ? sh.n : sh.k);
    p.num_p = (p.cols + lt::BP - 1) / lt::BP;
    p.out_rows = (int)sh.n;
    p.chunk = weights_split(sh.m, sh.n, sh.k, sh.n_experts).chunk;
    p.partial = g.partial;
    p.db = g.db;
    p.bias_sums = g.bias_sums;
    p.bias_rows = g.bias_rows;
    p.contraction = (int)(mode == Product::kForward ? sh.k : sh.n);
    p.bias = g.bias;
    p.residual = g.residual;
    p.ldr = g.ldr;
    p.activation = g.activation;
    p.out = g.out;
    p.pre = g.pre;
    p.wide = rows16(g.out, p.cols) && (!g.pre || rows16(g.pre, p.cols)) && (!g.residual || rows16(g.residual, g.ldr));
    p.status = status;
    p.clear = clear;
    // test-only fault injection (no trap, no fault), as in the assignment: every
    // consumer's bounded wait runs out and the status word reports the timeout
    const char *starve = getenv("KMEANS_GB300_TEST_STARVE_PIPELINE");
    p.test_starve = (starve != nullptr && starve[0] == '1') ? 1 : 0;
    // Rows per unit.  As many as 256 for the fewest bytes per MMA (a stage of
    // 256 x 256 x 64 just fills shared memory's bandwidth); about an expert's
    // average rows where there are fewer, so that small groups do not load
    // their neighbours' rows; and no more than needed to keep everything in one
    // round of the CTA pairs: the smaller the unit then, the sooner it is done
    // (24 rows through 8192 x 2048 10.9 us, 15.3 in units of 256; the gradient's
    // two products of 257 rows, 1000 x 520, 12.9 and 10.0 us in units of 256, 9.5
    // and 8.2 as chosen).
    const int64_t pairs = std::min(device_sm_count() / 2, kPairs);
    auto one_round = [&](int64_t bn) {
        const int64_t tiles = mode == Product::kWeights ? (sh.n + bn - 1) / bn * (sh.n_experts + sh.m / p.chunk)
                                                        : (sh.m + bn - 1) / bn + (sh.offsets ? sh.n_experts : 0);
        return tiles * p.num_p <= pairs;
    };
    if (mode == Product::kWeights)
        return one_round(128) ? launch_typed<Product::kWeights, 128>(sh, g, p, s)
                              : launch_typed<Product::kWeights, 256>(sh, g, p, s);
    const int64_t rows = sh.m / sh.n_experts;
    const int bn = rows <= 64 || one_round(64) ? 64 : rows <= 128 || one_round(128) ? 128 : 256;
    return mode == Product::kForward ? launch_rows<Product::kForward>(bn, sh, g, p, s)
                                     : launch_rows<Product::kRows>(bn, sh, g, p, s);
}

}  // namespace km
