// What stands around the experts in a model: the gate that chooses them, the
// layer norm in front and the cross entropy at the end: layouts and launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace km {

// --------------------------------------------------------------------- gate
struct GateShape {
    int64_t n;
    int n_experts, topk;
    int groups, topk_groups;
    bool sigmoid;      // else softmax
    bool renormalize;
    float scale;
};

cudaError_t launch_gate(const GateShape &g, int dtype, const void *logits, int64_t ldl, const float *bias, int32_t *ids,
                        float *weights, cudaStream_t s);
cudaError_t launch_gate_grad(const GateShape &g, int dtype, const float *dweights, const void *logits, int64_t ldl,
                             const int32_t *ids, void *dlogits, cudaStream_t s);

// --------------------------------------------------------------- layer norm
struct NormShape {
    int64_t n, d;
    int dtype;
};

// Sums of dy and dy * normalised over some rows each, joined at the end.
struct NormLayout {
    int64_t off_partial;
    int64_t bytes;
};

NormLayout norm_layout(int64_t n, int64_t d);

cudaError_t launch_norm(const NormShape &sh, const void *x, int64_t ldx, const void *weight, const void *bias, float eps,
                        void *y, float *mean, float *rstd, cudaStream_t s);
cudaError_t launch_norm_grad(const NormShape &sh, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                             const float *mean, const float *rstd, const void *weight, const void *residual,
                             int64_t ldr, void *dx, void *dweight, void *dbias, const NormLayout &L, uint8_t *ws,
                             cudaStream_t s);

// ------------------------------------------------------------- cross entropy
struct XentShape {
    int64_t m, n, k;  // rows, classes, features
    const void *labels;
    int id_bytes;
    float scale;
    bool bf16;  // else fp16
};

// Starts with the header and a status word for the products.
struct XentLayout {
    int64_t off_info;    // how many rows count, dz's scale
    int64_t off_rows;    // what the products know of each row that counts
    int64_t off_tally;   // rows that count, per share of the rows
    int64_t off_x;       // the rows that count, on 16 bytes
    int64_t off_w;       // w likewise (0: its rows are a multiple of 16 bytes)
    int64_t off_target;  // forward: the labels' logits
    int64_t off_stats;   // forward: largest logit and sum of exponentials per class part and row
    int64_t off_share;   // gradient: each row's share of its gradient (xent.cu)
    int64_t off_xw;      // gradient: the rows times their share
    int64_t off_dz;      // gradient: a piece's
    int64_t off_sums;    // gradient: dx so far, where there are several pieces or parts
    int64_t off_partial; // gradient: sums of chunks of the rows
    int64_t bytes;
};

int64_t xent_piece(int64_t m, int64_t n);
XentLayout xent_layout(bool grad, int64_t m, int64_t n, int64_t k);

cudaError_t launch_xent(const XentShape &sh, const void *x, int64_t ldx, const void *w, float *loss, float *lse,
                        const XentLayout &L, uint8_t *ws, cudaStream_t s);
cudaError_t launch_xent_grad(const XentShape &sh, const float *dloss, const void *x, int64_t ldx, const void *w,
                             const float *lse, void *dx, void *dw, const XentLayout &L, uint8_t *ws, cudaStream_t s);

}  // namespace km
