// radamw_block.h -- structures shared by the block operators' C entry points
// (radamw_block_api.cpp) and their gfx950 kernels (radamw_dropout.hip,
// radamw_residual.hip, radamw_balance.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

namespace radamw {

// --------------------------------------------------------------- dropout --

// What the generator and its comparison need; threshold 0 keeps everything.
struct DropArgs {
    uint32_t key0, key1;    // seed
    uint32_t off0, off1;    // offset
    uint32_t first_row;
    uint32_t threshold;     // 0 .. 65536: a number below is dropped
    float factor;           // 65536 / (65536 - threshold)
};

struct DropoutArgs {
    const void *x;
    void *out;
    int64_t n, dim, stride, out_stride;  // strides in elements
    DropArgs drop;
};
hipError_t launch_dropout(const DropoutArgs &a, int dt, hipStream_t stream, int *launched);

// -------------------------------------------------------------- residual --

// The widest row that one workgroup holds in registers.
constexpr int64_t RESIDUAL_MAX_DIM = 32768;

struct ResidualArgs {
    const void *x, *branch, *gate, *post, *pre;  // branch, gate, post, pre may be null
    void *h, *out;                               // may be null
    float *rstd;                                 // 2 n, or null
    int64_t x_stride, branch_stride, gate_stride, h_stride, out_stride;
    int64_t n, dim, per;                         // per: rows that share a gate row
    int32_t gate_dt, weight_dt;
    float eps, weight_offset, scale;
    DropArgs drop;
};
hipError_t launch_residual(const ResidualArgs &a, int sdt, int bdt, hipStream_t stream, int *launched);

// Workers of the gradient (each sums its rows' columns) and its workspace in
// bytes.
struct ResidualPlan {
    int64_t rows;     // rows of a worker
    int64_t workers;
    int64_t width;    // floats of one partial row
    int64_t post, pre, gate;  // byte offsets of [workers][width] (gate: [workers][2][width]) FP32 sums
    int64_t bytes;
};
ResidualPlan residual_plan(int64_t n, int64_t dim, int64_t per);

struct ResidualGradArgs {
    const void *h, *branch, *gate, *post, *pre;
    const float *rstd;                 // 2 n
    const void *grad_h, *grad_out;     // either may be null
    void *grad_x, *grad_branch;
    void *grad_gate, *grad_post, *grad_pre;  // may be null
    int64_t h_stride, branch_stride, gate_stride, grad_h_stride, grad_out_stride, grad_x_stride, grad_branch_stride,
        grad_gate_stride;
    int64_t n, dim, per;
    int32_t gate_dt, weight_dt;
    float weight_offset, scale;
    DropArgs drop;
    char *workspace;
};
hipError_t launch_residual_grad(const ResidualGradArgs &a, const ResidualPlan &p, int sdt, int bdt, hipStream_t stream,
                                int *launched);

// --------------------------------------------------------------- balance --

// The most experts one wave holds: 64 lanes of eight eights.
constexpr int64_t BALANCE_MAX_EXPERTS = 4096;

// The rows are cut into pieces where a piece of `rows` rows ends and where a
// group ends: the part of group g in rows c * rows .. is piece c + g.
struct BalancePlan {
    int64_t rows;
    int64_t pieces;   // slots, some of them unused
    int64_t width;    // experts, rounded up to 16
    int64_t probs;    // byte offset of [pieces][width] FP32 sums of probabilities
    int64_t counts;   // of [pieces][width] int32 counts
    int64_t extra;    // of [pieces] {FP64 sum of squared log-sums, int64 rows that take part}
    int64_t bytes;
};
BalancePlan balance_plan(int64_t n, int64_t experts, int64_t groups);

struct BalanceArgs {
    const void *logits;
    const void *ids;          // n * top_k, or null (gradient from counts)
    const uint8_t *mask;      // may be null
    const void *offsets;      // groups + 1 of the ids' type, or null: one group
    const float *weights;     // may be null
    int64_t n, experts, stride, groups, top_k;
    int32_t wide;             // ids and offsets: 0 int32, 1 int64
    int32_t sigmoid;
    double balance_coef, z_coef;
    float *total, *loss, *mean_prob;
    int32_t *counts, *tokens;
    const float *upstream;    // may be null
    void *grad;               // may be null
    int64_t grad_stride;
    double grad_scale;
    char *workspace;
};
hipError_t launch_balance_loss(const BalanceArgs &a, const BalancePlan &p, int dt, hipStream_t stream, int *launched);
hipError_t launch_balance_grad(const BalanceArgs &a, const BalancePlan &p, int dt, hipStream_t stream, int *launched);

}  // namespace radamw
