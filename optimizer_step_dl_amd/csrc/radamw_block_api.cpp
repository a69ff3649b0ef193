// radamw_block_api.cpp -- the C ABI of the operators between the
// vocabulary's two ends of a training step: dropout, the residual stream's
// norms around a block with their gradient, and the routers' balance loss.
// Validation and launches only.
//
// Every entry point validates all of its arguments before it launches
// anything; the checks allocate nothing.
#include "radamw.h"
#include "radamw_block.h"
#include "radamw_host.h"

#include <cmath>

using namespace radamw;

namespace {

constexpr int64_t MAX_DROPOUT_DIM = int64_t(1) << 24;
// With the at most 1024 pieces of a batch this is below 2^24 workgroups.
constexpr int64_t MAX_GROUPS = (int64_t(1) << 24) - 2048;

int check_drop(const radamw_dropout_options &o, int64_t n, DropArgs *d) {
    if (!(o.p >= 0.0 && o.p <= 1.0) || o.first_row < 0) return RADAMW_ERR_INVALID;
    if (o.first_row > (int64_t(1) << 32) - n) return RADAMW_ERR_RANGE;
    const uint32_t t = static_cast<uint32_t>(std::floor(o.p * 65536.0 + 0.5));
    *d = {static_cast<uint32_t>(o.seed), static_cast<uint32_t>(o.seed >> 32), static_cast<uint32_t>(o.offset),
          static_cast<uint32_t>(o.offset >> 32), static_cast<uint32_t>(o.first_row), t,
          t < 65536 ? static_cast<float>(65536.0 / (65536.0 - t)) : 0.0f};
    return RADAMW_OK;
}

// Two arrays of rows that may be exactly the same one, which is then written.
int add_pair(Buffers &b, const void *in, int64_t in_stride, const void *out, int64_t out_stride, int64_t n, int64_t dim,
             size_t es) {
    int rc;
    const bool same = in == out && in_stride == out_stride;
    if ((rc = b.add(in, es, span(n, dim, in_stride, es), same))) return rc;
    return same ? RADAMW_OK : b.add(out, es, span(n, dim, out_stride, es), true);
}

int64_t gate_rows(int64_t n, int64_t per) { return (n + per - 1) / per; }

// Types, sizes and options of a residual call.
int check_residual(const radamw_residual_block *k, const radamw_residual_options *o, DropArgs *d) {
    int rc;
    if (!k || !o || !valid_dtype(k->stream_dtype) || !valid_dtype(k->branch_dtype)) return RADAMW_ERR_INVALID;
    if (k->stream_dtype != k->branch_dtype && k->stream_dtype != RADAMW_F32) return RADAMW_ERR_INVALID;
    if (!std::isfinite(o->eps) || !(static_cast<float>(o->eps) > 0.0f) || !std::isfinite(static_cast<float>(o->eps)))
        return RADAMW_ERR_INVALID;
    if ((rc = finite_scale(o->weight_offset)) || (rc = finite_scale(o->residual_scale))) return rc;
    // arrays of no rows may be NULL
    if (k->n > 0 && !k->branch && (k->gate || k->post_weight || !k->pre_weight)) return RADAMW_ERR_INVALID;
    if ((k->post_weight || k->pre_weight) && !valid_dtype(k->weight_dtype)) return RADAMW_ERR_INVALID;
    if ((rc = check_rows(k->n, k->dim, k->dim, RESIDUAL_MAX_DIM))) return rc;
    if (k->branch && (rc = check_rows(k->n, k->dim, k->branch_stride, RESIDUAL_MAX_DIM))) return rc;
    if (k->gate) {
        if (!valid_dtype(k->gate_dtype) || k->rows_per_gate < 1) return RADAMW_ERR_INVALID;
        if ((rc = check_rows(gate_rows(k->n, std::min(k->rows_per_gate, MAX_ROWS)), k->dim, k->gate_stride,
                             RESIDUAL_MAX_DIM)))
            return rc;
    }
    return check_drop(o->dropout, k->n, d);
}

// What both residual calls read.
int add_block(Buffers &b, const radamw_residual_block *k, int64_t per) {
    int rc;
    const size_t ws = grad_bytes(k->weight_dtype);
    if (k->gate) {
        const size_t gs = grad_bytes(k->gate_dtype);
        if ((rc = b.add(k->gate, gs, span(gate_rows(k->n, per), k->dim, k->gate_stride, gs), false))) return rc;
    }
    if (k->post_weight && (rc = b.add(k->post_weight, ws, k->dim * static_cast<int64_t>(ws), false))) return rc;
    if (k->pre_weight && (rc = b.add(k->pre_weight, ws, k->dim * static_cast<int64_t>(ws), false))) return rc;
    return RADAMW_OK;
}

int check_balance(int64_t n, int64_t experts, int64_t stride, int dt, int idt, int64_t top_k, const void *offsets,
                  int64_t groups, const radamw_balance_options *o, double grad_scale) {
    int rc;
    if (!o || !valid_dtype(dt) || !valid_index(idt)) return RADAMW_ERR_INVALID;
    if (!std::isfinite(o->balance_coef) || !(o->balance_coef >= 0.0) || !std::isfinite(o->z_coef) || !(o->z_coef >= 0.0))
        return RADAMW_ERR_INVALID;
    if (o->score != RADAMW_SCORE_SOFTMAX && o->score != RADAMW_SCORE_SIGMOID) return RADAMW_ERR_INVALID;
    if (o->score == RADAMW_SCORE_SIGMOID && o->z_coef != 0.0) return RADAMW_ERR_INVALID;
    if ((rc = finite_scale(grad_scale))) return rc;
    if (top_k < 1 || groups < 1 || (!offsets && groups != 1)) return RADAMW_ERR_INVALID;
    if ((rc = check_rows(n, experts, stride, BALANCE_MAX_EXPERTS))) return rc;
    return top_k > MAX_ROWS || n > MAX_ROWS / top_k || groups > MAX_GROUPS ? RADAMW_ERR_RANGE : RADAMW_OK;
}

}  // namespace

extern "C" {

radamw_dropout_options radamw_dropout_options_default(void) { return radamw_dropout_options{0.0, 0, 0, 0}; }

int radamw_dropout(const void *x, radamw_dtype dtype, int64_t n, int64_t dim, int64_t stride,
                   const radamw_dropout_options *opts, void *out, int64_t out_stride, radamw_stream_t stream_) {
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    int rc;
    if (!opts || !valid_dtype(dtype)) return RADAMW_ERR_INVALID;
    if ((rc = check_rows(n, dim, stride, MAX_DROPOUT_DIM))) return rc;
    if ((rc = check_rows(n, dim, out_stride, MAX_DROPOUT_DIM))) return rc;
    DropoutArgs a{x, out, n, dim, stride, out_stride, {}};
    if ((rc = check_drop(*opts, n, &a.drop))) return rc;
    if (n == 0) return RADAMW_OK;
    int dev;
    if ((rc = stream_device(stream, &dev))) return rc;
    DeviceScope scope(dev);
    Buffers b(dev);
    if ((rc = add_pair(b, x, stride, out, out_stride, n, dim, grad_bytes(dtype)))) return rc;
    if ((rc = b.alias())) return rc;
    int launched = 0;
    rc = hip_status(launch_dropout(a, dtype, stream, &launched));
    count_launches(launched);
    return rc;
}

radamw_residual_options radamw_residual_options_default(void) {
    return radamw_residual_options{1e-6, 0.0, 1.0, radamw_dropout_options_default()};
}

int radamw_residual_norm(const radamw_residual_block *k, const void *x, int64_t x_stride,
                         const radamw_residual_options *opts, void *h, int64_t h_stride, void *out, int64_t out_stride,
                         float *rstd, radamw_stream_t stream_) {
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    int rc;
    DropArgs drop{};
    if ((rc = check_residual(k, opts, &drop))) return rc;
    if (k->n > 0 && ((!k->branch && h) || (!k->pre_weight && out))) return RADAMW_ERR_INVALID;
    if ((rc = check_rows(k->n, k->dim, x_stride, RESIDUAL_MAX_DIM))) return rc;
    if (k->branch && (rc = check_rows(k->n, k->dim, h_stride, RESIDUAL_MAX_DIM))) return rc;
    if (k->pre_weight && (rc = check_rows(k->n, k->dim, out_stride, RESIDUAL_MAX_DIM))) return rc;
    if (k->n == 0) return RADAMW_OK;
    int dev;
    if ((rc = stream_device(stream, &dev))) return rc;
    DeviceScope scope(dev);
    Buffers b(dev);
    const int64_t per = k->gate ? std::min(k->rows_per_gate, MAX_ROWS) : 1;
    const size_t ss = grad_bytes(k->stream_dtype), bs = grad_bytes(k->branch_dtype);
    if (k->branch) {
        if ((rc = add_pair(b, x, x_stride, h, h_stride, k->n, k->dim, ss))) return rc;
        if (k->pre_weight) {
            if ((rc = add_pair(b, k->branch, k->branch_stride, out, out_stride, k->n, k->dim, bs))) return rc;
        } else if ((rc = b.add(k->branch, bs, span(k->n, k->dim, k->branch_stride, bs), false))) {
            return rc;
        }
    } else {
        if ((rc = b.add(x, ss, span(k->n, k->dim, x_stride, ss), false))) return rc;
        if ((rc = b.add(out, bs, span(k->n, k->dim, out_stride, bs), true))) return rc;
    }
    if ((rc = add_block(b, k, per))) return rc;
    if (rstd && (rc = b.add(rstd, 4, 2 * k->n * 4, true))) return rc;
    if ((rc = b.alias())) return rc;
    ResidualArgs a{x, k->branch, k->gate, k->post_weight, k->pre_weight, h, out, rstd,
                   x_stride, k->branch_stride, k->gate_stride, h_stride, out_stride, k->n, k->dim, per,
                   k->gate_dtype, k->weight_dtype, static_cast<float>(opts->eps),
                   static_cast<float>(opts->weight_offset), static_cast<float>(opts->residual_scale), drop};
    int launched = 0;
    rc = hip_status(launch_residual(a, k->stream_dtype, k->branch_dtype, stream, &launched));
    count_launches(launched);
    return rc;
}

int64_t radamw_residual_grad_workspace_bytes(int64_t n, int64_t dim, int64_t rows_per_gate) {
    int rc;
    if ((rc = check_rows(n, dim, dim, RESIDUAL_MAX_DIM))) return rc;
    if (rows_per_gate < 1) return RADAMW_ERR_INVALID;
    return residual_plan(n, dim, rows_per_gate).bytes;
}

int radamw_residual_norm_grad(const radamw_residual_block *k, const void *h, int64_t h_stride, const float *rstd,
                              const radamw_residual_options *opts, const void *grad_h, int64_t grad_h_stride,
                              const void *grad_out, int64_t grad_out_stride, void *grad_x, int64_t grad_x_stride,
                              void *grad_branch, int64_t grad_branch_stride, void *grad_gate, int64_t grad_gate_stride,
                              void *grad_post_weight, void *grad_pre_weight, void *workspace, int64_t workspace_bytes,
                              radamw_stream_t stream_) {
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    int rc;
    DropArgs drop{};
    if ((rc = check_residual(k, opts, &drop))) return rc;
    if ((!k->post_weight && grad_post_weight) || (!k->pre_weight && grad_pre_weight)) return RADAMW_ERR_INVALID;
    if (k->n > 0 && ((!k->branch && grad_branch) || (!k->gate && grad_gate) || (!k->pre_weight && (grad_out || !grad_h))))
        return RADAMW_ERR_INVALID;
    const int64_t n = k->n, dim = k->dim;
    if (k->pre_weight && (rc = check_rows(n, dim, h_stride, RESIDUAL_MAX_DIM))) return rc;
    if (k->pre_weight && (rc = check_rows(n, dim, grad_out_stride, RESIDUAL_MAX_DIM))) return rc;
    if (grad_h && (rc = check_rows(n, dim, grad_h_stride, RESIDUAL_MAX_DIM))) return rc;
    if ((rc = check_rows(n, dim, grad_x_stride, RESIDUAL_MAX_DIM))) return rc;
    if (k->branch && (rc = check_rows(n, dim, grad_branch_stride, RESIDUAL_MAX_DIM))) return rc;
    const int64_t per = k->gate ? std::min(k->rows_per_gate, MAX_ROWS) : 1;
    if (grad_gate && (rc = check_rows(gate_rows(n, per), dim, grad_gate_stride, RESIDUAL_MAX_DIM))) return rc;
    const ResidualPlan plan = residual_plan(n, dim, per);
    const bool sums = grad_post_weight || grad_pre_weight || (grad_gate && per != 1);
    if (n == 0 && !sums) return RADAMW_OK;
    if (sums && workspace_bytes < plan.bytes) return RADAMW_ERR_RANGE;
    int dev;
    if ((rc = stream_device(stream, &dev))) return rc;
    DeviceScope scope(dev);
    Buffers b(dev);
    const size_t ss = grad_bytes(k->stream_dtype), bs = grad_bytes(k->branch_dtype), ws = grad_bytes(k->weight_dtype);
    if (k->pre_weight && (rc = b.add(h, ss, span(n, dim, h_stride, ss), false))) return rc;
    if ((k->post_weight || k->pre_weight) && (rc = b.add(rstd, 4, 2 * n * 4, false))) return rc;
    if (grad_h) {
        if ((rc = add_pair(b, grad_h, grad_h_stride, grad_x, grad_x_stride, n, dim, ss))) return rc;
    } else if ((rc = b.add(grad_x, ss, span(n, dim, grad_x_stride, ss), true))) {
        return rc;
    }
    if (k->branch && (rc = b.add(k->branch, bs, span(n, dim, k->branch_stride, bs), false))) return rc;
    if (k->branch && k->pre_weight) {
        if ((rc = add_pair(b, grad_out, grad_out_stride, grad_branch, grad_branch_stride, n, dim, bs))) return rc;
    } else {
        if (k->pre_weight && (rc = b.add(grad_out, bs, span(n, dim, grad_out_stride, bs), false))) return rc;
        if (k->branch && (rc = b.add(grad_branch, bs, span(n, dim, grad_branch_stride, bs), true))) return rc;
    }
    if ((rc = add_block(b, k, per))) return rc;
    if (grad_gate) {
        const size_t gs = grad_bytes(k->gate_dtype);
        if ((rc = b.add(grad_gate, gs, span(gate_rows(n, per), dim, grad_gate_stride, gs), true))) return rc;
    }
    if (grad_post_weight && (rc = b.add(grad_post_weight, ws, dim * static_cast<int64_t>(ws), true))) return rc;
    if (grad_pre_weight && (rc = b.add(grad_pre_weight, ws, dim * static_cast<int64_t>(ws), true))) return rc;
    if (sums && (rc = b.add(workspace, 16, plan.bytes, true))) return rc;
    if ((rc = b.alias())) return rc;
    ResidualGradArgs a{h, k->branch, k->gate, k->post_weight, k->pre_weight, rstd, grad_h, grad_out, grad_x, grad_branch,
                       grad_gate, grad_post_weight, grad_pre_weight, h_stride, k->branch_stride, k->gate_stride,
                       grad_h_stride, grad_out_stride, grad_x_stride, grad_branch_stride, grad_gate_stride, n, dim, per,
                       k->gate_dtype, k->weight_dtype, static_cast<float>(opts->weight_offset),
                       static_cast<float>(opts->residual_scale), drop, static_cast<char *>(workspace)};
    int launched = 0;
    rc = hip_status(launch_residual_grad(a, plan, k->stream_dtype, k->branch_dtype, stream, &launched));
    count_launches(launched);
    return rc;
}

radamw_balance_options radamw_balance_options_default(void) {
    return radamw_balance_options{0.01, 0.0, RADAMW_SCORE_SOFTMAX};
}

int64_t radamw_balance_workspace_bytes(int64_t n, int64_t experts, int64_t groups) {
    int rc;
    if ((rc = check_rows(n, experts, experts, BALANCE_MAX_EXPERTS))) return rc;
    if (groups < 1) return RADAMW_ERR_INVALID;
    if (groups > MAX_GROUPS) return RADAMW_ERR_RANGE;
    return balance_plan(n, experts, groups).bytes;
}

int radamw_balance_loss(const void *logits, radamw_dtype dtype, int64_t n, int64_t experts, int64_t stride,
                        const void *ids, radamw_index_type index_type, int64_t top_k, const uint8_t *mask,
                        const void *offsets, int64_t groups, const float *weights, const radamw_balance_options *opts,
                        double grad_scale, float *total, float *loss, int32_t *counts, int32_t *tokens,
                        float *mean_prob, void *grad, int64_t grad_stride, void *workspace, int64_t workspace_bytes,
                        radamw_stream_t stream_) {
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    int rc;
    if ((rc = check_balance(n, experts, stride, dtype, index_type, top_k, offsets, groups, opts, grad_scale))) return rc;
    if (grad && (rc = check_rows(n, experts, grad_stride, BALANCE_MAX_EXPERTS))) return rc;
    const BalancePlan plan = balance_plan(n, experts, groups);
    if (workspace_bytes < plan.bytes) return RADAMW_ERR_RANGE;
    int dev;
    if ((rc = stream_device(stream, &dev))) return rc;
    DeviceScope scope(dev);
    Buffers b(dev);
    const size_t es = grad_bytes(dtype);
    const int64_t is = static_cast<int64_t>(index_bytes(index_type));
    if (grad) {
        if ((rc = add_pair(b, logits, stride, grad, grad_stride, n, experts, es))) return rc;
    } else if ((rc = b.add(logits, es, span(n, experts, stride, es), false))) {
        return rc;
    }
    if ((rc = b.add(ids, index_bytes(index_type), n * top_k * is, false))) return rc;
    if (mask && (rc = b.add(mask, 1, n, false))) return rc;
    if (offsets && (rc = b.add(offsets, index_bytes(index_type), (groups + 1) * is, false))) return rc;
    if (weights && (rc = b.add(weights, 4, groups * 4, false))) return rc;
    if ((rc = b.add(total, 4, 4, true))) return rc;
    if ((rc = b.add(loss, 4, groups * 4, true))) return rc;
    if ((rc = b.add(counts, 4, groups * experts * 4, true))) return rc;
    if ((rc = b.add(tokens, 4, groups * 4, true))) return rc;
    if ((rc = b.add(mean_prob, 4, groups * experts * 4, true))) return rc;
    if ((rc = b.add(workspace, 16, plan.bytes, true))) return rc;
    if ((rc = b.alias())) return rc;
    BalanceArgs a{logits, ids, mask, offsets, weights, n, experts, stride, groups, top_k, index_type == RADAMW_I64,
                  opts->score == RADAMW_SCORE_SIGMOID, opts->balance_coef, opts->z_coef, total, loss, mean_prob, counts,
                  tokens, nullptr, grad, grad_stride, static_cast<double>(static_cast<float>(grad_scale)),
                  static_cast<char *>(workspace)};
    int launched = 0;
    rc = hip_status(launch_balance_loss(a, plan, dtype, stream, &launched));
    count_launches(launched);
    return rc;
}

int radamw_balance_grad(const void *logits, radamw_dtype dtype, int64_t n, int64_t experts, int64_t stride,
                        int64_t top_k, const uint8_t *mask, const void *offsets, radamw_index_type offsets_type,
                        int64_t groups, const float *weights, const radamw_balance_options *opts, const int32_t *counts,
                        const int32_t *tokens, const float *upstream, double grad_scale, void *grad,
                        int64_t grad_stride, radamw_stream_t stream_) {
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    int rc;
    if ((rc = check_balance(n, experts, stride, dtype, offsets_type, top_k, offsets, groups, opts, grad_scale))) return rc;
    if ((rc = check_rows(n, experts, grad_stride, BALANCE_MAX_EXPERTS))) return rc;
    if (n == 0) return RADAMW_OK;
    int dev;
    if ((rc = stream_device(stream, &dev))) return rc;
    DeviceScope scope(dev);
    Buffers b(dev);
    const size_t es = grad_bytes(dtype);
    const int64_t is = static_cast<int64_t>(index_bytes(offsets_type));
    if ((rc = add_pair(b, logits, stride, grad, grad_stride, n, experts, es))) return rc;
    if (mask && (rc = b.add(mask, 1, n, false))) return rc;
    if (offsets && (rc = b.add(offsets, index_bytes(offsets_type), (groups + 1) * is, false))) return rc;
    if (weights && (rc = b.add(weights, 4, groups * 4, false))) return rc;
    if ((rc = b.add(counts, 4, groups * experts * 4, false))) return rc;
    if ((rc = b.add(tokens, 4, groups * 4, false))) return rc;
    if (upstream && (rc = b.add(upstream, 4, 4, false))) return rc;
    if ((rc = b.alias())) return rc;
    BalanceArgs a{logits, nullptr, mask, offsets, weights, n, experts, stride, groups, top_k, offsets_type == RADAMW_I64,
                  opts->score == RADAMW_SCORE_SIGMOID, opts->balance_coef, opts->z_coef, nullptr, nullptr, nullptr,
                  const_cast<int32_t *>(counts), const_cast<int32_t *>(tokens), upstream, grad, grad_stride,
                  static_cast<double>(static_cast<float>(grad_scale)), nullptr};
    int launched = 0;
    rc = hip_status(launch_balance_grad(a, balance_plan(n, experts, groups), dtype, stream, &launched));
    count_launches(launched);
    return rc;
}

}  // extern "C"
