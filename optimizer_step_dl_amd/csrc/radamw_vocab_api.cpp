// radamw_vocab_api.cpp -- the C ABI of the operators at the vocabulary's two
// ends of a training step: the embedding lookup and its gradient, the
// clipped policy loss, the preference loss and the logits' gradient from
// saved records.  Validation and launches only.
//
// Every entry point validates all of its arguments before it launches
// anything; the checks allocate nothing.
#include "radamw.h"
#include "radamw_host.h"
#include "radamw_vocab.h"

#include <cmath>

using namespace radamw;

namespace {

// The buffers of one call: each is queried once per allocation, and written
// ranges may overlap nothing.
class Buffers {
  public:
    explicit Buffers(int dev) : dev_(dev) {}

    int add(const void *p, size_t align, int64_t bytes, bool written) {
        if (bytes <= 0) return RADAMW_OK;
        if (!p) return RADAMW_ERR_INVALID;
        const uintptr_t a = reinterpret_cast<uintptr_t>(p);
        if (a % align != 0) return RADAMW_ERR_ALIGN;
        const uintptr_t end = a + static_cast<uintptr_t>(bytes);
        if (end < a) return RADAMW_ERR_INVALID;
        bool known = false;
        for (int i = 0; i < extents_; ++i) {
            if (a < extent_[i].lo || a >= extent_[i].hi) continue;
            if (end > extent_[i].hi) return RADAMW_ERR_INVALID;
            known = true;
            break;
        }
        if (!known) {
            uintptr_t lo = 0, hi = 0;
            const int rc = query_extent(dev_, p, &lo, &hi);
            if (rc != RADAMW_OK) return rc;
            if (hi != 0) {
                if (end > hi) return RADAMW_ERR_INVALID;
                extent_[extents_++] = {lo, hi, false};
            }
        }
        range_[ranges_++] = {a, end, written};
        return RADAMW_OK;
    }

    // RADAMW_ERR_ALIAS when a written range overlaps another one.
    int alias() {
        for (int i = 0; i < ranges_; ++i)
            for (int j = i + 1; j < ranges_; ++j)
                if ((range_[i].written || range_[j].written) && range_[i].lo < range_[j].hi &&
                    range_[j].lo < range_[i].hi)
                    return RADAMW_ERR_ALIAS;
        return RADAMW_OK;
    }

  private:
    static constexpr int MOST = 16;
    int dev_;
    int extents_ = 0, ranges_ = 0;
    Range extent_[MOST], range_[MOST];
};

// Dimensions and vocabularies above these are rejected: grid dimensions other
// than x hold 65535 workgroups.
constexpr int64_t MAX_DIM = int64_t(1) << 24;
constexpr int64_t MAX_VOCAB = int64_t(1) << 27;

bool valid_index(int idt) { return idt == RADAMW_I32 || idt == RADAMW_I64; }
size_t index_bytes(int idt) { return idt == RADAMW_I64 ? 8 : 4; }

// Bytes a [n, width] array with row stride `stride` spans.
int64_t span(int64_t n, int64_t width, int64_t stride, size_t elem) {
    return n > 0 && width > 0 ? ((n - 1) * stride + width) * static_cast<int64_t>(elem) : 0;
}

// Counts, widths and strides that index without overflow.
int check_rows(int64_t n, int64_t width, int64_t stride, int64_t max_width) {
    if (n < 0 || width < 1 || stride < width) return RADAMW_ERR_INVALID;
    if (n > VOCAB_MAX_ROWS || width > max_width || stride > MAX_ELEMENTS) return RADAMW_ERR_RANGE;
    if (n > 0 && stride > MAX_ELEMENTS / n) return RADAMW_ERR_RANGE;
    return RADAMW_OK;
}

void count_launches(int k) { g_launches.fetch_add(static_cast<uint64_t>(k), std::memory_order_relaxed); }

int finite_scale(double s) { return std::isfinite(s) && std::isfinite(static_cast<float>(s)) ? RADAMW_OK : RADAMW_ERR_INVALID; }

// The logits, labels and (optional) gradient of a loss.
int check_logits(const LogitsArgs &x, int dt, int idt, Buffers &b) {
    const size_t es = grad_bytes(dt);
    int rc;
    const bool in_place = x.grad == x.logits && x.grad_stride == x.stride;
    if ((rc = b.add(x.logits, es, span(x.n, x.vocab, x.stride, es), in_place))) return rc;
    if ((rc = b.add(x.labels, index_bytes(idt), x.n * static_cast<int64_t>(index_bytes(idt)), false))) return rc;
    if (x.grad && !in_place && (rc = b.add(x.grad, es, span(x.n, x.vocab, x.grad_stride, es), true))) return rc;
    return RADAMW_OK;
}

int check_logits_shape(int64_t n, int64_t vocab, int64_t stride, const void *grad, int64_t grad_stride) {
    int rc;
    if ((rc = check_rows(n, vocab, stride, MAX_VOCAB))) return rc;
    if (grad && (rc = check_rows(n, vocab, grad_stride, MAX_VOCAB))) return rc;
    return RADAMW_OK;
}

}  // namespace

extern "C" {

int radamw_embedding_lookup(const void *table, radamw_dtype table_dtype, int64_t rows, int64_t dim,
                            int64_t table_stride, const void *ids, radamw_index_type ids_type, int64_t n, double scale,
                            void *out, radamw_dtype out_dtype, int64_t out_stride, radamw_stream_t stream_) {
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    int rc;
    if (!valid_dtype(table_dtype) || !valid_dtype(out_dtype) || !valid_index(ids_type)) return RADAMW_ERR_INVALID;
    if ((rc = finite_scale(scale))) return rc;
    if ((rc = check_rows(rows, dim, table_stride, MAX_DIM))) return rc;
    if ((rc = check_rows(n, dim, out_stride, MAX_DIM))) return rc;
    if (n == 0) return RADAMW_OK;
    if (lookup_blocks(n, dim) > LAUNCH_MAX_BLOCKS) return RADAMW_ERR_RANGE;
    int dev;
    if ((rc = stream_device(stream, &dev))) return rc;
    DeviceScope scope(dev);
    Buffers b(dev);
    if ((rc = b.add(table, grad_bytes(table_dtype), span(rows, dim, table_stride, grad_bytes(table_dtype)), false)))
        return rc;
    if ((rc = b.add(ids, index_bytes(ids_type), n * static_cast<int64_t>(index_bytes(ids_type)), false))) return rc;
    if ((rc = b.add(out, grad_bytes(out_dtype), span(n, dim, out_stride, grad_bytes(out_dtype)), true))) return rc;
    if ((rc = b.alias())) return rc;
    LookupArgs a{table, ids, out, table_stride, out_stride, n, rows, dim, static_cast<float>(scale),
                 ids_type == RADAMW_I64};
    if ((rc = hip_status(launch_embedding_lookup(a, table_dtype, out_dtype, stream)))) return rc;
    count_launches(1);
    return RADAMW_OK;
}

int64_t radamw_embedding_grad_workspace_bytes(int64_t n, int64_t rows, int64_t dim) {
    int rc;
    if ((rc = check_rows(n, dim, dim, MAX_DIM))) return rc;
    if ((rc = check_rows(rows, dim, dim, MAX_DIM))) return rc;
    return embedding_plan(n, rows, dim).bytes;
}

int radamw_embedding_grad(const void *grad_out, radamw_dtype grad_dtype, int64_t grad_stride, const void *ids,
                          radamw_index_type ids_type, int64_t n, int64_t rows, int64_t dim, double scale,
                          int64_t padding_id, int32_t accumulate, void *table_grad, radamw_dtype table_dtype,
                          int64_t table_stride, void *workspace, int64_t workspace_bytes, radamw_stream_t stream_) {
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    int rc;
    if (!valid_dtype(grad_dtype) || !valid_dtype(table_dtype) || !valid_index(ids_type)) return RADAMW_ERR_INVALID;
    if ((rc = finite_scale(scale))) return rc;
    if (padding_id < -1 || (accumulate != 0 && accumulate != 1)) return RADAMW_ERR_INVALID;
    if ((rc = check_rows(n, dim, grad_stride, MAX_DIM))) return rc;
    if ((rc = check_rows(rows, dim, table_stride, MAX_DIM))) return rc;
    if (padding_id >= rows) return RADAMW_ERR_RANGE;
    if (rows == 0 || (n == 0 && accumulate)) return RADAMW_OK;
    const EmbeddingPlan plan = embedding_plan(n, rows, dim);
    if (workspace_bytes < plan.bytes) return RADAMW_ERR_RANGE;
    // the sums' grid is the largest: a chunk holds 64 tokens at these sizes, so
    // that the join has at most 2^25 / 8 workgroups of 512 lanes and the sort
    // 2^20 tiles beside 2^20 that clear
    if (plan.sum_blocks > LAUNCH_MAX_BLOCKS) return RADAMW_ERR_RANGE;
    int dev;
    if ((rc = stream_device(stream, &dev))) return rc;
    DeviceScope scope(dev);
    Buffers b(dev);
    if ((rc = b.add(grad_out, grad_bytes(grad_dtype), span(n, dim, grad_stride, grad_bytes(grad_dtype)), false)))
        return rc;
    if ((rc = b.add(ids, index_bytes(ids_type), n * static_cast<int64_t>(index_bytes(ids_type)), false))) return rc;
    if ((rc = b.add(table_grad, grad_bytes(table_dtype), span(rows, dim, table_stride, grad_bytes(table_dtype)), true)))
        return rc;
    if ((rc = b.add(workspace, 16, plan.bytes, true))) return rc;
    if ((rc = b.alias())) return rc;
    EmbeddingGradArgs a{grad_out, ids, table_grad, grad_stride, table_stride, n, rows, dim, padding_id,
                        static_cast<float>(scale), ids_type == RADAMW_I64, accumulate,
                        static_cast<char *>(workspace)};
    int launched = 0;
    rc = hip_status(launch_embedding_grad(a, plan, grad_dtype, table_dtype, stream, &launched));
    count_launches(launched);
    return rc;
}

radamw_policy_options radamw_policy_options_default(void) { return radamw_policy_options{0.2, 0.2, 0.0}; }

int radamw_policy_loss(const void *logits, radamw_dtype dtype, int64_t n, int64_t vocab, int64_t stride,
                       const void *labels, radamw_index_type labels_type, const float *old_logp, const float *ref_logp,
                       const float *advantages, const float *weights, const radamw_policy_options *opts,
                       double grad_scale, float *total, float *loss, float *logp, float *row_stats, void *grad,
                       int64_t grad_stride, radamw_stream_t stream_) {
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    int rc;
    if (!opts || !valid_dtype(dtype) || !valid_index(labels_type)) return RADAMW_ERR_INVALID;
    if (!(opts->clip_low >= 0.0 && opts->clip_low <= 1.0) || !(opts->clip_high >= 0.0) ||
        !std::isfinite(opts->clip_high) || !(opts->kl_coef >= 0.0) || !std::isfinite(opts->kl_coef))
        return RADAMW_ERR_INVALID;
    if (opts->kl_coef != 0.0 && !ref_logp && n != 0) return RADAMW_ERR_INVALID;
    if ((rc = finite_scale(grad_scale))) return rc;
    if ((rc = check_logits_shape(n, vocab, stride, grad, grad_stride))) return rc;
    int dev;
    if ((rc = stream_device(stream, &dev))) return rc;
    DeviceScope scope(dev);
    Buffers b(dev);
    LogitsArgs x{logits, labels, n, vocab, stride, grad, grad_stride, static_cast<float>(grad_scale),
                 labels_type == RADAMW_I64, reinterpret_cast<RowStats *>(row_stats), logp, 0};
    const bool kl = opts->kl_coef != 0.0;
    if ((rc = check_logits(x, dtype, labels_type, b))) return rc;
    if (old_logp && (rc = b.add(old_logp, 4, n * 4, false))) return rc;
    if (kl && (rc = b.add(ref_logp, 4, n * 4, false))) return rc;
    if ((rc = b.add(advantages, 4, n * 4, false))) return rc;
    if (weights && (rc = b.add(weights, 4, n * 4, false))) return rc;
    if ((rc = b.add(total, 4, 4, true))) return rc;
    if ((rc = b.add(loss, 4, n * 4, true))) return rc;
    if ((rc = b.add(logp, 4, n * 4, true))) return rc;
    if (row_stats && (rc = b.add(row_stats, 16, n * 16, true))) return rc;
    if ((rc = b.alias())) return rc;
    PolicyArgs a{x, old_logp, kl ? ref_logp : nullptr, advantages, weights, opts->clip_low, opts->clip_high,
                 opts->kl_coef, loss, total};
    int launched = 0;
    rc = hip_status(launch_policy_loss(a, dtype, stream, &launched));
    count_launches(launched);
    return rc;
}

radamw_preference_options radamw_preference_options_default(void) { return radamw_preference_options{0.1, 0.0}; }

int radamw_preference_loss(const void *logits, radamw_dtype dtype, int64_t n, int64_t vocab, int64_t stride,
                           const void *labels, radamw_index_type index_type, const void *offsets, int64_t pairs,
                           const float *ref_logp, const float *weights, const radamw_preference_options *opts,
                           double grad_scale, float *total, float *loss, float *seq_logp, float *logp,
                           float *row_stats, void *grad, int64_t grad_stride, radamw_stream_t stream_) {
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    int rc;
    if (!opts || !valid_dtype(dtype) || !valid_index(index_type)) return RADAMW_ERR_INVALID;
    if (!std::isfinite(opts->beta) || !(opts->beta >= 0.0) ||
        !(opts->label_smoothing >= 0.0 && opts->label_smoothing <= 1.0))
        return RADAMW_ERR_INVALID;
    if ((rc = finite_scale(grad_scale))) return rc;
    if (pairs < 1) return RADAMW_ERR_INVALID;
    if (pairs > LAUNCH_MAX_BLOCKS) return RADAMW_ERR_RANGE;
    if ((rc = check_logits_shape(n, vocab, stride, grad, grad_stride))) return rc;
    int dev;
    if ((rc = stream_device(stream, &dev))) return rc;
    DeviceScope scope(dev);
    Buffers b(dev);
    LogitsArgs x{logits, labels, n, vocab, stride, grad, grad_stride, static_cast<float>(grad_scale),
                 index_type == RADAMW_I64, reinterpret_cast<RowStats *>(row_stats), logp, 0};
    if ((rc = check_logits(x, dtype, index_type, b))) return rc;
    const int64_t is = static_cast<int64_t>(index_bytes(index_type));
    if ((rc = b.add(offsets, index_bytes(index_type), (2 * pairs + 1) * is, false))) return rc;
    if ((rc = b.add(ref_logp, 4, 2 * pairs * 4, false))) return rc;
    if (weights && (rc = b.add(weights, 4, pairs * 4, false))) return rc;
    if ((rc = b.add(total, 4, 4, true))) return rc;
    if ((rc = b.add(loss, 4, pairs * 4, true))) return rc;
    if ((rc = b.add(seq_logp, 4, 2 * pairs * 4, true))) return rc;
    if ((rc = b.add(logp, 4, n * 4, true))) return rc;
    if ((rc = b.add(row_stats, 16, n * 16, true))) return rc;
    if ((rc = b.alias())) return rc;
    PreferenceArgs a{x, offsets, pairs, ref_logp, weights, opts->beta, opts->label_smoothing, loss, seq_logp, total};
    int launched = 0;
    rc = hip_status(launch_preference_loss(a, dtype, stream, &launched));
    count_launches(launched);
    return rc;
}

int radamw_logits_grad(const void *logits, radamw_dtype dtype, int64_t n, int64_t vocab, int64_t stride,
                       const void *labels, radamw_index_type labels_type, const float *row_stats,
                       const float *upstream, double grad_scale, void *grad, int64_t grad_stride,
                       radamw_stream_t stream_) {
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    int rc;
    if (!valid_dtype(dtype) || !valid_index(labels_type)) return RADAMW_ERR_INVALID;
    if ((rc = finite_scale(grad_scale))) return rc;
    if (!grad && n != 0) return RADAMW_ERR_INVALID;
    if ((rc = check_logits_shape(n, vocab, stride, grad, grad_stride))) return rc;
    if (n == 0) return RADAMW_OK;
    int dev;
    if ((rc = stream_device(stream, &dev))) return rc;
    DeviceScope scope(dev);
    Buffers b(dev);
    LogitsArgs x{logits, labels, n, vocab, stride, grad, grad_stride, static_cast<float>(grad_scale),
                 labels_type == RADAMW_I64, reinterpret_cast<RowStats *>(const_cast<float *>(row_stats)), nullptr, 0};
    if ((rc = check_logits(x, dtype, labels_type, b))) return rc;
    if ((rc = b.add(row_stats, 16, n * 16, false))) return rc;
    if (upstream && (rc = b.add(upstream, 4, 4, false))) return rc;
    if ((rc = b.alias())) return rc;
    int launched = 0;
    rc = hip_status(launch_logits_grad(x, upstream, dtype, stream, &launched));
    count_launches(launched);
    return rc;
}

}  // extern "C"
