// radamw_vocab.h -- structures shared by the vocabulary operators' C entry
// points (radamw_vocab_api.cpp) and their gfx950 kernels
// (radamw_embedding.hip, radamw_loss.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

namespace radamw {

// A launch addresses fewer than 2^32 work-items along x: workgroups of up to
// 256 lanes.
constexpr int64_t LAUNCH_MAX_BLOCKS = (int64_t(1) << 24) - 1;

// ------------------------------------------------------------- embedding --

struct LookupArgs {
    const void *table;
    const void *ids;
    void *out;
    int64_t table_stride, out_stride;  // elements
    int64_t n, rows, dim;
    float scale;
    int32_t wide_ids;  // 0: int32, 1: int64
};
// Workgroups (along x) of a lookup.
int64_t lookup_blocks(int64_t n, int64_t dim);
hipError_t launch_embedding_lookup(const LookupArgs &a, int tdt, int odt, hipStream_t stream);

// Tokens one workgroup sorts in LDS, in one launch; longer lists take the
// tiled sort.  Up to SORT_TINY_MAX it has four waves, which wait less for one
// another, else sixteen.
constexpr int SORT_SMALL_MAX = 8192;
constexpr int SORT_TINY_MAX = 1024;
// Tokens of one tile of the tiled sort.
constexpr int64_t SORT_TILE = 2048;
constexpr int SORT_MAX_DIGIT_BITS = 10;

// Workspace of an embedding gradient over n tokens (byte offsets).
struct EmbeddingPlan {
    int64_t keys[2], pos[2];  // two buffers each of sorted ids and token positions (u32)
    int64_t counts;           // digit counts of the tiled sort's passes (u32)
    int64_t present;          // one byte per table row
    int64_t partials;         // FP32 sums of runs that cross a chunk: [chunks][2][dim]
    int64_t bytes;
    int32_t chunk;            // sorted tokens per chunk
    int64_t chunks;
    int32_t lg;               // 2^lg lanes own 8 columns each of one chunk's column tile
    int32_t tiles;            // column tiles per row
    int64_t sum_blocks;       // workgroups that sum
};

struct EmbeddingGradArgs {
    const void *grad_out;
    const void *ids;
    void *table_grad;
    int64_t grad_stride, table_stride;  // elements
    int64_t n, rows, dim;
    int64_t padding_id;  // -1: none
    float scale;
    int32_t wide_ids;
    int32_t accumulate;
    char *workspace;
};
EmbeddingPlan embedding_plan(int64_t n, int64_t rows, int64_t dim);
// *launched counts the kernels submitted.
hipError_t launch_embedding_grad(const EmbeddingGradArgs &a, const EmbeddingPlan &p, int gdt, int tgdt,
                                 hipStream_t stream, int *launched);

// ---------------------------------------------------------------- losses --

// Per-row record the losses keep for the backward pass.
struct RowStats {
    float max;        // a logit m near the largest
    float inv_sum;    // 1 / sum of exponentials relative to m
    float coef;       // d total / d log-probability of the label
    float one_less_p; // 1 - probability of the label
};
static_assert(sizeof(RowStats) == 16, "one 16-byte load");

struct LogitsArgs {
    const void *logits;
    const void *labels;
    int64_t n, vocab, stride;  // stride in elements
    void *grad;                // may be null
    int64_t grad_stride;
    float grad_scale;
    int32_t wide_ids;
    RowStats *stats;           // may be null for a policy loss
    float *logp;
    int64_t row0;              // first row of a launch
};

struct PolicyArgs {
    LogitsArgs x;
    const float *old_logp, *ref_logp, *advantages, *weights;  // old / ref / weights may be null
    double clip_low, clip_high, kl_coef;
    float *loss, *total;
};
hipError_t launch_policy_loss(const PolicyArgs &a, int dt, hipStream_t stream, int *launched);

struct PreferenceArgs {
    LogitsArgs x;
    const void *offsets;  // 2 * pairs + 1, of the labels' index type
    int64_t pairs;
    const float *ref_logp, *weights;  // weights may be null
    double beta, label_smoothing;
    float *loss, *seq_logp, *total;
};
hipError_t launch_preference_loss(const PreferenceArgs &a, int dt, hipStream_t stream, int *launched);

// grad = upstream * grad_scale * coef * (1[label] - p) from saved records.
hipError_t launch_logits_grad(const LogitsArgs &a, const float *upstream, int dt, hipStream_t stream, int *launched);

}  // namespace radamw
