/*
 * radamw.h -- C ABI of libradamw.so, the fused AdamW / AMSGrad optimizer
 * step for AMD Instinct MI355X (gfx950).
 *
 * Page abbreviations used in the citations below:
 *   FA-ja  = RUDA docs page "実験的なデバイス上の融合 AdamW / AMSGrad"
 *   FA-zh  = RUDA docs page "实验性融合 AdamW / AMSGrad"
 *   TR-zh  = RUDA docs page "训练与状态保存"
 *
 * General conventions (all entry points):
 *   - Every array pointer is a DEVICE pointer (hipMalloc / torch CUDA
 *     memory) unless the argument says "host".  Host pointers are rejected
 *     (FA-ja "サポートされている契約": no arbitrary host pointers).
 *   - Arrays are dense and contiguous, 1-D, indexed 0..n-1.  Parameters and
 *     moments are FP32; gradients are FP32, FP16 or BF16 (FA-zh
 *     "增加的实际能力").  Pointers must be aligned to their element size.
 *   - All device work is enqueued on `stream` (a hipStream_t; NULL is the
 *     legacy default stream) and is asynchronous: a RADAMW_OK return means
 *     the work was SUBMITTED, not that it completed (FA-ja "低レベルの使用").
 *     The caller keeps every buffer alive until the stream has passed the
 *     work, and synchronises before reading results or saving a checkpoint.
 *   - Any non-zero return other than RADAMW_ERR_HIP and RADAMW_ERR_DECISION
 *     means nothing was launched and nothing (device memory, state structs,
 *     step counts, output flags) was modified (FA-ja "低レベルの使用": validation leaves
 *     every input unchanged).  RADAMW_ERR_HIP reports a failing HIP runtime
 *     call; a multi-kernel entry point may have submitted earlier kernels,
 *     and the caller should treat the device state as unconfirmed (FA-ja
 *     "低レベルの使用": discard unconfirmed outputs after a device fault).
 *     The library keeps no pointer after a call returns, except a
 *     persistent tensor list (radamw_list_create), which keeps its
 *     segments' pointers until radamw_list_destroy.
 *   - There is no device-side step counter: the completed-step count lives
 *     in host memory owned by the caller, and the bias-correction
 *     coefficients are computed on the host for every call, so a captured
 *     graph replay would repeat one step's coefficients (FA-zh
 *     "增加的实际能力"); graph capture is not supported: a stream being
 *     captured is refused with RADAMW_ERR_INVALID before anything is
 *     launched or recorded.
 *   - Thread safety: calls may come from several host threads; each call is
 *     independent apart from the launch counter and the per-device caches
 *     (segment-table staging, the mapped report page, the second update
 *     stream), which are internally locked.  Multi-tensor calls on
 *     different caller streams of one device share that device's second
 *     stream, so their update launches may wait for one another.
 */
#ifndef RADAMW_H
#define RADAMW_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* hipStream_t without requiring the HIP headers in C callers. */
typedef struct ihipStream_t *radamw_stream_t;

/* ----------------------------------------------------------- status codes */
enum {
    RADAMW_OK = 0,
    RADAMW_ERR_INVALID = -1, /* null pointer, n < 0, unknown dtype, host pointer,
                                pointer of another device, an array running
                                past the end of its allocation, hyper-
                                parameter out of range, non-finite or
                                non-positive gradient_scale, flag not 0/1,
                                a stream being captured into a graph          */
    RADAMW_ERR_STATE = -2,   /* AMSGrad flag and v_max presence disagree, or
                                the step count would overflow                 */
    RADAMW_ERR_ALIAS = -3,   /* a written range overlaps another range         */
    RADAMW_ERR_ALIGN = -4,   /* pointer not aligned to its element size        */
    RADAMW_ERR_RANGE = -5,   /* row count / capacity / scratch size out of
                                range; an element count above 2^48 (any
                                entry point taking n)                         */
    RADAMW_ERR_HIP = -6,     /* a HIP runtime call failed (see
                                radamw_last_hip_error)                         */
    RADAMW_ERR_DECISION = -7 /* fused steps only: the host's skip / clip
                                decision from the read-back report differs
                                from the one the device took and applied (a
                                library fault; never expected).  Unlike the
                                other errors the step DID run as the device
                                decided: the result struct and the step count
                                follow the device's decision.                 */
};

/* Gradient storage type (FA-zh "增加的实际能力"). */
typedef enum {
    RADAMW_F32 = 0,
    RADAMW_F16 = 1,  /* IEEE binary16 */
    RADAMW_BF16 = 2  /* bfloat16: the upper 16 bits of a binary32 */
} radamw_dtype;

/*
 * Hyper-parameters of the update (FA-ja "この演算子を使用する理由": formula
 * and defaults; FA-ja "低レベルの使用": the options struct).  Checked:
 * lr >= 0, eps >= 0, weight_decay >= 0, 0 <= beta1, beta2 < 1, all finite;
 * amsgrad and maximize are 0 or 1.
 */
typedef struct {
    double lr;
    double beta1;
    double beta2;
    double eps;
    double weight_decay;
    int32_t amsgrad;
    int32_t maximize;
} radamw_options;

/*
 * Per-call control (FA-ja "低レベルの使用": StepControl).  The stored
 * gradient is divided by gradient_scale (finite, > 0).  skip_update = 1 is
 * the caller's found_inf decision: no launch, no write, no step increment
 * (FA-zh "增加的实际能力").  The library never scans for non-finite values
 * inside the update itself.
 */
typedef struct {
    double gradient_scale;
    int32_t skip_update;
} radamw_control;

/*
 * Optimizer state of one tensor (FA-ja "低レベルの使用": the state exposes
 * the step and the moment buffers).  step is the number of completed
 * updates; step == 0 is the pages' "no state yet": the next update is t = 1
 * and initialises the moments inside the kernel without reading them
 * (FA-zh "增加的实际能力").  exp_avg / exp_avg_sq / max_exp_avg_sq are
 * device FP32 arrays of n elements; max_exp_avg_sq is non-NULL exactly when
 * AMSGrad is on.
 */
typedef struct {
    uint64_t step;
    float *exp_avg;
    float *exp_avg_sq;
    float *max_exp_avg_sq;
} radamw_state;

/* One contiguous tensor of a multi-tensor update (in place). */
typedef struct {
    float *param;
    const void *grad;
    float *exp_avg;
    float *exp_avg_sq;
    float *max_exp_avg_sq; /* NULL unless AMSGrad */
    int64_t n;
} radamw_segment;

/*
 * 12-byte gradient-statistics record (TR-zh "在 ruda:0 上进行原生 PyTorch
 * 训练": a 12-byte report is read back before the update).  Layout chosen
 * here (the pages fix only the size): w[0] | w[1] << 32 is the IEEE binary64
 * sum of squares of the finite stored gradient values; w[2] is the count of
 * non-finite values, saturating at 2^32 - 1.  The same record is used for
 * the per-workgroup rows, the intermediate merge levels and the report.
 */
typedef struct {
    uint32_t w[3];
} radamw_stats;

/* Result of radamw_fused_step_multi (host struct). */
typedef struct {
    int32_t updated;     /* 1 when the update was launched                  */
    int32_t found_inf;   /* 1 when the report counted non-finite values     */
    uint32_t nonfinite;  /* the report's non-finite count                   */
    uint32_t reserved;
    double sumsq;        /* the report's sum of squares (stored scale)      */
    double total_norm;   /* sqrt(sumsq) / gradient_scale                    */
    double clip_coef;    /* min(1, max_norm / (total_norm + 1e-6)), or 1    */
} radamw_fused_result;

/* Defaults of FA-ja "この演算子を使用する理由": betas (0.9, 0.999),
 * eps 1e-5, weight decay 1e-4; lr 1e-3 as in the pages' usage examples;
 * amsgrad = maximize = 0.  Returns the struct by value. */
radamw_options radamw_options_default(void);

/*
 * Out-of-place update of one tensor (FA-ja "低レベルの使用": adamw_step;
 * FA-ja "割り当てとパフォーマンスのモデル": out-of-place outputs).
 *   p, g      : inputs, n elements; g has dtype gdt.  Never written.
 *   in        : host struct; in->step completed steps.  When in->step == 0
 *               the input moment pointers are not read (may be NULL).
 *   p_out     : output params (device, n FP32), caller-allocated.
 *   out       : host struct with caller-allocated output moment arrays
 *               (n FP32 each; max_exp_avg_sq iff amsgrad).  On launch,
 *               out->step = in->step + 1; otherwise out is not touched.
 *   updated   : host int32, set to 1 on launch, 0 on skip / n == 0.
 * No output range may overlap any input or other output (RADAMW_ERR_ALIAS).
 * skip_update or n == 0: nothing is launched or written (FA-zh
 * "增加的实际能力"), so the caller may allocate outputs only after a call
 * with ctrl->skip_update known to be 0.
 */
int radamw_step(const float *p, const void *g, radamw_dtype gdt, int64_t n,
                const radamw_state *in, float *p_out, radamw_state *out,
                const radamw_options *opts, const radamw_control *ctrl,
                radamw_stream_t stream, int32_t *updated);

/*
 * In-place update over caller-owned storage (FA-ja "ネイティブ PyTorch
 * ストレージと階層統計": the storage kernel adamw_scaled).  p, st->exp_avg,
 * st->exp_avg_sq (and st->max_exp_avg_sq iff AMSGrad) are read and written;
 * g is read only.  st->step is incremented only when the kernel is launched.
 */
int radamw_step_inplace(float *p, const void *g, radamw_dtype gdt, int64_t n,
                        radamw_state *st, const radamw_options *opts,
                        const radamw_control *ctrl, radamw_stream_t stream,
                        int32_t *updated);

/*
 * The staged (unfused) baseline, for measurement only (FA-ja
 * "割り当てとパフォーマンスのモデル", FA-zh "优化点与边界": a benchmark-only
 * baseline of four kernels, five with AMSGrad, that re-reads the gradient
 * and goes through a delta buffer; 48 bytes per parameter instead of 28, 60
 * instead of 36).  Same arguments and semantics as radamw_step_inplace,
 * plus delta: a caller-owned device scratch array of n FP32 (written).  The
 * per-element arithmetic is the fused kernel's, split across the launches
 * m -> v -> [v_max] -> delta -> p, so results are identical to
 * radamw_step_inplace.  Every array must be 16-byte aligned (RADAMW_ERR_ALIGN),
 * gradients of 16-bit types 8-byte aligned.
 */
/*
 * Placement of the streams of one flattened bucket (FA-ja
 * "サポートされている契約": a pre-flattened bucket whose elements share the
 * options and the step count) in a single allocation.  The update's
 * bandwidth depends on where its streams lie relative to one another in
 * HBM: on MI355X, p, g, m and v of a 2^28-element bucket exactly 1 GiB apart
 * update at ~6.44-6.55 TB/s, in separate allocations at ~6.54-6.59 TB/s,
 * and back to back in one allocation with each stream's start shifted by a
 * further 12 KiB at ~6.76-6.83 TB/s (3-4.5% faster for AdamW, AMSGrad and
 * 16-bit gradients; 3.6% at 1e8+7 elements).  The gain is for streams up to
 * about 1 GiB: streams of 5-27 GB came within +-2% of separate allocations.
 * The rule is measured, not derived: stream k starts at byte offset
 * k * pitch, with pitch = (n * max element size rounded up to 2 MiB) +
 * 12 KiB.
 *   n              : elements of every stream (0 <= n <= 2^48).
 *   element_bytes  : host array of nstreams element sizes (1, 2, 4 or 8),
 *                    in the order the caller wants the streams placed
 *                    (for example p, g, m, v, v_max); 1 <= nstreams <= 16.
 *   offsets        : host array of nstreams byte offsets (written).
 *   arena_bytes    : host, the allocation size the layout needs (written).
 * The arena's base should be 2 MiB-aligned (large hipMalloc allocations
 * are).  Host only; allocates nothing.  Any layout of the streams gives the
 * same results; this one is only faster.
 */
int radamw_bucket_layout(int64_t n, const int32_t *element_bytes, int32_t nstreams, int64_t *offsets,
                         int64_t *arena_bytes);

/*
 * Streaming ceiling, for measurement only.  FA-ja "残りゲート" asks that
 * performance work follow measured profiles rather than the traffic model;
 * this call measures what the memory system gives the update's access
 * pattern.  It moves nreads FP32 read streams and nwrites FP32 write streams
 * of n elements with the update kernel's geometry, cache hints and
 * occupancy rule, and one add per stream instead of the optimizer's
 * arithmetic: out[w][i] = ((in[0][i] + in[1][i]) + ...) + w (the empty sum
 * is 0).  AdamW with an FP32 gradient is the 4-read / 3-write pattern,
 * AMSGrad 5 / 4, a first step 2 / 3.
 *   in        : host array of nreads device pointers (0 <= nreads <= 5).
 *   out       : host array of max(nwrites, 1) device pointers
 *               (0 <= nwrites <= 4).  With nwrites == 0, out[0] is a sink of
 *               n floats that is never written in practice (a store guarded
 *               by a comparison with NaN keeps the loads live).
 *   n         : elements per stream, a multiple of 4; every array 16-byte
 *               aligned (RADAMW_ERR_ALIGN).
 *   cap_per_cu: resident workgroups per compute unit, 1..32, or 0 for the
 *               update kernels' own rule applied to 4 * (nreads + nwrites)
 *               bytes per element.
 * nreads + nwrites >= 1.  An output may be exactly one of the inputs
 * (in place, as the in-place update writes p, m and v: every element is
 * loaded before the same lane stores it); otherwise written arrays may
 * overlap nothing (RADAMW_ERR_ALIAS).  Read arrays may overlap each other.
 * n == 0 launches nothing.  radamw_time_next_update applies to this launch.
 */
int radamw_stream_probe(const float *const *in, int32_t nreads, float *const *out, int32_t nwrites,
                        int64_t n, int32_t cap_per_cu, radamw_stream_t stream);

int radamw_step_staged_inplace(float *p, const void *g, radamw_dtype gdt, int64_t n,
                               radamw_state *st, float *delta, const radamw_options *opts,
                               const radamw_control *ctrl, radamw_stream_t stream,
                               int32_t *updated);

/*
 * In-place update of a list of tensors that share one options struct and
 * one step count (FA-ja "サポートされている契約": a pre-flattened bucket
 * works only when every element shares the options and the step count).  A
 * flattened bucket is nseg == 1.  Launches: every tensor of at least 2^22
 * elements gets a launch of its own and all smaller tensors share a single
 * launch, so a list of many small tensors costs one launch, while large
 * tensors keep the single-tensor kernel (which measured faster than sharing
 * a launch).  All launches use the same constants and the step count
 * advances once.  With two or more launches, every other one runs on a
 * second stream the library keeps per device, so that the drain of one
 * launch overlaps the start of the next: that stream first waits for all
 * work queued on `stream` before the call, and `stream` waits for all of it
 * before anything queued after the call, so the call still orders on
 * `stream` exactly like a single launch.  The fused and list entry points
 * below submit their update launches the same way.
 *   segs  : host array of nseg descriptors (device pointers inside).
 *   step  : host, the shared completed-step count; incremented on launch.
 * Segments with n == 0 are ignored; when every segment is empty nothing is
 * launched and *step is unchanged.  No written range may overlap any other
 * range of any segment (RADAMW_ERR_ALIAS).  nseg >= 0.
 */
int radamw_step_multi(const radamw_segment *segs, int32_t nseg, radamw_dtype gdt,
                      uint64_t *step, const radamw_options *opts,
                      const radamw_control *ctrl, radamw_stream_t stream,
                      int32_t *updated);

/*
 * radamw_step_multi that also writes a 16-bit model copy of the updated
 * parameters in the same pass: models[i] (device, segs[i].n elements of
 * model_dtype, written) receives segs[i].param after the update, rounded to
 * nearest even (the FP16 / BF16 model weights of an FP32-master optimizer,
 * TR-zh "训练与状态保存": FP32 master parameters, 16-bit model storage).
 * models[i] may be NULL (no copy for that tensor).  model_dtype is
 * RADAMW_F16 or RADAMW_BF16.  Adds 2 bytes per parameter of traffic; the
 * update itself is identical to radamw_step_multi's.  Copies may overlap
 * nothing (RADAMW_ERR_ALIAS).
 */
int radamw_step_multi_writeback(const radamw_segment *segs, void *const *models, int32_t nseg,
                                radamw_dtype gdt, radamw_dtype model_dtype, uint64_t *step,
                                const radamw_options *opts, const radamw_control *ctrl,
                                radamw_stream_t stream, int32_t *updated);

/*
 * Merge plan for rows statistics records (FA-ja "ネイティブ PyTorch
 * ストレージと階層統計": StatsPlan; TR-zh "在 ruda:0 上进行原生 PyTorch
 * 训练": fan-in 1024, at most two extra merge kernels, at most 49,200 bytes
 * of reusable scratch).  rows must be in 1..4,194,304 (else
 * RADAMW_ERR_RANGE).  *scratch_elements receives the FP32-element count of
 * the intermediate levels (3 per record; initial rows and final report not
 * included); *extra_merge_kernels the number of fan-in-1024 levels before
 * the final merge (0 when rows <= 1024).  Host only; no device access.
 */
int radamw_stats_plan(int64_t rows, int64_t *scratch_elements,
                      int32_t *extra_merge_kernels);

/* Number of records one radamw_grad_stats call writes for n elements of
 * dtype gdt (a deterministic function of n and gdt alone; 0 when n == 0).
 * Returns a negative status for n < 0 or an unknown dtype.  Host only. */
int64_t radamw_grad_stats_rows(int64_t n, radamw_dtype gdt);

/*
 * Read-only analysis of one gradient (FA-ja "ネイティブ PyTorch ストレージと
 * 階層統計": analyze_gradient; TR-zh: gradient storage stays unchanged).
 * Writes radamw_grad_stats_rows(n, gdt) records to rows_out (device), each
 * the sum of squares of the finite values and the non-finite count of one
 * workgroup's share.  rows_capacity < that count -> RADAMW_ERR_RANGE.
 * *rows_written (host) receives the count (0 when n == 0: nothing launched).
 * The reduction order is fixed, so repeated calls give identical bits.
 */
int radamw_grad_stats(const void *g, radamw_dtype gdt, int64_t n,
                      radamw_stats *rows_out, int64_t rows_capacity,
                      int64_t *rows_written, radamw_stream_t stream);

/*
 * Reduce nrows records to the 12-byte report (FA-ja "ネイティブ PyTorch
 * ストレージと階層統計": merge_gradient_stats_chunks then
 * merge_gradient_stats; TR-zh: hierarchical fan-in 1024 changes only the
 * reduction order).  nrows in 1..4,194,304.
 *   hierarchical = 1: the radamw_stats_plan levels, each reducing groups of
 *     up to 1024 records into scratch, then one final merge into report.
 *     scratch (device, FP32 elements, 4-byte aligned) must hold
 *     scratch_elements >= the plan's count; it may be NULL when that count
 *     is 0.
 *   hierarchical = 0: one final merge over all rows (scratch unused).
 * Counts are bit-identical between the two modes; sums differ only by
 * FP64 rounding order.  report: 12 device bytes owned by the caller.
 */
int radamw_merge_stats(const radamw_stats *rows, int64_t nrows, float *scratch,
                       int64_t scratch_elements, radamw_stats *report,
                       int32_t hierarchical, radamw_stream_t stream);

/*
 * Read a device report back to the host (hipMemcpyAsync through a pinned
 * staging buffer, then stream synchronisation): the read-back of the step
 * composed from separate calls (TR-zh: the report is read back before any
 * update).  host_report: host struct.
 */
int radamw_read_report(const radamw_stats *report, radamw_stats *host_report,
                       radamw_stream_t stream);

/*
 * Host decision after the report (TR-zh "在 ruda:0 上进行原生 PyTorch 训练":
 * any non-finite gradient skips the whole step; optional global L2 clipping
 * after unscaling).  norm = sqrt(sumsq) / gradient_scale; clip = min(1,
 * max_grad_norm / (norm + 1e-6)) when max_grad_norm > 0, else 1.
 * Fills ctrl: skip_update = (count > 0); gradient_scale = gradient_scale /
 * clip (exactly gradient_scale when clip == 1).  result (optional, may be
 * NULL) receives the decoded report and the decision.  Host only.
 */
int radamw_decide(const radamw_stats *host_report, double gradient_scale,
                  double max_grad_norm, radamw_control *ctrl,
                  radamw_fused_result *result);

/*
 * The check every fused step makes after its read-back (TR-zh "在 ruda:0 上
 * 进行原生 PyTorch 训练": the report read back decides whether and how the
 * step updates): the host's decision from host_report (radamw_decide) must
 * equal the device's, device_decision = {skip, bits of the FP32 unscale
 * factor 1 / (gradient_scale / clip)} as the final merge wrote it.  result
 * (host, required) is filled from the report as by radamw_decide, with
 * result->updated taken from the DEVICE's decision, which is the one the
 * queued update kernels applied.  Returns RADAMW_OK when the two agree
 * (same skip; for an update, the same FP32 factor bit for bit) and
 * RADAMW_ERR_DECISION otherwise.  Host only.
 */
int radamw_check_decision(const radamw_stats *host_report, const uint32_t *device_decision,
                          double gradient_scale, double max_grad_norm,
                          radamw_fused_result *result);

/*
 * The whole fused step over a tensor list, the ruda_torch.AdamW
 * fused_step path of TR-zh: statistics of every active gradient ->
 * (hierarchical) merge -> 12-byte report read back -> skip or clip decision
 * -> the in-place update of radamw_step_multi.
 *   workspace : device, >= radamw_fused_workspace_bytes(...) bytes, 8-byte
 *               aligned (RADAMW_ERR_ALIGN otherwise), caller-owned: the
 *               rows, the merge scratch and a decision slot in its last 12
 *               bytes (an 8-byte record at an 8-byte boundary).
 *   max_grad_norm <= 0 disables clipping.
 *   result    : host struct, always filled on RADAMW_OK.
 * The final merge writes the report into host memory the library maps for
 * the device, and takes the same skip / clip decision as radamw_decide on
 * the device as well (the same binary64 operations, each correctly
 * rounded), writing it to the decision slot.  The update launches are
 * queued right behind the merge and read that slot, so the GPU never waits
 * for the host; the host waits once, for the merge, reads the report, takes
 * the decision itself and advances *step when the update ran.  When the
 * report counts a non-finite value the queued update kernels write nothing
 * (they have already issued their reads, so a skipped step costs one read
 * pass of the update's inputs; skips are rare).  The two decisions always
 * agree (radamw_check_decision); if they did not, the call returns
 * RADAMW_ERR_DECISION with *step and *result following the decision the
 * device applied.  The workspace stays in use until the stream has passed
 * the update kernels.
 */
int64_t radamw_fused_workspace_bytes(const radamw_segment *segs, int32_t nseg,
                                     radamw_dtype gdt);
int radamw_fused_step_multi(const radamw_segment *segs, int32_t nseg,
                            radamw_dtype gdt, uint64_t *step,
                            const radamw_options *opts, double gradient_scale,
                            double max_grad_norm, int32_t hierarchical,
                            void *workspace, int64_t workspace_bytes,
                            radamw_stream_t stream, radamw_fused_result *result);

/*
 * The fused step for callers that cannot allocate device memory: tight
 * serving loops, harnesses that forbid hipMalloc, and programs that replay
 * captured HIP graphs around it and may not allocate between replays.  The
 * call itself waits for its stream (it reads the report back), so it cannot
 * be recorded into a graph.
 * radamw_fused_step_multi over ONE flattened bucket (nseg <= 1; more is
 * RADAMW_ERR_RANGE) with no workspace argument: the statistics rows, merge
 * scratch, decision slot and report live in a static device array of the
 * library (98,560 bytes per device, held until the process ends), which fits
 * every bucket the library accepts (a tensor writes at most 8192 statistics
 * rows).  The call allocates no device or pinned host memory (its host-side
 * validation uses small host containers); on its first call on a device it
 * looks up that device's copy of the array.  Same arguments, checks,
 * arithmetic and results as radamw_fused_step_multi, bit for bit; the update
 * is one launch on `stream`.  The report and the device's decision are read
 * back behind the update, so the call returns when the step has completed
 * on the GPU.  Calls on one device share the array and are serialised by a
 * lock inside the library; work of another process has its own copy.
 * Nothing in the array needs clearing between calls: every call writes the
 * rows, records and report it reads.
 */
int radamw_fused_step_multi_noalloc(const radamw_segment *segs, int32_t nseg,
                                    radamw_dtype gdt, uint64_t *step,
                                    const radamw_options *opts, double gradient_scale,
                                    double max_grad_norm, int32_t hierarchical,
                                    radamw_stream_t stream, radamw_fused_result *result);

/*
 * Persistent tensor lists.  A training run updates the same tensors step
 * after step, and validating a list of a few hundred separately allocated
 * tensors (two HIP pointer queries per allocation, the overlap sweep)
 * costs about 0.6 ms of host time per call before the first kernel can
 * start.  radamw_list_create validates a segment list once and computes
 * everything that depends only on the tensors: the launch split of
 * radamw_step_multi, the update descriptors, the statistics rows of
 * radamw_fused_step_multi and their coarse indexes.  The device tables, the
 * statistics rows and the merge scratch live in one device allocation the
 * list owns, so a step only launches.  The arithmetic, the launch policy and
 * every result are those of radamw_step_multi / radamw_step_multi_writeback
 * / radamw_fused_step_multi on the same segments, bit for bit.
 *
 * OWNERSHIP (the one exception to "the library keeps no pointer"): a list
 * keeps the segment and model-copy pointers it was created with.  The
 * caller keeps every one of those buffers allocated, at the same address
 * and size, until radamw_list_destroy; stepping a list whose buffers were
 * freed or moved is undefined (the kernels would touch freed memory).  A
 * gradient that moves to a new buffer needs a new list.
 *
 * radamw_list_create(segs, nseg, gdt, amsgrad, models, model_dtype, stream,
 *                    list_out)
 *   segs, nseg, gdt : as radamw_step_multi (host array, device buffers,
 *                     in place); validated here exactly as there, with the
 *                     AMSGrad flag `amsgrad` (0/1) fixed for the list.
 *   models          : host array of nseg device pointers to FP16 / BF16
 *                     model copies (entries may be NULL), or NULL for none;
 *                     model_dtype is then RADAMW_F16 or RADAMW_BF16.
 *   stream          : fixes the device; the tables are uploaded on it
 *                     from pinned memory the list keeps (the call does not
 *                     wait for the stream).
 *   list_out        : host; receives the handle.  Allocates device memory
 *                     (tables + 12 B per statistics row + merge scratch).
 *   Errors as radamw_step_multi, plus RADAMW_ERR_RANGE when the rows exceed
 *   the merge plan's limit.  On error nothing is allocated.
 *
 * radamw_list_step(list, step, opts, ctrl, stream, updated)
 *   radamw_step_multi (or the write-back variant, when the list has model
 *   copies) over the list's segments.  opts->amsgrad must equal the list's
 *   flag (RADAMW_ERR_STATE otherwise); the stream must be on the list's
 *   device (RADAMW_ERR_INVALID otherwise).
 *
 * radamw_list_fused_step(list, step, opts, gradient_scale, max_grad_norm,
 *                        hierarchical, stream, result)
 *   radamw_fused_step_multi over the list's segments, using the list's own
 *   rows, scratch and decision slot as the workspace; the host waits once,
 *   for the final merge.
 *
 * Calls on one list serialise on a lock inside it, and each step's first
 * kernel waits (hipStreamWaitEvent) for the list's previous work, the table
 * upload or the last update, even when that went to another stream; calls
 * on different lists are independent.  radamw_time_next_update applies to the update
 * launches of a list step as to radamw_step_multi's.
 *
 * radamw_list_destroy(list): waits for the last submitted kernel that reads
 * the list's device memory, frees it and the handle.  NULL is accepted.
 */
typedef struct radamw_list_s *radamw_list;

int radamw_list_create(const radamw_segment *segs, int32_t nseg, radamw_dtype gdt,
                       int32_t amsgrad, void *const *models, radamw_dtype model_dtype,
                       radamw_stream_t stream, radamw_list *list_out);
int radamw_list_step(radamw_list list, uint64_t *step, const radamw_options *opts,
                     const radamw_control *ctrl, radamw_stream_t stream, int32_t *updated);
int radamw_list_fused_step(radamw_list list, uint64_t *step, const radamw_options *opts,
                           double gradient_scale, double max_grad_norm,
                           int32_t hierarchical, radamw_stream_t stream,
                           radamw_fused_result *result);
int radamw_list_destroy(radamw_list list);

/*
 * One fused step over several lists that take one decision together: the
 * parameter groups of a torch optimizer (for example weights with weight
 * decay and norms without), each with its own options and step count, under
 * one global-norm clip and one non-finite skip (TR-zh "在 ruda:0 上进行原生
 * PyTorch 训练": the statistics of every active group are reduced before any
 * parameter is updated).
 *
 * radamw_lists_fused_step(lists, nlists, steps, opts, gradient_scale,
 *                         max_grad_norm, hierarchical, stream, result)
 *   lists  : host array of nlists distinct list handles (1..65536), all on
 *            the stream's device.
 *   steps  : host array of nlists completed-step counts, one per list; a
 *            list that updates advances its own entry by one.
 *   opts   : host array of nlists option structs; opts[k].amsgrad must
 *            equal list k's flag.
 *   Every list's gradients are analysed (one launch per list); each list's
 *   rows are merged to one record (with the fan-in-1024 levels when
 *   hierarchical = 1), and those records, in array order, take one final
 *   merge into the report.  With a single non-empty list this is exactly
 *   radamw_list_fused_step.  The decision is taken once on that report
 *   (on the device by the final merge, into the first non-empty list's
 *   decision slot, which every list's queued update kernels read; and on
 *   the host after the one wait): a non-finite value anywhere skips every
 *   list; otherwise every list updates with the same clipped scale and its
 *   own options and step.
 *   Lists with no non-empty tensor neither launch nor step.
 *   Errors as radamw_list_fused_step, checked for every list before any
 *   launch; a handle given twice is RADAMW_ERR_INVALID.
 */
int radamw_lists_fused_step(const radamw_list *lists, int32_t nlists, uint64_t *steps,
                            const radamw_options *opts, double gradient_scale,
                            double max_grad_norm, int32_t hierarchical,
                            radamw_stream_t stream, radamw_fused_result *result);

/*
 * The FP32 constants one update launches with, formed on the host in FP64
 * and cast (FA-ja "この演算子を使用する理由": bias corrections by an FP64
 * integer power, cast to FP32), for update number t >= 1:
 *   out9 = {beta1, 1 - beta1, beta2, 1 - beta2, (maximize ? -1 : 1) /
 *           gradient_scale, 1 - lr * weight_decay, lr / (1 - beta1^t),
 *           1 / (1 - beta2^t), eps}.
 * Host only (out9: host array of 9 floats); lets the coefficients be
 * checked without a device.
 */
int radamw_host_coefficients(const radamw_options *opts, uint64_t t, double gradient_scale,
                             float *out9);

/*
 * ---------------------------------------------------- vocabulary operators --
 *
 * The two ends of the training step that the optimizer closes: the embedding
 * lookup with its gradient, and the losses over the vocabulary's logits with
 * theirs.  Both are indexed by token ids and both move arrays of the
 * vocabulary's size.  Their gradients go where the update reads them: the
 * embedding gradient into a dense gradient (of a bucket, too), the logits'
 * gradient scaled by the loss scale the update divides out again
 * (radamw_control.gradient_scale).
 *
 * Conventions beyond the general ones:
 *   - Two-dimensional arrays are row-major with unit column stride; `stride`
 *     counts the elements between row starts (stride >= row width), so a row
 *     may start at any element.  Spans are checked as (n - 1) * stride +
 *     width elements, and a written span may overlap no other span.
 *   - Index arrays hold 32- or 64-bit integers (radamw_index_type).  Their
 *     VALUES are read on the device only: an id or label outside its range
 *     is not an error but takes no part, as stated at each call.
 *   - Sums, softmax statistics and losses are formed in FP32 or FP64;
 *     outputs of a 16-bit type are rounded once, to nearest even.
 *   - No atomics on values: every sum has a fixed order, so repeated calls
 *     on the same inputs give identical bits.
 *   - Like every entry point they refuse a stream under graph capture.
 *   - Calls keep nothing: two calls may run at once, on any streams, as long
 *     as they share no output and no workspace.
 *   - Limits (RADAMW_ERR_RANGE): dim <= 2^24, vocab <= 2^27, rows and n up to
 *     2^31 - 16, pairs below 2^24; a lookup or embedding gradient that needs
 *     more than 2^24 - 1 workgroups (n below 2^24 always fits the lookup, n
 *     below 2^30 with n * dim below 2^40 the gradient).
 */
typedef enum {
    RADAMW_I32 = 0,
    RADAMW_I64 = 1
} radamw_index_type;

/*
 * Scaled embedding lookup:
 *   out[t, :] = scale * table[ids[t], :],   t = 0 .. n-1
 * in FP32, rounded once to out_dtype; a row of zeros where ids[t] is outside
 * 0 .. rows-1.
 *   table : [rows, dim] of table_dtype (FP32 masters, or their 16-bit model
 *           copy), row stride table_stride.
 *   ids   : n indices.   out : [n, dim] of out_dtype, row stride out_stride.
 * scale is finite, also as FP32.  n == 0 launches nothing.  rows may be 0
 * (every output row is zeros).
 */
int radamw_embedding_lookup(const void *table, radamw_dtype table_dtype, int64_t rows, int64_t dim,
                            int64_t table_stride, const void *ids, radamw_index_type ids_type, int64_t n, double scale,
                            void *out, radamw_dtype out_dtype, int64_t out_stride, radamw_stream_t stream);

/*
 * Gradient of the lookup with respect to the table:
 *   table_grad[v, :] = (accumulate ? table_grad[v, :] : 0)
 *                      + scale * sum of grad_out[t, :] over ids[t] == v
 * Each id's rows are summed in FP32 in an order that the arguments fix, so
 * that equal calls give equal bits; the result is rounded once.  Tokens whose
 * id is padding_id (-1: none) or outside 0 .. rows-1 add nothing.
 *   accumulate = 0 : all rows of table_grad are written (zeros where no token
 *                    adds).  Columns between dim and table_stride are left.
 *   accumulate = 1 : only rows that some token names are read and written,
 *                    the form that adds into a gradient bucket.
 *   workspace      : device, 16-byte aligned, at least
 *                    radamw_embedding_grad_workspace_bytes(n, rows, dim);
 *                    its contents need no preparation and mean nothing
 *                    afterwards.  In use until the stream has passed the call.
 * The workspace size returns a negative status for arguments out of range.
 */
int64_t radamw_embedding_grad_workspace_bytes(int64_t n, int64_t rows, int64_t dim);
int radamw_embedding_grad(const void *grad_out, radamw_dtype grad_dtype, int64_t grad_stride, const void *ids,
                          radamw_index_type ids_type, int64_t n, int64_t rows, int64_t dim, double scale,
                          int64_t padding_id, int32_t accumulate, void *table_grad, radamw_dtype table_dtype,
                          int64_t table_stride, void *workspace, int64_t workspace_bytes, radamw_stream_t stream);

/*
 * Clipped policy loss with a KL term, over n token rows of logits:
 *   logp_i  = logits[i, labels[i]] - log sum_j exp(logits[i, j])
 *   r_i     = exp(logp_i - old_logp_i)
 *   loss_i  = -min(r_i A_i, min(max(r_i, 1 - clip_low), 1 + clip_high) A_i)
 *             + kl_coef * (exp(ref_logp_i - logp_i) - (ref_logp_i - logp_i) - 1)
 *   total   = sum of weights_i * loss_i
 *   grad    = grad_scale * d total / d logits
 * The gradient passes where A_i >= 0 ? r_i <= 1 + clip_high : r_i >= 1 -
 * clip_low.  A row takes no part when its label is outside 0 .. vocab-1 or
 * its weight is 0: its logits are not read (they may hold anything), its
 * loss and logp are 0 and its gradient is a row of zeros.
 *   logits     : [n, vocab] of dtype, row stride `stride`.
 *   old_logp   : n FP32, or NULL: the row's own logp (r_i = 1).
 *   ref_logp   : n FP32; required when kl_coef != 0, else not read.
 *   advantages : n FP32.     weights : n FP32, or NULL: all 1.
 *   opts       : host; 0 <= clip_low <= 1, clip_high >= 0, kl_coef >= 0,
 *                finite.
 *   total      : 1 FP32.     loss, logp : n FP32.
 *   row_stats  : 4 n FP32, 16-byte aligned, the records radamw_logits_grad
 *                reads; or NULL.
 *   grad       : [n, vocab] of dtype, row stride grad_stride; NULL for the
 *                loss alone.  May be exactly the logits (same pointer and
 *                stride), which it then replaces.
 * Everything per row is formed in FP64 from the row's sum of exponentials
 * (FP32 by lane, joined in FP64); the total adds the FP32 losses in FP64.
 * Where the gradient is asked for, the logits of rows up to 256 KiB are read
 * once, by another kernel than without: logp, loss and total then agree to
 * the rounding of the sum of exponentials (about 1e-7 of it), not bit for
 * bit.  A ratio that shall be exactly 1 is had by old_logp = NULL.
 */
typedef struct {
    double clip_low;
    double clip_high;
    double kl_coef;
} radamw_policy_options;
/* clip 0.2 on both sides, no KL term. */
radamw_policy_options radamw_policy_options_default(void);
int radamw_policy_loss(const void *logits, radamw_dtype dtype, int64_t n, int64_t vocab, int64_t stride,
                       const void *labels, radamw_index_type labels_type, const float *old_logp, const float *ref_logp,
                       const float *advantages, const float *weights, const radamw_policy_options *opts,
                       double grad_scale, float *total, float *loss, float *logp, float *row_stats, void *grad,
                       int64_t grad_stride, radamw_stream_t stream);

/*
 * Preference loss of `pairs` pairs of sequences, packed along the rows:
 * sequence s holds rows offsets[s] .. offsets[s + 1] - 1; sequence p is pair
 * p's chosen one and sequence pairs + p its rejected one.
 *   S_s    = sum of logp_i over the rows of s whose label is inside
 *            0 .. vocab-1 (prompt rows carry a label outside)
 *   h_p    = beta * ((S_p - ref_logp_p) - (S_(pairs+p) - ref_logp_(pairs+p)))
 *   loss_p = -(1 - label_smoothing) log sigmoid(h_p)
 *            - label_smoothing log sigmoid(-h_p)
 *   total  = sum of weights_p * loss_p
 *   grad   = grad_scale * d total / d logits
 * Rows whose label is outside take no part (as in radamw_policy_loss), nor do
 * rows outside every sequence (their logp is still computed; their gradient
 * is zeros).  A pair of weight 0 adds nothing to the total and has a zero
 * gradient.
 *   offsets   : 2 * pairs + 1 indices of index_type, non-decreasing, within
 *               0 .. n (read on the device; other values are clamped to that
 *               range for every access, but the result is unspecified).
 *   ref_logp  : 2 * pairs FP32, the reference model's S_s.
 *   weights   : pairs FP32, or NULL: all 1.
 *   opts      : host; beta >= 0 finite, 0 <= label_smoothing <= 1.
 *   total     : 1 FP32.  loss : pairs FP32.  seq_logp : 2 * pairs FP32 (S_s).
 *   logp      : n FP32.  row_stats : 4 n FP32, 16-byte aligned; required.
 *   logits, labels, grad, strides : as in radamw_policy_loss.
 * pairs >= 1.  S_s is summed in FP64 from unrounded logp.
 */
typedef struct {
    double beta;
    double label_smoothing;
} radamw_preference_options;
/* beta 0.1, no label smoothing. */
radamw_preference_options radamw_preference_options_default(void);
int radamw_preference_loss(const void *logits, radamw_dtype dtype, int64_t n, int64_t vocab, int64_t stride,
                           const void *labels, radamw_index_type index_type, const void *offsets, int64_t pairs,
                           const float *ref_logp, const float *weights, const radamw_preference_options *opts,
                           double grad_scale, float *total, float *loss, float *seq_logp, float *logp,
                           float *row_stats, void *grad, int64_t grad_stride, radamw_stream_t stream);

/*
 * The logits' gradient of either loss from the records its forward call
 * left, for a backward pass that learns its scale only then:
 *   grad[i, j] = upstream * grad_scale * coef_i * (1[j = labels_i] - p_ij)
 *   row_stats : 4 n FP32, per row {m, 1 / sum of exponentials relative to m,
 *               coef, 1 - p_label}, m a logit near the largest; as written
 *               by the forward call, whose dtype this one shares.
 *   upstream  : 1 FP32 on the device, or NULL: 1.
 * logits and labels are those of the forward call, unchanged.  grad may be
 * exactly the logits.
 */
int radamw_logits_grad(const void *logits, radamw_dtype dtype, int64_t n, int64_t vocab, int64_t stride,
                       const void *labels, radamw_index_type labels_type, const float *row_stats,
                       const float *upstream, double grad_scale, void *grad, int64_t grad_stride,
                       radamw_stream_t stream);

/*
 * ------------------------------------------------------- block operators --
 *
 * Between the vocabulary's two ends: what a training step does around every
 * block of a model.  Dropout from a counter-based generator (of the looked-up
 * embedding, and inside the next operator); the residual stream's norms
 * behind and before a block, fused with the block's dropout, gate and scale,
 * and their gradient; the balance loss of a router with its per-expert counts
 * and gradient.  The conventions are those of the vocabulary operators: row
 * strides, index types, FP32 or FP64 sums in a fixed order, one rounding,
 * streams, no capture, nothing kept.
 */

/*
 * Dropout:
 *   out[t, j] = kept ? x[t, j] * 65536 / (65536 - m) : 0,   m = round(65536 p)
 * The probability is that of 16 bits, m / 65536 (halves round up); the factor
 * is that probability's, in FP32.  The gradient is the same call on the
 * output's gradient: the mask is formed again, not stored.
 *
 * An element's 16-bit number depends on seed, offset, its row and its column
 * alone, and it is dropped where the number is below m: Philox 4x32 with ten
 * rounds, the key {seed's low word, high word}, the counter {column / 8,
 * first_row + row, offset's low word, high word}; column 8 q + 2 i + b has
 * the half b (0: low) of output word i.  So a part of a batch (first_row), a
 * strided view or a recomputed pass has the numbers of the whole, and calls
 * that shall differ (layers, steps) have to differ in seed or offset.
 * A dropped element is 0 whatever x holds there.
 *   x, out  : [n, dim] of dtype; out may be exactly x (pointer and stride).
 *   opts    : host; 0 <= p <= 1, first_row >= 0; first_row + n <= 2^32
 *             (RADAMW_ERR_RANGE).  p = 1 gives zeros.
 * dim <= 2^24.
 */
typedef struct {
    double p;
    uint64_t seed;
    uint64_t offset;
    int64_t first_row;
} radamw_dropout_options;
/* No dropout, all else 0. */
radamw_dropout_options radamw_dropout_options_default(void);
int radamw_dropout(const void *x, radamw_dtype dtype, int64_t n, int64_t dim, int64_t stride,
                   const radamw_dropout_options *opts, void *out, int64_t out_stride, radamw_stream_t stream);

/*
 * The residual stream from one block's output to the next block's input:
 *   u[t]   = post_weight ? norm(branch[t]) * (weight_offset + post_weight)
 *                        : branch[t]
 *   h[t]   = x[t] + residual_scale * gate[t / rows_per_gate] * drop(u[t])
 *   out[t] = norm(h[t]) * (weight_offset + pre_weight)
 *   norm(v) = v / sqrt(mean(v^2) + eps)
 * all in FP32 from h's unrounded value; products are elementwise; drop is
 * radamw_dropout's (opts->dropout, 0 for none).
 *   branch : [n, dim] of branch_dtype, the block's output.  NULL: no block
 *            before the norm; then h = x is not written (h, gate and
 *            post_weight have to be NULL) and pre_weight is required.
 *   gate   : [ceil(n / rows_per_gate), dim] of gate_dtype, or NULL: 1.  One
 *            row for all rows (rows_per_gate >= n), one per sequence of equal
 *            lengths, or one per row (rows_per_gate = 1).
 *   post_weight, pre_weight : dim values of weight_dtype each, or NULL: no
 *            such norm.  Without pre_weight there is no out (NULL).
 *   x, h   : [n, dim] of stream_dtype, which is branch_dtype or RADAMW_F32.
 *            h may be exactly x.
 *   out    : [n, dim] of branch_dtype; may be exactly the branch.
 *   rstd   : 2 n FP32, or NULL: 1 / sqrt(mean + eps) of the branch's rows
 *            (written with a post_weight), then of h's (with a pre_weight),
 *            for the gradient.
 * dim <= 32768 (RADAMW_ERR_RANGE).  eps > 0, also as FP32.  A mean square
 * beyond FP32 counts as infinite (values from about 1.8e19 / sqrt(dim) on).
 */
typedef struct {
    int64_t n, dim;
    radamw_dtype stream_dtype, branch_dtype, gate_dtype, weight_dtype;
    const void *branch;
    int64_t branch_stride;
    const void *gate;
    int64_t gate_stride;
    int64_t rows_per_gate;
    const void *post_weight;
    const void *pre_weight;
} radamw_residual_block;
typedef struct {
    double eps;
    double weight_offset;
    double residual_scale;
    radamw_dropout_options dropout;
} radamw_residual_options;
/* eps 1e-6, weight_offset 0, residual_scale 1, no dropout. */
radamw_residual_options radamw_residual_options_default(void);
int radamw_residual_norm(const radamw_residual_block *block, const void *x, int64_t x_stride,
                         const radamw_residual_options *opts, void *h, int64_t h_stride, void *out, int64_t out_stride,
                         float *rstd, radamw_stream_t stream);

/*
 * The gradient of radamw_residual_norm, from grad_h (of h's later uses) and
 * grad_out:
 *   D           = grad_h + the gradient of out = norm(h) * (...) by h
 *   grad_x      = D
 *   grad_branch, grad_gate, grad_post_weight = those of
 *                 residual_scale * gate * drop(u) under D
 *   grad_pre_weight[j] = sum over rows of grad_out * norm(h)
 * block and opts are the forward call's, h and rstd what it wrote (h unused
 * without a pre_weight; where there was no branch, h is its x).
 *   grad_h   : [n, dim] of stream_dtype, or NULL (zeros) with a pre_weight.
 *   grad_out : [n, dim] of branch_dtype; exactly with a pre_weight.
 *   grad_x   : [n, dim] of stream_dtype; may be exactly grad_h.
 *   grad_branch : [n, dim] of branch_dtype, exactly with a branch; may be
 *                 exactly grad_out.
 *   grad_gate   : as the gate, of gate_dtype (all of its rows are written), or
 *                 NULL.
 *   grad_post_weight, grad_pre_weight : dim values of weight_dtype, or NULL.
 *   workspace : device, 16-byte aligned, at least
 *               radamw_residual_grad_workspace_bytes(n, dim, rows_per_gate)
 *               (rows_per_gate 1 without a gate); in use until the stream has
 *               passed the call.  May be NULL where no weight's gradient and
 *               no shared gate's is asked for.
 * Sums over rows are formed in FP32 by parts of the rows, which are joined in
 * FP64, in an order that n and dim fix.  A dropped element passes nothing on,
 * whatever the branch holds there.  With n = 0 the weights' gradients are
 * zeros.
 */
int64_t radamw_residual_grad_workspace_bytes(int64_t n, int64_t dim, int64_t rows_per_gate);
int radamw_residual_norm_grad(const radamw_residual_block *block, const void *h, int64_t h_stride, const float *rstd,
                              const radamw_residual_options *opts, const void *grad_h, int64_t grad_h_stride,
                              const void *grad_out, int64_t grad_out_stride, void *grad_x, int64_t grad_x_stride,
                              void *grad_branch, int64_t grad_branch_stride, void *grad_gate, int64_t grad_gate_stride,
                              void *grad_post_weight, void *grad_pre_weight, void *workspace, int64_t workspace_bytes,
                              radamw_stream_t stream);

/*
 * Balance loss of a router over groups of token rows, with a z-loss and the
 * per-expert counts.  Per group, over its T rows that take part:
 *   P_te   = softmax of logits[t], or sigmoid(logits[t, e]) divided by the
 *            row's sum of them (opts->score)
 *   c_e    = how many of the rows' top_k ids are e
 *   loss   = balance_coef * E / (top_k * T) * sum_e c_e * mean_t P_te
 *            + z_coef * mean_t (log sum_e exp logits[t, e])^2
 *   total  = sum of weights_g * loss_g
 *   grad   = grad_scale * d total / d logits (the counts are constants)
 * (balance_coef where every expert is chosen equally often.)
 *   logits  : [n, experts] of dtype, row stride `stride`; experts <= 4096.
 *   ids     : n * top_k indices, the experts each row chose; one outside
 *             0 .. experts-1 is not counted, one given twice counts twice.
 *   mask    : n bytes, or NULL: all 1.  A row of mask 0 takes no part: its
 *             logits and ids may hold anything, its gradient is zeros.
 *   offsets : groups + 1 indices of index_type, non-decreasing, within 0 ..
 *             n: group g holds rows offsets[g] .. offsets[g + 1] - 1 (read on
 *             the device; other values are clamped to 0 .. n for every
 *             access, but the result is unspecified).  Rows outside every
 *             group take no part.  NULL: one group (groups = 1) of all rows.
 *   weights : groups FP32, or NULL: all 1.  A group of weight 0 adds nothing to
 *             the total, and its gradient is zeros, whatever its logits hold.
 *   opts    : host; coefficients >= 0, finite; z_coef 0 with sigmoid scores.
 *   total   : 1 FP32.  loss : groups FP32.
 *   counts  : [groups, experts] int32.  tokens : groups int32 (T).
 *   mean_prob : [groups, experts] FP32, mean_t P_te.
 *   grad    : [n, experts] of dtype, or NULL; may be exactly the logits.
 *   workspace : device, 16-byte aligned, at least
 *               radamw_balance_workspace_bytes(n, experts, groups).
 * A group without rows has loss 0.  A row whose logits are all -inf (or whose
 * scores are all 0, as FP64 numbers: sigmoid logits below -709.78) adds no
 * probability and has a zero gradient.
 * n * top_k <= 2^31 - 16 and groups <= 2^24 - 2048 (RADAMW_ERR_RANGE).
 *
 * radamw_balance_grad is the gradient from the forward call's counts and
 * tokens, for a backward pass that learns its scale (upstream, 1 FP32 on the
 * device, or NULL: 1) only then.  counts and tokens may be sums over the
 * ranks of a data-parallel job: the loss is then the whole batch's.
 */
typedef enum {
    RADAMW_SCORE_SOFTMAX = 0,
    RADAMW_SCORE_SIGMOID = 1
} radamw_score_type;
typedef struct {
    double balance_coef;
    double z_coef;
    int32_t score; /* radamw_score_type */
} radamw_balance_options;
/* balance 0.01, no z-loss, softmax. */
radamw_balance_options radamw_balance_options_default(void);
int64_t radamw_balance_workspace_bytes(int64_t n, int64_t experts, int64_t groups);
int radamw_balance_loss(const void *logits, radamw_dtype dtype, int64_t n, int64_t experts, int64_t stride,
                        const void *ids, radamw_index_type index_type, int64_t top_k, const uint8_t *mask,
                        const void *offsets, int64_t groups, const float *weights, const radamw_balance_options *opts,
                        double grad_scale, float *total, float *loss, int32_t *counts, int32_t *tokens,
                        float *mean_prob, void *grad, int64_t grad_stride, void *workspace, int64_t workspace_bytes,
                        radamw_stream_t stream);
int radamw_balance_grad(const void *logits, radamw_dtype dtype, int64_t n, int64_t experts, int64_t stride,
                        int64_t top_k, const uint8_t *mask, const void *offsets, radamw_index_type offsets_type,
                        int64_t groups, const float *weights, const radamw_balance_options *opts, const int32_t *counts,
                        const int32_t *tokens, const float *upstream, double grad_scale, void *grad,
                        int64_t grad_stride, radamw_stream_t stream);

/* Utilities. */
const char *radamw_status_string(int status);
/* Last HIP error code seen by this thread inside the library (0 = none). */
int radamw_last_hip_error(void);
/* Total kernel launches made by the library in this process (test hook:
 * proves skip / empty calls launch nothing). */
uint64_t radamw_launch_count(void);

/*
 * Measurement hook (not part of the method): the next radamw_step,
 * radamw_step_inplace, radamw_step_multi, radamw_fused_step_multi or list
 * step call on this thread that launches an update records start_event
 * when its first update kernel starts (hipExtLaunchKernelGGL), so the
 * host's submission latency is not timed, and stop_event when its update
 * kernels have ended: at the end of a single launch, or, when the launches
 * are spread over two streams, on the caller's stream right after it has
 * joined the second one.
 * The events are caller-created hipEvent_t of the stream's device; passing
 * NULL, NULL clears the request.  Always returns RADAMW_OK.
 */
int radamw_time_next_update(void *start_event, void *stop_event);

#ifdef __cplusplus
}
#endif

#endif /* RADAMW_H */
