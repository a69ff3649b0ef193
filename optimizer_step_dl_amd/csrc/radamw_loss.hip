// radamw_loss.hip -- the losses over a vocabulary's logits for gfx950: the
// clipped policy loss with a KL term and the preference loss of sequence
// pairs, with the gradient of the logits.
//
// For a row of logits x with label a:
//   m = max x,  s = sum exp(x - m),  logp = (x_a - m) - log s
//   d total / d x_j = coef * (1[j = a] - exp(x_j - m) / s)
// where coef = d total / d logp is a number per row that each loss forms in
// its own way.  Everything that is one number per row is formed in binary64
// by one wave; the exponentials and their sums by lane are FP32.
//
// An exponential is exp2(x * L - c), one FMA (two where it is summed) and one
// v_exp_f32, with c = fl(m * L) and L = log2 e: the rounding of c shifts every
// exponent of the row alike and cancels in p_j = e_j / s and, in binary64, in
// logp.
// For the same reason m need not be the maximum: any logit that the maximum
// exceeds by little enough for the sum to stay finite does.  All of that
// holds while |m| < 2^24 (c is then off by at most 1); other rows, and those
// whose sum leaves the range, take slow_row, which finds the maximum, forms
// x - m first and reads the row again.
//
// What bounds it is HBM: the logits are read once and their gradient written
// once.  A workgroup holds a whole row in registers (up to 256 KiB: 1024
// lanes x 16 chunks of 16 bytes), so that the sum and the gradient need one
// read; longer rows are read twice.  m is the largest of the row's first
// NT chunks and the label's logit, so the exponentials are summed while the
// other chunks are still arriving.
#include "radamw_rows.h"
#include "radamw_vocab.h"

// c = fl(m * LOG2E) has to be the same number wherever it is used: a product
// fused into one of its uses would not be.
#pragma clang fp contract(off)

namespace radamw {

namespace {

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

constexpr double LN2 = 0.6931471805599453;
constexpr double LOG2E_64 = 1.4426950408889634;

// Sums below this have no exponential near FP32's largest value, and their
// reciprocals times a coefficient none near its smallest.
constexpr double SUM_LIMIT = 0x1p60;

// Rows whose exponents are shifted by c = fl(m * LOG2E).
constexpr float SHIFT_LIMIT = 16777216.0f;
__device__ __forceinline__ bool shiftable(float top) { return fabsf(top) < SHIFT_LIMIT; }

// Rows that lanes with a shift each may sum: the values of a lane that has
// none, all at most -2^24, are left out of the sum, which is right where the
// row's maximum exceeds them by 256 or more (e^-256 of it, each).
__device__ __forceinline__ bool shiftable_by_lane(float top) { return shiftable(top) && top >= 256.0f - SHIFT_LIMIT; }

// The gradient's exponentials, exp2(x * LOG2E - c).  LOG2E alone is off by
// 1.3e-8, so that p_j = e_j / s is by that much of x_j - m, behind the
// rounding of the exponent.
__device__ __forceinline__ float exp_shifted(float x, float c) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(x, LOG2E, -c));
}

// A sum's exponentials carry all of log2 e, as hi + lo: LOG2E alone would move
// every logp by 1.3e-8 (x_a - mean x), to the same side.  The second product
// has to be many steps of the exponent's last digit, or its rounding is no
// more even than what it mends (x lo of 0.6 steps always becomes 1), and small
// enough that the first FMA's rounding does not matter: hi has 13 bits where
// |m| < 4096, else 24.  Over 8192 rows of 131072 BF16 logits the mean error of
// logp is 4e-9, against 3.9e-8 with 24 bits for all and -2.7e-8 with LOG2E
// alone.  The second FMA costs the fused loss 1.2% where a row fills the
// registers (766 us against 757 for these rows), nothing elsewhere.
struct Shift {
    float c, hi, lo;
};
constexpr float LOG2E_13 = 5909.0f / 4096;

__device__ __forceinline__ Shift shift_by(float m) {
    const bool small = fabsf(m) < 4096.0f;
    return {m * LOG2E, small ? LOG2E_13 : LOG2E,
            small ? static_cast<float>(LOG2E_64 - double(LOG2E_13)) : static_cast<float>(LOG2E_64 - double(LOG2E))};
}
__device__ __forceinline__ float exp_sum(float x, Shift s) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(x, s.lo, __builtin_fmaf(x, s.hi, -s.c)));
}

// exp(y) for y <= 0, the slow rows' form.
__device__ __forceinline__ float exp_neg(float y) { return __builtin_amdgcn_exp2f(y * LOG2E); }

// -inf in every value of a chunk.
template <int DT>
__device__ __forceinline__ u32x4 lowest_chunk() {
    const uint32_t w = DT == G_F32 ? 0xff800000u : DT == G_F16 ? 0xfc00fc00u : 0xff80ff80u;
    return u32x4{w, w, w, w};
}

// How a row is cut: chunks of 16 bytes that start on a cache line, and the
// values before the first and behind the last of them (`edges`), one to a
// lane.  A row of 16-bit values may start at any even address; 16-byte
// accesses from an odd multiple of two bytes cost 17% of the fused loss
// (4097 rows of 50001 FP16 logits: 157 us, against 134 us for 50000), those
// from a cache line 6% less than from elsewhere (50048: 125 us).  Cut this way
// the three take the same.
template <int DT>
struct RowShape {
    static constexpr int E = chunk_elems<DT>;
    int head;      // values before the first chunk (fewer than 128 bytes)
    int full;      // chunks
    int tail_at;   // first value behind them
    int vocab;

    __device__ __forceinline__ RowShape(const void *row, int64_t vocab_) {
        vocab = static_cast<int>(vocab_);
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 127);
        const int lead = ((128 - off) & 127) / elem_bytes<DT>;
        head = lead < vocab ? lead : vocab;
        full = (vocab - head) / E;
        tail_at = head + full * E;
    }
    // Value number of chunk k's first value.
    __device__ __forceinline__ int64_t chunk_at(int64_t k) const { return head + k * E; }
    // The chunk of value v, or -1 for an edge.
    __device__ __forceinline__ int chunk_of(int v) const { return v >= head && v < tail_at ? (v - head) / E : -1; }
    // The edge value lane t holds, or -1: the head from lane 0 on, the tail
    // from lane 64 on, and from lane 128 on the values of chunk `apart`, which
    // is then no lane's chunk (-1: none).
    __device__ __forceinline__ int edge(int t, int apart) const {
        if (t < 64) return t < head ? t : -1;
        if (t < 128) {
            const int e = tail_at + (t - 64);
            return e < vocab ? e : -1;
        }
        return apart >= 0 && t < 128 + E ? head + apart * E + (t - 128) : -1;
    }
};

template <int DT>
__device__ __forceinline__ void store_values(void *p, int64_t e, const float *v) {
    if constexpr (DT == G_F32) {
        const f32x4 x = {v[0], v[1], v[2], v[3]};
        stream_out<DT>(p, e, __builtin_bit_cast(u32x4, x));
    } else {
        const f32x8 x = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
        if constexpr (DT == G_F16) stream_out<DT>(p, e, __builtin_bit_cast(u32x4, __builtin_convertvector(x, f16x8)));
        else stream_out<DT>(p, e, __builtin_bit_cast(u32x4, __builtin_convertvector(x, bf16x8)));
    }
}

// A row that takes no part: a gradient of zeros.
template <int DT, int NT>
__device__ __forceinline__ void zero_row(void *row, int64_t vocab) {
    const u32x4 z = {0, 0, 0, 0};
    const RowShape<DT> s(row, vocab);
    for (int k = threadIdx.x; k < s.full; k += NT) stream_out<DT>(row, s.chunk_at(k), z);
    const int e = s.edge(threadIdx.x, -1);
    if (e >= 0) store_value<DT>(row, e, 0.0f);
}

// What a row's own scalars give: formed by one wave.
struct RowResult {
    double coef;       // d total / d logp
    double one_less_p; // 1 - exp(logp)
};

// The clipped policy loss of one row.
struct PolicyRow {
    const float *old_logp, *ref_logp, *advantages, *weights;
    float *loss;
    double clip_low, clip_high, kl_coef;

    // Lane 0 of the calling wave writes the row's loss.  The three
    // exponentials of a row are evaluated at once, in lanes 0, 1 and 2.
    __device__ __forceinline__ RowResult operator()(int64_t row, double logp) const {
        const int lane = threadIdx.x & 63;
        // without old_logp the ratio is 1, also where logp is -inf; a NaN stays one
        const double moved = old_logp ? logp - double(old_logp[row]) : logp == logp ? 0.0 : logp;
        const double away = kl_coef != 0.0 ? double(ref_logp[row]) - logp : 0.0;
        const double arg = lane == 0 ? moved : lane == 1 ? away : logp;
        const double em1 = expm1(arg);
        const double r1 = __shfl(em1, 0, 64), k1 = __shfl(em1, 1, 64), p1 = __shfl(em1, 2, 64);
        const double ratio = r1 + 1.0, adv = advantages[row], w = weights ? double(weights[row]) : 1.0;
        const double lo = 1.0 - clip_low, hi = 1.0 + clip_high;
        const double clipped = ratio < lo ? lo : ratio > hi ? hi : ratio;
        const double plain = ratio * adv, held = clipped * adv;
        // a NaN ratio or advantage stays NaN: neither comparison holds for it
        double l = -(held < plain ? held : plain);
        const bool active = adv >= 0.0 ? !(ratio > hi) : !(ratio < lo);
        double d = active ? -plain : 0.0;
        if (kl_coef != 0.0) {
            l += kl_coef * (k1 - away);
            d -= kl_coef * k1;
        }
        if (lane == 0) loss[row] = static_cast<float>(l);
        return {d * w, -p1};
    }
};

// The preference loss's first pass keeps logp alone: what FP32 drops of it
// goes into the record, so that sequence sums have all of it.
struct LogpRow {};

template <typename ROW>
struct IsPolicy {
    static constexpr bool value = false;
};
template <>
struct IsPolicy<PolicyRow> {
    static constexpr bool value = true;
};

template <typename ROW>
__device__ __forceinline__ bool takes_part(const ROW &f, const LogitsArgs &x, int64_t row, int64_t *label) {
    // both loads leave before either is looked at
    const int64_t a = load_index(x.labels, x.wide_ids, row);
    float w = 1.0f;
    if constexpr (IsPolicy<ROW>::value) {
        if (f.weights) w = f.weights[row];
    }
    *label = a;
    return a >= 0 && a < x.vocab && w != 0.0f;
}

template <typename ROW>
__device__ __forceinline__ void absent_row(const ROW &f, const LogitsArgs &x, int64_t row) {
    if (threadIdx.x == 0) {
        x.logp[row] = 0.0f;
        if constexpr (IsPolicy<ROW>::value) f.loss[row] = 0.0f;
        if (x.stats) x.stats[row] = RowStats{0.0f, 0.0f, 0.0f, 0.0f};
    }
}

// The label's own exponential, formed in binary64: the label is most of many
// a row's sum, and an FP32 sum that held it would leave few digits of the
// others, that is of logp and 1 - p where p is near 1 (8.5863e-5 for a logp of
// 8.5831e-5).  It takes no time that shows (770 us against 768 for 8192 x
// 131072 BF16).
struct LabelTerm {
    double log2;     // of the exponential
    double inverse;  // 1 / the exponential
    double own;      // the exponential
    double factor;   // to the sum that goes with the gradient's exponentials
};

// By a whole wave, relative to the shift c of `top` (`shifted`) or to `top`
// itself.  The gradient's exponentials lack what LOG2E does: the part of m is
// taken out of their sum (that of x - m is below the exponent's rounding).
// The three exponentials are evaluated at once, by lanes 0, 1 and 2.
__device__ __forceinline__ LabelTerm label_term(float at_label, float top, float c, bool shifted) {
    const int lane = threadIdx.x & 63;
    const double t = shifted ? double(at_label) * LOG2E_64 - double(c) : (double(at_label) - double(top)) * LOG2E_64;
    const double lacks = shifted ? -double(top) * (LOG2E_64 - double(LOG2E)) : 0.0;
    const double e = exp2(lane == 0 ? t : lane == 1 ? -t : lacks);
    return {t, __shfl(e, 1, 64), __shfl(e, 0, 64), __shfl(e, 2, 64)};
}

struct RowSum {
    double logp;
    double of_grad;
};
__device__ __forceinline__ RowSum with_label(double others, const LabelTerm &l) {
    const double sum = others + l.own;
    // an exponential below 2^-500 adds nothing to the others, which hold m's
    const double logp = l.log2 > -500.0 ? -log1p(others * l.inverse) : l.log2 * LN2 - log(sum);
    return {logp, sum * l.factor};
}

// The row's scalars from its maximum, log-probability and sum, by a whole
// wave, whose lane 0 stores them.
template <typename ROW>
__device__ __forceinline__ RowResult finish_row(const ROW &f, const LogitsArgs &x, int64_t row, float top, double sum,
                                                double logp) {
    const float lp = static_cast<float>(logp);
    const bool lead = (threadIdx.x & 63) == 0;
    if (lead) x.logp[row] = lp;
    RowResult r{0.0, 0.0};
    if constexpr (IsPolicy<ROW>::value) {
        r = f(row, logp);
        if (x.stats && lead)
            x.stats[row] = RowStats{top, static_cast<float>(1.0 / sum), static_cast<float>(r.coef),
                                    static_cast<float>(r.one_less_p)};
    } else {
        const float less = static_cast<float>(-expm1(logp));
        const float rest = __builtin_isfinite(lp) ? static_cast<float>(logp - double(lp)) : 0.0f;
        if (lead) x.stats[row] = RowStats{top, static_cast<float>(1.0 / sum), rest, less};
    }
    return r;
}

// Sum over a workgroup, to every lane, in a fixed order.
template <int NT>
__device__ __forceinline__ double block_sum(double v, double *part) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v += part[w];
    return v;
}

// Maximum over a workgroup, to every lane; `part` is LDS.  The barrier waits
// for LDS alone, not for loads on their way to registers.
template <int NT>
__device__ __forceinline__ float block_max(float v, float *part) {
    v = wave_max(v);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v = fmaxf(v, part[w]);
    return v;
}

// A workgroup's shared words for one row.
template <int NT>
struct RowShared {
    float tops[NT / 64];
    double sums[NT / 64];
    float factor;    // of exp(x - m), for the gradient
    float at_label;  // the label's gradient
};

// The factors of the gradient from a row's scalars (one lane).
template <int NT>
__device__ __forceinline__ void put_factors(RowShared<NT> &sh, const RowResult &r, double scale, double sum) {
    const double g = r.coef * scale;
    sh.factor = static_cast<float>(-g / sum);
    sh.at_label = static_cast<float>(g * r.one_less_p);
}

// A row that shifted exponents do not serve: three more reads, one value at a
// time.  An infinite or NaN maximum makes its results NaN.
template <int DT, int NT, bool GRAD, typename ROW>
__device__ __forceinline__ void slow_row(const LogitsArgs &x, const ROW &f, int64_t row, int64_t label,
                                         RowShared<NT> &sh) {
    const char *in = static_cast<const char *>(x.logits) + row * x.stride * elem_bytes<DT>;
    const float at_label = load_value<DT>(in, label);
    float top = -__builtin_inff();
#pragma clang loop unroll(disable)
    for (int64_t k = threadIdx.x; k < x.vocab; k += NT) top = fmaxf(top, load_value<DT>(in, k));
    __syncthreads();  // past every use of sh so far
    top = block_max<NT>(top, sh.tops);
    const bool shifted = shiftable(top);  // the records' readers go by the same rule
    const Shift to = shift_by(top);
    const float shift = to.c;
    double sum = 0.0;
#pragma clang loop unroll(disable)
    for (int64_t k = threadIdx.x; k < x.vocab; k += NT) {
        const float z = load_value<DT>(in, k);
        if (k != label) sum += double(shifted ? exp_sum(z, to) : exp_neg(z - top));
    }
    sum = block_sum<NT>(sum, sh.sums);
    if (threadIdx.x < 64) {
        const RowSum w = with_label(sum, label_term(at_label, top, shift, shifted));
        const RowResult r = finish_row(f, x, row, top, w.of_grad, w.logp);
        if (GRAD && threadIdx.x == 0) put_factors(sh, r, x.grad_scale, w.of_grad);
    }
    if constexpr (GRAD) {
        char *out = static_cast<char *>(x.grad) + row * x.grad_stride * elem_bytes<DT>;
        __syncthreads();
#pragma clang loop unroll(disable)
        for (int64_t k = threadIdx.x; k < x.vocab; k += NT) {
            const float z = load_value<DT>(in, k);
            const float v = (shifted ? exp_shifted(z, shift) : exp_neg(z - top)) * sh.factor;
            store_value<DT>(out, k, k == label ? sh.at_label : v);
        }
    }
}

// ------------------------------------------------- rows held in registers --

// One workgroup per row; lane tid holds chunks tid, tid + NT, ...
template <int DT, int NT, int CH, bool GRAD, typename ROW>
__global__ __launch_bounds__(NT) void loss_rows(LogitsArgs x, ROW f) {
    constexpr int E = chunk_elems<DT>;
    __shared__ RowShared<NT> sh;
    const int64_t row = x.row0 + blockIdx.x;
    const int tid = threadIdx.x, wave = tid >> 6;
    char *out = static_cast<char *>(x.grad) + row * x.grad_stride * elem_bytes<DT>;
    int64_t label;
    if (!takes_part(f, x, row, &label)) {
        absent_row(f, x, row);
        if constexpr (GRAD) zero_row<DT, NT>(out, x.vocab);
        return;
    }
    const char *in = static_cast<const char *>(x.logits) + row * x.stride * elem_bytes<DT>;
    const RowShape<DT> s(in, x.vocab);
    const int used = (s.full + NT - 1) / NT;  // chunks of the busiest lane
    const float at_label = load_value<DT>(in, label);
    // the label's chunk is held value by value, and its value left out of the sum
    const int apart = s.chunk_of(static_cast<int>(label));
    u32x4 c[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = tid + i * NT;
        if (k < s.full && k != apart) c[i] = stream_chunk<DT>(in, s.chunk_at(k));
        else c[i] = lowest_chunk<DT>();
    }
    const int edge = s.edge(tid, apart);
    const float at_edge = edge >= 0 && edge != label ? load_value<DT>(in, edge) : -__builtin_inff();
    float top = at_edge;
#pragma unroll
    for (int j = 0; j < E; ++j) top = fmaxf(top, chunk_value<DT>(c[0], j));
    top = fmaxf(block_max<NT>(top, sh.tops), at_label);
    const Shift to = shift_by(top);
    const float shift = to.c;
    LabelTerm own{};  // while the row is still arriving
    if (wave == 0) own = label_term(at_label, top, shift, true);
    float part[4] = {exp_sum(at_edge, to), 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        if (i < used) {
#pragma unroll
            for (int j = 0; j < E; ++j) part[j & 3] += exp_sum(chunk_value<DT>(c[i], j), to);
        }
    }
    const double sum = block_sum<NT>((double(part[0]) + double(part[1])) + (double(part[2]) + double(part[3])), sh.sums);
    if (!shiftable(top) || !(sum < SUM_LIMIT)) {
        slow_row<DT, NT, GRAD>(x, f, row, label, sh);
        return;
    }
    if (wave == 0) {
        const RowSum w = with_label(sum, own);
        const RowResult r = finish_row(f, x, row, top, w.of_grad, w.logp);
        if (GRAD && tid == 0) put_factors(sh, r, x.grad_scale, w.of_grad);
    }
    if constexpr (GRAD) {
        __syncthreads();
        const float k = sh.factor;
        if (k == 0.0f && sh.at_label == 0.0f) {  // a clipped row
            zero_row<DT, NT>(out, x.vocab);
            return;
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int at = tid + i * NT;
            if (i < used) {
                float v[E];
#pragma unroll
                for (int j = 0; j < E; ++j) v[j] = exp_shifted(chunk_value<DT>(c[i], j), shift) * k;
                if (at < s.full && at != apart) store_values<DT>(out, s.chunk_at(at), v);
            }
        }
        if (edge >= 0) store_value<DT>(out, edge, edge == label ? sh.at_label : exp_shifted(at_edge, shift) * k);
    }
}

// ----------------------------------------------------------- longer rows --

// A sum relative to exponent `from`, relative to `to`.  A lane without a
// value yet has the sum 0 and no exponent; a NaN stays one.
__device__ __forceinline__ double rescaled(double sum, float from, float to) {
    return sum == 0.0 ? 0.0 : sum * double(__builtin_amdgcn_exp2f(from - to));
}

constexpr int STREAM_BLOCK = 1024;
constexpr int STREAM_UNROLL = 4;  // chunks in flight per lane

// The running maximum and sum by lane in one read; with the gradient, a
// second one.
template <int DT, bool GRAD, typename ROW>
__global__ __launch_bounds__(STREAM_BLOCK) void loss_rows_long(LogitsArgs x, ROW f) {
    constexpr int E = chunk_elems<DT>, NT = STREAM_BLOCK, U = STREAM_UNROLL;
    __shared__ RowShared<NT> sh;
    const int64_t row = x.row0 + blockIdx.x;
    const int tid = threadIdx.x, wave = tid >> 6;
    char *out = static_cast<char *>(x.grad) + row * x.grad_stride * elem_bytes<DT>;
    int64_t label;
    if (!takes_part(f, x, row, &label)) {
        absent_row(f, x, row);
        if constexpr (GRAD) zero_row<DT, NT>(out, x.vocab);
        return;
    }
    const char *in = static_cast<const char *>(x.logits) + row * x.stride * elem_bytes<DT>;
    const RowShape<DT> s(in, x.vocab);
    const float at_label = load_value<DT>(in, label);
    // top: the lane's largest value so far; shift: what its sum is relative
    // to.  A value of 2^24 or more makes the row's maximum such a one, and the
    // row slow; a lane whose values are all -2^24 or less adds nothing, and the
    // row is slow unless its maximum is far above; a NaN makes the sum one.
    float top = -__builtin_inff(), shift = 0.0f;
    double sum = 0.0;
    const auto take = [&](const u32x4 (&c)[U]) {
        float t = top;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j) t = fmaxf(t, chunk_value<DT>(c[u], j));
        const Shift to = shift_by(shiftable(t) ? t : 0.0f);
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < E; ++j) part[j & 3] += exp_sum(chunk_value<DT>(c[u], j), to);
        sum = rescaled(sum, shift, to.c) + ((double(part[0]) + double(part[1])) + (double(part[2]) + double(part[3])));
        top = t;
        shift = to.c;
    };
    const int apart = s.chunk_of(static_cast<int>(label));  // as in loss_rows
    const int edge = s.edge(tid, apart);
    const float at_edge = edge >= 0 && edge != label ? load_value<DT>(in, edge) : -__builtin_inff();
    for (int k0 = 0; k0 < s.full; k0 += NT * U) {
        u32x4 c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * NT + tid;
            if (k >= s.full || k == apart) c[u] = lowest_chunk<DT>();
            else c[u] = GRAD ? load_chunk<DT>(in, s.chunk_at(k)) : stream_chunk<DT>(in, s.chunk_at(k));
        }
        take(c);
    }
    if (edge >= 0) {
        const float t = fmaxf(top, at_edge);
        const Shift to = shift_by(shiftable(t) ? t : 0.0f);
        sum = rescaled(sum, shift, to.c) + double(exp_sum(at_edge, to));
        top = t;
        shift = to.c;
    }
    const float all = fmaxf(block_max<NT>(top, sh.tops), at_label);
    if (!shiftable_by_lane(all)) {
        slow_row<DT, NT, GRAD>(x, f, row, label, sh);
        return;
    }
    const float to = all * LOG2E;
    sum = block_sum<NT>(rescaled(sum, shift, to), sh.sums);
    shift = to;
    if (wave == 0) {
        const RowSum w = with_label(sum, label_term(at_label, all, shift, true));
        const RowResult r = finish_row(f, x, row, all, w.of_grad, w.logp);
        if (GRAD && tid == 0) put_factors(sh, r, x.grad_scale, w.of_grad);
    }
    if constexpr (GRAD) {
        __syncthreads();
        const float k = sh.factor;
        if (k == 0.0f && sh.at_label == 0.0f) {
            zero_row<DT, NT>(out, x.vocab);
            return;
        }
        for (int k0 = 0; k0 < s.full; k0 += NT * U) {
            u32x4 c[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = k0 + u * NT + tid;
                if (at < s.full && at != apart) c[u] = stream_chunk<DT>(in, s.chunk_at(at));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = k0 + u * NT + tid;
                if (at >= s.full || at == apart) continue;
                float v[E];
#pragma unroll
                for (int j = 0; j < E; ++j) v[j] = exp_shifted(chunk_value<DT>(c[u], j), shift) * k;
                store_values<DT>(out, s.chunk_at(at), v);
            }
        }
        if (edge >= 0) store_value<DT>(out, edge, edge == label ? sh.at_label : exp_shifted(at_edge, shift) * k);
    }
}

// ------------------------------------------- gradient from saved records --

// One chunk per lane and 1024 lanes measured 574 us for 7847 rows of 131072 BF16
// logits, 5492 of them live (3.5 GB, 6.1 TB/s), against 616 us with two
// chunks and 635 us with 256 lanes of four.
constexpr int GRAD_BLOCK = 1024;

// Workgroup (row, part): GRAD_BLOCK chunks of one row, part 0 its edges too.
template <int DT>
__global__ __launch_bounds__(GRAD_BLOCK) void logits_grad(LogitsArgs x, const float *upstream) {
    constexpr int E = chunk_elems<DT>;
    const int64_t row = x.row0 + blockIdx.x;
    const int tid = threadIdx.x, at = static_cast<int>(blockIdx.y) * GRAD_BLOCK + tid;
    char *out = static_cast<char *>(x.grad) + row * x.grad_stride * elem_bytes<DT>;
    const char *in = static_cast<const char *>(x.logits) + row * x.stride * elem_bytes<DT>;
    const RowShape<DT> s(in, x.vocab);
    const RowStats r = x.stats[row];
    const float up = upstream ? *upstream : 1.0f;
    const double g = double(r.coef) * double(x.grad_scale) * double(up);
    const int64_t label = load_index(x.labels, x.wide_ids, row);
    // no part in the loss (its record is all zeros), or clipped
    const bool dead = r.coef == 0.0f || label < 0 || label >= x.vocab;
    const float k = dead ? 0.0f : static_cast<float>(-g * double(r.inv_sum));
    const float at_label = static_cast<float>(g * double(r.one_less_p));
    // x - m first where the forward pass summed so
    const bool shifted = dead || shiftable(r.max);
    const float shift = dead ? 0.0f : r.max * LOG2E;
    const int edge = blockIdx.y == 0 ? s.edge(tid, -1) : -1;
    if (edge >= 0) {
        const float z = dead ? -__builtin_inff() : load_value<DT>(in, edge);
        const float v = (shifted ? exp_shifted(z, shift) : exp_neg(z - r.max)) * k;
        store_value<DT>(out, edge, !dead && edge == label ? at_label : v);
    }
    if (at >= s.full) return;
    u32x4 c = lowest_chunk<DT>();  // exponentials of zero
    if (!dead) c = stream_chunk<DT>(in, s.chunk_at(at));
    float v[E];
    if (shifted) {
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = exp_shifted(chunk_value<DT>(c, j), shift) * k;
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = exp_neg(chunk_value<DT>(c, j) - r.max) * k;
    }
    store_values<DT>(out, s.chunk_at(at), v);
    // the label's value, behind its own lane's store of the chunk
    if (!dead && label >= s.chunk_at(at) && label < s.chunk_at(at + 1)) store_value<DT>(out, label, at_label);
}

// ----------------------------------------------------------- small sums --

constexpr int TOTAL_BLOCK = 1024;

// total = sum of weights[i] * loss[i] in a fixed order; entries of weight
// zero add nothing, whatever their loss, nor do rows whose label is outside
// 0 .. vocab - 1 (labels may be null), whatever their weight.
__global__ __launch_bounds__(TOTAL_BLOCK) void weighted_total(const float *loss, const float *weights, int64_t n,
                                                              const void *labels, int32_t wide, int64_t vocab,
                                                              float *total) {
    __shared__ double part[TOTAL_BLOCK / 64];
    double s = 0.0;
    for (int64_t i0 = threadIdx.x; i0 < n; i0 += TOTAL_BLOCK * 4) {
        float w[4], l[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i0 + u * TOTAL_BLOCK;
            l[u] = i < n ? loss[i] : 0.0f;
            w[u] = i >= n ? 0.0f : weights ? weights[i] : 1.0f;
            if (labels && i < n) {
                const int64_t a = load_index(labels, wide, i);
                if (a < 0 || a >= vocab) w[u] = 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (w[u] != 0.0f) s += double(w[u]) * double(l[u]);
    }
    s = block_sum<TOTAL_BLOCK>(s, part);
    if (threadIdx.x == 0) *total = static_cast<float>(s);
}

constexpr int PAIR_BLOCK = 256;

// Offset s, held to the rows there are.
__device__ __forceinline__ int64_t row_offset(const PreferenceArgs &a, int64_t s) {
    const int64_t o = load_index(a.offsets, a.x.wide_ids, s);
    return o < 0 ? 0 : o > a.x.n ? a.x.n : o;
}

// A lane's part of a sequence's log-probability: rows begin, begin + step, ...
// `coef` still holds what FP32 dropped of logp.
__device__ __forceinline__ double sequence_part(const PreferenceArgs &a, int64_t begin, int64_t end, int step) {
    double v = 0.0;
    for (int64_t i0 = begin; i0 < end; i0 += step * 4) {
        float hi[4], lo[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i0 + int64_t(u) * step;
            hi[u] = i < end ? a.x.logp[i] : 0.0f;
            lo[u] = i < end ? a.x.stats[i].coef : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) v += double(hi[u]) + double(lo[u]);
    }
    return v;
}

// A pair's loss, and the coefficient of its chosen rows (the rejected rows'
// is the opposite), from its two sums.
__device__ __forceinline__ void pair_loss(const PreferenceArgs &a, int64_t pair, double chosen, double rejected,
                                          float *loss, float *coef) {
    const double h = a.beta * ((chosen - double(a.ref_logp[pair])) - (rejected - double(a.ref_logp[pair + a.pairs])));
    // log sigmoid(h) = min(h, 0) - log1p(exp(-|h|))
    const double q = exp(-fabs(h)), tail = log1p(q);
    const double up = (h >= 0.0 ? 1.0 : q) / (1.0 + q), down = (h >= 0.0 ? q : 1.0) / (1.0 + q);  // sigmoid(h), sigmoid(-h)
    const double ls = a.label_smoothing, w = a.weights ? double(a.weights[pair]) : 1.0;
    const double plus = h > 0.0 ? 0.0 : -h, minus = h < 0.0 ? 0.0 : h;
    // a term without weight adds nothing, infinite or not
    *loss = static_cast<float>((ls < 1.0 ? (1.0 - ls) * (plus + tail) : 0.0) + (ls > 0.0 ? ls * (minus + tail) : 0.0));
    *coef = w == 0.0 ? 0.0f : static_cast<float>(w * a.beta * (ls * up - (1.0 - ls) * down));
}

// The coefficient of every row of a sequence that takes part.
__device__ __forceinline__ void put_coef(const PreferenceArgs &a, int64_t begin, int64_t end, int step, float coef) {
#pragma unroll 4
    for (int64_t i = begin; i < end; i += step)
        a.x.stats[i].coef = a.x.stats[i].inv_sum != 0.0f ? coef : 0.0f;
}

// Rows outside every sequence have no coefficient.
__device__ __forceinline__ void clear_outside(const PreferenceArgs &a, int block) {
    const int64_t first = row_offset(a, 0), last = row_offset(a, 2 * a.pairs);
    for (int64_t i = threadIdx.x; i < first; i += block) a.x.stats[i].coef = 0.0f;
    for (int64_t i = last + threadIdx.x; i < a.x.n; i += block) a.x.stats[i].coef = 0.0f;
}

// One pair per workgroup: the sums of its two sequences, its loss, and the
// rows' coefficients.
__global__ __launch_bounds__(PAIR_BLOCK) void preference_pairs(PreferenceArgs a) {
    __shared__ double part[2][PAIR_BLOCK / 64];
    const int64_t pair = blockIdx.x;
    int64_t begin[2], end[2];
    double sum[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const int64_t s = pair + side * a.pairs;
        begin[side] = row_offset(a, s);
        end[side] = row_offset(a, s + 1);
        sum[side] = block_sum<PAIR_BLOCK>(sequence_part(a, begin[side] + threadIdx.x, end[side], PAIR_BLOCK), part[side]);
    }
    float loss, coef;
    pair_loss(a, pair, sum[0], sum[1], &loss, &coef);
    if (threadIdx.x == 0) {
        a.loss[pair] = loss;
        a.seq_logp[pair] = static_cast<float>(sum[0]);
        a.seq_logp[pair + a.pairs] = static_cast<float>(sum[1]);
    }
#pragma unroll
    for (int side = 0; side < 2; ++side)
        put_coef(a, begin[side] + threadIdx.x, end[side], PAIR_BLOCK, side ? -coef : coef);
    if (pair == 0) clear_outside(a, PAIR_BLOCK);
}

// Pairs that one workgroup serves with a wave per sequence, total and all: it
// saves the launch that sums the losses (8 pairs of up to 513 rows: 5.4 and
// 4.5 us for the two launches, 7.6 us for the one).
constexpr int FEW_PAIRS = 8;
constexpr int FEW_BLOCK = 2 * FEW_PAIRS * 64;

__global__ __launch_bounds__(FEW_BLOCK) void preference_few(PreferenceArgs a) {
    __shared__ double sums[2 * FEW_PAIRS];
    __shared__ double terms[FEW_PAIRS];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, pairs = static_cast<int>(a.pairs);
    int64_t begin = 0, end = 0;
    if (wave < 2 * pairs) {
        begin = row_offset(a, wave);
        end = row_offset(a, wave + 1);
        const double s = wave_sum(sequence_part(a, begin + lane, end, 64));
        if (lane == 0) {
            sums[wave] = s;
            a.seq_logp[wave] = static_cast<float>(s);
        }
    }
    __syncthreads();
    if (wave < 2 * pairs) {
        const int pair = wave < pairs ? wave : wave - pairs;
        float loss, coef;
        pair_loss(a, pair, sums[pair], sums[pair + pairs], &loss, &coef);
        if (lane == 0 && wave < pairs) {
            const float w = a.weights ? a.weights[pair] : 1.0f;
            a.loss[pair] = loss;
            terms[pair] = w != 0.0f ? double(w) * double(loss) : 0.0;
        }
        put_coef(a, begin + lane, end, 64, wave < pairs ? coef : -coef);
    }
    clear_outside(a, FEW_BLOCK);
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int p = 0; p < pairs; ++p) s += terms[p];
        *a.total = static_cast<float>(s);
    }
}

}  // namespace

// ------------------------------------------------------------- launchers --

// Rows of one launch: 2^21 workgroups of 1024 lanes stay below the 2^32
// work-items that a launch addresses.
constexpr int64_t ROWS_PER_LAUNCH = int64_t(1) << 21;

// launch(x, rows) for all rows, in as many launches as that takes.
template <typename LAUNCH>
static hipError_t over_rows(LogitsArgs x, int *launched, LAUNCH launch) {
    for (x.row0 = 0; x.row0 < x.n; x.row0 += ROWS_PER_LAUNCH) {
        const int64_t rows = x.n - x.row0 < ROWS_PER_LAUNCH ? x.n - x.row0 : ROWS_PER_LAUNCH;
        launch(x, static_cast<unsigned>(rows));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        ++*launched;
    }
    return hipSuccess;
}

template <int DT, bool GRAD, typename ROW>
static void launch_rows(const LogitsArgs &x, unsigned rows, const ROW &f, hipStream_t stream) {
    const int64_t chunks = (x.vocab + chunk_elems<DT> - 1) / chunk_elems<DT>;
    const dim3 grid(rows);
#define RADAMW_ROWS(NT, CH) \
    hipLaunchKernelGGL((loss_rows<DT, NT, CH, GRAD, ROW>), grid, dim3(NT), 0, stream, x, f)
#define RADAMW_LONG() \
    hipLaunchKernelGGL((loss_rows_long<DT, GRAD, ROW>), grid, dim3(STREAM_BLOCK), 0, stream, x, f)
    // Without a gradient nothing has to be held: a read that streams reaches
    // 6.8 TB/s (5492 rows of 131072 BF16 logits: 212 us, against 362 us from
    // registers, one workgroup per CU).  Short rows waste its 1024 lanes.
    if (chunks <= 256 * 4) {
        RADAMW_ROWS(256, 4);
    } else if constexpr (!GRAD) {
        RADAMW_LONG();
    } else {
        if (chunks <= 256 * 8) RADAMW_ROWS(256, 8);
        else if (chunks <= 256 * 16) RADAMW_ROWS(256, 16);
        else if (chunks <= 512 * 16) RADAMW_ROWS(512, 16);
        else if (chunks <= 1024 * 16) RADAMW_ROWS(1024, 16);
        else RADAMW_LONG();
    }
#undef RADAMW_LONG
#undef RADAMW_ROWS
}

template <int DT>
static void policy_rows(const LogitsArgs &x, unsigned rows, const PolicyRow &f, hipStream_t stream) {
    if (x.grad) launch_rows<DT, true>(x, rows, f, stream);
    else launch_rows<DT, false>(x, rows, f, stream);
}

hipError_t launch_policy_loss(const PolicyArgs &a, int dt, hipStream_t stream, int *launched) {
    const PolicyRow f{a.old_logp, a.ref_logp, a.advantages, a.weights, a.loss, a.clip_low, a.clip_high, a.kl_coef};
    hipError_t e = over_rows(a.x, launched, [&](const LogitsArgs &x, unsigned rows) {
        switch (dt) {
        case G_F32: policy_rows<G_F32>(x, rows, f, stream); break;
        case G_F16: policy_rows<G_F16>(x, rows, f, stream); break;
        default: policy_rows<G_BF16>(x, rows, f, stream); break;
        }
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(weighted_total, dim3(1), dim3(TOTAL_BLOCK), 0, stream, a.loss, a.weights, a.x.n,
                       a.x.labels, a.x.wide_ids, a.x.vocab, a.total);
    if ((e = hipGetLastError()) == hipSuccess) ++*launched;
    return e;
}

hipError_t launch_logits_grad(const LogitsArgs &a, const float *upstream, int dt, hipStream_t stream, int *launched) {
    const int64_t chunks = (a.vocab + (dt == G_F32 ? 3 : 7)) / (dt == G_F32 ? 4 : 8);
    const unsigned parts = static_cast<unsigned>((chunks + GRAD_BLOCK - 1) / GRAD_BLOCK);
    return over_rows(a, launched, [&](const LogitsArgs &x, unsigned rows) {
        const dim3 grid(rows, parts), block(GRAD_BLOCK);
        switch (dt) {
        case G_F32: hipLaunchKernelGGL(logits_grad<G_F32>, grid, block, 0, stream, x, upstream); break;
        case G_F16: hipLaunchKernelGGL(logits_grad<G_F16>, grid, block, 0, stream, x, upstream); break;
        default: hipLaunchKernelGGL(logits_grad<G_BF16>, grid, block, 0, stream, x, upstream); break;
        }
    });
}

hipError_t launch_preference_loss(const PreferenceArgs &a, int dt, hipStream_t stream, int *launched) {
    const LogpRow f{};
    hipError_t e = over_rows(a.x, launched, [&](const LogitsArgs &x, unsigned rows) {
        switch (dt) {
        case G_F32: launch_rows<G_F32, false>(x, rows, f, stream); break;
        case G_F16: launch_rows<G_F16, false>(x, rows, f, stream); break;
        default: launch_rows<G_BF16, false>(x, rows, f, stream); break;
        }
    });
    if (e != hipSuccess) return e;
    if (a.pairs <= FEW_PAIRS) {
        hipLaunchKernelGGL(preference_few, dim3(1), dim3(FEW_BLOCK), 0, stream, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        ++*launched;
    } else {
        hipLaunchKernelGGL(preference_pairs, dim3(static_cast<unsigned>(a.pairs)), dim3(PAIR_BLOCK), 0, stream, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL(weighted_total, dim3(1), dim3(TOTAL_BLOCK), 0, stream, a.loss, a.weights, a.pairs,
                           nullptr, 0, 0, a.total);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        *launched += 2;
    }
    if (a.x.grad) e = launch_logits_grad(a.x, nullptr, dt, stream, launched);
    return e;
}

}  // namespace radamw
