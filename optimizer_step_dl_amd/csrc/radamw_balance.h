// radamw_balance.h -- the rows of the balance loss (radamw_balance.hip) for
// gfx950: pieces of rows, their probabilities, sums and gradient, and all of a
// small batch in one workgroup.  The two scores are compiled beside one another
// (radamw_balance.hip, radamw_balance_sigmoid.hip), each without what the other
// alone holds in registers: in one kernel 8192 x 4096 FP32 logits with softmax
// took 253 us, against 198 us, and 353 us with far_scores() for the sigmoid.
#pragma once

#include "radamw_residual.h"

namespace radamw {

constexpr int BALANCE_BLOCK = 256;

struct BalanceExtra {
    double squares;
    int64_t rows;
};
static_assert(sizeof(BalanceExtra) == 16, "");

// ---------------------------------------------------------------- pieces --

// Offset g, clamped to the rows for every access.
__device__ __forceinline__ int64_t row_offset(const BalanceArgs &a, int64_t g) {
    const int64_t v = load_index(a.offsets, a.wide, g);
    return v < 0 ? 0 : v > a.n ? a.n : v;
}

struct BalanceRows {
    int64_t group, begin, end;  // empty where begin >= end
};
__device__ __forceinline__ BalanceRows piece_of(const BalanceArgs &a, const BalancePlan &p, int64_t b) {
    if (!a.offsets) return {0, b * p.rows, min((b + 1) * p.rows, a.n)};
    // the last group whose first piece is not behind b
    int64_t lo = 0, hi = a.groups;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (row_offset(a, mid) / p.rows + mid <= b) lo = mid;
        else hi = mid;
    }
    const int64_t c = b - lo;
    return {lo, max(row_offset(a, lo), c * p.rows), min(row_offset(a, lo + 1), (c + 1) * p.rows)};
}
// The pieces of a group: first and number.
__device__ __forceinline__ void pieces_of(const BalanceArgs &a, const BalancePlan &p, int64_t g, int64_t *first,
                                          int64_t *count) {
    const int64_t begin = a.offsets ? row_offset(a, g) : 0, end = a.offsets ? row_offset(a, g + 1) : a.n;
    *first = begin / p.rows + g;
    *count = end > begin ? (end - 1) / p.rows + g - *first + 1 : 0;
}

// -------------------------------------------------------------- counting --

// Counts of a piece's chosen experts and its rows that take part, in LDS.
__device__ __forceinline__ void count_piece(const BalanceArgs &a, const BalanceRows &piece, int32_t *hist, int32_t *rows) {
    const int experts = static_cast<int>(a.experts);
    for (int e = threadIdx.x; e < experts; e += BALANCE_BLOCK) hist[e] = 0;
    if (threadIdx.x == 0) *rows = 0;
    __syncthreads();
    const uint32_t top_k = static_cast<uint32_t>(a.top_k), count = static_cast<uint32_t>(piece.end - piece.begin) * top_k;
    for (uint32_t i = threadIdx.x; i < count; i += BALANCE_BLOCK) {
        const uint32_t r = i / top_k;
        if (a.mask && !a.mask[piece.begin + r]) continue;
        const int64_t id = load_index(a.ids, a.wide, piece.begin * a.top_k + i);
        if (id >= 0 && id < a.experts) atomicAdd(&hist[id], 1);
        if (i == r * top_k) atomicAdd(rows, 1);
    }
    __syncthreads();
}

// ------------------------------------------------------------------ rows --

// Reductions over the 2^lg lanes of a row.
__device__ __forceinline__ float lanes_sum(float v, int lg) {
    for (int s = 0; s < lg; ++s) v += __shfl_xor(v, 1 << s, 64);
    return v;
}
__device__ __forceinline__ float lanes_max(float v, int lg) {
    for (int s = 0; s < lg; ++s) v = fmaxf(v, __shfl_xor(v, 1 << s, 64));
    return v;
}

// A lane's eight columns; of FP32 logits two fours that are 4 * 2^lg apart, so
// that a row's lanes lie side by side in every load and store.
struct Piece8 : radamw::Piece {
    __device__ int32_t at(int j) const { return j < 4 ? e + j : e2 + j - 4; }
};
template <bool SPLIT>
__device__ __forceinline__ Piece8 columns_of(int lane, int k, int lg) {
    if constexpr (SPLIT) return {{(lane + (2 * k << lg)) * 4, (lane + ((2 * k + 1) << lg)) * 4}};
    else return {{(lane + (k << lg)) * 8, (lane + (k << lg)) * 8 + 4}};
}

// exp(d) for d <= 0.  log2 e is in two parts: as one FP32 number it is too
// small by 1.3e-8, and every exponential of d too large by that much of -d.
// The first has 13 bits, so that the second is many steps of the exponent's
// last digit and rounds evenly.
constexpr float LOG2E_HI = 5909.0f / 4096, LOG2E_LO = static_cast<float>(1.4426950408889634 - 5909.0 / 4096);
__device__ __forceinline__ float exp_of(float d) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(d, LOG2E_LO, d * LOG2E_HI));
}

// The scores of a row that are all far below one, anew and in proportion: with
// the largest logit m taken off every exponent, exp(x - m) / (1 + exp(x)), what
// FP32 would hold as zeros (logits below -87) keeps its share of the sum, which
// is what divides it.  A score is 0 where 1 / (1 + exp(-x)) is in 64 bits:
// exp(709.7828) is beyond their range.  Such rows are told by their sum: from
// FAR_SUM on, what is flushed to zero is below 2^-126 / FAR_SUM = 2^-120 of it.
constexpr float FAR_SUM = 0x1p-6f;
constexpr float FAR_LOGIT = -709.78271484375f;

template <int DT, int K, bool TAIL>
__device__ __forceinline__ float far_scores(const void *row, int lane, int lg, int32_t experts, f32x8 (&x)[K]) {
    constexpr bool SPLIT = split_stream<DT>;
    float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Piece8 e = columns_of<SPLIT>(lane, k, lg);
        Raw8<DT> r{};
        if (e.e < experts) r = load_piece<DT, SPLIT, TAIL>(row, e, experts);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = raw_value<DT>(r, j);
            x[k][j] = e.at(j) < experts && v > FAR_LOGIT ? v : -__builtin_inff();
            top = fmaxf(top, x[k][j]);
        }
        __builtin_amdgcn_sched_barrier(0);  // eight values at a time: registers are short
    }
    top = lanes_max(top, lg);
    if (top == -__builtin_inff()) top = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = x[k][j];
            x[k][j] = exp_of(v - top) * __builtin_amdgcn_rcpf(1.0f + exp_of(v));  // exp(v) < 2^-6
            sum += x[k][j];
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    return lanes_sum(sum, lg);
}

// The rows of a piece.  SUMS: leave the sums of their probabilities and of the
// squared log-sums in the workspace's `slot`.  GRAD: write the logits'
// gradient from the groups' counts.  `part` is LDS of p.width values, `squares`
// of one per wave (SUMS).
template <int DT, int K, bool SIGMOID, bool SUMS, bool GRAD, bool TAIL>
__device__ __forceinline__ void rows_of_piece(const BalanceArgs &a, const BalancePlan &p, const BalanceRows &piece,
                                              int64_t slot, int lg, float *part, double *squares) {
    constexpr bool SPLIT = split_stream<DT>;
    const int lane = threadIdx.x & ((1 << lg) - 1), mine = threadIdx.x >> lg;
    const int per = BALANCE_BLOCK >> lg;  // rows at a time
    const int32_t experts = static_cast<int32_t>(a.experts);
    f32x8 cost[K], acc[K];
    float zc = 0.0f, sq = 0.0f;
    bool counted = true;  // whether the group's loss is part of the total
#pragma unroll
    for (int k = 0; k < K; ++k) acc[k] = f32x8{};
    if constexpr (GRAD) {
        // The probabilities add up to one, so that a number taken off every
        // count leaves the gradient as it is.  Taken off as whole numbers, the
        // count of a balanced router leaves the small differences that the
        // gradient is made of with all their digits: a balanced one is zero.
        const int32_t even = static_cast<int32_t>(a.tokens[piece.group] * a.top_k / a.experts);
        const double t = max(a.tokens[piece.group], 1);
        double up = a.grad_scale / t;
        if (a.weights) {
            up *= a.weights[piece.group];
            counted = a.weights[piece.group] != 0.0f;
        }
        if (a.upstream) up *= *a.upstream;
        zc = static_cast<float>(2.0 * a.z_coef * up);
        const float f = static_cast<float>(up * a.balance_coef * static_cast<double>(a.experts) /
                                           (static_cast<double>(a.top_k) * t));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Piece8 e = columns_of<SPLIT>(lane, k, lg);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                cost[k][j] = e.at(j) < experts ? f * static_cast<float>(a.counts[piece.group * a.experts + e.at(j)] - even) : 0.0f;
        }
    }
    for (int64_t t = piece.begin + mine; t < piece.end; t += per) {
        const bool live = !a.mask || a.mask[t];
        f32x8 x[K];
        float top = -__builtin_inff();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Piece8 e = columns_of<SPLIT>(lane, k, lg);
            Raw8<DT> r{};
            if (live && e.e < experts) r = load_piece<DT, SPLIT, TAIL>(elem_at(a.logits, DT, t * a.stride), e, experts);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] = live && e.at(j) < experts ? raw_value<DT>(r, j) : -__builtin_inff();
                top = fmaxf(top, x[k][j]);
            }
        }
        // probabilities in x, for sigmoid their factor 1 - s in rest
        f32x8 rest[SIGMOID ? K : 1];
        float sum = 0.0f, lse = 0.0f;
        if constexpr (SIGMOID) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = x[k][j], e = exp_of(-fabsf(v)), r = 1.0f / (1.0f + e);
                    x[k][j] = v >= 0.0f ? r : e * r;  // NaN stays NaN: e is
                    rest[k][j] = v >= 0.0f ? e * r : r;
                    sum += x[k][j];
                }
            sum = lanes_sum(sum, lg);
            if (live && sum < FAR_SUM)
                sum = far_scores<DT, K, TAIL>(elem_at(a.logits, DT, t * a.stride), lane, lg, experts, x);
        } else {
            top = lanes_max(top, lg);
            const float m = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[k][j] = exp_of(x[k][j] - m);
                    sum += x[k][j];
                }
            sum = lanes_sum(sum, lg);
            lse = sum == 0.0f ? 0.0f : m + __logf(sum);
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a row of -inf has no probabilities
        float inner = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[k][j] *= inv;
                if constexpr (SUMS) acc[k][j] += x[k][j];
                if constexpr (GRAD) inner = __builtin_fmaf(cost[k][j], x[k][j], inner);
            }
        if constexpr (SUMS) {
            if (lane == 0 && live) sq = __builtin_fmaf(lse, lse, sq);
        }
        if constexpr (GRAD) {
            inner = lanes_sum(inner, lg) - zc * lse;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const Piece8 e = columns_of<SPLIT>(lane, k, lg);
                if (e.e >= experts) continue;
                f32x8 g;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    g[j] = x[k][j] * (cost[k][j] - inner);
                    if constexpr (SIGMOID) g[j] *= rest[k][j];
                    if (!live || !counted) g[j] = 0.0f;  // whatever the logits hold
                }
                store_piece<DT, SPLIT, TAIL>(elem_at(a.grad, DT, t * a.grad_stride), e, experts, g);
            }
        }
    }
    if constexpr (SUMS) {
        // rows of one wave, then the waves in turn
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                for (int s = lg; s < 6; ++s) acc[k][j] += __shfl_xor(acc[k][j], 1 << s, 64);
        double q = sq;
        for (int s = 32; s > 0; s >>= 1) q += __shfl_xor(q, s, 64);
        if ((threadIdx.x & 63) == 0) squares[threadIdx.x >> 6] = q;
        for (int w = 0; w < BALANCE_BLOCK / 64; ++w) {
            if (threadIdx.x >> 6 == w && (threadIdx.x & 63) < (1 << lg)) {
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int e = columns_of<SPLIT>(lane, k, lg).at(j);
                        if (e < p.width) part[e] = w == 0 ? acc[k][j] : part[e] + acc[k][j];
                    }
            }
            __syncthreads();
        }
        float *out = reinterpret_cast<float *>(a.workspace + p.probs) + slot * p.width;
        for (int e = threadIdx.x; e < experts; e += BALANCE_BLOCK) out[e] = part[e];
        if (threadIdx.x == 0)
            reinterpret_cast<BalanceExtra *>(a.workspace + p.extra)[slot].squares =
                (squares[0] + squares[1]) + (squares[2] + squares[3]);
    }
}

template <int DT, int K, bool SIGMOID, bool SUMS, bool GRAD, bool TAIL>
__global__ __launch_bounds__(BALANCE_BLOCK) void balance_rows(BalanceArgs a, BalancePlan p, int lg) {
    constexpr bool SPLIT = split_stream<DT>;
    __shared__ float part[SUMS ? BALANCE_MAX_EXPERTS : 1];
    __shared__ double squares[BALANCE_BLOCK / 64];
    const int lane = threadIdx.x & ((1 << lg) - 1), mine = threadIdx.x >> lg;
    const int per = BALANCE_BLOCK >> lg;  // rows at a time
    const int32_t experts = static_cast<int32_t>(a.experts);
    if constexpr (GRAD) {
        if (a.offsets) {
            // rows outside every group: before the first, behind the last
            const int64_t from = int64_t(blockIdx.x) * p.rows, to = min(from + p.rows, a.n);
            const int64_t lo = row_offset(a, 0), hi = row_offset(a, a.groups);
            for (int64_t t = from + mine; t < to; t += per) {
                if (t >= lo && t < hi) continue;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const Piece8 e = columns_of<SPLIT>(lane, k, lg);
                    if (e.e < experts) store_piece<DT, SPLIT, TAIL>(elem_at(a.grad, DT, t * a.grad_stride), e, experts, f32x8{});
                }
            }
        }
    }
    const BalanceRows piece = piece_of(a, p, blockIdx.x);
    if (piece.begin < piece.end) rows_of_piece<DT, K, SIGMOID, SUMS, GRAD, TAIL>(a, p, piece, blockIdx.x, lg, part, squares);
}

__device__ __forceinline__ double wave_sum64(double v) {
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s, 64);
    return v;
}

// A group's loss, by one wave.
__device__ __forceinline__ double group_loss(const BalanceArgs &a, const BalancePlan &p, int64_t g, int lane) {
    double dot = 0.0, squares = 0.0;
    for (int64_t e = lane; e < a.experts; e += 64)
        dot += static_cast<double>(a.counts[g * a.experts + e]) * static_cast<double>(a.mean_prob[g * a.experts + e]);
    const double t = max(a.tokens[g], 1);
    double loss = a.balance_coef * static_cast<double>(a.experts) / (static_cast<double>(a.top_k) * t) * wave_sum64(dot);
    if (a.z_coef != 0.0) {
        int64_t first, count;
        pieces_of(a, p, g, &first, &count);
        const BalanceExtra *extra = reinterpret_cast<const BalanceExtra *>(a.workspace + p.extra);
        for (int64_t i = lane; i < count; i += 64) squares += extra[first + i].squares;
        loss += a.z_coef / t * wave_sum64(squares);
    }
    return loss;
}

__device__ __forceinline__ double weighted(const BalanceArgs &a, int64_t g, float loss) {
    const float w = a.weights ? a.weights[g] : 1.0f;
    return w != 0.0f ? static_cast<double>(w) * static_cast<double>(loss) : 0.0;
}

// All of a batch that is one piece of one group: what the workgroup writes to
// memory in one step it reads in the next, behind a barrier.
template <int DT, int K, bool SIGMOID, bool GRAD, bool TAIL>
__global__ __launch_bounds__(BALANCE_BLOCK) void balance_single(BalanceArgs a, BalancePlan p, int lg) {
    __shared__ int32_t hist[BALANCE_MAX_EXPERTS];
    __shared__ float part[BALANCE_MAX_EXPERTS];
    __shared__ double squares[BALANCE_BLOCK / 64];
    __shared__ int32_t rows;
    const int experts = static_cast<int>(a.experts);
    const BalanceRows piece = {0, 0, a.n};
    count_piece(a, piece, hist, &rows);
    for (int e = threadIdx.x; e < experts; e += BALANCE_BLOCK) a.counts[e] = hist[e];
    if (threadIdx.x == 0) a.tokens[0] = rows;
    __threadfence_block();
    __syncthreads();
    rows_of_piece<DT, K, SIGMOID, true, GRAD, TAIL>(a, p, piece, 0, lg, part, squares);
    __threadfence_block();
    __syncthreads();
    const double t = max(rows, 1);
    for (int e = threadIdx.x; e < experts; e += BALANCE_BLOCK) a.mean_prob[e] = static_cast<float>(static_cast<double>(part[e]) / t);
    __threadfence_block();
    __syncthreads();
    if (threadIdx.x < 64) {
        const float loss = static_cast<float>(group_loss(a, p, 0, threadIdx.x));
        if (threadIdx.x == 0) {
            a.loss[0] = loss;
            *a.total = static_cast<float>(weighted(a, 0, loss));
        }
    }
}

// ---------------------------------------------------------------- launch --

// One workgroup does all in one launch: 256 x 8 BF16 logits in 12 us a call
// instead of 28 us with six launches.
inline bool balance_at_once(const BalanceArgs &a, const BalancePlan &p) {
    return a.n > 0 && p.pieces == 1 && !a.offsets && a.experts <= 512;
}

template <int DT, int K, bool SIGMOID, bool SUMS, bool GRAD>
void balance_rows_at(const BalanceArgs &a, const BalancePlan &p, int lg, hipStream_t stream) {
    auto kernel = a.experts % 8 ? balance_rows<DT, K, SIGMOID, SUMS, GRAD, true> : balance_rows<DT, K, SIGMOID, SUMS, GRAD, false>;
    if constexpr (SUMS && K == 1) {
        if (balance_at_once(a, p))
            kernel = a.experts % 8 ? balance_single<DT, K, SIGMOID, GRAD, true> : balance_single<DT, K, SIGMOID, GRAD, false>;
    }
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(p.pieces)), dim3(BALANCE_BLOCK), 0, stream, a, p, lg);
}

template <int DT, bool SIGMOID, bool SUMS, bool GRAD>
void balance_rows_with(const BalanceArgs &a, const BalancePlan &p, hipStream_t stream) {
    const int64_t eights = ceil_div(a.experts, 8);
    int lg = 0;
    while (lg < 6 && (int64_t(1) << lg) < eights) ++lg;
    if (eights <= 64) balance_rows_at<DT, 1, SIGMOID, SUMS, GRAD>(a, p, lg, stream);
    else if (eights <= 128) balance_rows_at<DT, 2, SIGMOID, SUMS, GRAD>(a, p, lg, stream);
    else if (eights <= 256) balance_rows_at<DT, 4, SIGMOID, SUMS, GRAD>(a, p, lg, stream);
    else balance_rows_at<DT, 8, SIGMOID, SUMS, GRAD>(a, p, lg, stream);
}

template <bool SIGMOID, bool SUMS, bool GRAD>
void balance_rows_type(const BalanceArgs &a, const BalancePlan &p, int dt, hipStream_t stream) {
    switch (dt) {
    case G_F32: balance_rows_with<G_F32, SIGMOID, SUMS, GRAD>(a, p, stream); break;
    case G_F16: balance_rows_with<G_F16, SIGMOID, SUMS, GRAD>(a, p, stream); break;
    default: balance_rows_with<G_BF16, SIGMOID, SUMS, GRAD>(a, p, stream); break;
    }
}

// One launch: the sums (with the gradient where one is asked for), or without
// `sums` the gradient from the counts.
template <bool SIGMOID>
hipError_t balance_rows_of(const BalanceArgs &a, const BalancePlan &p, bool sums, int dt, hipStream_t stream) {
    if (!sums) balance_rows_type<SIGMOID, false, true>(a, p, dt, stream);
    else if (a.grad) balance_rows_type<SIGMOID, true, true>(a, p, dt, stream);
    else balance_rows_type<SIGMOID, true, false>(a, p, dt, stream);
    return hipGetLastError();
}
hipError_t balance_rows_sigmoid(const BalanceArgs &a, const BalancePlan &p, bool sums, int dt, hipStream_t stream);

}  // namespace radamw
