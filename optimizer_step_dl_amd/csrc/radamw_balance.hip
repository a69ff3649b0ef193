// radamw_balance.hip -- the balance loss of a router with its per-expert
// counts, the z-loss and the logits' gradient for gfx950.
//
//   P_te = softmax of row t, or s_te / sum_e s_te with s = sigmoid
//   c_e  = how often the rows' chosen experts are e,  T = rows that take part
//   loss = a E / (k T^2) sum_e c_e sum_t P_te  +  z / T sum_t lse_t^2
//   grad = P (f_e - sum_e f_e P + 2 z / T lse),   f_e = a E c_e / (k T^2);
//          sigmoid: P (1 - s) (f_e - sum_e f_e P)
//
// per group of rows.  A row is held by 2^lg lanes of one wave, eight values
// to a lane (or 16, 32, 64).  The sums over rows have a fixed order: each
// workgroup takes a piece of rows (radamw_block.h), sums its columns in
// registers and leaves one row of FP32 sums, which are joined in FP64.
//
// The gradient needs all counts, so ids are counted first (they are an eighth
// of the logits' bytes or less); then loss and gradient take one read of the
// logits and one write.  Bound by HBM where the batch is long: 262144 x 256
// FP32 logits with their gradient take 132 us (554 MB: 4.2 TB/s), 112 us of it
// in balance_rows, the rest in the count and the two joins; by the latency of
// five dependent launches where it is not (16383 x 160 in 13 groups: 34 us).
#include "radamw_residual.h"

namespace radamw {

namespace {

constexpr int BLOCK = 256;

constexpr int64_t max_of(int64_t a, int64_t b) { return a > b ? a : b; }
constexpr int64_t min_of(int64_t a, int64_t b) { return a < b ? a : b; }

struct Extra {
    double squares;
    int64_t rows;
};
static_assert(sizeof(Extra) == 16, "");

int64_t up256(int64_t v) { return ceil_div(v, 256) * 256; }

}  // namespace

BalancePlan balance_plan(int64_t n, int64_t experts, int64_t groups) {
    BalancePlan p{};
    // one piece of up to 16384 values, which one workgroup does in one launch;
    // of more, at least 512 pieces where that leaves each 2048 values, and
    // about 1024 of a long batch: 16383 x 160 take 34 us, against 40 us with
    // 256 pieces; 262144 x 256 take 132 us, against 157 us with 2048
    if (n <= ceil_div(16384, experts)) p.rows = max_of(1, n);
    else p.rows = max_of(ceil_div(n, 1024), max_of(ceil_div(2048, experts), min_of(ceil_div(n, 512), ceil_div(16384, experts))));
    p.pieces = ceil_div(n, p.rows) + (groups > 1 ? groups : 0);
    p.width = ceil_div(experts, 16) * 16;
    p.probs = 0;
    p.counts = up256(p.pieces * p.width * 4);
    p.extra = p.counts + up256(p.pieces * p.width * 4);
    p.bytes = max_of(256, p.extra + up256(p.pieces * 16));
    return p;
}

// ---------------------------------------------------------------- pieces --

// Offset g, clamped to the rows for every access.
__device__ __forceinline__ int64_t row_offset(const BalanceArgs &a, int64_t g) {
    const int64_t v = load_index(a.offsets, a.wide, g);
    return v < 0 ? 0 : v > a.n ? a.n : v;
}

struct Rows {
    int64_t group, begin, end;  // empty where begin >= end
};
__device__ __forceinline__ Rows piece_of(const BalanceArgs &a, const BalancePlan &p, int64_t b) {
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
__device__ __forceinline__ void count_piece(const BalanceArgs &a, const Rows &piece, int32_t *hist, int32_t *rows) {
    const int experts = static_cast<int>(a.experts);
    for (int e = threadIdx.x; e < experts; e += BLOCK) hist[e] = 0;
    if (threadIdx.x == 0) *rows = 0;
    __syncthreads();
    const uint32_t top_k = static_cast<uint32_t>(a.top_k), count = static_cast<uint32_t>(piece.end - piece.begin) * top_k;
    for (uint32_t i = threadIdx.x; i < count; i += BLOCK) {
        const uint32_t r = i / top_k;
        if (a.mask && !a.mask[piece.begin + r]) continue;
        const int64_t id = load_index(a.ids, a.wide, piece.begin * a.top_k + i);
        if (id >= 0 && id < a.experts) atomicAdd(&hist[id], 1);
        if (i == r * top_k) atomicAdd(rows, 1);
    }
    __syncthreads();
}

__global__ __launch_bounds__(BLOCK) void balance_count(BalanceArgs a, BalancePlan p) {
    __shared__ int32_t hist[BALANCE_MAX_EXPERTS];
    __shared__ int32_t rows;
    const Rows piece = piece_of(a, p, blockIdx.x);
    if (piece.begin >= piece.end) return;
    count_piece(a, piece, hist, &rows);
    int32_t *out = reinterpret_cast<int32_t *>(a.workspace + p.counts) + blockIdx.x * p.width;
    for (int e = threadIdx.x; e < a.experts; e += BLOCK) out[e] = hist[e];
    if (threadIdx.x == 0) reinterpret_cast<Extra *>(a.workspace + p.extra)[blockIdx.x].rows = rows;
}

// Sixteen columns of one group: 16 columns x 64 strips of pieces.
constexpr int JOIN = 1024, STRIPS = JOIN / 16;

__global__ __launch_bounds__(JOIN) void balance_join_counts(BalanceArgs a, BalancePlan p, int64_t g0) {
    __shared__ int32_t strip[STRIPS][16];
    __shared__ int64_t rows[STRIPS];
    const int64_t g = g0 + blockIdx.y;
    int64_t first, count;
    pieces_of(a, p, g, &first, &count);
    const int c = threadIdx.x & 15, s = threadIdx.x >> 4;
    const int64_t e = int64_t(blockIdx.x) * 16 + c;
    const int32_t *counts = reinterpret_cast<const int32_t *>(a.workspace + p.counts);
    const Extra *extra = reinterpret_cast<const Extra *>(a.workspace + p.extra);
    int32_t sum = 0;
    int64_t taken = 0;
    if (e < a.experts) {
#pragma unroll 4
        for (int64_t i = s; i < count; i += STRIPS) sum += counts[(first + i) * p.width + e];
    }
    if (blockIdx.x == 0 && c == 0) {
#pragma unroll 4
        for (int64_t i = s; i < count; i += STRIPS) taken += extra[first + i].rows;
    }
    strip[s][c] = sum;
    if (c == 0) rows[s] = taken;
    __syncthreads();
    if (s != 0) return;
    for (int k = 1; k < STRIPS; ++k) sum += strip[k][c];
    if (e < a.experts) a.counts[g * a.experts + e] = sum;
    if (blockIdx.x == 0 && c == 0) {
        for (int k = 1; k < STRIPS; ++k) taken += rows[k];
        a.tokens[g] = static_cast<int32_t>(taken);
    }
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

// The rows of a piece.  SUMS: leave the sums of their probabilities and of the
// squared log-sums in the workspace's `slot`.  GRAD: write the logits'
// gradient from the groups' counts.  `part` is LDS of p.width values, `squares`
// of one per wave (SUMS).
template <int DT, int K, bool SUMS, bool GRAD, bool TAIL>
__device__ __forceinline__ void rows_of_piece(const BalanceArgs &a, const BalancePlan &p, const Rows &piece, int64_t slot,
                                              int lg, float *part, double *squares) {
    constexpr bool SPLIT = split_stream<DT>;
    const int lane = threadIdx.x & ((1 << lg) - 1), mine = threadIdx.x >> lg;
    const int per = BLOCK >> lg;  // rows at a time
    const int32_t experts = static_cast<int32_t>(a.experts);
    f32x8 cost[K], acc[K];
    float zc = 0.0f, sq = 0.0f;
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
        if (a.weights) up *= a.weights[piece.group];
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
        f32x8 rest[K];
        float sum = 0.0f, lse = 0.0f;
        if (a.sigmoid) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = x[k][j], e = __builtin_amdgcn_exp2f(-fabsf(v) * LOG2E), r = 1.0f / (1.0f + e);
                    x[k][j] = v >= 0.0f ? r : e * r;  // NaN stays NaN: e is
                    rest[k][j] = v >= 0.0f ? e * r : r;
                    sum += x[k][j];
                }
            sum = lanes_sum(sum, lg);
        } else {
            top = lanes_max(top, lg);
            const float m = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[k][j] = __builtin_amdgcn_exp2f((x[k][j] - m) * LOG2E);
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
                    if (a.sigmoid) g[j] *= rest[k][j];
                    if (!live) g[j] = 0.0f;
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
        for (int w = 0; w < BLOCK / 64; ++w) {
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
        for (int e = threadIdx.x; e < experts; e += BLOCK) out[e] = part[e];
        if (threadIdx.x == 0)
            reinterpret_cast<Extra *>(a.workspace + p.extra)[slot].squares =
                (squares[0] + squares[1]) + (squares[2] + squares[3]);
    }
}

template <int DT, int K, bool SUMS, bool GRAD, bool TAIL>
__global__ __launch_bounds__(BLOCK) void balance_rows(BalanceArgs a, BalancePlan p, int lg) {
    constexpr bool SPLIT = split_stream<DT>;
    __shared__ float part[SUMS ? BALANCE_MAX_EXPERTS : 1];
    __shared__ double squares[BLOCK / 64];
    const int lane = threadIdx.x & ((1 << lg) - 1), mine = threadIdx.x >> lg;
    const int per = BLOCK >> lg;  // rows at a time
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
    const Rows piece = piece_of(a, p, blockIdx.x);
    if (piece.begin < piece.end) rows_of_piece<DT, K, SUMS, GRAD, TAIL>(a, p, piece, blockIdx.x, lg, part, squares);
}

// Mean probabilities of one group's sixteen columns.
__global__ __launch_bounds__(JOIN) void balance_join_probs(BalanceArgs a, BalancePlan p, int64_t g0) {
    __shared__ double strip[STRIPS][16];
    const int64_t g = g0 + blockIdx.y;
    int64_t first, count;
    pieces_of(a, p, g, &first, &count);
    const int c = threadIdx.x & 15, s = threadIdx.x >> 4;
    const int64_t e = int64_t(blockIdx.x) * 16 + c;
    const float *probs = reinterpret_cast<const float *>(a.workspace + p.probs);
    double sum = 0.0;
    if (e < a.experts) {
#pragma unroll 4
        for (int64_t i = s; i < count; i += STRIPS) sum += static_cast<double>(probs[(first + i) * p.width + e]);
    }
    strip[s][c] = sum;
    __syncthreads();
    if (s != 0 || e >= a.experts) return;
    for (int k = 1; k < STRIPS; ++k) sum += strip[k][c];
    a.mean_prob[g * a.experts + e] = static_cast<float>(sum / static_cast<double>(max(a.tokens[g], 1)));
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
        const Extra *extra = reinterpret_cast<const Extra *>(a.workspace + p.extra);
        for (int64_t i = lane; i < count; i += 64) squares += extra[first + i].squares;
        loss += a.z_coef / t * wave_sum64(squares);
    }
    return loss;
}

constexpr int LOSS_WAVES = 16;

__device__ __forceinline__ double weighted(const BalanceArgs &a, int64_t g, float loss) {
    const float w = a.weights ? a.weights[g] : 1.0f;
    return w != 0.0f ? static_cast<double>(w) * static_cast<double>(loss) : 0.0;
}

// The groups' losses, a wave to each, and where one workgroup has all of them
// the total, which adds the FP32 losses in FP64.
__global__ __launch_bounds__(LOSS_WAVES * 64) void balance_losses(BalanceArgs a, BalancePlan p) {
    __shared__ double part[LOSS_WAVES];
    const int wave = threadIdx.x >> 6;
    const int64_t g = int64_t(blockIdx.x) * LOSS_WAVES + wave;
    const bool here = g < a.groups;
    const float loss = here ? static_cast<float>(group_loss(a, p, g, threadIdx.x & 63)) : 0.0f;
    if ((threadIdx.x & 63) == 0) {
        if (here) a.loss[g] = loss;
        part[wave] = here ? weighted(a, g, loss) : 0.0;
    }
    if (gridDim.x > 1) return;
    __syncthreads();
    if (threadIdx.x == 0) {
        double sum = 0.0;
        for (int w = 0; w < LOSS_WAVES; ++w) sum += part[w];
        *a.total = static_cast<float>(sum);
    }
}

__global__ __launch_bounds__(LOSS_WAVES * 64) void balance_total(BalanceArgs a) {
    __shared__ double part[LOSS_WAVES];
    double sum = 0.0;
    for (int64_t g = threadIdx.x; g < a.groups; g += LOSS_WAVES * 64) sum += weighted(a, g, a.loss[g]);
    sum = wave_sum64(sum);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < LOSS_WAVES; ++w) sum += part[w];
        *a.total = static_cast<float>(sum);
    }
}

// All of a batch that is one piece of one group: what the workgroup writes to
// memory in one step it reads in the next, behind a barrier.
template <int DT, int K, bool GRAD, bool TAIL>
__global__ __launch_bounds__(BLOCK) void balance_single(BalanceArgs a, BalancePlan p, int lg) {
    __shared__ int32_t hist[BALANCE_MAX_EXPERTS];
    __shared__ float part[BALANCE_MAX_EXPERTS];
    __shared__ double squares[BLOCK / 64];
    __shared__ int32_t rows;
    const int experts = static_cast<int>(a.experts);
    const Rows piece = {0, 0, a.n};
    count_piece(a, piece, hist, &rows);
    for (int e = threadIdx.x; e < experts; e += BLOCK) a.counts[e] = hist[e];
    if (threadIdx.x == 0) a.tokens[0] = rows;
    __threadfence_block();
    __syncthreads();
    rows_of_piece<DT, K, true, GRAD, TAIL>(a, p, piece, 0, lg, part, squares);
    __threadfence_block();
    __syncthreads();
    const double t = max(rows, 1);
    for (int e = threadIdx.x; e < experts; e += BLOCK) a.mean_prob[e] = static_cast<float>(static_cast<double>(part[e]) / t);
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
static bool single(const BalanceArgs &a, const BalancePlan &p) {
    return a.n > 0 && p.pieces == 1 && !a.offsets && a.experts <= 512;
}

template <int DT, int K, bool SUMS, bool GRAD>
static void rows_at(const BalanceArgs &a, const BalancePlan &p, int lg, hipStream_t stream) {
    auto kernel = a.experts % 8 ? balance_rows<DT, K, SUMS, GRAD, true> : balance_rows<DT, K, SUMS, GRAD, false>;
    if constexpr (SUMS && K == 1) {
        if (single(a, p)) kernel = a.experts % 8 ? balance_single<DT, K, GRAD, true> : balance_single<DT, K, GRAD, false>;
    }
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(p.pieces)), dim3(BLOCK), 0, stream, a, p, lg);
}

template <int DT, bool SUMS, bool GRAD>
static void rows_with(const BalanceArgs &a, const BalancePlan &p, hipStream_t stream) {
    const int64_t eights = ceil_div(a.experts, 8);
    int lg = 0;
    while (lg < 6 && (int64_t(1) << lg) < eights) ++lg;
    if (eights <= 64) rows_at<DT, 1, SUMS, GRAD>(a, p, lg, stream);
    else if (eights <= 128) rows_at<DT, 2, SUMS, GRAD>(a, p, lg, stream);
    else if (eights <= 256) rows_at<DT, 4, SUMS, GRAD>(a, p, lg, stream);
    else rows_at<DT, 8, SUMS, GRAD>(a, p, lg, stream);
}

template <bool SUMS, bool GRAD>
static hipError_t rows_of(const BalanceArgs &a, const BalancePlan &p, int dt, hipStream_t stream, int *launched) {
    switch (dt) {
    case G_F32: rows_with<G_F32, SUMS, GRAD>(a, p, stream); break;
    case G_F16: rows_with<G_F16, SUMS, GRAD>(a, p, stream); break;
    default: rows_with<G_BF16, SUMS, GRAD>(a, p, stream); break;
    }
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) ++*launched;
    return e;
}

constexpr int64_t MAX_GRID_Y = 65535;

template <class KERNEL>
static hipError_t over_groups(KERNEL kernel, const BalanceArgs &a, const BalancePlan &p, hipStream_t stream, int *launched) {
    for (int64_t g0 = 0; g0 < a.groups; g0 += MAX_GRID_Y) {
        const dim3 grid(static_cast<unsigned>(p.width / 16), static_cast<unsigned>(min_of(a.groups - g0, MAX_GRID_Y)));
        hipLaunchKernelGGL(kernel, grid, dim3(JOIN), 0, stream, a, p, g0);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        ++*launched;
    }
    return hipSuccess;
}

hipError_t launch_balance_loss(const BalanceArgs &a, const BalancePlan &p, int dt, hipStream_t stream, int *launched) {
    hipError_t e;
    const dim3 grid(static_cast<unsigned>(p.pieces));
    if (single(a, p))
        return a.grad ? rows_of<true, true>(a, p, dt, stream, launched) : rows_of<true, false>(a, p, dt, stream, launched);
    if (a.n > 0) {
        hipLaunchKernelGGL(balance_count, grid, dim3(BLOCK), 0, stream, a, p);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        ++*launched;
    }
    if ((e = over_groups(balance_join_counts, a, p, stream, launched)) != hipSuccess) return e;
    if (a.n > 0) {
        e = a.grad ? rows_of<true, true>(a, p, dt, stream, launched) : rows_of<true, false>(a, p, dt, stream, launched);
        if (e != hipSuccess) return e;
    }
    if ((e = over_groups(balance_join_probs, a, p, stream, launched)) != hipSuccess) return e;
    hipLaunchKernelGGL(balance_losses, dim3(static_cast<unsigned>(ceil_div(a.groups, LOSS_WAVES))), dim3(LOSS_WAVES * 64), 0,
                       stream, a, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    ++*launched;
    if (a.groups <= LOSS_WAVES) return hipSuccess;
    hipLaunchKernelGGL(balance_total, dim3(1), dim3(LOSS_WAVES * 64), 0, stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    ++*launched;
    return hipSuccess;
}

hipError_t launch_balance_grad(const BalanceArgs &a, const BalancePlan &p, int dt, hipStream_t stream, int *launched) {
    return rows_of<false, true>(a, p, dt, stream, launched);
}

}  // namespace radamw
