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
// logits and one write.  262144 x 256 FP32 logits with their gradient take 132
// us (554 MB: 4.2 TB/s), 107 us of it in balance_rows (537 MB: 5.0 TB/s), the
// rest in the count, the joins and the loss.  16383 x 160 in 13 groups take 33
// us, 19 us of it in balance_rows: there a row's mask, logits, sums over lanes
// and store wait for one another, and five launches do.
#include "radamw_balance.h"

namespace radamw {

namespace {

constexpr int64_t max_of(int64_t a, int64_t b) { return a > b ? a : b; }
constexpr int64_t min_of(int64_t a, int64_t b) { return a < b ? a : b; }

int64_t up256(int64_t v) { return ceil_div(v, 256) * 256; }

}  // namespace

BalancePlan balance_plan(int64_t n, int64_t experts, int64_t groups) {
    BalancePlan p{};
    // one piece of up to 16384 values, which one workgroup does in one launch;
    // of more, at least 512 pieces where that leaves each 2048 values, and
    // about 1024 of a long batch: 16383 x 160 take 33 us, against 40 us with
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

// -------------------------------------------------------------- counting --

__global__ __launch_bounds__(BALANCE_BLOCK) void balance_count(BalanceArgs a, BalancePlan p) {
    __shared__ int32_t hist[BALANCE_MAX_EXPERTS];
    __shared__ int32_t rows;
    const BalanceRows piece = piece_of(a, p, blockIdx.x);
    if (piece.begin >= piece.end) return;
    count_piece(a, piece, hist, &rows);
    int32_t *out = reinterpret_cast<int32_t *>(a.workspace + p.counts) + blockIdx.x * p.width;
    for (int e = threadIdx.x; e < a.experts; e += BALANCE_BLOCK) out[e] = hist[e];
    if (threadIdx.x == 0) reinterpret_cast<BalanceExtra *>(a.workspace + p.extra)[blockIdx.x].rows = rows;
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
    const BalanceExtra *extra = reinterpret_cast<const BalanceExtra *>(a.workspace + p.extra);
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

constexpr int LOSS_WAVES = 16;

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

// ---------------------------------------------------------------- launch --

static hipError_t rows_of(const BalanceArgs &a, const BalancePlan &p, bool sums, int dt, hipStream_t stream,
                          int *launched) {
    const hipError_t e = a.sigmoid ? balance_rows_sigmoid(a, p, sums, dt, stream)
                                   : balance_rows_of<false>(a, p, sums, dt, stream);
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
    if (balance_at_once(a, p)) return rows_of(a, p, true, dt, stream, launched);
    if (a.n > 0) {
        hipLaunchKernelGGL(balance_count, grid, dim3(BALANCE_BLOCK), 0, stream, a, p);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        ++*launched;
    }
    if ((e = over_groups(balance_join_counts, a, p, stream, launched)) != hipSuccess) return e;
    if (a.n > 0 && (e = rows_of(a, p, true, dt, stream, launched)) != hipSuccess) return e;
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
    return rows_of(a, p, false, dt, stream, launched);
}

}  // namespace radamw
