// radamw_residual_grad.hip -- the gradient of the residual stream's norms
// around one block for gfx950 (the kernel is in radamw_residual_grad.h): the
// workers, FP32 alone, the join of the workers' sums, the launches.
#include "radamw_residual_grad.h"

namespace radamw {

// Waves per CU of the gradient (128 registers each leave room for sixteen), and
// the least rows of a worker (a row's lanes) where there are more rows than
// CUs: a worker leaves 4 bytes per column and sum, read again by the join,
// against 12 to 24 bytes per column and row.
constexpr int64_t GRAD_WAVES = 16;
constexpr int64_t GRAD_ROWS = 4;

ResidualPlan residual_plan(int64_t n, int64_t dim, int64_t) {
    ResidualPlan p{};
    int64_t lanes = 64;
    while (lanes < 1024 && lanes * 8 < dim) lanes *= 2;
    const int64_t resident = 256 * GRAD_WAVES * 64 / lanes;
    const int64_t most = n < 256 ? n : n / GRAD_ROWS < 256 ? 256 : n / GRAD_ROWS < resident ? n / GRAD_ROWS : resident;
    p.rows = n > 0 ? ceil_div(n, most) : 1;
    p.workers = ceil_div(n, p.rows);
    p.width = ceil_div(dim, 64) * 64;
    const int64_t one = p.workers * p.width * 4;
    p.post = 0;
    p.pre = one;
    p.gate = 2 * one;
    p.bytes = 4 * one > 0 ? 4 * one : 16;
    return p;
}

// Sums of partial rows in FP64, 32 columns (a cache line) to a workgroup: 8
// lanes of four columns, 32 strips of partial rows.
constexpr int JOIN_BLOCK = 256;
constexpr int JOIN_COLUMNS = 32;
constexpr int JOIN_STRIPS = JOIN_BLOCK / (JOIN_COLUMNS / 4);

__device__ __forceinline__ void join_rows(const float *first, const float *rest, int64_t count, int64_t step, int64_t dim,
                                          void *out, int32_t dt, int64_t row) {
    // partial row 0 is `first`, partial row i > 0 is rest + (i - 1) * step
    __shared__ double strip[JOIN_STRIPS][JOIN_COLUMNS];
    const int c = (threadIdx.x % (JOIN_COLUMNS / 4)) * 4, s = threadIdx.x / (JOIN_COLUMNS / 4);
    const int64_t e = int64_t(blockIdx.x) * JOIN_COLUMNS + c;
    const auto at = [&](int64_t i) {
        const float *src = i == 0 ? first : rest + (i - 1) * step;
        return *(const RADAMW_GLOBAL f32x4 *)(src + e);
    };
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    int64_t i = s;
    for (; i + 3 * JOIN_STRIPS < count; i += 4 * JOIN_STRIPS) {
        f32x4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = at(i + u * JOIN_STRIPS);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] += static_cast<double>(v[u][j]);
    }
    for (; i < count; i += JOIN_STRIPS) {
        const f32x4 v = at(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += static_cast<double>(v[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) strip[s][c + j] = acc[j];
    __syncthreads();
    if (threadIdx.x < JOIN_COLUMNS) {
        double v = 0.0;
#pragma unroll
        for (int k = 0; k < JOIN_STRIPS; ++k) v += strip[k][threadIdx.x];
        const int64_t col = int64_t(blockIdx.x) * JOIN_COLUMNS + threadIdx.x;
        if (col < dim) {
            const float f = static_cast<float>(v);
            if (dt == G_F32) store_value<G_F32>(out, row + col, f);
            else if (dt == G_F16) store_value<G_F16>(out, row + col, f);
            else store_value<G_BF16>(out, row + col, f);
        }
    }
}

// blockIdx.y: 0 and 1 the weights, then the gate rows that several workers
// share: gate row y - 2 where `by_group`, else the last one of worker y - 2.
__global__ __launch_bounds__(JOIN_BLOCK) void residual_join(ResidualGradArgs a, ResidualPlan p, int64_t y0, int by_group) {
    const int64_t y = y0 + blockIdx.y;
    if (y < 2) {
        void *out = y == 0 ? a.grad_post : a.grad_pre;
        const float *rows = reinterpret_cast<const float *>(a.workspace + (y == 0 ? p.post : p.pre));
        if (out) join_rows(rows, rows + p.width, p.workers, p.width, a.dim, out, a.weight_dt, 0);
        return;
    }
    int64_t group = y - 2;
    if (!by_group) {
        const int64_t last = (y - 1) * p.rows - 1;
        if (last >= a.n) return;
        group = last / a.per;
    }
    const int64_t from = group * a.per, to = from + a.per < a.n ? from + a.per : a.n;
    const int64_t w0 = from / p.rows, w1 = (to - 1) / p.rows;
    if (w0 == w1 || (!by_group && w0 != y - 2)) return;
    const float *rows = reinterpret_cast<const float *>(a.workspace + p.gate);
    join_rows(rows + (2 * w0 + 1) * p.width, rows + 2 * (w0 + 1) * p.width, w1 - w0 + 1, 2 * p.width, a.dim, a.grad_gate,
              a.gate_dt, group * a.grad_gate_stride);
}

hipError_t launch_residual_grad(const ResidualGradArgs &a, const ResidualPlan &p, int sdt, int bdt, hipStream_t stream,
                                int *launched) {
    hipError_t e = hipSuccess;
    if (a.n > 0) {
        if (sdt == G_F32 && bdt == G_F32) e = residual_grad_rows<G_F32, G_F32>(a, p, stream);
        else if (sdt == G_F32) e = bdt == G_F16 ? residual_grad_f32_f16(a, p, stream) : residual_grad_f32_bf16(a, p, stream);
        else e = bdt == G_F16 ? residual_grad_f16(a, p, stream) : residual_grad_bf16(a, p, stream);
        if (e != hipSuccess) return e;
        ++*launched;
    }
    const bool weights = a.grad_post || a.grad_pre;
    const int64_t groups = a.grad_gate && a.per != 1 ? ceil_div(a.n, a.per) : 0;
    const int by_group = groups <= p.workers;
    // no gate row is shared where a worker has all rows
    const int64_t shared = p.workers > 1 ? (by_group ? groups : p.workers) : 0;
    const int64_t from = weights ? 0 : 2, to = 2 + shared;
    if (from >= to) return hipSuccess;
    hipLaunchKernelGGL(residual_join, dim3(static_cast<unsigned>(p.width / JOIN_COLUMNS), static_cast<unsigned>(to - from)),
                       dim3(JOIN_BLOCK), 0, stream, a, p, from, by_group);
    if ((e = hipGetLastError()) == hipSuccess) ++*launched;
    return e;
}

}  // namespace radamw
