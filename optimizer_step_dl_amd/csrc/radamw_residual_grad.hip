// radamw_residual_grad.hip -- the gradient of the residual stream's norms
// around one block (radamw_residual.hip) for gfx950.
//
//   D        = dh + r_h (q - hat_h mean(q hat_h)),  q = dout (o + w_pre),
//                                                   hat_h = h r_h
//   dx       = D
//   b        = scale * drop'(D),  dgate = b u,  du = b gate
//   dbranch  = r_b (s - hat_b mean(s hat_b)),       s = du (o + w_post),
//                                                   hat_b = branch r_b
//   dw_pre   = sum over rows of dout hat_h,  dw_post = of du hat_b
//
// Bound by HBM: four or five arrays in, two or three out, each moved once.
// A worker (a row's lanes) takes a run of rows and keeps its columns' sums in
// registers; what it leaves per column is joined by a second launch.  An
// absent norm or gate is arithmetic with 1 and 0 rather than a branch around
// each value.
#include "radamw_residual.h"

namespace radamw {

// The most workers (each a row's lanes), and the least rows of one where
// there are more rows than CUs: a worker leaves 4 bytes per column and sum,
// read again by the join, against 12 to 24 bytes per column and row.
constexpr int64_t GRAD_WORKERS = 1024;
constexpr int64_t GRAD_ROWS = 4;

ResidualPlan residual_plan(int64_t n, int64_t dim, int64_t) {
    ResidualPlan p{};
    const int64_t most = n < 256 ? n : n / GRAD_ROWS < 256 ? 256 : n / GRAD_ROWS < GRAD_WORKERS ? n / GRAD_ROWS : GRAD_WORKERS;
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

// A worker's column sums, whole pieces: a partial row has room for them.
template <int NT, int K>
__device__ __forceinline__ void put_partial(char *base, int64_t slot, int64_t width, int lane, const f32x8 (&acc)[K]) {
    float *row = reinterpret_cast<float *>(base) + slot * width;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int32_t e = (lane + k * NT) * 8;
        if (e < width) store8<G_F32>(row, e, acc[k]);
    }
}

// One worker's rows, in order.  The gate's sum is one per gate row: where the
// gate row's rows all belong to this worker it is stored, else it is left in
// slot 0 (the gate row began before this worker) or 1 (it goes on behind it).
template <int SDT, int BDT, int NT, int K, bool TAIL>
__global__ __launch_bounds__(row_block<NT>) void residual_norm_grad(ResidualGradArgs a, ResidualPlan p) {
    __shared__ float part[2][row_block<NT> / 64];
    const int lane = threadIdx.x % NT;
    const int32_t dim = static_cast<int32_t>(a.dim);
    const int64_t w = int64_t(blockIdx.x) * (row_block<NT> / NT) + wave_row<NT>();
    const int64_t begin = w * p.rows, end = begin + p.rows < a.n ? begin + p.rows : a.n;
    if (begin >= end) return;  // whole waves; with NT > 64 whole workgroups
    const float inv_dim = 1.0f / static_cast<float>(dim);
    const float drop_scale = a.scale * a.drop.factor;
    f32x8 post[K], pre[K], gate[K], sum_post[K], sum_pre[K], sum_gate[K];
    Raw8<BDT> g[K], y[K];
    Raw8<SDT> h[K], dh[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int32_t e = (lane + k * NT) * 8;
        post[k] = pre[k] = gate[k] = all_of(1.0f);
        sum_post[k] = sum_pre[k] = sum_gate[k] = f32x8{};
        g[k] = y[k] = Raw8<BDT>{};
        h[k] = dh[k] = Raw8<SDT>{};
        if (e >= dim) continue;
        if (a.post) post[k] = load_any<TAIL>(static_cast<const char *>(a.post), a.weight_dt, e, dim, a.weight_offset);
        if (a.pre) pre[k] = load_any<TAIL>(static_cast<const char *>(a.pre), a.weight_dt, e, dim, a.weight_offset);
    }
    // the gate row of row t, and the first row behind it
    int64_t group = a.gate ? begin / a.per : 0, next = begin;
    for (int64_t t = begin; t < end; ++t) {
        if (a.gate && t == next) {
            if (t != begin) ++group;
            next = (group + 1) * a.per;
            const char *row = elem_at(a.gate, a.gate_dt, group * a.gate_stride);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int32_t e = (lane + k * NT) * 8;
                if (e < dim) gate[k] = load_any<TAIL>(row, a.gate_dt, e, dim, 0.0f);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int32_t e = (lane + k * NT) * 8;
            if (e >= dim) continue;
            if (a.pre) {
                g[k] = load_piece<BDT, TAIL>(elem_at(a.grad_out, BDT, t * a.grad_out_stride), e, dim);
                h[k] = load_piece<SDT, TAIL>(elem_at(a.h, SDT, t * a.h_stride), e, dim);
            }
            if (a.grad_h) dh[k] = load_piece<SDT, TAIL>(elem_at(a.grad_h, SDT, t * a.grad_h_stride), e, dim);
            if (a.branch) y[k] = load_piece<BDT, TAIL>(elem_at(a.branch, BDT, t * a.branch_stride), e, dim);
        }
        // D, and the sums of the norm behind the stream's sum
        float rh = 0.0f, mean = 0.0f;
        if (a.pre) {
            rh = a.rstd[a.n + t];
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float c = raw_value<BDT>(g[k], j) * (raw_value<SDT>(h[k], j) * rh);
                    sum_pre[k][j] += c;
                    s = __builtin_fmaf(c, pre[k][j], s);
                }
            mean = row_sum<NT>(s, part[0]) * inv_dim;
        }
        const float rb = a.post ? a.rstd[t] : 1.0f;
        float s = 0.0f;
        f32x8 du[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int32_t e = (lane + k * NT) * 8;
            if (e >= dim) continue;
            f32x8 d;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float q = raw_value<BDT>(g[k], j) * pre[k][j], hat = raw_value<SDT>(h[k], j) * rh;
                d[j] = __builtin_fmaf(rh, __builtin_fmaf(-hat, mean, q), raw_value<SDT>(dh[k], j));
            }
            store_piece<SDT, TAIL>(elem_at(a.grad_x, SDT, t * a.grad_x_stride), e, dim, d);
            if (!a.branch) continue;
            u32x4 words = {0, 0, 0, 0};
            if (a.drop.threshold) words = random_words(static_cast<uint32_t>(e >> 3), static_cast<uint32_t>(t), a.drop);
            f32x8 dg;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // a dropped place passes nothing on, whatever the branch holds there
                const bool keep = kept(words, j, a.drop.threshold);
                const float hat = raw_value<BDT>(y[k], j) * rb, b = d[j] * drop_scale;
                dg[j] = keep ? b * (hat * post[k][j]) : 0.0f;
                sum_gate[k][j] += dg[j];
                const float c = keep ? b * gate[k][j] : 0.0f;
                sum_post[k][j] = __builtin_fmaf(c, hat, sum_post[k][j]);
                du[k][j] = c * post[k][j];
                s = __builtin_fmaf(du[k][j], hat, s);
            }
            if (a.grad_gate && a.per == 1)
                store_any<TAIL>(elem_at(a.grad_gate, a.gate_dt, t * a.grad_gate_stride), a.gate_dt, e, dim, dg);
        }
        if (a.branch) {
            float mb = 0.0f;
            if (a.post) mb = row_sum<NT>(s, part[1]) * inv_dim * rb;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int32_t e = (lane + k * NT) * 8;
                if (e >= dim) continue;
                if (a.post) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        du[k][j] = rb * __builtin_fmaf(-raw_value<BDT>(y[k], j), mb, du[k][j]);
                }
                store_piece<BDT, TAIL>(elem_at(a.grad_branch, BDT, t * a.grad_branch_stride), e, dim, du[k]);
            }
        }
        if constexpr (NT > 64) {
            // the next row's first sum writes part[0] again: with one norm
            // alone no other barrier stands between its reads and that write
            if (!(a.pre && a.post)) __syncthreads();
        }
        if (a.grad_gate && (t + 1 == end || t + 1 == next)) {
            const int64_t from = group * a.per, to = next < a.n ? next : a.n;
            if (a.per == 1) {
                // stored above
            } else if (from >= begin && to <= end) {
                char *row = elem_at(a.grad_gate, a.gate_dt, group * a.grad_gate_stride);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int32_t e = (lane + k * NT) * 8;
                    if (e < dim) store_any<TAIL>(row, a.gate_dt, e, dim, sum_gate[k]);
                }
            } else {
                put_partial<NT>(a.workspace + p.gate, 2 * w + (from >= begin), p.width, lane, sum_gate);
            }
#pragma unroll
            for (int k = 0; k < K; ++k) sum_gate[k] = f32x8{};
        }
    }
    if (a.grad_post) put_partial<NT>(a.workspace + p.post, w, p.width, lane, sum_post);
    if (a.grad_pre) put_partial<NT>(a.workspace + p.pre, w, p.width, lane, sum_pre);
}

// Sums of partial rows, 64 columns to a workgroup: 16 lanes of four columns,
// 16 strips of partial rows; FP64.
constexpr int JOIN_BLOCK = 256;
constexpr int JOIN_COLUMNS = 64;

__device__ __forceinline__ void join_rows(const float *first, const float *rest, int64_t count, int64_t step, int64_t dim,
                                          void *out, int32_t dt, int64_t row) {
    // partial row 0 is `first`, partial row i > 0 is rest + (i - 1) * step
    __shared__ double strip[16][JOIN_COLUMNS];
    const int c = (threadIdx.x & 15) * 4, s = threadIdx.x >> 4;
    const int64_t e = int64_t(blockIdx.x) * JOIN_COLUMNS + c;
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    for (int64_t i = s; i < count; i += 16) {
        const float *src = i == 0 ? first : rest + (i - 1) * step;
        const f32x4 v = *(const RADAMW_GLOBAL f32x4 *)(src + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += static_cast<double>(v[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) strip[s][c + j] = acc[j];
    __syncthreads();
    if (threadIdx.x < JOIN_COLUMNS) {
        double v = 0.0;
#pragma unroll
        for (int k = 0; k < 16; ++k) v += strip[k][threadIdx.x];
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

template <int SDT, int BDT, int NT, int K>
static void residual_grad_at(const ResidualGradArgs &a, const ResidualPlan &p, hipStream_t stream) {
    const auto kernel = a.dim % 8 ? residual_norm_grad<SDT, BDT, NT, K, true> : residual_norm_grad<SDT, BDT, NT, K, false>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(ceil_div(p.workers, row_block<NT> / NT))), dim3(row_block<NT>), 0,
                       stream, a, p);
}

template <int SDT, int BDT>
static hipError_t residual_grad_rows(const ResidualGradArgs &a, const ResidualPlan &p, hipStream_t stream) {
#define RADAMW_CALL(NT, K) residual_grad_at<SDT, BDT, NT, K>(a, p, stream)
    RADAMW_ROW_SHAPES(a.dim, RADAMW_CALL)
#undef RADAMW_CALL
    return hipGetLastError();
}

hipError_t launch_residual_grad(const ResidualGradArgs &a, const ResidualPlan &p, int sdt, int bdt, hipStream_t stream,
                                int *launched) {
    hipError_t e = hipSuccess;
    if (a.n > 0) {
        if (sdt == bdt) {
            switch (bdt) {
            case G_F32: e = residual_grad_rows<G_F32, G_F32>(a, p, stream); break;
            case G_F16: e = residual_grad_rows<G_F16, G_F16>(a, p, stream); break;
            default: e = residual_grad_rows<G_BF16, G_BF16>(a, p, stream); break;
            }
        } else if (bdt == G_F16) {
            e = residual_grad_rows<G_F32, G_F16>(a, p, stream);
        } else {
            e = residual_grad_rows<G_F32, G_BF16>(a, p, stream);
        }
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
