// radamw_residual.hip -- the residual stream around one block for gfx950:
// the norm behind the block, its dropout, gate and scale, the sum, and the
// norm before the next block, in one pass.
//
//   u   = branch * r_b * (o + w_post),   r_b = 1 / sqrt(mean branch^2 + eps)
//   h   = x + scale * gate * drop(u)
//   out = h * r_h * (o + w_pre),         r_h = 1 / sqrt(mean h^2 + eps)
//
// A row is held in registers between its two sums, so each array is moved
// once; all of it is bound by HBM.  32768 x 8192 BF16 rows with both norms and
// a gate per sequence take 365 us (2.15 GB: 5.9 TB/s), 8192 x 4096 with an FP32
// stream, FP32 weights and dropout 77 us (403 MB: 5.2 TB/s; 72 us with 16-bit
// weights, whose loads are half as long).
//
// What was measured against this shape at those two sizes (365 and 77 us):
// workgroups that stay and load the next row ahead 360 and 75 to 84 us, but 53
// against 49 us for 65536 x 512 and 66 against 55 us without norms; a wave to
// each row, no barriers, 450 and 86 us; four rows at a time 440 and 94 us;
// fewer workgroups per CU no gain.
#include "radamw_residual.h"

namespace radamw {

// Of a branch whose reciprocal root is NaN dropout may drop every column of the
// row and yet keep some that lie behind it in the last lanes' pieces, which are
// no part of the row's sum.  So such a root is taken into the row's own values,
// all of them NaN then, and 1 is left of it.
template <int DT>
__device__ __forceinline__ void take_nan(Raw8<DT> &r, float &root, Piece e, int32_t dim) {
    root = 1.0f;
#pragma unroll
    for (int j = 0; j < 8; j += DT == G_F32 ? 1 : 2) {
        const int32_t c = j < 4 ? e.e + j : e.e2 + j - 4;
        if constexpr (DT == G_F32) r.c[j / 4][j % 4] = c < dim ? 0x7fc00000u : 0u;
        else r.c[0][j / 2] = (c < dim ? 0x7fffu : 0u) | (c + 1 < dim ? 0x7fff0000u : 0u);
    }
}

// NT lanes hold a row, K pieces of eight each.
template <int SDT, int BDT, int NT, int K, bool TAIL>
__global__ __launch_bounds__(row_block<NT>) void residual_norm(ResidualArgs a, int64_t row0) {
    constexpr bool SPLIT = split_stream<SDT>;
    __shared__ float part[2][row_block<NT> / 64];
    const int lane = threadIdx.x % NT;
    const int32_t dim = static_cast<int32_t>(a.dim);
    const int64_t t = row0 + int64_t(blockIdx.x) * (row_block<NT> / NT) + wave_row<NT>();
    if (t >= a.n) return;  // whole waves; with NT > 64 whole workgroups
    const char *xr = elem_at(a.x, SDT, t * a.x_stride), *yr = elem_at(a.branch, BDT, t * a.branch_stride);
    const char *gr = elem_at(a.gate, a.gate_dt, a.gate ? t / a.per * a.gate_stride : 0);
    const auto post_at = [&](Piece e) {
        return a.post ? load_weight<SPLIT, TAIL>(a.post, a.weight_dt, e, dim, a.weight_offset) : all_of(1.0f);
    };
    const auto pre_at = [&](Piece e) {
        return load_weight<SPLIT, TAIL>(a.pre, a.weight_dt, e, dim, a.weight_offset);
    };
    const auto gate_at = [&](Piece e) {
        return a.gate ? load_weight<SPLIT, TAIL>(gr, a.gate_dt, e, dim, 0.0f) : all_of(1.0f);
    };
    Raw8<SDT> x[K];
    Raw8<BDT> y[K];
    // with one piece to a lane there is room to load everything at once
    f32x8 gate, post, pre;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Piece e = piece_at<SPLIT, NT>(lane, k);
        y[k] = Raw8<BDT>{};
        if (e.e >= dim) continue;
        if (a.branch) y[k] = load_piece<BDT, SPLIT, TAIL>(yr, e, dim);
        x[k] = load_piece<SDT, SPLIT, TAIL>(xr, e, dim);
        if constexpr (K == 1) {
            post = post_at(e);
            gate = gate_at(e);
            if (a.pre) pre = pre_at(e);
        }
    }
    const float inv_dim = 1.0f / static_cast<float>(dim);
    float rb = 1.0f;
    if (a.post) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = raw_value<BDT>(y[k], j);
                s = __builtin_fmaf(v, v, s);
            }
        s = row_sum<NT>(s, part[0]);
        rb = rsqrtf(__builtin_fmaf(s, inv_dim, a.eps));
        if (a.rstd && lane == 0) a.rstd[t] = rb;
        if ((SPLIT || TAIL) && rb != rb) {
#pragma unroll
            for (int k = 0; k < K; ++k) take_nan<BDT>(y[k], rb, piece_at<SPLIT, NT>(lane, k), dim);
        }
    }
    f32x8 h[K];
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Piece e = piece_at<SPLIT, NT>(lane, k);
        if (e.e >= dim) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[k][j] = raw_value<SDT>(x[k], j);
        if (a.branch) {
            if constexpr (K > 1) {
                post = post_at(e);
                gate = gate_at(e);
            }
            u32x4 words = {0, 0, 0, 0};
            if (a.drop.threshold) words = piece_words<SPLIT>(e, t, a.drop);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = raw_value<BDT>(y[k], j) * rb * post[j] * gate[j] * a.drop.factor;
                h[k][j] = __builtin_fmaf(a.scale, kept(words, j, a.drop.threshold) ? u : 0.0f, h[k][j]);
            }
            store_piece<SDT, SPLIT, TAIL>(elem_at(a.h, SDT, t * a.h_stride), e, dim, h[k]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __builtin_fmaf(h[k][j], h[k][j], s);
    }
    if (!a.pre) return;
    s = row_sum<NT>(s, part[1]);
    const float rh = rsqrtf(__builtin_fmaf(s, inv_dim, a.eps));
    if (a.rstd && lane == 0) a.rstd[a.n + t] = rh;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Piece e = piece_at<SPLIT, NT>(lane, k);
        if (e.e >= dim) continue;
        if constexpr (K > 1) pre = pre_at(e);
        f32x8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = h[k][j] * rh * pre[j];
        store_piece<BDT, SPLIT, TAIL>(elem_at(a.out, BDT, t * a.out_stride), e, dim, v);
    }
}

// Two rows at a time, a piece of each to a lane: they share the weights' loads
// and the barriers.
template <int SDT, int BDT, int NT, bool TAIL>
__global__ __launch_bounds__(row_block<NT>) void residual_norm_pair(ResidualArgs a, int64_t row0) {
    constexpr bool SPLIT = split_stream<SDT>;
    __shared__ float part[2][2 * row_block<NT> / 64];
    const int lane = threadIdx.x % NT;
    const int32_t dim = static_cast<int32_t>(a.dim);
    const Piece e = piece_at<SPLIT, NT>(lane, 0);
    const int64_t t0 = row0 + (int64_t(blockIdx.x) * (row_block<NT> / NT) + wave_row<NT>()) * 2;
    if (t0 >= a.n) return;  // whole waves; with NT > 64 whole workgroups
    // behind the last row that row is read again and nothing stored
    const bool both = t0 + 1 < a.n, here = e.e < dim;
    const int64_t t[2] = {t0, both ? t0 + 1 : t0};
    Raw8<SDT> x[2];
    Raw8<BDT> y[2] = {};
    f32x8 gate[2], post, pre;
    post = gate[0] = gate[1] = all_of(1.0f);
    if (here) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (a.branch) y[m] = load_piece<BDT, SPLIT, TAIL>(elem_at(a.branch, BDT, t[m] * a.branch_stride), e, dim);
            x[m] = load_piece<SDT, SPLIT, TAIL>(elem_at(a.x, SDT, t[m] * a.x_stride), e, dim);
        }
        if (a.post) post = load_weight<SPLIT, TAIL>(a.post, a.weight_dt, e, dim, a.weight_offset);
        if (a.gate) {
            const uint32_t g0 = static_cast<uint32_t>(t[0]) / static_cast<uint32_t>(a.per),
                           g1 = static_cast<uint32_t>(t[1]) / static_cast<uint32_t>(a.per);
            gate[0] = load_weight<SPLIT, TAIL>(elem_at(a.gate, a.gate_dt, g0 * a.gate_stride), a.gate_dt, e, dim, 0.0f);
            gate[1] = g1 == g0 ? gate[0]
                               : load_weight<SPLIT, TAIL>(elem_at(a.gate, a.gate_dt, g1 * a.gate_stride), a.gate_dt, e, dim, 0.0f);
        }
        if (a.pre) pre = load_weight<SPLIT, TAIL>(a.pre, a.weight_dt, e, dim, a.weight_offset);
    }
    const float inv_dim = 1.0f / static_cast<float>(dim);
    float rb[2] = {1.0f, 1.0f}, s[2] = {0.0f, 0.0f};
    if (a.post) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = raw_value<BDT>(y[m], j);
                s[m] = __builtin_fmaf(v, v, s[m]);
            }
        row_sums<NT>(s[0], s[1], part[0]);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            rb[m] = rsqrtf(__builtin_fmaf(s[m], inv_dim, a.eps));
            if (a.rstd && lane == 0) a.rstd[t[m]] = rb[m];
            s[m] = 0.0f;
        }
        if ((SPLIT || TAIL) && (rb[0] != rb[0] || rb[1] != rb[1])) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
                if (rb[m] != rb[m]) take_nan<BDT>(y[m], rb[m], e, dim);
        }
    }
    f32x8 h[2];
    if (here) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[m][j] = raw_value<SDT>(x[m], j);
            if (a.branch) {
                u32x4 words = {0, 0, 0, 0};
                if (a.drop.threshold)
                    words = piece_words<SPLIT>(e, t[m], a.drop);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float u = raw_value<BDT>(y[m], j) * rb[m] * post[j] * gate[m][j] * a.drop.factor;
                    h[m][j] = __builtin_fmaf(a.scale, kept(words, j, a.drop.threshold) ? u : 0.0f, h[m][j]);
                }
                if (m == 0 || both) store_piece<SDT, SPLIT, TAIL>(elem_at(a.h, SDT, t[m] * a.h_stride), e, dim, h[m]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s[m] = __builtin_fmaf(h[m][j], h[m][j], s[m]);
        }
    }
    if (!a.pre) return;
    row_sums<NT>(s[0], s[1], part[1]);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const float rh = rsqrtf(__builtin_fmaf(s[m], inv_dim, a.eps));
        if (a.rstd && lane == 0) a.rstd[a.n + t[m]] = rh;
        if (!here || (m == 1 && !both)) continue;
        f32x8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = h[m][j] * rh * pre[j];
        store_piece<BDT, SPLIT, TAIL>(elem_at(a.out, BDT, t[m] * a.out_stride), e, dim, v);
    }
}

// Two rows at a time where that leaves four workgroups per CU (up to 512
// columns one, of eight rows): 8192 x 4096
// (FP32 stream, BF16 branch, FP32 weights) takes 77 us, against 84 us, 65536 x
// 2048 BF16 186 against 197 us.  Wider rows have no registers for two.
constexpr int64_t PAIR_ROWS = 2048;
// Rows of one launch.
constexpr int64_t RESIDUAL_LAUNCH_ROWS = int64_t(1) << 21;

template <int SDT, int BDT, int NT, int K>
static hipError_t residual_at(const ResidualArgs &a, hipStream_t stream, int *launched) {
    auto kernel = a.dim % 8 ? residual_norm<SDT, BDT, NT, K, true> : residual_norm<SDT, BDT, NT, K, false>;
    int rows_of_block = row_block<NT> / NT;
    if constexpr (K == 1) {
        if (a.n >= PAIR_ROWS) {
            kernel = a.dim % 8 ? residual_norm_pair<SDT, BDT, NT, true> : residual_norm_pair<SDT, BDT, NT, false>;
            rows_of_block *= 2;
        }
    }
    for (int64_t row0 = 0; row0 < a.n; row0 += RESIDUAL_LAUNCH_ROWS) {
        const int64_t rows = a.n - row0 < RESIDUAL_LAUNCH_ROWS ? a.n - row0 : RESIDUAL_LAUNCH_ROWS;
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(ceil_div(rows, rows_of_block))), dim3(row_block<NT>), 0,
                           stream, a, row0);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        ++*launched;
    }
    return hipSuccess;
}

template <int SDT, int BDT>
static hipError_t residual_shape(const ResidualArgs &a, hipStream_t stream, int *launched) {
#define RADAMW_CALL(NT, K) return residual_at<SDT, BDT, NT, K>(a, stream, launched)
    // 32768 x 8192 BF16 rows take 365 us, against 432 us with 1024 lanes of one
    // piece and 381 us with 256 of four
    RADAMW_ROW_SHAPES(a.dim, RADAMW_CALL, RADAMW_CALL(512, 2))
#undef RADAMW_CALL
}

hipError_t launch_residual(const ResidualArgs &a, int sdt, int bdt, hipStream_t stream, int *launched) {
    if (sdt == bdt) {
        switch (bdt) {
        case G_F32: return residual_shape<G_F32, G_F32>(a, stream, launched);
        case G_F16: return residual_shape<G_F16, G_F16>(a, stream, launched);
        default: return residual_shape<G_BF16, G_BF16>(a, stream, launched);
        }
    }
    return bdt == G_F16 ? residual_shape<G_F32, G_F16>(a, stream, launched)
                        : residual_shape<G_F32, G_BF16>(a, stream, launched);
}

}  // namespace radamw
