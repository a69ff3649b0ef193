// radamw_residual.hip -- the residual stream around one block for gfx950:
// the norm behind the block, its dropout, gate and scale, the sum, and the
// norm before the next block, in one pass.
//
//   u   = branch * r_b * (o + w_post),   r_b = 1 / sqrt(mean branch^2 + eps)
//   h   = x + scale * gate * drop(u)
//   out = h * r_h * (o + w_pre),         r_h = 1 / sqrt(mean h^2 + eps)
//
// A row is held in registers between its two sums, so each array is moved
// once; all of it is bound by HBM.
#include "radamw_residual.h"

namespace radamw {

// NT lanes hold a row, K pieces of eight each.
template <int SDT, int BDT, int NT, int K, bool TAIL>
__global__ __launch_bounds__(row_block<NT>) void residual_norm(ResidualArgs a, int64_t row0) {
    __shared__ float part[2][row_block<NT> / 64];
    const int lane = threadIdx.x % NT;
    const int32_t dim = static_cast<int32_t>(a.dim);
    const int64_t t = row0 + int64_t(blockIdx.x) * (row_block<NT> / NT) + wave_row<NT>();
    if (t >= a.n) return;  // whole waves; with NT > 64 whole workgroups
    const char *xr = elem_at(a.x, SDT, t * a.x_stride), *yr = elem_at(a.branch, BDT, t * a.branch_stride);
    const char *gr = elem_at(a.gate, a.gate_dt, a.gate ? t / a.per * a.gate_stride : 0);
    const auto post_at = [&](int32_t e) {
        return a.post ? load_any<TAIL>(static_cast<const char *>(a.post), a.weight_dt, e, dim, a.weight_offset) : all_of(1.0f);
    };
    const auto pre_at = [&](int32_t e) {
        return load_any<TAIL>(static_cast<const char *>(a.pre), a.weight_dt, e, dim, a.weight_offset);
    };
    const auto gate_at = [&](int32_t e) {
        return a.gate ? load_any<TAIL>(gr, a.gate_dt, e, dim, 0.0f) : all_of(1.0f);
    };
    Raw8<SDT> x[K];
    Raw8<BDT> y[K];
    // with one piece to a lane there is room to load everything at once
    f32x8 gate, post, pre;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int32_t e = (lane + k * NT) * 8;
        y[k] = Raw8<BDT>{};
        if (e >= dim) continue;
        if (a.branch) y[k] = load_piece<BDT, TAIL>(yr, e, dim);
        x[k] = load_piece<SDT, TAIL>(xr, e, dim);
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
    }
    f32x8 h[K];
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int32_t e = (lane + k * NT) * 8;
        if (e >= dim) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[k][j] = raw_value<SDT>(x[k], j);
        if (a.branch) {
            if constexpr (K > 1) {
                post = post_at(e);
                gate = gate_at(e);
            }
            u32x4 words = {0, 0, 0, 0};
            if (a.drop.threshold) words = random_words(static_cast<uint32_t>(e >> 3), static_cast<uint32_t>(t), a.drop);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = raw_value<BDT>(y[k], j) * rb * post[j] * gate[j] * a.drop.factor;
                h[k][j] = __builtin_fmaf(a.scale, kept(words, j, a.drop.threshold) ? u : 0.0f, h[k][j]);
            }
            store_piece<SDT, TAIL>(elem_at(a.h, SDT, t * a.h_stride), e, dim, h[k]);
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
        const int32_t e = (lane + k * NT) * 8;
        if (e >= dim) continue;
        if constexpr (K > 1) pre = pre_at(e);
        f32x8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = h[k][j] * rh * pre[j];
        store_piece<BDT, TAIL>(elem_at(a.out, BDT, t * a.out_stride), e, dim, v);
    }
}

// Rows of one launch.
constexpr int64_t RESIDUAL_LAUNCH_ROWS = int64_t(1) << 21;

template <int SDT, int BDT, int NT, int K>
static hipError_t residual_at(const ResidualArgs &a, hipStream_t stream, int *launched) {
    const auto kernel = a.dim % 8 ? residual_norm<SDT, BDT, NT, K, true> : residual_norm<SDT, BDT, NT, K, false>;
    for (int64_t row0 = 0; row0 < a.n; row0 += RESIDUAL_LAUNCH_ROWS) {
        const int64_t rows = a.n - row0 < RESIDUAL_LAUNCH_ROWS ? a.n - row0 : RESIDUAL_LAUNCH_ROWS;
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(ceil_div(rows, row_block<NT> / NT))), dim3(row_block<NT>), 0,
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
    RADAMW_ROW_SHAPES(a.dim, RADAMW_CALL)
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
