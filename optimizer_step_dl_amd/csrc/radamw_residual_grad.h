// radamw_residual_grad.h -- the kernel of the gradient of the residual stream's norms
// around one block (radamw_residual.hip) for gfx950; radamw_residual_grad.hip
// has the join, the launches and FP32 alone, the other types are compiled beside
// it (radamw_residual_grad_*.hip).
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
//
// 8192 x 4096 with an FP32 stream, both norms, one gate and dropout take 111 us
// (604 MB: 5.4 TB/s), 32768 x 8192 BF16 with a gate per element 805 us (4.3 GB:
// 5.3 TB/s), 32768 x 4096 BF16 without one 312 us (1.6 GB: 5.2 TB/s).  About 35
// vector operations per value run beside the memory's time.
//
// Two or four pieces to a lane (more than 8192 columns) are more than the 128
// registers hold: 23 to 1284 of them are spilled.  8192 x 16384 BF16 take 385
// us, with an FP32 stream 1960 us, against 240 and 361 us for their bytes.
#pragma once

#include "radamw_residual.h"

namespace radamw {

// A worker's column sums, whole pieces: a partial row has room for them.
template <bool SPLIT, int NT, int K>
__device__ __forceinline__ void put_partial(char *base, int64_t slot, int64_t width, int lane, const f32x8 (&acc)[K]) {
    float *row = reinterpret_cast<float *>(base) + slot * width;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Piece e = piece_at<SPLIT, NT>(lane, k);
        const f32x4 lo = {acc[k][0], acc[k][1], acc[k][2], acc[k][3]}, hi = {acc[k][4], acc[k][5], acc[k][6], acc[k][7]};
        if (e.e < width) store_chunk<G_F32>(row, e.e, __builtin_bit_cast(u32x4, lo));
        if (e.e2 < width) store_chunk<G_F32>(row, e.e2, __builtin_bit_cast(u32x4, hi));
    }
}

// Parts of a call, as bits.
// EACH_ROW: every row has a gate row of its own; EACH_GATE and SUM_GATE: the
// gate's gradient is asked for, by row or summed.
enum : uint32_t {
    HAS_PRE = 1, HAS_POST = 2, HAS_GATE = 4, HAS_BRANCH = 8, HAS_GRAD_H = 16, EACH_ROW = 32, EACH_GATE = 64, SUM_GATE = 128
};

// What a lane reads of one row.
template <int SDT, int BDT, int K>
struct GradRow {
    Raw8<BDT> g[K], y[K];
    Raw8<SDT> h[K], dh[K];
    Any8 gate[K];
};

// The kernel's arguments where the hardware has put them, at its first
// argument's place.  Read through a pointer that the compiler takes for a new
// one at every row, they need scalar registers only where they are used; kept
// over the whole loop they were 60 to 120 registers too many, each spilled to
// a vector lane and back.
typedef const __attribute__((address_space(4))) ResidualGradArgs *GradArgsPtr;
__device__ __forceinline__ GradArgsPtr args_again(GradArgsPtr p) {
    asm volatile("" : "+s"(p));
    return p;
}

// A value that the kernel does not write, by a scalar load: a vector load would
// be waited for with the next row's, which are issued before it.
__device__ __forceinline__ float row_constant(const float *p, int64_t i) {
    return ((const __attribute__((address_space(4))) float *)p)[i];
}

// One worker's rows, in order.  AHEAD: the next row's loads are under way
// while this row's sums are formed.  The weights wait in LDS, each lane's own,
// so that the registers hold the column sums and the rows; of lanes with two
// pieces the weights' sums are in LDS instead.  The gate's sum is one per gate
// row: where the gate row's rows all belong to this worker it is stored, else
// it is left in slot 0 (the gate row began before this worker) or 1 (it goes
// on behind it).
//
// KNOWN: the parts that are known to be there, all lanes with columns.  Only
// then is the number of stores behind the next row's loads known as well, so
// that those loads are waited for without the stores, with which they share a
// counter; else 0.
template <int SDT, int BDT, int NT, int K, bool TAIL, uint32_t KNOWN>
__global__ __launch_bounds__(row_block<NT>, 4) void residual_norm_grad(ResidualGradArgs args, ResidualPlan p,
                                                                       uint32_t parts) {
    constexpr bool SPLIT = split_stream<SDT>;
    // an FP32 row and the next one have the registers only where parts are
    // known to be absent; with a gate row for each row it costs more than it
    // gives (32768 x 8192 BF16: 850 us, against 802 us)
    constexpr bool AHEAD = K == 1 && (KNOWN ? !(KNOWN & EACH_ROW) : SDT != G_F32);
    constexpr uint32_t RARE = HAS_GATE | SUM_GATE;  // of no load or store in most rows
    const uint32_t has = KNOWN ? KNOWN | (parts & RARE) : parts;
    constexpr int BLOCK = row_block<NT>, WAVES = BLOCK / 64;
    __shared__ float part[2][2][WAVES];
    // K == 1: weights; K == 2: sums of both; K == 4: sums of the norm behind the stream's sum
    __shared__ f32x4 own[K == 1 ? 4 : 8][BLOCK];
    const GradArgsPtr kernarg = (GradArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
    const int lane = threadIdx.x % NT;
    const int32_t dim = KNOWN ? NT * K * 8 : static_cast<int32_t>(args.dim);
    const int64_t w = int64_t(blockIdx.x) * (BLOCK / NT) + wave_row<NT>();
    const int64_t begin = w * p.rows, end = begin + p.rows < args.n ? begin + p.rows : args.n;
    if (begin >= end) return;  // whole waves; with NT > 64 whole workgroups
    const float inv_dim = 1.0f / static_cast<float>(dim);
    f32x8 sum_post[K], sum_pre[K], sum_gate[K];
    GradRow<SDT, BDT, K> row, next;
    const auto put_own = [&](int i, f32x8 v) {
        own[2 * i][threadIdx.x] = f32x4{v[0], v[1], v[2], v[3]};
        own[2 * i + 1][threadIdx.x] = f32x4{v[4], v[5], v[6], v[7]};
    };
    const auto get_own = [&](int i) {
        const f32x4 lo = own[2 * i][threadIdx.x], hi = own[2 * i + 1][threadIdx.x];
        return f32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    // the weights of piece k: 0 behind the branch, 1 behind the stream's sum
    const auto global_weight = [&](GradArgsPtr a, int which, Piece e) -> f32x8 {
        if (!(has & (which ? HAS_PRE : HAS_POST)) || e.e >= dim) return all_of(1.0f);
        return load_weight<SPLIT, TAIL>(which ? a->pre : a->post, a->weight_dt, e, dim, a->weight_offset);
    };
    const auto weight = [&](GradArgsPtr a, int which, Piece e) -> f32x8 {
        if constexpr (K == 1) return get_own(which);
        else return global_weight(a, which, e);
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Piece e = piece_at<SPLIT, NT>(lane, k);
        sum_post[k] = sum_pre[k] = sum_gate[k] = f32x8{};
        row.g[k] = row.y[k] = Raw8<BDT>{};
        row.h[k] = row.dh[k] = Raw8<SDT>{};
        row.gate[k] = Any8{};
        if constexpr (K == 1) {
            put_own(0, global_weight(kernarg, 0, e));
            put_own(1, global_weight(kernarg, 1, e));
        } else if constexpr (K == 2) {
            put_own(k, f32x8{});
            put_own(2 + k, f32x8{});
        } else {
            put_own(k, f32x8{});
        }
    }
    // adds to piece k's sum, where it is held
    const auto add_pre = [&](int k, f32x8 v) {
        if constexpr (K == 1) sum_pre[k] += v;
        else put_own(k, get_own(k) + v);
    };
    const auto add_post = [&](int k, f32x8 v) {
        if constexpr (K == 2) put_own(2 + k, get_own(2 + k) + v);
        else sum_post[k] += v;
    };
    const auto load_gate = [&](GradArgsPtr a, GradRow<SDT, BDT, K> &r, int64_t group) {
        const char *from = elem_at(a->gate, a->gate_dt, group * a->gate_stride);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Piece e = piece_at<SPLIT, NT>(lane, k);
            if (e.e < dim) r.gate[k] = load_any<SPLIT, TAIL>(from, a->gate_dt, e, dim);
        }
    };
    const auto load = [&](GradArgsPtr a, GradRow<SDT, BDT, K> &r, int64_t t) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Piece e = piece_at<SPLIT, NT>(lane, k);
            if (e.e >= dim) continue;
            if (has & HAS_PRE) {
                r.g[k] = load_piece<BDT, SPLIT, TAIL>(elem_at(a->grad_out, BDT, t * a->grad_out_stride), e, dim);
                r.h[k] = load_piece<SDT, SPLIT, TAIL>(elem_at(a->h, SDT, t * a->h_stride), e, dim);
            }
            if (has & HAS_GRAD_H)
                r.dh[k] = load_piece<SDT, SPLIT, TAIL>(elem_at(a->grad_h, SDT, t * a->grad_h_stride), e, dim);
            if (has & HAS_BRANCH)
                r.y[k] = load_piece<BDT, SPLIT, TAIL>(elem_at(a->branch, BDT, t * a->branch_stride), e, dim);
        }
        if (has & EACH_ROW) load_gate(a, r, t);
    };
    if constexpr (AHEAD) {
        next = row;
        load(kernarg, next, begin);
    }
    // the gate row of row t, and the first row behind it
    int64_t group = has & HAS_GATE ? begin / args.per : 0, behind = begin;
    int odd = 0;
    for (int64_t t = begin; t < end; ++t, odd ^= 1) {
        const GradArgsPtr a = args_again(kernarg);
        if constexpr (AHEAD) {
            row.g[0] = next.g[0];
            row.y[0] = next.y[0];
            row.h[0] = next.h[0];
            row.dh[0] = next.dh[0];
            if (has & EACH_ROW) row.gate[0] = next.gate[0];
            if (t + 1 < end) load(a, next, t + 1);
        } else {
            load(a, row, t);
        }
        if ((has & HAS_GATE) && t == behind) {
            if (t != begin) ++group;
            behind = (group + 1) * a->per;
            if (!(has & EACH_ROW)) load_gate(a, row, group);
        }
        // D, and the sums of the norm behind the stream's sum
        float rh = 0.0f, mean = 0.0f;
        if (has & HAS_PRE) {
            rh = row_constant(a->rstd, a->n + t);
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const f32x8 pre = weight(a, 1, piece_at<SPLIT, NT>(lane, k));
                f32x8 c;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    c[j] = raw_value<BDT>(row.g[k], j) * (raw_value<SDT>(row.h[k], j) * rh);
                    s = __builtin_fmaf(c[j], pre[j], s);
                }
                add_pre(k, c);
            }
            mean = row_sum<NT>(s, part[odd][0]) * inv_dim;
        }
        const float rb = has & HAS_POST ? row_constant(a->rstd, t) : 1.0f;
        float s = 0.0f;
        f32x8 du[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Piece e = piece_at<SPLIT, NT>(lane, k);
            if (e.e >= dim) continue;
            f32x8 d;
            const f32x8 pre = weight(a, 1, e);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float q = raw_value<BDT>(row.g[k], j) * pre[j], hat = raw_value<SDT>(row.h[k], j) * rh;
                d[j] = __builtin_fmaf(rh, __builtin_fmaf(-hat, mean, q), raw_value<SDT>(row.dh[k], j));
            }
            store_piece<SDT, SPLIT, TAIL>(elem_at(a->grad_x, SDT, t * a->grad_x_stride), e, dim, d);
            if (!(has & HAS_BRANCH)) continue;
            f32x8 gate = has & HAS_GATE ? any_values(row.gate[k], a->gate_dt, 0.0f) : all_of(1.0f), hat;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                hat[j] = raw_value<BDT>(row.y[k], j) * rb;
                d[j] *= a->scale;
            }
            if (a->drop.threshold) {
                // a dropped place passes nothing on, whatever the branch and the gate hold there
                const DropArgs drop = {a->drop.key0, a->drop.key1, a->drop.off0, a->drop.off1, a->drop.first_row,
                                       a->drop.threshold, a->drop.factor};
                const u32x4 words = piece_words<SPLIT>(e, t, drop);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool keep = kept(words, j, drop.threshold);
                    d[j] = keep ? d[j] * drop.factor : 0.0f;
                    hat[j] = keep ? hat[j] : 0.0f;
                    gate[j] = keep ? gate[j] : 0.0f;
                }
            }
            const f32x8 post = weight(a, 0, e);
            f32x8 dg, c;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dg[j] = d[j] * (hat[j] * post[j]);
                du[k][j] = d[j] * gate[j];
                c[j] = du[k][j] * hat[j];
                du[k][j] *= post[j];
                s = __builtin_fmaf(c[j], post[j], s);
            }
            if (has & HAS_POST) add_post(k, c);
            if (has & EACH_GATE)
                store_any<SPLIT, TAIL>(elem_at(a->grad_gate, a->gate_dt, t * a->grad_gate_stride), a->gate_dt, e, dim, dg);
            if (has & SUM_GATE) sum_gate[k] += dg;
        }
        if (has & HAS_BRANCH) {
            float mb = 0.0f;
            if (has & HAS_POST) mb = row_sum<NT>(s, part[odd][1]) * inv_dim * rb;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const Piece e = piece_at<SPLIT, NT>(lane, k);
                if (e.e >= dim) continue;
                if (has & HAS_POST) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        du[k][j] = rb * __builtin_fmaf(-raw_value<BDT>(row.y[k], j), mb, du[k][j]);
                }
                store_piece<BDT, SPLIT, TAIL>(elem_at(a->grad_branch, BDT, t * a->grad_branch_stride), e, dim, du[k]);
            }
        }
        if ((has & SUM_GATE) && (t + 1 == end || t + 1 == behind)) {
            const int64_t from = group * a->per, to = behind < a->n ? behind : a->n;
            if (from >= begin && to <= end) {
                char *out = elem_at(a->grad_gate, a->gate_dt, group * a->grad_gate_stride);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const Piece e = piece_at<SPLIT, NT>(lane, k);
                    if (e.e < dim) store_any<SPLIT, TAIL>(out, a->gate_dt, e, dim, sum_gate[k]);
                }
            } else {
                put_partial<SPLIT, NT>(a->workspace + p.gate, 2 * w + (from >= begin), p.width, lane, sum_gate);
            }
#pragma unroll
            for (int k = 0; k < K; ++k) sum_gate[k] = f32x8{};
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if constexpr (K > 1) sum_pre[k] = get_own(k);
        if constexpr (K == 2) sum_post[k] = get_own(2 + k);
    }
    if (args.grad_post) put_partial<SPLIT, NT>(args.workspace + p.post, w, p.width, lane, sum_post);
    if (args.grad_pre) put_partial<SPLIT, NT>(args.workspace + p.pre, w, p.width, lane, sum_pre);
}

template <int SDT, int BDT, int NT, int K>
void residual_grad_at(const ResidualGradArgs &a, const ResidualPlan &p, hipStream_t stream) {
    auto kernel = a.dim % 8 ? residual_norm_grad<SDT, BDT, NT, K, true, 0> : residual_norm_grad<SDT, BDT, NT, K, false, 0>;
    const uint32_t has = (a.pre ? HAS_PRE : 0) | (a.post ? HAS_POST : 0) | (a.gate ? HAS_GATE : 0) |
                         (a.branch ? HAS_BRANCH : 0) | (a.grad_h ? HAS_GRAD_H : 0) |
                         (a.gate && a.per == 1 ? EACH_ROW : 0) |
                         (a.grad_gate ? a.per == 1 ? EACH_GATE : SUM_GATE : 0);
    if constexpr (K == 1) {
        if (a.dim == NT * 8) {
            constexpr uint32_t PLAIN = HAS_PRE | HAS_BRANCH | HAS_GRAD_H, BOTH = PLAIN | HAS_POST,
                               EACH = BOTH | HAS_GATE | EACH_ROW | EACH_GATE;
            if (has == EACH) kernel = residual_norm_grad<SDT, BDT, NT, K, false, EACH>;
            else if ((has & ~(HAS_GATE | SUM_GATE)) == BOTH) kernel = residual_norm_grad<SDT, BDT, NT, K, false, BOTH>;
            else if ((has & ~(HAS_GATE | SUM_GATE)) == PLAIN) kernel = residual_norm_grad<SDT, BDT, NT, K, false, PLAIN>;
        }
    }
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(ceil_div(p.workers, row_block<NT> / NT))), dim3(row_block<NT>), 0,
                       stream, a, p, has);
}

template <int SDT, int BDT>
hipError_t residual_grad_rows(const ResidualGradArgs &a, const ResidualPlan &p, hipStream_t stream) {
#define RADAMW_CALL(NT, K) residual_grad_at<SDT, BDT, NT, K>(a, p, stream)
    RADAMW_ROW_SHAPES(a.dim, RADAMW_CALL, RADAMW_CALL(1024, 1))
#undef RADAMW_CALL
    return hipGetLastError();
}

// FP32 streams under 16-bit branches.
hipError_t residual_grad_f32_f16(const ResidualGradArgs &a, const ResidualPlan &p, hipStream_t stream);
hipError_t residual_grad_f32_bf16(const ResidualGradArgs &a, const ResidualPlan &p, hipStream_t stream);
// 16-bit streams.
hipError_t residual_grad_f16(const ResidualGradArgs &a, const ResidualPlan &p, hipStream_t stream);
hipError_t residual_grad_bf16(const ResidualGradArgs &a, const ResidualPlan &p, hipStream_t stream);

}  // namespace radamw
