// radamw_residual.h -- device helpers shared by the residual stream's norms
// (radamw_residual.hip) and their gradient (radamw_residual_grad.hip).
#pragma once

#include "radamw_random.h"

namespace radamw {

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The sum over a wave, in every lane: butterflies inside rows of 16 lanes by
// DPP, then the four rows' sums.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0xB1>(v);   // lanes 1 apart
    v = dpp_add<0x4E>(v);   // 2 apart
    v = dpp_add<0x141>(v);  // the other half of eight
    v = dpp_add<0x140>(v);  // the other half of sixteen
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// The sum over a row's NT lanes.  `part` is LDS of NT / 64 values that no
// other sum since the last but one barrier has used.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float *part) {
    v = wave_sum(v);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) v += part[w];
    }
    return v;
}

// The sums of two rows, likewise; `part` has room for both.
template <int NT>
__device__ __forceinline__ void row_sums(float &v, float &w, float *part) {
    constexpr int WAVES = NT / 64;
    v = wave_sum(v);
    w = wave_sum(w);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) {
            part[threadIdx.x >> 6] = v;
            part[WAVES + (threadIdx.x >> 6)] = w;
        }
        __syncthreads();
        v = w = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            v += part[i];
            w += part[WAVES + i];
        }
    }
}

// A lane's piece: eight columns.  Where the stream is FP32 they are two fours,
// 4 NT columns apart, so that the wave's lanes lie side by side in every load
// and store: 32 bytes to a lane are two half-filled 16-byte accesses, whose
// nontemporal stores reach memory in parts (8192 x 4096 took 75 to 90 us, with
// the order the compiler chose for them).
template <int SDT>
constexpr bool split_stream = SDT == G_F32;
struct Piece {
    int32_t e, e2;  // first columns of its fours
};
template <bool SPLIT, int NT>
__device__ __forceinline__ Piece piece_at(int lane, int k) {
    if constexpr (SPLIT) return {(lane + 2 * k * NT) * 4, (lane + (2 * k + 1) * NT) * 4};
    else return {(lane + k * NT) * 8, (lane + k * NT) * 8 + 4};
}
template <int DT, bool SPLIT, bool TAIL, bool SHARED = false>
__device__ __forceinline__ Raw8<DT> load_piece(const void *row, Piece c, int32_t dim) {
    if constexpr (!SPLIT) return load_piece<DT, TAIL, SHARED>(row, c.e, dim);
    const u32x4 lo = load_four<DT, TAIL, SHARED>(row, c.e, dim), hi = load_four<DT, TAIL, SHARED>(row, c.e2, dim);
    Raw8<DT> r;
    if constexpr (DT == G_F32) {
        r.c[0] = lo;
        r.c[1] = hi;
    } else {
        r.c[0] = u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
    return r;
}
template <int DT, bool SPLIT, bool TAIL>
__device__ __forceinline__ void store_piece(void *row, Piece c, int32_t dim, f32x8 v) {
    if constexpr (!SPLIT) {
        store_piece<DT, TAIL>(row, c.e, dim, v);
    } else {
        store_four<DT, TAIL>(row, c.e, dim, f32x4{v[0], v[1], v[2], v[3]});
        store_four<DT, TAIL>(row, c.e2, dim, f32x4{v[4], v[5], v[6], v[7]});
    }
}
// The random words of a piece's eight columns.
template <bool SPLIT>
__device__ __forceinline__ u32x4 piece_words(Piece c, int64_t row, const DropArgs &d) {
    const u32x4 a = random_words(static_cast<uint32_t>(c.e) >> 3, static_cast<uint32_t>(row), d);
    if constexpr (!SPLIT) return a;
    // a four is half of a counter's eight columns
    const u32x4 b = random_words(static_cast<uint32_t>(c.e2) >> 3, static_cast<uint32_t>(row), d);
    return c.e & 4 ? u32x4{a[2], a[3], b[2], b[3]} : u32x4{a[0], a[1], b[0], b[1]};
}

// Eight values of an array whose type is known at run time (a weight's, a
// gate's), as they are stored, so that many such loads are under way before
// the first is waited for; many workgroups read its rows.
struct Any8 {
    u32x4 c[2];  // 16-bit types: the first alone
};
template <bool SPLIT, bool TAIL>
__device__ __forceinline__ Any8 load_any(const void *row, int32_t dt, Piece c, int32_t dim) {
    Any8 r;
    if (dt == G_F32) {
        const Raw8<G_F32> w = load_piece<G_F32, SPLIT, TAIL, true>(row, c, dim);
        r.c[0] = w.c[0];
        r.c[1] = w.c[1];
    } else {
        r.c[0] = load_piece<G_BF16, SPLIT, TAIL, true>(row, c, dim).c[0];
    }
    return r;
}
// As FP32, plus `offset`.
__device__ __forceinline__ f32x8 any_values(const Any8 &r, int32_t dt, float offset) {
    f32x8 v;
    if (dt == G_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = chunk_value<G_F32>(r.c[j >> 2], j & 3) + offset;
    } else if (dt == G_F16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = chunk_value<G_F16>(r.c[0], j) + offset;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = chunk_value<G_BF16>(r.c[0], j) + offset;
    }
    return v;
}
template <bool SPLIT, bool TAIL>
__device__ __forceinline__ f32x8 load_weight(const void *row, int32_t dt, Piece c, int32_t dim, float offset) {
    return any_values(load_any<SPLIT, TAIL>(row, dt, c, dim), dt, offset);
}
template <bool SPLIT, bool TAIL>
__device__ __forceinline__ void store_any(char *row, int32_t dt, Piece c, int32_t dim, f32x8 v) {
    if (dt == G_F32) store_piece<G_F32, SPLIT, TAIL>(row, c, dim, v);
    else if (dt == G_F16) store_piece<G_F16, SPLIT, TAIL>(row, c, dim, v);
    else store_piece<G_BF16, SPLIT, TAIL>(row, c, dim, v);
}

__device__ __forceinline__ f32x8 all_of(float v) { return f32x8{v, v, v, v, v, v, v, v}; }

// Threads of a workgroup whose rows have NT lanes: at least four waves where
// a row is one wave's.
template <int NT>
constexpr int row_block = NT == 64 ? 256 : NT;
// The row (or worker) of this wave within its workgroup, in a scalar register.
template <int NT>
__device__ __forceinline__ int wave_row() {
    return NT == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
}

// Calls F(NT, K) with the lanes of a row and the pieces of a lane.  One piece
// to a lane needs the fewest registers and has the most loads of a row in
// flight; WIDE is the call for rows of 4104 to 8192 columns.
#define RADAMW_ROW_SHAPES(dim, F, WIDE)          \
    {                                            \
        const int64_t pieces_ = ((dim) + 7) / 8; \
        if (pieces_ <= 64) {                     \
            F(64, 1);                            \
        } else if (pieces_ <= 128) {             \
            F(128, 1);                           \
        } else if (pieces_ <= 256) {             \
            F(256, 1);                           \
        } else if (pieces_ <= 512) {             \
            F(512, 1);                           \
        } else if (pieces_ <= 1024) {            \
            WIDE;                                \
        } else if (pieces_ <= 2048) {            \
            F(1024, 2);                          \
        } else {                                 \
            F(1024, 4);                          \
        }                                        \
    }

}  // namespace radamw
