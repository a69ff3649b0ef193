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

// Eight values of an array whose type is known at run time (a weight's, a
// gate's), plus `offset`; the row's values are read by many workgroups.
template <bool TAIL>
__device__ __forceinline__ f32x8 load_any(const char *row, int32_t dt, int32_t e, int32_t dim, float offset) {
    f32x8 v;
    if (dt == G_F32) {
        const Raw8<G_F32> r = load_piece<G_F32, TAIL, true>(row, e, dim);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = raw_value<G_F32>(r, j) + offset;
    } else {
        const Raw8<G_BF16> r = load_piece<G_BF16, TAIL, true>(row, e, dim);
        if (dt == G_F16) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = chunk_value<G_F16>(r.c[0], j) + offset;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = chunk_value<G_BF16>(r.c[0], j) + offset;
        }
    }
    return v;
}
template <bool TAIL>
__device__ __forceinline__ void store_any(char *row, int32_t dt, int32_t e, int32_t dim, f32x8 v) {
    if (dt == G_F32) store_piece<G_F32, TAIL>(row, e, dim, v);
    else if (dt == G_F16) store_piece<G_F16, TAIL>(row, e, dim, v);
    else store_piece<G_BF16, TAIL>(row, e, dim, v);
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

// Calls f<NT, K> with the lanes of a row and the pieces of a lane.  One piece
// to a lane as long as a workgroup has the lanes: it needs the fewest
// registers, and the most loads of a row are in flight.
#define RADAMW_ROW_SHAPES(dim, F)                                  \
    {                                                              \
        const int64_t pieces_ = ((dim) + 7) / 8;                   \
        if (pieces_ <= 64) F(64, 1);                               \
        else if (pieces_ <= 128) F(128, 1);                        \
        else if (pieces_ <= 256) F(256, 1);                        \
        else if (pieces_ <= 512) F(512, 1);                        \
        else if (pieces_ <= 1024) F(1024, 1);                      \
        else if (pieces_ <= 2048) F(1024, 2);                      \
        else F(1024, 4);                                           \
    }

}  // namespace radamw
