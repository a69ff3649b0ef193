// radamw_rows.h -- device helpers of the vocabulary operators: values of the
// three storage types moved eight at a time, rows whose start need only be
// aligned to its element.
//
// gfx950 loads and stores 16 bytes at any element address (a row of an odd
// length starts anywhere), so one path serves aligned and unaligned rows.
#pragma once

#include "radamw_internal.h"

namespace radamw {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any2 __attribute__((aligned(2)));
typedef u32x4 u32x4_any4 __attribute__((aligned(4)));
#define RADAMW_GLOBAL __attribute__((address_space(1)))

constexpr float LOG2E = 1.4426950408889634f;

template <int DT>
constexpr int elem_bytes = DT == G_F32 ? 4 : 2;
// Values of one 16-byte chunk.
template <int DT>
constexpr int chunk_elems = 16 / elem_bytes<DT>;

// 16 bytes at element e.
template <int DT>
__device__ __forceinline__ u32x4 load_chunk(const void *p, int64_t e) {
    if constexpr (DT == G_F32) return *(const RADAMW_GLOBAL u32x4_any4 *)(static_cast<const float *>(p) + e);
    else return *(const RADAMW_GLOBAL u32x4_any2 *)(static_cast<const uint16_t *>(p) + e);
}
// The same, with the nontemporal hint, for data that is touched once.
template <int DT>
__device__ __forceinline__ u32x4 stream_chunk(const void *p, int64_t e) {
    if constexpr (DT == G_F32)
        return __builtin_nontemporal_load((const RADAMW_GLOBAL u32x4_any4 *)(static_cast<const float *>(p) + e));
    else return __builtin_nontemporal_load((const RADAMW_GLOBAL u32x4_any2 *)(static_cast<const uint16_t *>(p) + e));
}
template <int DT>
__device__ __forceinline__ void stream_out(void *p, int64_t e, u32x4 v) {
    if constexpr (DT == G_F32)
        __builtin_nontemporal_store(v, (RADAMW_GLOBAL u32x4_any4 *)(static_cast<float *>(p) + e));
    else __builtin_nontemporal_store(v, (RADAMW_GLOBAL u32x4_any2 *)(static_cast<uint16_t *>(p) + e));
}
template <int DT>
__device__ __forceinline__ void store_chunk(void *p, int64_t e, u32x4 v) {
    if constexpr (DT == G_F32) *(RADAMW_GLOBAL u32x4_any4 *)(static_cast<float *>(p) + e) = v;
    else *(RADAMW_GLOBAL u32x4_any2 *)(static_cast<uint16_t *>(p) + e) = v;
}

// The bits of one value, in the low half for a 16-bit type.
template <int DT>
__device__ __forceinline__ uint32_t load_bits(const void *p, int64_t e) {
    if constexpr (DT == G_F32) return gl(static_cast<const uint32_t *>(p))[e];
    else return gl(static_cast<const uint16_t *>(p))[e];
}
template <int DT>
__device__ __forceinline__ float from_bits(uint32_t b) {
    if constexpr (DT == G_F32) return __builtin_bit_cast(float, b);
    else if constexpr (DT == G_F16) return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b)));
    else return __builtin_bit_cast(float, b << 16);
}
template <int DT>
__device__ __forceinline__ float load_value(const void *p, int64_t e) {
    return from_bits<DT>(load_bits<DT>(p, e));
}
// Rounded to nearest even.
template <int DT>
__device__ __forceinline__ void store_value(void *p, int64_t e, float v) {
    if constexpr (DT == G_F32) gl(static_cast<float *>(p))[e] = v;
    else if constexpr (DT == G_F16) gl(static_cast<_Float16 *>(p))[e] = static_cast<_Float16>(v);
    else gl(static_cast<__bf16 *>(p))[e] = static_cast<__bf16>(v);
}

// Value j of a chunk, widened exactly.
template <int DT>
__device__ __forceinline__ float chunk_value(u32x4 c, int j) {
    if constexpr (DT == G_F32) {
        const uint32_t w = c[j];
        return __builtin_bit_cast(float, w);
    } else {
        const uint32_t w = c[j >> 1];
        if constexpr (DT == G_F16)
            return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(j & 1 ? w >> 16 : w)));
        else return __builtin_bit_cast(float, j & 1 ? w & 0xffff0000u : w << 16);
    }
}

// A row of at least eight values is cut into eights, a lane to each; where
// they do not go up evenly, the last lane serves the row's last eight values,
// some of them beside the lane before it, so that no lane moves values one by
// one.  Only rows of fewer than eight take e itself.
__device__ __forceinline__ int64_t first_of_eight(int64_t e, int64_t dim) {
    return e + 8 <= dim || dim < 8 ? e : dim - 8;
}

// Eight consecutive values at element e.
template <int DT>
struct Raw8 {
    u32x4 c[DT == G_F32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const void *p, int64_t e) {
    Raw8<DT> r;
    r.c[0] = load_chunk<DT>(p, e);
    if constexpr (DT == G_F32) r.c[1] = load_chunk<DT>(p, e + 4);
    return r;
}
template <int DT>
__device__ __forceinline__ Raw8<DT> stream_raw8(const void *p, int64_t e) {
    Raw8<DT> r;
    r.c[0] = stream_chunk<DT>(p, e);
    if constexpr (DT == G_F32) r.c[1] = stream_chunk<DT>(p, e + 4);
    return r;
}
template <int DT>
__device__ __forceinline__ float raw_value(const Raw8<DT> &r, int j) {
    if constexpr (DT == G_F32) return chunk_value<DT>(r.c[j >> 2], j & 3);
    else return chunk_value<DT>(r.c[0], j);
}
template <int DT>
__device__ __forceinline__ void store8(void *p, int64_t e, f32x8 v) {
    if constexpr (DT == G_F32) {
        const f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
        store_chunk<DT>(p, e, __builtin_bit_cast(u32x4, lo));
        store_chunk<DT>(p, e + 4, __builtin_bit_cast(u32x4, hi));
    } else if constexpr (DT == G_F16) {
        store_chunk<DT>(p, e, __builtin_bit_cast(u32x4, __builtin_convertvector(v, f16x8)));
    } else {
        store_chunk<DT>(p, e, __builtin_bit_cast(u32x4, __builtin_convertvector(v, bf16x8)));
    }
}

template <int DT>
__device__ __forceinline__ void stream8(void *p, int64_t e, f32x8 v) {
    if constexpr (DT == G_F32) {
        const f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
        stream_out<DT>(p, e, __builtin_bit_cast(u32x4, lo));
        stream_out<DT>(p, e + 4, __builtin_bit_cast(u32x4, hi));
    } else if constexpr (DT == G_F16) {
        stream_out<DT>(p, e, __builtin_bit_cast(u32x4, __builtin_convertvector(v, f16x8)));
    } else {
        stream_out<DT>(p, e, __builtin_bit_cast(u32x4, __builtin_convertvector(v, bf16x8)));
    }
}

// Entry i of an index array, as 64 bits.
__device__ __forceinline__ int64_t load_index(const void *p, int32_t wide, int64_t i) {
    return wide ? gl(static_cast<const int64_t *>(p))[i] : int64_t(gl(static_cast<const int32_t *>(p))[i]);
}

}  // namespace radamw
