// radamw_dropout.hip -- dropout from a counter-based generator for gfx950.
//
//   out[t, j] = kept(seed, offset, first_row + t, j) ? factor * x[t, j] : 0
//
// The mask is never stored: the gradient is the same call on the output's
// gradient.  Bound by HBM: a lane forms one counter's numbers for eight
// columns, which hides behind the loads (32768 x 8192 BF16: 178 us, 6.0 TB/s,
// at p = 0.1; 4097 x 1111 FP32: 8.2 us).
#include "radamw_random.h"

namespace radamw {

namespace {

constexpr int DROPOUT_BLOCK = 256;
// Pieces of eight per lane: four where that leaves eight workgroups per CU.
constexpr int DROPOUT_DEEP = 4;
constexpr int64_t DROPOUT_DEEP_BLOCKS = 8 * 256;
// Pieces of one launch: an index and its quotient stay in 31 bits.
constexpr int64_t DROPOUT_MAX_PIECES = (int64_t(1) << 31) - 4 * DROPOUT_BLOCK * DROPOUT_DEEP;

// i / d for i < 2^31: with d <= 2^s, m = ceil(2^(31 + s) / d) exceeds the
// exact quotient by less than 2^s / d, which i * m >> (31 + s) does not see.
struct Divisor {
    uint32_t m;
    int32_t shift;
};

Divisor divisor(int64_t d) {
    int s = 0;
    while ((int64_t(1) << s) < d) ++s;
    return {static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + static_cast<uint64_t>(d) - 1) / static_cast<uint64_t>(d)),
            31 + s};
}

}  // namespace

template <int DT, int UNROLL, bool TAIL>
__global__ __launch_bounds__(DROPOUT_BLOCK) void dropout_rows(DropoutArgs a, uint32_t row0, uint32_t pieces,
                                                              uint32_t per_row, Divisor by_row) {
    const uint32_t first = blockIdx.x * (DROPOUT_BLOCK * UNROLL) + threadIdx.x;
    const int32_t dim = static_cast<int32_t>(a.dim);
    Raw8<DT> r[UNROLL];
    uint32_t row[UNROLL], col[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const uint32_t i = first + u * DROPOUT_BLOCK;
        row[u] = static_cast<uint32_t>((uint64_t(i) * by_row.m) >> by_row.shift);
        col[u] = i - row[u] * per_row;
        row[u] += row0;
        if (i < pieces)
            r[u] = load_piece<DT, TAIL>(elem_at(a.x, DT, row[u] * a.stride), static_cast<int32_t>(col[u] * 8), dim);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        if (first + u * DROPOUT_BLOCK >= pieces) continue;
        const u32x4 words = random_words(col[u], row[u], a.drop);
        f32x8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = kept(words, j, a.drop.threshold) ? raw_value<DT>(r[u], j) * a.drop.factor : 0.0f;
        store_piece<DT, TAIL>(elem_at(a.out, DT, row[u] * a.out_stride), static_cast<int32_t>(col[u] * 8), dim, v);
    }
}

template <int DT, int UNROLL>
static void dropout_of(const DropoutArgs &a, int64_t row0, int64_t pieces, int64_t per_row, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>((pieces + DROPOUT_BLOCK * UNROLL - 1) / (DROPOUT_BLOCK * UNROLL)));
    const auto kernel = a.dim % 8 ? dropout_rows<DT, UNROLL, true> : dropout_rows<DT, UNROLL, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(DROPOUT_BLOCK), 0, stream, a, static_cast<uint32_t>(row0),
                       static_cast<uint32_t>(pieces), static_cast<uint32_t>(per_row), divisor(per_row));
}

template <int DT>
static hipError_t dropout_at(const DropoutArgs &a, hipStream_t stream, int *launched) {
    const int64_t per_row = (a.dim + 7) / 8;
    const int64_t rows = DROPOUT_MAX_PIECES / per_row;  // of a launch
    for (int64_t row0 = 0; row0 < a.n; row0 += rows) {
        const int64_t pieces = (a.n - row0 < rows ? a.n - row0 : rows) * per_row;
        if (pieces >= DROPOUT_DEEP_BLOCKS * DROPOUT_BLOCK * DROPOUT_DEEP)
            dropout_of<DT, DROPOUT_DEEP>(a, row0, pieces, per_row, stream);
        else dropout_of<DT, 1>(a, row0, pieces, per_row, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        ++*launched;
    }
    return hipSuccess;
}

hipError_t launch_dropout(const DropoutArgs &a, int dt, hipStream_t stream, int *launched) {
    switch (dt) {
    case G_F32: return dropout_at<G_F32>(a, stream, launched);
    case G_F16: return dropout_at<G_F16>(a, stream, launched);
    default: return dropout_at<G_BF16>(a, stream, launched);
    }
}

}  // namespace radamw
