// radamw_embedding.hip -- the embedding lookup and its gradient for gfx950.
//
//   lookup    out[t, :] = scale * table[id_t, :]
//   gradient  dW[v, :] (+)= scale * sum over t with id_t = v of dY[t, :]
//
// Both only move rows: one product or one sum per value read, so they are
// bound by HBM and every lane moves eight values (16 or 32 bytes) at a time.
//
// The gradient sums in a fixed order, without atomics on values: the token
// positions are sorted by id (a stable radix sort), the sorted list is cut
// into chunks of equal length, and each chunk is summed by waves that own
// 64 x 8 columns.  A run of equal ids inside one chunk is finished there; a
// run that crosses chunks leaves FP32 partial sums, which a second launch
// joins in the order of the chunks.  Equal chunks keep the waves balanced
// however uneven the ids are.  A list of up to 512 tokens needs no sort: each
// token's workgroup finds its equals among all ids.
//
// The sort is a few microseconds' latency of few workgroups, so the rows
// that no token names are cleared by the other workgroups of its launches.
// Measured on MI355X, BF16 gradients: 131072 tokens into 131072 x 4096 BF16
// rows take 447 us (2.15 GB: 4.8 TB/s, of which clearing 160 us and summing
// 265 us at 5.2 TB/s each); 8192 tokens into 32000 x 4096 FP32 rows 121 us
// (583 MB: 4.8 TB/s).
#include "radamw_rows.h"
#include "radamw_vocab.h"

namespace radamw {

namespace {

constexpr int ROW_BLOCK = 256;

int log2_ceil(int64_t v) {
    int b = 0;
    while ((int64_t(1) << b) < v) ++b;
    return b;
}

}  // namespace

// ---------------------------------------------------------------- lookup --

// Pieces per lane.  Four where that still leaves eight workgroups per CU:
// 65536 x 8192 BF16 rows take 256 us, against 266 with two and 339 with one.
// One below: 64 x 4096 take 2.5 us, against 2.9 and 3.5.  The output is
// written with the nontemporal hint (255 us against 284), so that the table
// keeps the caches.
constexpr int LOOKUP_DEEP = 4;
constexpr int64_t LOOKUP_DEEP_BLOCKS = 8 * 256;

// x * scale as an FP32 value: the empty asm keeps the compiler from fusing
// the product with a conversion to FP16, which would round the exact product
// in some places and its FP32 value in others.
__device__ __forceinline__ float scaled(float x, float scale) {
    float p = x * scale;
    asm("" : "+v"(p));
    return p;
}

// A group of 2^lg lanes serves one row's UNROLL * 2^lg pieces of 8 values of
// the column tile blockIdx.y.
template <int TDT, int ODT, int UNROLL>
__global__ __launch_bounds__(ROW_BLOCK) void embedding_lookup(LookupArgs a, int lg) {
    const int lanes = 1 << lg;
    const int64_t t = (int64_t(blockIdx.x) << (8 - lg)) + (threadIdx.x >> lg);
    if (t >= a.n) return;
    const int64_t id = load_index(a.ids, a.wide_ids, t);
    const bool inside = id >= 0 && id < a.rows;
    const char *src = static_cast<const char *>(a.table) + (inside ? id : 0) * a.table_stride * elem_bytes<TDT>;
    char *dst = static_cast<char *>(a.out) + t * a.out_stride * elem_bytes<ODT>;
    const int64_t first = int64_t(blockIdx.y) * UNROLL * lanes + (threadIdx.x & (lanes - 1));
    Raw8<TDT> r[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int64_t e = (first + u * lanes) * 8;
        if (inside && e < a.dim && a.dim >= 8) r[u] = load_raw8<TDT>(src, first_of_eight(e, a.dim));
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int64_t e = (first + u * lanes) * 8;
        if (e >= a.dim) continue;
        if (a.dim >= 8) {
            f32x8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = inside ? scaled(raw_value<TDT>(r[u], j), a.scale) : 0.0f;
            stream8<ODT>(dst, first_of_eight(e, a.dim), v);
        } else {
            for (int64_t k = e; k < a.dim; ++k)
                store_value<ODT>(dst, k, inside ? scaled(load_value<TDT>(src, k), a.scale) : 0.0f);
        }
    }
}

// Pieces per lane and lanes (as a power of two) per row.
struct LookupShape {
    int unroll, lg;
    int64_t blocks, tiles;
};

static LookupShape lookup_shape(int64_t n, int64_t dim) {
    const int64_t pieces = (dim + 7) / 8;
    const auto shape = [&](int unroll) {
        const int lg = log2_ceil((pieces + unroll - 1) / unroll);
        LookupShape s{unroll, lg < 3 ? 3 : lg > 8 ? 8 : lg, 0, 0};
        s.blocks = (n + (int64_t(1) << (8 - s.lg)) - 1) >> (8 - s.lg);
        const int64_t tile = int64_t(unroll) << s.lg;
        s.tiles = (pieces + tile - 1) / tile;
        return s;
    };
    const LookupShape deep = shape(LOOKUP_DEEP);
    return deep.blocks * deep.tiles >= LOOKUP_DEEP_BLOCKS ? deep : shape(1);
}

int64_t lookup_blocks(int64_t n, int64_t dim) { return lookup_shape(n, dim).blocks; }

template <int TDT, int ODT>
static void lookup_at(const LookupArgs &a, hipStream_t stream) {
    const LookupShape s = lookup_shape(a.n, a.dim);
    const dim3 grid(static_cast<unsigned>(s.blocks), static_cast<unsigned>(s.tiles));
    if (s.unroll == LOOKUP_DEEP)
        hipLaunchKernelGGL((embedding_lookup<TDT, ODT, LOOKUP_DEEP>), grid, dim3(ROW_BLOCK), 0, stream, a, s.lg);
    else hipLaunchKernelGGL((embedding_lookup<TDT, ODT, 1>), grid, dim3(ROW_BLOCK), 0, stream, a, s.lg);
}

template <int TDT>
static hipError_t lookup_out(const LookupArgs &a, int odt, hipStream_t stream) {
    switch (odt) {
    case G_F32: lookup_at<TDT, G_F32>(a, stream); break;
    case G_F16: lookup_at<TDT, G_F16>(a, stream); break;
    default: lookup_at<TDT, G_BF16>(a, stream); break;
    }
    return hipGetLastError();
}

hipError_t launch_embedding_lookup(const LookupArgs &a, int tdt, int odt, hipStream_t stream) {
    switch (tdt) {
    case G_F32: return lookup_out<G_F32>(a, odt, stream);
    case G_F16: return lookup_out<G_F16>(a, odt, stream);
    default: return lookup_out<G_BF16>(a, odt, stream);
    }
}

// ------------------------------------------------------------- clearing --

// Table rows to be cleared by the workgroups of a launch that sorts: sorting
// is a few workgroups' latency, clearing all the others' bandwidth.
struct ClearArgs {
    void *table;
    const uint8_t *present;  // rows to leave, or null: none
    int64_t stride, dim;     // elements
    int64_t begin, end;      // rows of this launch
    int64_t rows_per_block;
    int32_t dtype;
    int32_t lg;              // 2^lg lanes share a row
};

// Values one clearing workgroup covers: 65536 measured 90.7 us for 32000 x
// 4096 FP32 rows (5.8 TB/s), 32768 96 us, 16384 106 us.
constexpr int64_t CLEAR_ELEMS = 65536;
// Small tables are spread over at least this many workgroups.
constexpr int64_t CLEAR_BLOCKS = 1024;

template <int TDT, int BLOCK>
__device__ __forceinline__ void clear_rows_of(const ClearArgs &a, int64_t block) {
    constexpr int E = chunk_elems<TDT>;
    const int lanes = 1 << a.lg, per = BLOCK >> a.lg;  // rows at a time
    const int mine = threadIdx.x >> a.lg, lane = threadIdx.x & 63;
    const int64_t begin = a.begin + block * a.rows_per_block;
    const int64_t end = begin + a.rows_per_block < a.end ? begin + a.rows_per_block : a.end;
    const auto clear = [&](int64_t r) {
        const u32x4 z = {0, 0, 0, 0};
        char *dst = static_cast<char *>(a.table) + r * a.stride * elem_bytes<TDT>;
        for (int64_t e = int64_t(threadIdx.x & (lanes - 1)) * E; e < a.dim; e += lanes * E) {
            if (a.dim >= E) {
                stream_out<TDT>(dst, e + E <= a.dim ? e : a.dim - E, z);
            } else {
                for (int64_t k = e; k < a.dim; ++k) store_value<TDT>(dst, k, 0.0f);
            }
        }
    };
    if (!a.present || per >= 64) {
        for (int64_t r = begin + mine; r < end; r += per)
            if (!a.present || !a.present[r]) clear(r);
        return;
    }
    for (int64_t r0 = begin; r0 < end; r0 += 64) {
        // few rows at a time: the flags of 64 in one load
        const int rows = static_cast<int>(end - r0 < 64 ? end - r0 : 64);
        const uint64_t left = __ballot(lane < rows && a.present[lane < rows ? r0 + lane : r0] != 0);
        for (int r = mine; r < rows; r += per)
            if (!((left >> r) & 1)) clear(r0 + r);
    }
}

// Zeros have the same bits in both 16-bit types.
template <int BLOCK>
__device__ __forceinline__ void clear_rows(const ClearArgs &a, int64_t block) {
    if (a.dtype == G_F32) clear_rows_of<G_F32, BLOCK>(a, block);
    else clear_rows_of<G_BF16, BLOCK>(a, block);
}

// ------------------------------------------------------------------ sort --
//
// Least-significant-digit radix sort of (id, position), stable, so that
// equal ids keep the order of their tokens.  An id that takes no part
// (outside the table, or the padding id) gets the key `rows` and sorts last.
// Digits have up to 10 bits: two passes for vocabularies below 2^20.

struct SortKeys {
    const void *ids;  // pass 0 reads the ids, later passes keys / pos
    const uint32_t *keys;
    const uint32_t *pos;
    int64_t n, rows, padding_id;
    int32_t wide_ids;
};

// Keys of tokens first, first + 64, ...: all loads are issued before the
// first is used (tokens behind the last reload the last).
template <int ROUNDS>
__device__ __forceinline__ void token_keys(const SortKeys &s, int64_t first, int rounds, uint32_t (&key)[ROUNDS]) {
    int64_t id[ROUNDS];
    const int64_t last = s.n - 1;
    if (s.wide_ids) {
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
            if (r < rounds) id[r] = gl(static_cast<const int64_t *>(s.ids))[first + r * 64 < last ? first + r * 64 : last];
    } else {
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
            if (r < rounds) id[r] = gl(static_cast<const int32_t *>(s.ids))[first + r * 64 < last ? first + r * 64 : last];
    }
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
        key[r] = static_cast<uint32_t>(r < rounds && id[r] >= 0 && id[r] < s.rows && id[r] != s.padding_id ? id[r]
                                                                                                         : s.rows);
}

// Among the lanes of a wave with `in` set: how many before this one have the
// same digit, and how many have it at all.
__device__ __forceinline__ void match_digit(uint32_t digit, int bits, bool in, int *before, int *total) {
    const uint64_t live = __ballot(in);
    uint32_t lo = static_cast<uint32_t>(live), hi = static_cast<uint32_t>(live >> 32);
#pragma unroll
    for (int b = 0; b < SORT_MAX_DIGIT_BITS; ++b) {
        if (b < bits) {
            const uint32_t mine = static_cast<uint32_t>(static_cast<int32_t>(digit << (31 - b)) >> 31);  // 0 or ~0
            const uint64_t set = __ballot(mine != 0);
            lo &= ~(static_cast<uint32_t>(set) ^ mine);
            hi &= ~(static_cast<uint32_t>(set >> 32) ^ mine);
        }
    }
    *before = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));
    *total = __builtin_popcount(lo) + __builtin_popcount(hi);
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t u = __shfl_up(v, off, 64);
        if (lane >= off) v += u;
    }
    return v;
}

// Exclusive sum over a workgroup of WAVES waves; *all receives the total.
// `part` is LDS of WAVES words; ends with every lane past its last read.
template <int WAVES>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *part, uint32_t *all) {
    const uint32_t inc = wave_scan(v);
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 63) part[wave] = inc;
    __syncthreads();
    uint32_t base = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const uint32_t p = part[w];
        base += w < wave ? p : 0;
        sum += p;
    }
    *all = sum;
    __syncthreads();
    return base + inc - v;
}

// One pass's place of every key of a workgroup: waves own consecutive parts
// of the keys and walk them 64 at a time; hist[wave][digit] counts the keys
// of a wave seen so far, then holds the wave's first place for the digit.
template <int WAVES, int ROUNDS>
struct Ranker {
    uint32_t digit[ROUNDS];
    int32_t rank[ROUNDS];  // among the wave's keys of that digit

    __device__ __forceinline__ void count(const uint32_t (&key)[ROUNDS], int rounds, int64_t first, int64_t n, int shift,
                                          int bits, uint32_t *hist, int bins) {
        for (int i = threadIdx.x; i < WAVES * bins; i += WAVES * 64) hist[i] = 0;
        __syncthreads();
        uint32_t *mine = hist + (threadIdx.x >> 6) * bins;
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            if (r >= rounds) break;
            const bool in = first + r * 64 < n;
            digit[r] = (key[r] >> shift) & (bins - 1);
            int before, total;
            match_digit(digit[r], bits, in, &before, &total);
            const uint32_t seen = in ? mine[digit[r]] : 0;
            rank[r] = static_cast<int>(seen) + before;
            // every lane has read before the last of its equals adds them
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (in && before + 1 == total) mine[digit[r]] = seen + total;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        __syncthreads();
    }
};

constexpr int SORT_SMALL_BITS = 9;

// The whole sort of up to BLOCK * ROUNDS tokens by workgroup 0: the keys stay
// in LDS between the passes.  The other workgroups clear the table.
template <int BLOCK, int ROUNDS>
__global__ __launch_bounds__(BLOCK) void sort_small(SortKeys s, int bits, int passes, uint32_t *keys_out,
                                                    uint32_t *pos_out, ClearArgs clear) {
    constexpr int WAVES = BLOCK / 64;
    constexpr int OWN = (1 << SORT_SMALL_BITS) > BLOCK ? (1 << SORT_SMALL_BITS) / BLOCK : 1;  // digits per thread
    static_assert(OWN * BLOCK >= 1 << SORT_SMALL_BITS, "every digit has a thread");
    if (blockIdx.x > 0) {
        clear_rows<BLOCK>(clear, blockIdx.x - 1);
        return;
    }
    __shared__ uint32_t lkey[BLOCK * ROUNDS];
    __shared__ uint16_t lpos[BLOCK * ROUNDS];
    __shared__ uint32_t hist[WAVES << SORT_SMALL_BITS];
    __shared__ uint32_t part[WAVES];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int rounds = static_cast<int>((s.n + BLOCK - 1) / BLOCK);
    const int64_t first = int64_t(wave) * rounds * 64 + lane;
    uint32_t key[ROUNDS];
    uint32_t pos[ROUNDS];
    if (s.n > 0) token_keys(s, first, rounds, key);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) pos[r] = static_cast<uint32_t>(first + r * 64);
    const int bins = 1 << bits;
    Ranker<WAVES, ROUNDS> rk;
    for (int pass = 0; pass < passes; ++pass) {
        rk.count(key, rounds, first, s.n, pass * bits, bits, hist, bins);
        // thread t owns digits OWN t .. OWN t + OWN - 1: their keys over the
        // waves, then over the digits
        uint32_t of[OWN][WAVES], mine = 0;
#pragma unroll
        for (int o = 0; o < OWN; ++o)
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                of[o][w] = tid * OWN + o < bins ? hist[w * bins + tid * OWN + o] : 0;
                mine += of[o][w];
            }
        uint32_t all;
        uint32_t at = block_scan<WAVES>(mine, part, &all);
#pragma unroll
        for (int o = 0; o < OWN; ++o)
            if (tid * OWN + o < bins) {
#pragma unroll
                for (int w = 0; w < WAVES; ++w) {
                    hist[w * bins + tid * OWN + o] = at;
                    at += of[o][w];
                }
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            if (r < rounds && first + r * 64 < s.n) {
                const uint32_t to = hist[wave * bins + rk.digit[r]] + rk.rank[r];
                lkey[to] = key[r];
                lpos[to] = static_cast<uint16_t>(pos[r]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            if (r < rounds && first + r * 64 < s.n) {
                key[r] = lkey[first + r * 64];
                pos[r] = lpos[first + r * 64];
            }
        }
    }
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int64_t i = first + r * 64;
        if (r >= rounds || i >= s.n) continue;
        keys_out[i] = key[r];
        pos_out[i] = pos[r];
    }
}

constexpr int SORT_BLOCK = 512;
constexpr int SORT_WAVES = SORT_BLOCK / 64;
constexpr int SORT_ROUNDS = int(SORT_TILE / SORT_BLOCK);
constexpr int SORT_MAX_BINS = 1 << SORT_MAX_DIGIT_BITS;

// Tiles up to which a tile finds its places from all tiles' counts by itself;
// beyond, one workgroup sums the counts first.
constexpr int64_t SORT_SELF_TILES = 256;

// Keys and positions of a tile's tokens, wave by wave.
template <bool FIRST>
__device__ __forceinline__ void tile_keys(const SortKeys &s, int64_t first, uint32_t (&key)[SORT_ROUNDS]) {
    if constexpr (FIRST) {
        token_keys(s, first, SORT_ROUNDS, key);
    } else {
#pragma unroll
        for (int r = 0; r < SORT_ROUNDS; ++r) key[r] = s.keys[first + r * 64 < s.n ? first + r * 64 : s.n - 1];
    }
}

// One byte per table row: 0 until the first pass's counts have seen a token
// of it.  The tokens of one id all store the same 1, which needs no atomic.
__global__ __launch_bounds__(256) void clear_flags(uint8_t *present, int64_t rows) {
    const u32x4 z = {0, 0, 0, 0};
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i * 16 < rows) gl(reinterpret_cast<u32x4 *>(present))[i] = z;  // the array is padded to 256 bytes
}

// Digit counts of tile blockIdx.x, as counts[digit * tiles + tile], so that
// one exclusive sum over the array gives each tile its places.  The first
// pass sets the flags; workgroups behind the tiles clear table rows.
template <bool FIRST>
__global__ __launch_bounds__(SORT_BLOCK) void radix_count(SortKeys s, int shift, int bits, int64_t tiles,
                                                          uint32_t *counts, uint8_t *present, ClearArgs clear) {
    __shared__ uint32_t hist[SORT_MAX_BINS];
    if (blockIdx.x >= tiles) {
        clear_rows<SORT_BLOCK>(clear, blockIdx.x - tiles);
        return;
    }
    const int bins = 1 << bits;
    const int64_t first = int64_t(blockIdx.x) * SORT_TILE + int64_t(threadIdx.x >> 6) * SORT_ROUNDS * 64 + (threadIdx.x & 63);
    uint32_t key[SORT_ROUNDS];
    tile_keys<FIRST>(s, first, key);
    for (int i = threadIdx.x; i < bins; i += SORT_BLOCK) hist[i] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < SORT_ROUNDS; ++r) {
        if (first + r * 64 < s.n) {
            atomicAdd(&hist[(key[r] >> shift) & (bins - 1)], 1u);
            if (FIRST && present && key[r] < static_cast<uint32_t>(s.rows)) present[key[r]] = 1;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += SORT_BLOCK) counts[i * tiles + blockIdx.x] = hist[i];
}

constexpr int SCAN_BLOCK = 1024;

// Exclusive sum over m counts in place, by one workgroup.
__global__ __launch_bounds__(SCAN_BLOCK) void radix_scan(uint32_t *counts, int64_t m) {
    __shared__ uint32_t part[SCAN_BLOCK / 64];
    uint32_t carry = 0;
    for (int64_t base = 0; base < m; base += SCAN_BLOCK * 4) {
        const int64_t i = base + int64_t(threadIdx.x) * 4;
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = i + j < m ? counts[i + j] : 0;
        uint32_t all;
        uint32_t at = carry + block_scan<SCAN_BLOCK / 64>(v[0] + v[1] + v[2] + v[3], part, &all);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (i + j < m) counts[i + j] = at;
            at += v[j];
        }
        carry += all;
    }
}

// One pass of tile blockIdx.x: every key to its place.  `scanned`: counts
// holds their exclusive sum already.
template <bool FIRST>
__global__ __launch_bounds__(SORT_BLOCK) void radix_scatter(SortKeys s, int shift, int bits, int64_t tiles,
                                                            const uint32_t *counts, int scanned, uint32_t *keys_out,
                                                            uint32_t *pos_out, ClearArgs clear) {
    __shared__ uint32_t hist[SORT_WAVES * SORT_MAX_BINS];
    __shared__ uint32_t part[SORT_WAVES];
    if (blockIdx.x >= tiles) {
        clear_rows<SORT_BLOCK>(clear, blockIdx.x - tiles);
        return;
    }
    constexpr int OWN = SORT_MAX_BINS / SORT_BLOCK;  // digits per thread
    static_assert(OWN * SORT_BLOCK >= SORT_MAX_BINS, "every digit has a thread");
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int bins = 1 << bits;
    const int64_t tile = blockIdx.x;
    const int64_t first = tile * SORT_TILE + int64_t(wave) * SORT_ROUNDS * 64 + lane;
    uint32_t key[SORT_ROUNDS], pos[SORT_ROUNDS];
    tile_keys<FIRST>(s, first, key);
#pragma unroll
    for (int r = 0; r < SORT_ROUNDS; ++r) {
        const int64_t i = first + r * 64;
        pos[r] = FIRST ? static_cast<uint32_t>(i) : s.pos[i < s.n ? i : s.n - 1];
    }
    // thread t owns digits OWN t, OWN t + 1: their first places of this tile
    uint32_t place[OWN];
    if (scanned) {
#pragma unroll
        for (int o = 0; o < OWN; ++o)
            place[o] = tid * OWN + o < bins ? counts[(tid * OWN + o) * tiles + tile] : 0;
    } else {
        uint32_t before[OWN], of[OWN], sum = 0;
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            before[o] = of[o] = 0;
            if (tid * OWN + o < bins) {
                const uint32_t *c = counts + (tid * OWN + o) * tiles;
#pragma unroll 8
                for (int64_t t = 0; t < tiles; ++t) {
                    const uint32_t k = c[t];
                    before[o] += t < tile ? k : 0;
                    of[o] += k;
                }
            }
            sum += of[o];
        }
        uint32_t all;
        uint32_t at = block_scan<SORT_WAVES>(sum, part, &all);
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            place[o] = at + before[o];
            at += of[o];
        }
    }
    Ranker<SORT_WAVES, SORT_ROUNDS> rk;
    rk.count(key, SORT_ROUNDS, first, s.n, shift, bits, hist, bins);
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        const int b = tid * OWN + o;
        if (b < bins) {
            uint32_t of[SORT_WAVES];
#pragma unroll
            for (int w = 0; w < SORT_WAVES; ++w) of[w] = hist[w * bins + b];
#pragma unroll
            for (int w = 0; w < SORT_WAVES; ++w) {
                hist[w * bins + b] = place[o];
                place[o] += of[w];
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < SORT_ROUNDS; ++r) {
        if (first + r * 64 < s.n) {
            const uint32_t at = hist[wave * bins + rk.digit[r]] + rk.rank[r];
            keys_out[at] = key[r];
            pos_out[at] = pos[r];
        }
    }
}

// -------------------------------------------------------------- gradient --

struct SumArgs {
    const void *grad_out;
    void *table_grad;
    const uint32_t *keys, *pos;
    float *partials;
    int64_t grad_stride, table_stride, n, rows, dim, chunks;
    int32_t chunk, tiles;  // tokens per chunk; column tiles per row
    int32_t accumulate;
    float scale;
};

// v into the eight columns that the lane of columns e ... serves (from
// first_of_eight on) of table row `key`, rounded once.  A column that two
// lanes serve gets the same value from both; where that adds to the table,
// the second keeps it to itself.
template <int TDT, bool ACC>
__device__ __forceinline__ void write_row(const SumArgs &a, uint32_t key, int64_t e, f32x8 v) {
    char *dst = static_cast<char *>(a.table_grad) + int64_t(key) * a.table_stride * elem_bytes<TDT>;
    if (a.dim >= 8) {
        const int64_t from = first_of_eight(e, a.dim);
        if constexpr (ACC) {
            const Raw8<TDT> old = load_raw8<TDT>(dst, from);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __builtin_fmaf(v[j], a.scale, raw_value<TDT>(old, j));
            if (from != e) {
#pragma unroll
                for (int j = 1; j < 8; ++j)
                    if (from + j >= e) store_value<TDT>(dst, from + j, v[j]);
                return;
            }
        } else {
            v *= a.scale;
        }
        store8<TDT>(dst, from, v);
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j) {
            if (j < a.dim) {
                const float x = ACC ? __builtin_fmaf(v[j], a.scale, load_value<TDT>(dst, j)) : v[j] * a.scale;
                store_value<TDT>(dst, j, x);
            }
        }
    }
}

constexpr int SUM_UNROLL = 8;  // rows in flight per lane

// The `dim` values (fewer than eight) of a row, zeros behind.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_narrow8(const void *p, int64_t dim) {
    Raw8<DT> r;
#pragma unroll
    for (int c = 0; c < (DT == G_F32 ? 2 : 1); ++c) r.c[c] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 7; ++k) {
        const uint32_t b = k < dim ? load_bits<DT>(p, k) : 0;
        if constexpr (DT == G_F32) r.c[k >> 2][k & 3] = b;
        else r.c[0][k >> 1] |= k & 1 ? b << 16 : b;
    }
    return r;
}

// The lane's eight columns of one chunk of the sorted tokens.  The keys and
// positions of a group of SUM_UNROLL tokens come in two wide loads (scalar
// ones where a wave shares its chunk); entries behind the last token are read
// and not used, and a token that takes no part reads row 0 in its place, so
// that no load waits behind a branch.
template <int GDT, int TDT, bool ACC>
__device__ __forceinline__ void sum_chunk(const SumArgs &a, int64_t chunk, int64_t e) {
    const int64_t base = chunk * a.chunk;
    const int count = static_cast<int>(a.n - base < a.chunk ? a.n - base : a.chunk);
    const uint32_t *keys = a.keys + base, *pos = a.pos + base;
    const uint32_t rows = static_cast<uint32_t>(a.rows);
    if (keys[0] >= rows) return;  // sorted behind every id that takes part
    const bool whole = a.dim >= 8;
    const int64_t from = first_of_eight(e, a.dim);
    bool continued = base > 0 && a.keys[base - 1] == keys[0];  // the first run began in an earlier chunk
    const bool more = base + count < a.n && a.keys[base + count] == keys[count - 1];
    f32x8 acc = 0.0f;
    for (int j0 = 0; j0 < count; j0 += SUM_UNROLL) {
        uint32_t key[SUM_UNROLL + 1], at[SUM_UNROLL];
#pragma unroll
        for (int u = 0; u <= SUM_UNROLL; ++u) key[u] = keys[j0 + u];
#pragma unroll
        for (int u = 0; u < SUM_UNROLL; ++u) at[u] = pos[j0 + u];
#pragma unroll
        for (int u = 0; u <= SUM_UNROLL; ++u) key[u] = j0 + u < count ? key[u] : 0xffffffffu;
        Raw8<GDT> raw[SUM_UNROLL];
        const auto source = [&](int u) {
            return static_cast<const char *>(a.grad_out) +
                   int64_t(key[u] < rows ? at[u] : 0) * a.grad_stride * elem_bytes<GDT>;
        };
        if (whole) {
#pragma unroll
            for (int u = 0; u < SUM_UNROLL; ++u) raw[u] = stream_raw8<GDT>(source(u), from);
        } else {
#pragma unroll
            for (int u = 0; u < SUM_UNROLL; ++u) raw[u] = load_narrow8<GDT>(source(u), a.dim);
        }
#pragma unroll
        for (int u = 0; u < SUM_UNROLL; ++u) {
            if (key[u] >= rows) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] += raw_value<GDT>(raw[u], k);
            if (key[u + 1] != key[u]) {  // the run ends here, or crosses into the next chunk
                const bool open = j0 + u + 1 == count && more;
                if (!continued && !open) {
                    write_row<TDT, ACC>(a, key[u], e, acc);
                } else {
                    float *slot = a.partials + (2 * chunk + (continued ? 0 : 1)) * a.dim;
                    if (whole) {
                        store8<G_F32>(slot, from, acc);
                    } else {
#pragma unroll
                        for (int k = 0; k < 7; ++k)
                            if (k < a.dim) slot[k] = acc[k];
                    }
                }
                continued = false;
                acc = 0.0f;
            }
        }
    }
}

template <int GDT, int TDT, bool ACC>
__global__ __launch_bounds__(ROW_BLOCK) void embedding_sum(SumArgs a, int lg) {
    const int64_t unit = (int64_t(blockIdx.x) << (8 - lg)) + (threadIdx.x >> lg);
    if (lg == 6) {
        // a whole wave shares its chunk: ids and positions are scalar loads
        const uint32_t u = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(unit));
        const uint32_t chunk = u / a.tiles, tile = u % a.tiles;
        const int64_t e = (int64_t(tile) * 64 + (threadIdx.x & 63)) * 8;
        if (chunk < a.chunks && e < a.dim) sum_chunk<GDT, TDT, ACC>(a, chunk, e);
    } else {
        const int64_t e = int64_t(threadIdx.x & ((1 << lg) - 1)) * 8;
        if (unit < a.chunks && e < a.dim) sum_chunk<GDT, TDT, ACC>(a, unit, e);
    }
}

// Eight waves share a long run: 32705 tokens of FP32, 495 columns, whose most
// frequent id is in 4% of them, join in 5.8 us, against 7.1 us with four and
// 6.7 with sixteen; 30000 BF16 tokens of one id, 2048 columns, take 87 us in
// all, against 119 and 98.
constexpr int JOIN_BLOCK = 512;
constexpr int JOIN_WAVES = JOIN_BLOCK / 64;
constexpr int JOIN_UNROLL = 4;
// Partial sums up to which one wave joins a run by itself.
constexpr int64_t JOIN_ALONE = 16;

// Sum of the partial sums first, first + step, ... up to `last` of the run
// that begins in chunk c, the lane's eight columns, in that order.
__device__ __forceinline__ f32x8 sum_partials(const SumArgs &a, int64_t c, int64_t first, int64_t step, int64_t last,
                                              int64_t e) {
    f32x8 acc = 0.0f;
    const bool whole = a.dim >= 8;
    const int64_t from = first_of_eight(e, a.dim);
    for (int64_t i = first; i <= last; i += step * JOIN_UNROLL) {
        Raw8<G_F32> r[JOIN_UNROLL];
        const auto slot = [&](int u) {
            const int64_t k = i + u * step <= last ? i + u * step : last;
            return a.partials + (k == 0 ? 2 * c + 1 : 2 * (c + k)) * a.dim;
        };
        if (whole) {
#pragma unroll
            for (int u = 0; u < JOIN_UNROLL; ++u) r[u] = load_raw8<G_F32>(slot(u), from);
        } else {
#pragma unroll
            for (int u = 0; u < JOIN_UNROLL; ++u) r[u] = load_narrow8<G_F32>(slot(u), a.dim);
        }
#pragma unroll
        for (int u = 0; u < JOIN_UNROLL; ++u)
            if (i + u * step <= last)
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] += raw_value<G_F32>(r[u], k);
    }
    return acc;
}

// The runs that cross chunks: wave (c, tile) joins the run that begins in
// chunk c and continues past it, 512 columns, in the order of the chunks.  A
// long run is left to the whole workgroup, whose waves take its partial sums
// in turn and add their sums in the order of the waves.
template <int TDT, bool ACC>
__global__ __launch_bounds__(JOIN_BLOCK) void embedding_join(SumArgs a) {
    __shared__ float sums[JOIN_WAVES][64 * 8];
    __shared__ int64_t reaches[JOIN_WAVES];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t c = int64_t(blockIdx.x) * JOIN_WAVES + wave;
    const int64_t base = c * a.chunk, next = base + a.chunk;
    const int64_t e = (int64_t(blockIdx.y) * 64 + lane) * 8;
    int64_t reach = 0;  // chunks after c that a run beginning in c reaches
    uint32_t key = 0;
    if (next < a.n) {
        key = a.keys[next];
        const uint32_t end = a.keys[next - 1], begin = a.keys[base], before = a.keys[base > 0 ? base - 1 : 0];
        const bool earlier = base > 0 && begin == key && before == key;
        if (key < static_cast<uint32_t>(a.rows) && end == key && !earlier) {
            // the ids are sorted: behind the nearest 64 chunks, each round
            // narrows the place where the run ends to a 64th
            const auto reached = [&](int64_t i) {
                const int64_t k = next + i * a.chunk;
                return __ballot(k < a.n && a.keys[k < a.n ? k : 0] == key);
            };
            const uint64_t near = reached(lane);
            reach = ~near ? __builtin_ctzll(~near) : 64;
            if (reach == 64) {
                int64_t off = a.chunks - c;  // the run reaches `reach` chunks, not `off`
                while (off - reach > 1) {
                    const int64_t step = (off - reach + 63) / 64;
                    const int64_t i = reach + (lane + 1) * step - 1;
                    const uint64_t on = reached(i);
                    reach += (~on ? __builtin_ctzll(~on) : 64) * step;
                    off = reach + step < off ? reach + step : off;
                }
            }
        }
    }
    if (reach > 0 && reach < JOIN_ALONE && e < a.dim) write_row<TDT, ACC>(a, key, e, sum_partials(a, c, 0, 1, reach, e));
    if (lane == 0) reaches[wave] = reach;
    __syncthreads();
    for (int w = 0; w < JOIN_WAVES; ++w) {
        const int64_t far = reaches[w];
        if (far < JOIN_ALONE) continue;  // the same for every wave
        const int64_t of = c - wave + w;
        f32x8 acc = 0.0f;
        if (e < a.dim) acc = sum_partials(a, of, wave, JOIN_WAVES, far, e);
#pragma unroll
        for (int k = 0; k < 8; ++k) sums[wave][k * 64 + lane] = acc[k];
        __syncthreads();
        if (wave == w && e < a.dim) {
#pragma unroll
            for (int v = 0; v < JOIN_WAVES; ++v)
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = v == 0 ? sums[0][k * 64 + lane] : acc[k] + sums[v][k * 64 + lane];
            write_row<TDT, ACC>(a, key, e, acc);
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------- few tokens --

// A list of at most FEW_MAX tokens whose rows are at most FEW_SUMS column
// tiles is summed without a sort.  One launch instead of three: 511 x 2048
// FP16 added into 32000 rows take 9.9 us a call, against 16.6 (the kernel
// 6.6, against 14.6).  Every workgroup reads all ids, which is what more
// tokens or tiles cost: 4096 tiles take 9.0 us against 14.7, 8192 take 15.5
// against 14.9; one id in all of 512 tokens takes 14.6 against 14.9, of 1024
// tokens 26 against 18.5.  Eight waves a workgroup instead of four: 9.2
// against 7.6 us at 2044 tiles.
constexpr int FEW_MAX = 512;
constexpr int64_t FEW_SUMS = 4096;
constexpr int FEW_BLOCK = 256;
constexpr int FEW_WAVES = FEW_BLOCK / 64;
constexpr int FEW_ROUNDS = FEW_MAX / FEW_BLOCK;
constexpr int FEW_WORDS = FEW_MAX / 64;
// Table rows a clearing workgroup covers at most.
constexpr int64_t FEW_FLAGS = 4096;
// Tokens of one id that a single wave sums, all in flight at once.
constexpr int FEW_ALONE = SUM_UNROLL;

// Sum of the rows list[begin .. end), the lane's eight columns, in that order.  The
// last group reads its last row again for what it lacks.
template <int GDT>
__device__ __forceinline__ f32x8 sum_list(const SumArgs &a, const uint16_t *list, int begin, int end, int64_t e) {
    f32x8 acc = 0.0f;
    const bool whole = a.dim >= 8;
    const int64_t from = first_of_eight(e, a.dim);
    for (int j = begin; j < end; j += SUM_UNROLL) {
        Raw8<GDT> raw[SUM_UNROLL];
        const auto source = [&](int u) {
            const int t = __builtin_amdgcn_readfirstlane(list[j + u < end ? j + u : end - 1]);
            return static_cast<const char *>(a.grad_out) + int64_t(t) * a.grad_stride * elem_bytes<GDT>;
        };
        if (whole) {
#pragma unroll
            for (int u = 0; u < SUM_UNROLL; ++u) raw[u] = load_raw8<GDT>(source(u), from);
        } else {
#pragma unroll
            for (int u = 0; u < SUM_UNROLL; ++u) raw[u] = load_narrow8<GDT>(source(u), a.dim);
        }
#pragma unroll
        for (int u = 0; u < SUM_UNROLL; ++u) {
            if (j + u >= end) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] += raw_value<GDT>(raw[u], k);
        }
    }
    return acc;
}

// The whole gradient of up to FEW_MAX tokens in one launch, without a sort.
// Workgroup (t, tile) of the first `sums` compares every id with token t's;
// unless an earlier token has the same id, it sums the rows of all that have
// it, 512 columns.  The workgroups behind clear the rows that no token names.
template <int GDT, int TDT, bool ACC>
__global__ __launch_bounds__(FEW_BLOCK) void embedding_grad_few(SumArgs a, SortKeys s, uint32_t sums, ClearArgs clear) {
    __shared__ uint64_t masks[FEW_WORDS];  // bit i of word w: token 64 w + i has the id
    __shared__ uint16_t list[FEW_MAX];
    __shared__ float parts[FEW_WAVES][64 * 8];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int n = static_cast<int>(s.n), rounds = (n + FEW_BLOCK - 1) / FEW_BLOCK;
    const int first = wave * rounds * 64 + lane;
    uint32_t key[FEW_ROUNDS];
    if (n > 0) token_keys(s, first, rounds, key);
    if constexpr (!ACC) {
        if (blockIdx.x >= sums) {
            __shared__ u32x4 named[FEW_FLAGS / 16];
            uint8_t *flags = reinterpret_cast<uint8_t *>(named);
            const int64_t begin = clear.begin + int64_t(blockIdx.x - sums) * clear.rows_per_block;
            const int64_t left = clear.end - begin, count = left < clear.rows_per_block ? left : clear.rows_per_block;
            for (int i = tid; i * 16 < count; i += FEW_BLOCK) named[i] = u32x4{0, 0, 0, 0};
            __syncthreads();
#pragma unroll
            for (int r = 0; r < FEW_ROUNDS; ++r) {
                if (r >= rounds) break;
                const int64_t at = int64_t(key[r]) - begin;
                if (at >= 0 && at < count) flags[at] = 1;
            }
            __syncthreads();
            clear.table = static_cast<char *>(clear.table) + begin * clear.stride * elem_bytes<TDT>;
            clear.begin = 0;
            clear.end = clear.rows_per_block = count;
            clear.present = flags;
            clear_rows_of<TDT, FEW_BLOCK>(clear, 0);
            return;
        }
    }
    const uint32_t t = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int64_t e = (int64_t(tile) * 64 + lane) * 8;
    const bool on = e < a.dim;
    Raw8<GDT> own;  // wave 0: token t's row, needed unless an earlier token has the id
    if (wave == 0 && on) {
        const char *row = static_cast<const char *>(a.grad_out) + int64_t(t) * a.grad_stride * elem_bytes<GDT>;
        own = a.dim >= 8 ? load_raw8<GDT>(row, first_of_eight(e, a.dim)) : load_narrow8<GDT>(row, a.dim);
    }
    const int64_t id = load_index(s.ids, s.wide_ids, t);
    if (id < 0 || id >= s.rows || id == s.padding_id) return;
    const uint32_t mine = static_cast<uint32_t>(id);
#pragma unroll
    for (int r = 0; r < FEW_ROUNDS; ++r) {
        if (r >= rounds) break;
        const uint64_t same = __ballot(first + r * 64 < n && key[r] == mine);
        if (lane == 0) masks[wave * rounds + r] = same;
    }
    __syncthreads();
    int total = 0, earlier = 0, base = 0;  // tokens of the id: in all, before t, before this wave's
    for (int w = 0; w < FEW_WAVES * rounds; ++w) {
        const uint64_t m = masks[w];
        const int c = __builtin_popcountll(m);
        total += c;
        base += w < wave * rounds ? c : 0;
        earlier |= w * 64 + 63 < static_cast<int>(t) ? c
                   : w == static_cast<int>(t >> 6)  ? __builtin_popcountll(m & ((uint64_t(1) << (t & 63)) - 1))
                                                    : 0;
    }
    total = __builtin_amdgcn_readfirstlane(total);
    if (__builtin_amdgcn_readfirstlane(earlier)) return;
    f32x8 acc = 0.0f;
    if (total == 1) {
        if (wave > 0 || !on) return;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += raw_value<GDT>(own, k);
        write_row<TDT, ACC>(a, mine, e, acc);
        return;
    }
#pragma unroll
    for (int r = 0; r < FEW_ROUNDS; ++r) {
        if (r >= rounds) break;
        const bool same = first + r * 64 < n && key[r] == mine;
        const uint64_t m = __ballot(same);
        if (same) list[base + __builtin_popcountll(m & ((uint64_t(1) << lane) - 1))] = static_cast<uint16_t>(first + r * 64);
        base += __builtin_popcountll(m);
    }
    __syncthreads();
    if (total <= FEW_ALONE) {
        if (wave == 0 && on) write_row<TDT, ACC>(a, mine, e, sum_list<GDT>(a, list, 0, total, e));
        return;
    }
    if (on) acc = sum_list<GDT>(a, list, total * wave / FEW_WAVES, total * (wave + 1) / FEW_WAVES, e);
#pragma unroll
    for (int k = 0; k < 8; ++k) parts[wave][k * 64 + lane] = acc[k];
    __syncthreads();
    if (wave > 0 || !on) return;
#pragma unroll
    for (int w = 1; w < FEW_WAVES; ++w)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += parts[w][k * 64 + lane];
    write_row<TDT, ACC>(a, mine, e, acc);
}

// ------------------------------------------------------------- launchers --

// Waves that sum, where there are tokens enough: 2048 to 8192 measured alike.
constexpr int64_t SUM_WAVES = 4096;

EmbeddingPlan embedding_plan(int64_t n, int64_t rows, int64_t dim) {
    EmbeddingPlan p{};
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const int64_t pieces = (dim + 7) / 8;
    const int lg = log2_ceil(pieces);
    p.lg = lg < 3 ? 3 : lg > 6 ? 6 : lg;
    p.tiles = static_cast<int32_t>((pieces + 63) / 64);
    // chunks as long as leaves SUM_WAVES waves to sum, of 8 to 64 tokens
    const int64_t share = n * p.tiles / SUM_WAVES;
    p.chunk = share < 16 ? 8 : share < 32 ? 16 : share < 64 ? 32 : 64;
    p.chunks = (n + p.chunk - 1) / p.chunk;
    // the sums read whole groups of SUM_UNROLL keys and positions, and one key behind
    const int64_t list = (n + SUM_UNROLL + 1) * 4;
    p.keys[0] = take(list);
    p.pos[0] = take(list);
    if (n > SORT_SMALL_MAX) {
        p.keys[1] = take(list);
        p.pos[1] = take(list);
        p.counts = take((n + SORT_TILE - 1) / SORT_TILE * SORT_MAX_BINS * 4);
    }
    p.present = take(rows);
    p.partials = take(p.chunks * 2 * dim * 4);
    p.bytes = at;
    const int64_t units = p.lg == 6 ? p.chunks * p.tiles : p.chunks;
    p.sum_blocks = (units + (int64_t(1) << (8 - p.lg)) - 1) >> (8 - p.lg);
    return p;
}

template <int GDT>
static void launch_few_to(const SumArgs &a, int tgdt, const SortKeys &s, uint32_t sums, const ClearArgs &clear,
                          int64_t blocks, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(blocks)), block(FEW_BLOCK);
    const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, s, sums, clear); };
    switch (tgdt) {
    case G_F32: a.accumulate ? go(embedding_grad_few<GDT, G_F32, true>) : go(embedding_grad_few<GDT, G_F32, false>); break;
    case G_F16: a.accumulate ? go(embedding_grad_few<GDT, G_F16, true>) : go(embedding_grad_few<GDT, G_F16, false>); break;
    default: a.accumulate ? go(embedding_grad_few<GDT, G_BF16, true>) : go(embedding_grad_few<GDT, G_BF16, false>); break;
    }
}

template <int GDT, int TDT>
static hipError_t launch_sums(const SumArgs &a, int lg, dim3 grid, hipStream_t stream, int *launched) {
    const dim3 block(ROW_BLOCK), join(static_cast<unsigned>((a.chunks + JOIN_WAVES - 1) / JOIN_WAVES),
                                      static_cast<unsigned>((a.dim + 511) / 512));
    if (a.accumulate) hipLaunchKernelGGL((embedding_sum<GDT, TDT, true>), grid, block, 0, stream, a, lg);
    else hipLaunchKernelGGL((embedding_sum<GDT, TDT, false>), grid, block, 0, stream, a, lg);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    ++*launched;
    if (a.chunks < 2) return e;
    if (a.accumulate) hipLaunchKernelGGL((embedding_join<TDT, true>), join, dim3(JOIN_BLOCK), 0, stream, a);
    else hipLaunchKernelGGL((embedding_join<TDT, false>), join, dim3(JOIN_BLOCK), 0, stream, a);
    e = hipGetLastError();
    if (e == hipSuccess) ++*launched;
    return e;
}

template <int GDT>
static hipError_t launch_sums_to(const SumArgs &a, int tgdt, int lg, dim3 grid, hipStream_t stream, int *launched) {
    switch (tgdt) {
    case G_F32: return launch_sums<GDT, G_F32>(a, lg, grid, stream, launched);
    case G_F16: return launch_sums<GDT, G_F16>(a, lg, grid, stream, launched);
    default: return launch_sums<GDT, G_BF16>(a, lg, grid, stream, launched);
    }
}

hipError_t launch_embedding_grad(const EmbeddingGradArgs &g, const EmbeddingPlan &p, int gdt, int tgdt,
                                 hipStream_t stream, int *launched) {
    auto words = [&](int64_t off) { return reinterpret_cast<uint32_t *>(g.workspace + off); };
    SortKeys s{g.ids, nullptr, nullptr, g.n, g.rows, g.padding_id, g.wide_ids};
    const int key_bits = log2_ceil(g.rows + 1);
    const bool dense = !g.accumulate;
    ClearArgs clear{};
    clear.table = g.table_grad;
    clear.stride = g.table_stride;
    clear.dim = g.dim;
    clear.dtype = tgdt;
    const int piece_bits = log2_ceil((g.dim * (tgdt == G_F32 ? 4 : 2) + 15) / 16);
    clear.lg = piece_bits > 8 ? 8 : piece_bits;
    // Rows [begin, end) for one launch, CLEAR_ELEMS values per workgroup or
    // less and at most 2^20 workgroups; returns how many that takes.
    const auto take_rows = [&](int64_t begin, int64_t end, int64_t most) -> int64_t {
        clear.begin = begin;
        clear.end = end;
        const int64_t even = (end - begin + CLEAR_BLOCKS - 1) / CLEAR_BLOCKS;
        clear.rows_per_block = g.dim >= CLEAR_ELEMS ? 1 : CLEAR_ELEMS / g.dim;
        if (clear.rows_per_block > even) clear.rows_per_block = even > 0 ? even : 1;
        if (clear.rows_per_block > most) clear.rows_per_block = most;
        if (clear.rows_per_block <= ((end - begin) >> 20)) clear.rows_per_block = ((end - begin) >> 20) + 1;
        return dense ? (end - begin + clear.rows_per_block - 1) / clear.rows_per_block : 0;
    };
    SumArgs a{};
    a.grad_out = g.grad_out;
    a.table_grad = g.table_grad;
    a.partials = reinterpret_cast<float *>(g.workspace + p.partials);
    a.grad_stride = g.grad_stride;
    a.table_stride = g.table_stride;
    a.n = g.n;
    a.rows = g.rows;
    a.dim = g.dim;
    a.chunk = p.chunk;
    a.chunks = p.chunks;
    a.accumulate = g.accumulate;
    a.scale = g.scale;
    a.tiles = p.tiles;
    if (g.n <= FEW_MAX && g.n * p.tiles <= FEW_SUMS) {
        const int64_t sums = g.n * p.tiles, blocks = sums + take_rows(0, g.rows, FEW_FLAGS);
        switch (gdt) {
        case G_F32: launch_few_to<G_F32>(a, tgdt, s, static_cast<uint32_t>(sums), clear, blocks, stream); break;
        case G_F16: launch_few_to<G_F16>(a, tgdt, s, static_cast<uint32_t>(sums), clear, blocks, stream); break;
        default: launch_few_to<G_BF16>(a, tgdt, s, static_cast<uint32_t>(sums), clear, blocks, stream); break;
        }
        ++*launched;
        return hipGetLastError();
    }
    hipError_t e;
    int at = 0;  // the buffer that holds the sorted keys
    if (g.n <= SORT_SMALL_MAX) {
        // every row is cleared while one workgroup sorts
        const int passes = (key_bits + SORT_SMALL_BITS - 1) / SORT_SMALL_BITS;
        const int bits = (key_bits + passes - 1) / passes;
        const int64_t blocks = 1 + take_rows(0, g.rows, g.rows);
        const dim3 grid(static_cast<unsigned>(blocks));
        if (g.n <= SORT_TINY_MAX)
            hipLaunchKernelGGL((sort_small<256, SORT_TINY_MAX / 256>), grid, dim3(256), 0, stream, s, bits, passes,
                               words(p.keys[0]), words(p.pos[0]), clear);
        else
            hipLaunchKernelGGL((sort_small<1024, SORT_SMALL_MAX / 1024>), grid, dim3(1024), 0, stream, s, bits, passes,
                               words(p.keys[0]), words(p.pos[0]), clear);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        ++*launched;
    } else {
        const int passes = (key_bits + SORT_MAX_DIGIT_BITS - 1) / SORT_MAX_DIGIT_BITS;
        const int bits = (key_bits + passes - 1) / passes;
        const int64_t tiles = (g.n + SORT_TILE - 1) / SORT_TILE;
        const dim3 block(SORT_BLOCK);
        const int scanned = tiles > SORT_SELF_TILES;
        uint32_t *counts = words(p.counts);
        uint8_t *present = dense ? reinterpret_cast<uint8_t *>(g.workspace + p.present) : nullptr;
        if (dense) {
            hipLaunchKernelGGL(clear_flags, dim3(static_cast<unsigned>((g.rows + 4095) / 4096)), dim3(256), 0, stream,
                               present, g.rows);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            ++*launched;
        }
        clear.present = present;
        // The absent rows are cleared in equal shares by the launches behind
        // the first count, which finds them.
        const int64_t shares = 2 * passes - 1;
        int64_t share = 0;
        const auto grid = [&](bool first) {
            int64_t blocks = tiles;
            if (!first) {
                blocks += take_rows(g.rows * share / shares, g.rows * (share + 1) / shares, g.rows);
                ++share;
            }
            return dim3(static_cast<unsigned>(blocks));
        };
        for (int pass = 0; pass < passes; ++pass) {
            const int shift = pass * bits;
            at = pass & 1;
            const dim3 count_grid = grid(pass == 0);
            if (pass == 0)
                hipLaunchKernelGGL(radix_count<true>, count_grid, block, 0, stream, s, shift, bits, tiles, counts,
                                   present, clear);
            else
                hipLaunchKernelGGL(radix_count<false>, count_grid, block, 0, stream, s, shift, bits, tiles, counts,
                                   present, clear);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            ++*launched;
            if (scanned) {
                hipLaunchKernelGGL(radix_scan, dim3(1), dim3(SCAN_BLOCK), 0, stream, counts, tiles << bits);
                if ((e = hipGetLastError()) != hipSuccess) return e;
                ++*launched;
            }
            const dim3 scatter_grid = grid(false);
            if (pass == 0)
                hipLaunchKernelGGL(radix_scatter<true>, scatter_grid, block, 0, stream, s, shift, bits, tiles, counts,
                                   scanned, words(p.keys[at]), words(p.pos[at]), clear);
            else
                hipLaunchKernelGGL(radix_scatter<false>, scatter_grid, block, 0, stream, s, shift, bits, tiles, counts,
                                   scanned, words(p.keys[at]), words(p.pos[at]), clear);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            ++*launched;
            s.keys = words(p.keys[at]);
            s.pos = words(p.pos[at]);
        }
    }
    if (p.chunks == 0) return hipSuccess;
    a.keys = words(p.keys[at]);
    a.pos = words(p.pos[at]);
    const int lg = p.lg;
    const dim3 grid(static_cast<unsigned>(p.sum_blocks));
    switch (gdt) {
    case G_F32: return launch_sums_to<G_F32>(a, tgdt, lg, grid, stream, launched);
    case G_F16: return launch_sums_to<G_F16>(a, tgdt, lg, grid, stream, launched);
    default: return launch_sums_to<G_BF16>(a, tgdt, lg, grid, stream, launched);
    }
}

}  // namespace radamw
