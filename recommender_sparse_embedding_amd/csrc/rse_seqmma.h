// rse_seqmma.h -- 32 x 32 matrix-core tiles for the sequence attention:
// row-major tiles in LDS, the two products that read them, and the bucket
// arithmetic of a tile of event pairs.
//
// Every product has the events of one side ("columns", one per lane:
// column l % 32 of lane l) and of the other ("rows", one per accumulator
// register): register r of lane l holds row 8 (r / 4) + 4 (l / 32) + r % 4.
// X Y^T over dim (scores) leaves its result in that layout, and the same
// registers are, unmoved, an operand of the next product over the rows,
// because the order of a contraction is free as long as both operands agree.
#pragma once

#include "rse_seq.h"

namespace rse {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Row of register r for lanes of half h.
__device__ __forceinline__ constexpr int tile_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 v = __builtin_convertvector(f32x2{a, b}, bf16x2);   // to nearest even
    return __builtin_bit_cast(uint32_t, v);
}

// One value from the other half of the wave (lane l ^ 32).
__device__ __forceinline__ float other_half(float x) {
    const u32x2 s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(lane_id() < 32 ? s.y : s.x);
}

// Rows of D elements of T in LDS, in 16-byte chunks.  Chunk c of row r is
// kept at c ^ swz(r): a 16-byte read of one chunk of 16 rows, and a
// transposed read of 64 bytes of 8 rows, both fall in different banks.
template <typename T, int D>
struct Tile {
    static constexpr int CH = D * (int)sizeof(T) / 16;      // chunks of a row
    static constexpr int EPC = 16 / (int)sizeof(T);         // elements of a chunk
    static __device__ __forceinline__ int swz(int r) {
        if (CH == 4) return (r >> 2) & 3;
        if (CH == 8) return ((r >> 1) & 1) << 2 | ((r >> 2) & 1) << 1 | ((r >> 3) & 1);
        return (r & 1) << 2 | ((r >> 1) & 1) << 3 | ((r >> 2) & 1) | ((r >> 3) & 1) << 1;
    }
    static __device__ __forceinline__ int chunk_at(int r, int c) { return r * CH + (c ^ swz(r)); }
};

// The column operand of a product over dim: chunks 2 s + h of the lane's row.
template <typename T, int D>
struct ColFrag {
    u32x4 v[Tile<T, D>::CH / 2];
    __device__ __forceinline__ void load(const T* row, int h) {
#pragma unroll
        for (int s = 0; s < Tile<T, D>::CH / 2; ++s) v[s] = gload_u4(row + (2 * s + h) * Tile<T, D>::EPC);
    }
    __device__ __forceinline__ void load_lds(const u32x4* tile, int row, int h) {
#pragma unroll
        for (int s = 0; s < Tile<T, D>::CH / 2; ++s) v[s] = tile[Tile<T, D>::chunk_at(row, 2 * s + h)];
    }
    __device__ __forceinline__ void negate() {
#pragma unroll
        for (int s = 0; s < Tile<T, D>::CH / 2; ++s) v[s] ^= sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
    }
};

// Elements e .. e + 3 of a chunk as fp32.
template <typename T>
__device__ __forceinline__ f32x4 chunk_f32(u32x4 v, int e) {
    if (sizeof(T) == 4) return __builtin_bit_cast(f32x4, v);
    const uint32_t a = v[e / 2], b = v[e / 2 + 1];
    return f32x4{__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u), __uint_as_float(b << 16),
                 __uint_as_float(b & 0xFFFF0000u)};
}

template <typename T>
__device__ __forceinline__ f32x16 mma_chunk(u32x4 a, u32x4 b, f32x16 c);
template <>
__device__ __forceinline__ f32x16 mma_chunk<uint16_t>(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16 mma_chunk<float>(u32x4 a, u32x4 b, f32x16 c) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[e], y[e], c, 0, 0, 0);
    return c;
}

// rows r0 .. r0 + 31 of an LDS tile times the column operand, over dim.
template <typename T, int D>
__device__ __forceinline__ f32x16 mma_rows(const u32x4* tile, int r0, const ColFrag<T, D>& col, f32x16 c) {
    const int lane = lane_id(), row = r0 + (lane & 31), h = lane >> 5;
#pragma unroll
    for (int s = 0; s < Tile<T, D>::CH / 2; ++s)
        c = mma_chunk<T>(tile[Tile<T, D>::chunk_at(row, 2 * s + h)], col.v[s], c);
    return c;
}

// A 32 x 32 tile's values as the operand of a product over its rows.
template <typename T>
struct RowOperand;
template <>
struct RowOperand<float> {
    f32x16 v;
    __device__ __forceinline__ void set(const f32x16& x) { v = x; }
    __device__ __forceinline__ void set_rest(const f32x16&, const RowOperand&) { v = f32x16{}; }
};
template <>
struct RowOperand<uint16_t> {
    u32x4 v[2];
    __device__ __forceinline__ void set(const f32x16& x) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[s][i] = pack_bf16(x[8 * s + 2 * i], x[8 * s + 2 * i + 1]);
    }
    // what hi's rounding left of x (exact), rounded in turn
    __device__ __forceinline__ void set_rest(const f32x16& x, const RowOperand& hi) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[s][i] = pack_bf16(x[8 * s + 2 * i] - __uint_as_float(hi.v[s][i] << 16),
                                    x[8 * s + 2 * i + 1] - __uint_as_float(hi.v[s][i] & 0xFFFF0000u));
    }
};

// acc[d, column] += sum over rows r0 .. r0 + 31 of tile[row, 32 dt + d] x[row, column].
template <int D>
__device__ __forceinline__ f32x16 mma_over_rows(const u32x4* tile, int r0, int dt, const RowOperand<float>& x, f32x16 acc) {
    const int lane = lane_id(), d = 32 * dt + (lane & 31), h = lane >> 5;
    const float* f = reinterpret_cast<const float*>(tile);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int row = r0 + tile_row(r, h);
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(f[Tile<float, D>::chunk_at(row, d >> 2) * 4 + (d & 3)], x.v[r], acc, 0, 0, 0);
    }
    return acc;
}
// bf16: four rows of a column at a time by the transposing LDS read: in each
// group of 16 lanes, lane i supplies the address of row i / 4, elements
// 4 (i % 4) .., and receives column i of the four rows.
template <int D>
__device__ __forceinline__ f32x16 mma_over_rows(const u32x4* tile, int r0, int dt, const RowOperand<uint16_t>& x, f32x16 acc) {
    const int lane = lane_id(), h = lane >> 5, i = lane & 15;
    const int c = 4 * dt + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);       // chunk of elements 32 dt + 16 half + 4 (i % 4)
    const char* base = reinterpret_cast<const char*>(tile);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        s16x4 p[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int row = r0 + 16 * s + 8 * u + 4 * h + (i >> 2);
            const char* at = base + Tile<uint16_t, D>::chunk_at(row, c) * 16 + (i & 1) * 8;
            p[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((RSE_LDS s16x4*)at);
        }
        u32x4 a;
        a.xy = __builtin_bit_cast(u32x2, p[0]);
        a.zw = __builtin_bit_cast(u32x2, p[1]);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, x.v[s]), acc, 0, 0, 0);
    }
    return acc;
}

// Elements 32 dt .. 32 dt + 31 of the lane's column from acc, times f, to
// p[0 .. 31] of the column's row; 16 bytes a store.
__device__ __forceinline__ void store_column(float* p, const f32x16& acc, float f) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        gstore_f4(p + 8 * j + 4 * h, f32x4{acc[4 * j] * f, acc[4 * j + 1] * f, acc[4 * j + 2] * f, acc[4 * j + 3] * f});
}
__device__ __forceinline__ void store_column(uint16_t* p, const f32x16& acc, float f) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        // halves 0 / 1 hold elements 8 j + (0..3) / (4..7): swapped so that
        // half 0 holds the eight of j and half 1 those of j + 1
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t a = pack_bf16(acc[4 * j + 2 * i] * f, acc[4 * j + 2 * i + 1] * f);
            const uint32_t b = pack_bf16(acc[4 * j + 4 + 2 * i] * f, acc[4 * j + 5 + 2 * i] * f);
            const u32x2 s = __builtin_amdgcn_permlane32_swap(a, b, false, false);
            o[i] = s.x;
            o[2 + i] = s.y;
        }
        gstore_u4(p + 8 * (j + h), o);
    }
}

// ---------------------------------------------------------------- buckets --
// A wave's copy of one head's boundaries and bias (lane l: entries l and
// 64 + l): a wave-uniform distance finds its bucket by two comparisons and
// bit counts, and any entry is read as a scalar.
struct WaveBuckets {
    int32_t bnd[2];
    float bias[2];
    int n;
    __device__ __forceinline__ void load(const SeqHeader* hdr, const float* head_bias, int n_bounds, float factor) {
        n = n_bounds;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int at = 64 * u + lane_id();
            bnd[u] = hdr->bounds[at];
            bias[u] = at <= n_bounds ? head_bias[at] * factor : 0.f;
        }
    }
    __device__ __forceinline__ int bucket(int32_t d) const {
        const int b = __popcll(__ballot(bnd[0] <= d)) + __popcll(__ballot(bnd[1] <= d));
        return b < n ? b : n;       // the padding counts where d is INT32_MAX
    }
    __device__ __forceinline__ int32_t boundary(int m) const {
        return __builtin_amdgcn_readlane(m < 64 ? bnd[0] : bnd[1], m & 63);
    }
    __device__ __forceinline__ float value(int b) const {
        return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(b < 64 ? bias[0] : bias[1]), b & 63));
    }
};

__device__ __forceinline__ int32_t wave_min(int32_t x) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        const int32_t y = __shfl_xor(x, m, WAVE);
        x = y < x ? y : x;
    }
    return x;
}
__device__ __forceinline__ int32_t wave_max(int32_t x) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        const int32_t y = __shfl_xor(x, m, WAVE);
        x = y > x ? y : x;
    }
    return x;
}

constexpr float LOG2E = 1.4426950408889634f;
// More distinct buckets than this in a tile: looked up event by event.
constexpr int CHAIN = 6;

// Buckets of the lane's column and the 16 rows of a tile that spans buckets
// lo .. hi: compared with the boundaries between them, or searched.
template <bool column_first>
__device__ __forceinline__ void bucket_index(int (&idx)[16], const WaveBuckets& wb, int lo, int hi, const int32_t* row_pos,
                                             int32_t col_pos, bool cells, const uint32_t* s_cell,
                                             const int32_t* s_bounds) {
    const int h = lane_id() >> 5;
    int32_t dist[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const i32x4 p = *reinterpret_cast<const i32x4*>(row_pos + 8 * j + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) dist[4 * j + i] = column_first ? seq_dist(col_pos, p[i]) : seq_dist(p[i], col_pos);
    }
    if (hi - lo <= 2 * CHAIN) {
#pragma unroll
        for (int r = 0; r < 16; ++r) idx[r] = lo;
        for (int m = lo; m < hi; ++m) {
            const int32_t edge = wb.boundary(m);
#pragma unroll
            for (int r = 0; r < 16; ++r) idx[r] += dist[r] >= edge;
        }
    } else if (cells) {
        const uint8_t* cell = reinterpret_cast<const uint8_t*>(s_cell);
#pragma unroll
        for (int r = 0; r < 16; ++r) idx[r] = seq_bucket_cell(cell, s_bounds, wb.n, dist[r]);
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) idx[r] = seq_bucket(s_bounds, wb.n, dist[r]);
    }
}

// Bias (base 2) of the lane's column for the 16 rows of a 32 x 32 tile that
// may span buckets lo .. hi, added to s times c.  row_pos: positions of the
// tile's rows in LDS.  A tile of few buckets compares each distance with the
// boundaries between them; with many, each distance is searched in the LDS
// copy of the boundaries.
// `column_first`: the column event is the query (distance = column - row).
template <bool column_first>
__device__ __forceinline__ f32x16 add_bias(f32x16 s, float c, const WaveBuckets& wb, int lo, int hi, const int32_t* row_pos,
                                           int32_t col_pos, bool cells, const uint32_t* s_cell,
                                           const int32_t* s_bounds, const float* s_bias) {
    const int h = lane_id() >> 5;
    int32_t dist[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const i32x4 p = *reinterpret_cast<const i32x4*>(row_pos + 8 * j + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) dist[4 * j + i] = column_first ? seq_dist(col_pos, p[i]) : seq_dist(p[i], col_pos);
    }
    f32x16 b;
    if (hi - lo <= CHAIN) {
        const float b0 = wb.value(lo);
#pragma unroll
        for (int r = 0; r < 16; ++r) b[r] = b0;
        for (int m = lo; m < hi; ++m) {
            const int32_t edge = wb.boundary(m);
            const float bm = wb.value(m + 1);
#pragma unroll
            for (int r = 0; r < 16; ++r) b[r] = dist[r] >= edge ? bm : b[r];
        }
    } else if (cells) {
        const uint8_t* cell = reinterpret_cast<const uint8_t*>(s_cell);
#pragma unroll
        for (int r = 0; r < 16; ++r) b[r] = s_bias[seq_bucket_cell(cell, s_bounds, wb.n, dist[r])];
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) b[r] = s_bias[seq_bucket(s_bounds, wb.n, dist[r])];
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = __builtin_fmaf(s[r], c, b[r]);
    return s;
}

// ------------------------------------------------------------- tile finder --
// Tiles of TQ events of every sequence, numbered without a table: sequence b
// has the numbers offsets[b] / TQ + b and on, at least as many as its tiles
// (a number past its last tile is idle).  True with the sequence's range and
// the tile's index; also checks all offsets, a part in each block.
__host__ __device__ __forceinline__ int64_t tile_slots(int64_t n_events, int64_t batch, int tq) { return n_events / tq + batch; }

__device__ __forceinline__ bool find_tile(const SeqArgs& a, int64_t slot, int tq, int64_t& s, int& len, int& tile,
                                          bool check) {
    if (check) {
        const int64_t i = slot * blockDim.x + threadIdx.x;
        if (i < a.batch) {
            const int64_t x = a.offsets[i], y = a.offsets[i + 1];
            if (x > y || (i == 0 && x != 0) || (i == a.batch - 1 && y != a.n_events))
                set_status(&a.hdr->status, RSE_ERR_BAD_INPUT);
        }
    }
    const int64_t b = wave_last_le(a.batch, [&](int64_t x) { return a.offsets[x] / tq + x; }, slot);
    s = a.offsets[b];
    const int64_t e = a.offsets[b + 1];
    const int64_t t = slot - (s / tq + b);
    if (s < 0 || e < s || e > a.n_events || e - s > a.max_len) {
        if (lane_id() == 0) set_status(&a.hdr->status, RSE_ERR_BAD_INPUT);
        return false;
    }
    if (t < 0 || t * tq >= e - s) return false;
    len = (int)(e - s);
    tile = (int)t;
    return true;
}

}  // namespace rse
