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

#include <cstddef>

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

// The lane, formed anew where it stands (the compiler may not keep what it
// derives from it over a loop): addresses of lookups kept so were spilled, and
// a spill's reload waits for every load in flight, the next tile's among them.
__device__ __forceinline__ int lane_anew() {
    uint32_t none = 0;
    asm volatile("" : "+s"(none));
    return (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, none));
}

// One value from the other half of the wave (lane l ^ 32).
__device__ __forceinline__ float other_half(float x) {
    const u32x2 s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(lane_id() < 32 ? s.y : s.x);
}

// The sum of the registers, by halves: probabilities far below a row's largest
// are added to each other before they meet its running sum (4096 events of
// which 4095 weigh 2^-25: one by one half of them were lost; 218 -> 222 us on
// the forward of 16 histories of up to 4096).
__device__ __forceinline__ float sum_registers(const f32x16& x) {
    float s[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) s[r] = x[r] + x[r + 8];
#pragma unroll
    for (int n = 4; n > 0; n >>= 1)
#pragma unroll
        for (int r = 0; r < n; ++r) s[r] += s[r + n];
    return s[0];
}

// Rows of D elements of T in LDS, in 16-byte chunks.  Chunk c of row r is
// kept at c ^ swz(r): a 16-byte read of one chunk of 16 rows, and a
// transposed read of 64 bytes of 8 rows, both fall in different banks.
template <typename T, int D>
struct Tile {
    static constexpr int CH = D * (int)sizeof(T) / 16;      // chunks of a row
    static constexpr int EPC = 16 / (int)sizeof(T);         // elements of a chunk
    static __device__ __forceinline__ constexpr int swz(int r) {
        if (CH == 4) return (r >> 2) & 3;
        if (CH == 8) return ((r >> 1) & 1) << 2 | ((r >> 2) & 1) << 1 | ((r >> 3) & 1);
        return (r & 1) << 2 | ((r >> 1) & 1) << 3 | ((r >> 2) & 1) | ((r >> 3) & 1) << 1;
    }
    static __device__ __forceinline__ constexpr int chunk_at(int r, int c) { return r * CH + (c ^ swz(r)); }
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

// acc[dt][d, column] += sum over rows r0 .. r0 + 31 of tile[row, 32 dt + d] x[row, column].
template <typename T, int D, int TERMS = 2>
struct OverRows;
template <int D, int TERMS>
struct OverRows<float, D, TERMS> {
    static __device__ __forceinline__ void add(f32x16& acc, const u32x4* tile, int r0, int dt, const f32x16& x) {
        const int lane = lane_id(), h = lane >> 5, d = 32 * dt + (lane & 31);
        const float* f = reinterpret_cast<const float*>(tile);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = r0 + tile_row(r, h);
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(f[Tile<float, D>::chunk_at(row, d >> 2) * 4 + (d & 3)], x[r], acc, 0, 0, 0);
        }
    }
    static __device__ __forceinline__ void add(f32x16 (&acc)[D / 32], const u32x4* tile, int r0, const f32x16& x) {
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt) add(acc[dt], tile, r0, dt, x);
    }
};
// bf16: x enters as the sum of TERMS bf16 values, each the rounded remainder of
// those before it, and is left less what entered (exact).  Half of the rows
// after the other, so that few operands are held at once (both halves formed
// first: spills in the step, 256 users of 1..1000 events 34 us for 26).  Four
// rows of a column at a time by the transposing LDS read: in each group of 16 lanes,
// lane i supplies the address of row i / 4, elements 4 (i % 4) .., and receives
// column i of the four rows.
template <int D, int TERMS>
struct OverRows<uint16_t, D, TERMS> {
    static __device__ __forceinline__ void add(f32x16 (&acc)[D / 32], const u32x4* tile, int r0, f32x16& x) {
        const int lane = lane_id(), h = lane >> 5, i = lane & 15;
        const char* base = reinterpret_cast<const char*>(tile);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            u32x4 v[TERMS];
#pragma unroll
            for (int t = 0; t < TERMS; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[t][j] = pack_bf16(x[8 * s + 2 * j], x[8 * s + 2 * j + 1]);
                    x[8 * s + 2 * j] -= __uint_as_float(v[t][j] << 16);
                    x[8 * s + 2 * j + 1] -= __uint_as_float(v[t][j] & 0xFFFF0000u);
                }
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) {
                const int c = 4 * dt + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);       // chunk of elements 32 dt + 16 half + 4 (i % 4)
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
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
                    acc[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, v[t]), acc[dt], 0, 0, 0);
            }
        }
    }
};

// Elements 32 dt .. 32 dt + 31 of the lane's column from acc, times f, to
// p[0 .. 31] of the column's row; 16 bytes a store.
__device__ __forceinline__ void store_column(float* p, const f32x16& acc, float f) {
    const int h = lane_anew() >> 5;
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

__device__ __forceinline__ void store_four(float* p, f32x4 x) { gstore_f4(p, x); }
__device__ __forceinline__ void store_four(uint16_t* p, f32x4 x) {
    *(RSE_GLOBAL u32x2*)p = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
}

// ------------------------------------------------------------ async copies --
// 16 bytes (or 4) from memory straight to LDS: lane l's piece lands 16 l (4 l)
// bytes past `lds`, the same of all lanes.  In assembly, so that the compiler does not make every read of
// LDS wait for the loads in flight to other buffers; the waits are the
// caller's.  Nothing is returned to registers.  m0 is named as written (the compiler
// may keep a value there from one use to the next; it warns that it does not save
// registers of its own, which nothing here asks for).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ uint32_t lds_address(const void* lds) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(RSE_LDS const void*)lds);
}
__device__ __forceinline__ void to_lds(const void* p, const void* lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds_address(lds)) : "memory", "m0");
}
__device__ __forceinline__ void to_lds4(const void* p, const void* lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "s"(lds_address(lds)) : "memory", "m0");
}
// from `bytes` behind a place that the wave has in common.  A memory instruction
// may read a scalar register five wait states after a vector one wrote it, as `from`
// is, and the compiler does not count those inside the assembly: the move is one,
// s_nop 3 four.
__device__ __forceinline__ void to_lds(const void* base, uint32_t bytes, const void* lds) {
    const int64_t from = uniform((int64_t)(uintptr_t)base);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(bytes), "s"(from), "s"(lds_address(lds)) : "memory", "m0");
}
__device__ __forceinline__ void to_lds4(const void* base, uint32_t bytes, const void* lds) {
    const int64_t from = uniform((int64_t)(uintptr_t)base);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dword %0, %1" ::"v"(bytes), "s"(from), "s"(lds_address(lds)) : "memory", "m0");
}
#pragma clang diagnostic pop
// At most N of the wave's memory operations are still in flight.  The compiler
// does not see this wait: for what it loads to registers itself it adds its own
// where the value is first used, be it in a loop, unless none_left, which it
// sees, comes before.
template <int N>
__device__ __forceinline__ void loads_left() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
__device__ __forceinline__ void none_left() { __builtin_amdgcn_s_waitcnt(0x0F70); }        // vmcnt(0), the others free
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ---------------------------------------------------------------- buckets --
// A wave's copy of one head's boundaries and bias (lane l: entries l and
// 64 + l): a wave-uniform distance finds its bucket by two comparisons and
// bit counts, and any entry is read as a scalar.
struct WaveBuckets {
    int32_t bnd[2];
    float bias[2];
    int n;
    __device__ __forceinline__ void load(const SeqHeader* hdr, const float* head_bias, int n_bounds) {
        n = n_bounds;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int at = 64 * u + lane_id();
            bnd[u] = hdr->bounds[at];
            bias[u] = at <= n_bounds ? bias2(head_bias[at]) : 0.f;
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

// The same where the lanes' heads differ: `bias` is the lane's row of a table
// in LDS, in base 2.
struct LaneBuckets {
    int32_t bnd[2];
    const float* bias;
    int n;
    __device__ __forceinline__ void load(const SeqHeader* hdr, const float* lane_bias, int n_bounds) {
        n = n_bounds;
        bias = lane_bias;
#pragma unroll
        for (int u = 0; u < 2; ++u) bnd[u] = hdr->bounds[64 * u + lane_id()];
    }
    __device__ __forceinline__ int bucket(int32_t d) const {
        const int b = __popcll(__ballot(bnd[0] <= d)) + __popcll(__ballot(bnd[1] <= d));
        return b < n ? b : n;
    }
    __device__ __forceinline__ int32_t boundary(int m) const {
        return __builtin_amdgcn_readlane(m < 64 ? bnd[0] : bnd[1], m & 63);
    }
    __device__ __forceinline__ float value(int b) const { return bias[b]; }
};

// Lowest and highest of each half of the wave, by rotations within rows of 16
// lanes and one exchange of rows (no trip through LDS: five dependent
// shuffles took some 600 cycles of a tile).
template <int N>
__device__ __forceinline__ int32_t row_ror(int32_t x) { return __builtin_amdgcn_update_dpp(x, x, 0x120 + N, 0xF, 0xF, false); }
template <bool MAX>
__device__ __forceinline__ int32_t half_extreme(int32_t x) {
    auto pick = [](int32_t a, int32_t b) { return MAX ? (a > b ? a : b) : (a < b ? a : b); };
    x = pick(x, row_ror<8>(x));
    x = pick(x, row_ror<4>(x));
    x = pick(x, row_ror<2>(x));
    x = pick(x, row_ror<1>(x));
    const u32x2 s = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
    return pick((int32_t)s.x, (int32_t)s.y);
}
__device__ __forceinline__ int32_t half_min(int32_t x) { return half_extreme<false>(x); }
__device__ __forceinline__ int32_t half_max(int32_t x) { return half_extreme<true>(x); }

constexpr float LOG2E = 1.4426950408889634f;
// More boundaries than this inside a tile: looked up event by event.
constexpr int CHAIN = 6;

__device__ __forceinline__ int32_t sat_add(int32_t a, int32_t b) { return __builtin_elementwise_add_sat(a, b); }

// What a kernel holds in LDS to look buckets up pair by pair.
struct LdsBuckets {
    int32_t bounds[RSE_SEQ_MAX_BOUNDARIES + 1];
    uint32_t cell[128];
    __device__ __forceinline__ void load(const SeqHeader* h) {
        for (int t = threadIdx.x; t <= RSE_SEQ_MAX_BOUNDARIES; t += blockDim.x) {
            bounds[t] = h->bounds[t];
            cell[t] = reinterpret_cast<const uint32_t*>(h->cell)[t];
        }
    }
};

// The rows of a 32 x 32 tile span positions range[0] .. range[1]; its pairs'
// distances the buckets lo .. hi.  column_first: distance = column - row.
//  - one bucket (most tiles of a long history): the bias is a constant;
//  - up to CHAIN boundaries: each is passed by the rows on one side of a
//    position that is the lane's own (col_pos -/+ the boundary, saturated),
//    one comparison per pair and boundary (all sixteen before their uses: a
//    selection right behind its comparison waits for it).  A saturated threshold is met
//    wrongly only by a row at the very end of int32: such tiles go with
//  - many: every pair is looked up (find_pairs), into LDS as bytes in the
//    order of the registers, so that the heads share the work.
template <bool column_first>
struct TileBuckets {
    int lo, hi;
    bool many;
    template <typename WB>
    __device__ __forceinline__ void set(const WB& wb, int32_t col_lo, int32_t col_hi, const int32_t* range) {
        const int32_t r_lo = __builtin_amdgcn_readfirstlane(range[0]), r_hi = __builtin_amdgcn_readfirstlane(range[1]);
        lo = wb.bucket(column_first ? seq_dist(col_lo, r_hi) : seq_dist(r_lo, col_hi));
        hi = wb.bucket(column_first ? seq_dist(col_hi, r_lo) : seq_dist(r_hi, col_lo));
        many = lo != hi && (hi - lo > CHAIN || (column_first ? r_lo == INT32_MIN : r_hi == INT32_MAX));
    }
    template <typename WB>
    __device__ __forceinline__ int32_t threshold(const WB& wb, int m, int32_t col_pos) const {
        const int32_t edge = wb.boundary(m);
        return column_first ? seq_dist(col_pos, edge) : sat_add(col_pos, edge);
    }
    static __device__ __forceinline__ bool passed(int32_t row, int32_t threshold) {
        return column_first ? row <= threshold : row >= threshold;
    }
    // Of `many` tiles: registers 4 j .. 4 j + 3 for j = first, + step, ... < 4.
    static __device__ __forceinline__ void find_pairs(u32x4* bytes, int first, int step, const LdsBuckets& lb, int n, bool cells,
                                                      const int32_t* row_pos, int32_t col_pos) {
        const int lane = lane_anew(), h = lane >> 5;
        uint32_t* mine = reinterpret_cast<uint32_t*>(bytes + lane);
#pragma unroll 1
        for (int j = first; j < 4; j += step) {
            const i32x4 p = *reinterpret_cast<const i32x4*>(row_pos + 8 * j + 4 * h);
            uint32_t packed = 0;
            if (cells) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    packed |= seq_bucket_cell(reinterpret_cast<const uint8_t*>(lb.cell), lb.bounds, n,
                                              column_first ? seq_dist(col_pos, p[i]) : seq_dist(p[i], col_pos)) << (8 * i);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    packed |= seq_bucket(lb.bounds, n, column_first ? seq_dist(col_pos, p[i]) : seq_dist(p[i], col_pos)) << (8 * i);
            }
            mine[j] = packed;
        }
    }
    static __device__ __forceinline__ int pair(const u32x4& bytes, int r) { return (bytes[r >> 2] >> (8 * (r & 3))) & 255; }
    static __device__ __forceinline__ void positions(int32_t (&p)[16], const int32_t* row_pos) {
        const int h = lane_anew() >> 5;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const i32x4 v = *reinterpret_cast<const i32x4*>(row_pos + 8 * j + 4 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[4 * j + i] = v[i];
        }
    }
    // s c + bias + shift of every pair (WB: WaveBuckets, or LaneBuckets where the
    // lanes' heads differ)
    template <typename WB>
    __device__ __forceinline__ f32x16 logits(f32x16 s, float c, float shift, const WB& wb, const u32x4* bytes,
                                             const float* s_bias, const int32_t* row_pos, int32_t col_pos) const {
        if (lo == hi) {
            const float b = wb.value(lo) + shift;
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = __builtin_fmaf(s[r], c, b);
        } else if (!many) {
            int32_t p[16];
            positions(p, row_pos);
            float b[16];
            const float b0 = wb.value(lo) + shift;
            {
                const int32_t th = threshold(wb, lo, col_pos);
                const float bm = wb.value(lo + 1) + shift;
                bool c[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) c[r] = passed(p[r], th);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = 0; r < 16; ++r) b[r] = c[r] ? bm : b0;
            }
#pragma unroll 1
            for (int m = lo + 1; m < hi; ++m) {
                const int32_t th = threshold(wb, m, col_pos);
                const float bm = wb.value(m + 1) + shift;
                bool c[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) c[r] = passed(p[r], th);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = 0; r < 16; ++r) b[r] = c[r] ? bm : b[r];
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = __builtin_fmaf(s[r], c, b[r]);
        } else {
            const u32x4 at = bytes[lane_anew()];
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = __builtin_fmaf(s[r], c, s_bias[pair(at, r)] + shift);
        }
        return s;
    }
    // bucket of every pair (lo < hi)
    __device__ __forceinline__ void index(int (&idx)[16], const WaveBuckets& wb, const u32x4* bytes, const int32_t* row_pos,
                                          int32_t col_pos) const {
        if (!many) {
            int32_t p[16];
            positions(p, row_pos);
#pragma unroll
            for (int r = 0; r < 16; ++r) idx[r] = lo;
#pragma unroll 1
            for (int m = lo; m < hi; ++m) {
                const int32_t th = threshold(wb, m, col_pos);
#pragma unroll
                for (int r = 0; r < 16; ++r) idx[r] += passed(p[r], th);
            }
        } else {
            const u32x4 at = bytes[lane_anew()];
#pragma unroll
            for (int r = 0; r < 16; ++r) idx[r] = pair(at, r);
        }
    }
};

// ------------------------------------------------------------- tile finder --
// Tiles of tq events of every sequence, numbered in one of two ways.
//  - per_seq > 0 (no sequence has more tiles): items t * batch and on are the
//    tiles t of the sequences; idle where the sequence is shorter.  No search, and tiles of
//    equal index stand together, so that long work can start first.
//  - per_seq = 0, where that would leave most items idle: sequence b has the
//    numbers offsets[b] / tq + b and on, at least as many as its tiles, found
//    by a search.
// Every call checks a part of the offsets.
struct TileGrid {
    int64_t items;
    int64_t per_seq;
};
inline TileGrid tile_grid(int64_t n_events, int64_t batch, int64_t max_len, int tq) {
    const int64_t slots = n_events / tq + batch, longest = max_len < n_events ? max_len : n_events;
    const int64_t per_seq = (longest + tq - 1) / tq;
    if (per_seq <= 4 * slots / (batch > 0 ? batch : 1)) return {per_seq * batch, per_seq};
    return {slots, 0};
}

// The item's sequence (first event, length) and tile; false if it is idle.
// backwards: items of a grid by tile index start from the last tile.
__device__ __forceinline__ bool find_tile(const SeqArgs& a, const TileGrid& g, int64_t item, int tq, bool backwards,
                                          int64_t& s, int& len, int& tile, bool check) {
    if (check) {
        for (int64_t i = item * blockDim.x + threadIdx.x; i < a.batch; i += g.items * blockDim.x) {
            const int64_t x = a.offsets[i], y = a.offsets[i + 1];
            if (x > y || (i == 0 && x != 0) || (i == a.batch - 1 && y != a.n_events))
                set_status(&a.hdr->status, RSE_ERR_BAD_INPUT);
        }
    }
    int64_t b, t;
    if (g.per_seq) {
        t = item / a.batch;
        b = item - t * a.batch + t % a.batch;           // a sequence's tiles on different XCDs
        if (b >= a.batch) b -= a.batch;
        if (backwards) t = g.per_seq - 1 - t;
    } else {
        b = wave_last_le(a.batch, [&](int64_t x) { return a.offsets[x] / tq + x; }, item);
        t = item - (a.offsets[b] / tq + b);
    }
    s = uniform(a.offsets[b]);
    const int64_t e = uniform(a.offsets[b + 1]);
    t = uniform(t);
    if (s < 0 || e < s || e > a.n_events || e - s > a.max_len) {
        if (lane_id() == 0) set_status(&a.hdr->status, RSE_ERR_BAD_INPUT);
        return false;
    }
    if (t < 0 || t * tq >= e - s) return false;
    len = (int)(e - s);
    tile = (int)t;
    return true;
}

// The tiles a block works through, one after the other.  By sequence: block x
// takes sequences x, + blocks, ..., all their tiles in order; the next
// sequence's offsets are loaded one ahead, so that its first tile can be on
// its way while the last one of the current sequence is computed.
struct SeqTiles {
    int64_t s;
    int len, tile;
    bool valid;
    int64_t b, step;
    int phase, stride;                          // the block's tiles: phase, + stride, ...
    int64_t next0, next1;                       // offsets of sequence b + step, as loaded
    // `split` blocks share a sequence's tiles
    __device__ __forceinline__ void begin(const SeqArgs& a, int64_t block, int64_t n_blocks, int split, bool check) {
        const int64_t first = block / split, blocks = n_blocks / split;
        phase = (int)(block % split);
        stride = split;
        if (check)
            for (int64_t i = block * blockDim.x + threadIdx.x; i < a.batch; i += n_blocks * blockDim.x) {
                const int64_t x = a.offsets[i], y = a.offsets[i + 1];
                if (x > y || (i == 0 && x != 0) || (i == a.batch - 1 && y != a.n_events))
                    set_status(&a.hdr->status, RSE_ERR_BAD_INPUT);
            }
        b = first - blocks;
        step = blocks;
        fetch(a);
        next_sequence(a);
    }
    __device__ __forceinline__ void fetch(const SeqArgs& a) {
        const int64_t n = b + step < a.batch ? b + step : a.batch - 1;
        next0 = a.offsets[n];
        next1 = a.offsets[n + 1];
    }
    __device__ __forceinline__ void next_sequence(const SeqArgs& a) {
        for (;;) {
            b += step;
            valid = b < a.batch;
            if (!valid) return;
            s = uniform(next0);
            const int64_t e = uniform(next1);
            fetch(a);
            if (s < 0 || e < s || e > a.n_events || e - s > a.max_len) {
                if (lane_id() == 0) set_status(&a.hdr->status, RSE_ERR_BAD_INPUT);
                continue;
            }
            len = (int)(e - s);
            tile = phase;
            if (tile * 32 < len) return;
        }
    }
    __device__ __forceinline__ void advance(const SeqArgs& a) {
        if ((tile + stride) * 32 < len) tile += stride;
        else next_sequence(a);
    }
};

// Blocks of W waves that go through the short sequences, for `heads` of them
// side by side: four times as many as fit the GPU at once (what is left over
// evens out; with as many as fit, dq took 620 us for 553), a
// sequence's tiles shared by several where there are few sequences.
struct ShortGrid {
    int64_t blocks;
    int split;
};
inline ShortGrid short_grid(int64_t batch, int64_t heads, int64_t max_len, int waves) {
    const int64_t fit = (8192 / waves + heads - 1) / heads;
    const int64_t seqs = batch < fit ? batch : fit, tiles = (max_len + 31) / 32;
    int64_t split = seqs > 0 ? fit / seqs : 1;
    split = split > tiles ? tiles : split;
    if (split < 1) split = 1;
    return {seqs * split, (int)split};
}

// ------------------------------------------------------------------ shapes --
// A block's waves and what they share.  A team of waves stages tiles of rows
// together; WH waves take heads side by side, WQ waves tiles of 32 columns.
//  - long sequences: one team of 4, tiles of 64 rows (two buffers of two
//    tensors: at most 64 KiB), either 4 column tiles of one head, or one
//    column tile of 4 heads that share keys (equal work for every wave, and
//    the buckets of a tile looked up once for the 4);
//  - up to SHORT events, where such a block would mostly idle: every wave a
//    team of its own with one buffer, 4 heads of one column tile side by side.
//    Rows past 128 bytes do not pass through one wave's registers: long form.
template <typename T, int D, int TEAM_, int WH_, int WQ_>
struct Shape {
    static constexpr int TEAM = TEAM_, WH = WH_, WQ = WQ_, WAVES = WH * WQ, TEAMS = WAVES / TEAM;
    static constexpr int RB = D * (int)sizeof(T);       // bytes of a row
    static constexpr int KT = TEAM > 2 && RB <= 256 ? 64 : 32, NS = KT / 32, NB = TEAM > 1 ? 2 : 1;
    static constexpr int CH = Tile<T, D>::CH, NT = TEAM * WAVE;
};
// Long sequences whose heads do not share keys by fours:
//  - fp32 rows of 128 bytes: the matrix products are 8 times as long as in
//    bf16 and the staging beside them free, so waves apart (even work) win;
//  - else teams, each wave with a column tile of one head: of 2 where that
//    leaves room for several blocks, of 4 for wide rows.
// us, causal, 4 heads on 4, forward / training step:
//                   512 sequences of 1..203           24 of up to 1500
//               teams of 2  teams of 4  apart     of 2        of 4        apart
//   bf16   32     35 /  188   39 /  224   37 /  172   67 /  252   53 /  238   79 /  250
//   bf16   64     60 /  267   54 /  324   57 /  233   84 /  307   59 /  288   90 /  311
//   bf16  128     95 /  600   95 /  781  222 /  680  114 /  560   76 /  553  283 /  741
//   fp32   32     78 /  356   83 /  417   73 /  293  134 /  566  123 /  547  126 /  484
//   fp32   64    181 /  751  153 /  964  215 /  743  266 /  966  185 / 1000  302 /  948
//   fp32  128    289 / 1999  418 / 1999    -         301 / 2311  355 / 1899    -
// No one choice is the best for both batches of a row: teams of 4 suit the
// forward of long sequences, teams of 2 or waves apart the backward of
// shorter ones.
template <typename T, int D>
constexpr bool LONG_APART = sizeof(T) == 4 && D == 32;
template <typename T, int D>
constexpr int LONG_WAVES = D * sizeof(T) <= 128 ? 2 : 4;
template <typename T, int D>
constexpr bool HAS_SHORT = D * sizeof(T) <= 128;

// Orders a team's LDS writes before its reads.
template <int TEAM>
__device__ __forceinline__ void team_sync() {
    if (TEAM > 1) __syncthreads();
    else wave_lds_sync();
}

// ----------------------------------------------------------------- staging --
// Rows k0 .. k0 + KT - 1 of two tensors on their way to LDS: loaded into
// registers (thread t of the team: chunk t % CH of rows t / CH, + NT / CH,
// ...), stored after the current tile's work.  Hidden rows and rows past the
// end are stored as zeros, whatever they hold.  Nothing loaded is looked at
// before the store: a wait there would end the overlap.
template <typename T, int D, int NT, int KT>
struct RowStage {
    using TL = Tile<T, D>;
    static constexpr int CH = TL::CH, PER = KT * CH / NT, STEP = NT / CH;
    static_assert(KT * CH % NT == 0 && NT % CH == 0, "tile shape");
    u32x4 x[PER], y[PER];
    int32_t off[PER];                           // high half of the row's key_off, 0 without one
    int left;                                   // rows from the thread's first to the end
    __device__ __forceinline__ void load(const Rows<const T>& X, int hx, const Rows<const T>& Y, int hy, int64_t s, int k0,
                                         int end, const int64_t* key_off, int t) {
        const int row = t / CH, c = t % CH;
        left = end - k0 - row;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int kk = k0 + row + i * STEP;
            const int64_t j = s + (kk < end ? kk : end - 1);
            x[i] = gload_u4(X.at(j, hx) + c * TL::EPC);
            y[i] = gload_u4(Y.at(j, hy) + c * TL::EPC);
            off[i] = key_off ? reinterpret_cast<const int32_t*>(key_off + j)[1] : 0;
        }
    }
    __device__ __forceinline__ void store(u32x4* sx, u32x4* sy, int t) const {
        const int row = t / CH, c = t % CH;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = TL::chunk_at(row + i * STEP, c);
            const bool z = i * STEP >= left || off[i] < 0;
            sx[at] = z ? u32x4{0, 0, 0, 0} : x[i];
            sy[at] = z ? u32x4{0, 0, 0, 0} : y[i];
        }
    }
};

// The events of a tile of keys beside its rows (the team's first KT threads):
// positions, which may be seen, and of each 32 of them the lowest and highest
// position and whether any may not be seen.  mask and pos are read by 16 bytes,
// in every element of an array of these.
template <int KT>
struct alignas(16) KeySide {
    float mask[KT];
    int32_t pos[KT];
    int32_t range[KT / 32][2];
    uint32_t hidden[KT / 32];                   // bit per event
};
static_assert(sizeof(KeySide<32>) % 16 == 0 && offsetof(KeySide<32>, pos) % 16 == 0, "16-byte reads");
static_assert(sizeof(KeySide<64>) % 16 == 0 && offsetof(KeySide<64>, pos) % 16 == 0, "16-byte reads");
struct KeySideStage {
    int32_t p, off;
    bool in;
    __device__ __forceinline__ void load(const SeqArgs& a, int64_t s, int k0, int end, int kt, int t) {
        if (t < kt) {
            const int kk = k0 + t;
            const int64_t j = s + (kk < end ? kk : end - 1);
            p = a.pos[j];
            off = a.key_off ? reinterpret_cast<const int32_t*>(a.key_off + j)[1] : 0;
            in = kk < end;
        }
    }
    template <int KT>
    __device__ __forceinline__ void store(KeySide<KT>& ks, int t) const {
        if (t >= WAVE) return;
        const bool see = in && off >= 0;
        const int32_t lo = half_min(p), hi = half_max(p);
        const uint64_t hid = __ballot(t < KT && !see);
        if (t < KT) {
            ks.mask[t] = see ? 0.f : -INFINITY;
            ks.pos[t] = p;
            if ((t & 31) == 0) {
                ks.range[t / 32][0] = lo;
                ks.range[t / 32][1] = hi;
                ks.hidden[t / 32] = (uint32_t)(hid >> t);
            }
        }
    }
};

// -infinity where a key may not be seen: hidden ones, and those after the
// lane's query (lim: the last row the lane's half may see).
__device__ __forceinline__ void hide(f32x16& x, uint32_t hidden, const float* mask) {
    if (!__builtin_amdgcn_readfirstlane(hidden)) return;
    const int h = lane_id() >> 5;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f32x4 mk = *reinterpret_cast<const f32x4*>(mask + 8 * j + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * j + i] += mk[i];
    }
}

}  // namespace rse
