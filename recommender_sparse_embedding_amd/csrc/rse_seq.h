// rse_seq.h -- shared by the sequence operators' translation units: the
// handles, the views passed to kernels, the bucket lookup (not part of the
// public ABI).
#pragma once

#include <type_traits>

#include "rse_host.h"

namespace rse {

// Device memory of an attention handle.
struct SeqHeader {
    int32_t status;
    int32_t n_bounds;
    int32_t pad[62];
    int32_t bounds[RSE_SEQ_MAX_BOUNDARIES + 1];   // unused entries: INT32_MAX
    uint8_t cell[512];                            // by seq_cell: boundaries <= every distance of the cell
};
static_assert(sizeof(SeqHeader) == 256 + 512 + 512, "SeqHeader size");

// Distances in cells of an eighth of a power of two (positive and negative
// apart): sign, exponent and three more bits of the distance as a float.
__host__ __device__ __forceinline__ int seq_cell(int32_t d) {
    const float f = (float)d;
    const uint32_t u = __builtin_bit_cast(uint32_t, f);
    const int c = (int)((u >> 20) & 0x7FF) - 1015;      // 1 for a distance of 1, 249 for 2^31
    return (c > 0 ? c : 0) | (int)((u >> 31) << 8);
}

struct SeqCacheHeader {
    int32_t status;
    int32_t pad[63];
};
static_assert(sizeof(SeqCacheHeader) == 256, "SeqCacheHeader size");

// rse_seq_rows as a kernel sees them.
template <typename T>
struct Rows {
    T* p;
    int64_t row, head;
    __device__ __forceinline__ T* at(int64_t i, int64_t h) const { return p + i * row + h * head; }
};

// What every attention kernel is given about the batch and the layer.
struct SeqArgs {
    const int64_t* offsets;
    int64_t batch, n_events, max_len;
    const int32_t* pos;
    const int64_t* key_off;
    const float* bias;
    SeqHeader* hdr;
    int32_t n_heads, group;      // query heads, query heads per key/value head
    int32_t n_bounds, causal;
    int32_t cells;               // no cell holds two boundaries: seq_bucket_cell may be used
    float scale;
};

// pos_i - pos_j saturated to int32 (one instruction).
__device__ __forceinline__ int32_t seq_dist(int32_t a, int32_t b) { return __builtin_elementwise_sub_sat(a, b); }

// Number of boundaries <= d: binary search over a table padded to 128 entries
// with INT32_MAX (a distance of INT32_MAX would count the padding: capped).
__device__ __forceinline__ int seq_bucket(const int32_t* bounds, int n_bounds, int32_t d) {
    int b = 0;
#pragma unroll
    for (int step = 64; step > 0; step >>= 1)
        if (bounds[b + step - 1] <= d) b += step;
    return b < n_bounds ? b : n_bounds;
}

// The same by the distance's cell, where no cell holds two boundaries: all
// boundaries <= the whole cell, and perhaps the next one.
__device__ __forceinline__ int seq_bucket_cell(const uint8_t* cell, const int32_t* bounds, int n_bounds, int32_t d) {
    const int b = cell[seq_cell(d)];
    const int e = b + (bounds[b] <= d);         // the padding at n_bounds counts where d is INT32_MAX
    return e < n_bounds ? e : n_bounds;
}

// A bias in base 2.  One that far down, the type's lowest value as a mask for
// example, hides its pairs like -infinity: such a sum holds nothing of the
// score, and in base 2 the lowest value would overflow.
__device__ __forceinline__ float bias2(float b) { return b <= -1e30f ? -INFINITY : b * 1.4426950408889634f; }

// Wave-level ordering of a wave's own LDS writes before its other lanes read them.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A value that all lanes of the wave hold, as a scalar (branches on it stay
// scalar branches).
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// Elements of the two storage types as fp32, and back.
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ uint16_t f32_to_bf16(float x) {   // to nearest even; NaN stays NaN
    uint32_t u = __float_as_uint(x);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
    u += 0x7FFFu + ((u >> 16) & 1u);
    return (uint16_t)(u >> 16);
}
__device__ __forceinline__ void from_f32(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f32(uint16_t& y, float x) { y = f32_to_bf16(x); }

// The largest b in [0, batch) whose key f(b) <= x, for f ascending with
// f(0) <= x: 64 probes at a time, all lanes of the wave together.
template <typename F>
__device__ __forceinline__ int64_t wave_last_le(int64_t n, F f, int64_t x) {
    int64_t lo = 0, len = n;                 // the answer is in [lo, lo + len)
    const int lane = lane_id();
    while (len > 1) {
        const int64_t step = (len + WAVE - 1) / WAVE;
        const int64_t at = lo + lane * step;
        const bool le = lane * step < len && f(at) <= x;
        const int k = __popcll(__ballot(le));   // lanes 0 .. k-1 hold; k >= 1 for ascending f
        const int64_t first = lo + (int64_t)(k > 0 ? k - 1 : 0) * step;
        const int64_t end = lo + len;
        lo = first;
        len = end - first < step ? end - first : step;
    }
    return lo;
}

}  // namespace rse

struct rse_seqattn {
    int32_t n_heads, n_kv_heads, dim, dtype, causal, n_bounds, cells;
    float scale;
    rse::SeqHeader* hdr;
};

struct rse_seqcache {
    rse::SeqCacheHeader* hdr;
    void* k;
    void* v;
    int32_t* pos;
    int64_t n_pages;
    int32_t page_size, page_shift, n_kv_heads, dim, dtype;
};

namespace rse_host {

// A launch numbers its threads along an axis in 32 bits.
inline bool launch_holds(int64_t blocks, int threads) { return blocks <= UINT32_MAX / threads; }

// Rows of the handle's type: present, 16-byte aligned, strides in 16 bytes.
inline bool rows_ok(const rse_seq_rows* r, int32_t dtype) {
    const int64_t e = dtype == RSE_F32 ? 4 : 2;
    return r && r->data && reinterpret_cast<uintptr_t>(r->data) % 16 == 0 && r->row_stride % (16 / e) == 0 &&
           r->head_stride % (16 / e) == 0;
}

// Rows to be written: no element belongs to two events or heads.  Two of them,
// di events and dh heads apart, overlap where their distance is less than a
// head; of the di only those next to cancelling dh heads can be.
inline bool out_rows_ok(const rse_seq_rows* r, int32_t dtype, int64_t n, int64_t heads, int32_t dim) {
    if (!rows_ok(r, dtype)) return false;
    using Wide = __int128;
    const auto apart = [&](Wide di, int64_t dh) {
        if (di <= -(Wide)n || di >= n || (di == 0 && dh == 0)) return true;
        const Wide x = di * r->row_stride + (Wide)dh * r->head_stride;
        return x >= dim || x <= -dim;
    };
    for (int64_t dh = 0; dh < heads; ++dh) {
        Wide near = r->row_stride ? -((Wide)dh * r->head_stride) / r->row_stride : 0;
        near = near < 1 - (Wide)n ? 1 - (Wide)n : (near > (Wide)n - 1 ? (Wide)n - 1 : near);
        for (int u = -1; u <= 1; ++u)
            if (!apart(near + u, dh)) return false;
    }
    return true;
}

template <typename T>
inline rse::Rows<T> rows_view(const rse_seq_rows* r) {
    return {static_cast<T*>(r->data), r->row_stride, r->head_stride};
}

inline int batch_ok(const rse_seqattn* a, const rse_seq_batch* b) {
    if (!a || !b || !b->d_offsets || !b->d_bias) return RSE_ERR_INVALID_ARG;
    if (b->batch < 0 || b->n_events < 0 || b->max_len < 0) return RSE_ERR_INVALID_ARG;
    if (b->n_events > 0 && (!b->d_pos || b->batch == 0 || b->max_len == 0)) return RSE_ERR_INVALID_ARG;
    return RSE_OK;
}

inline rse::SeqArgs seq_args(const rse_seqattn* a, const rse_seq_batch* b) {
    rse::SeqArgs s;
    s.offsets = b->d_offsets;
    s.batch = b->batch;
    s.n_events = b->n_events;
    s.max_len = b->max_len < INT32_MAX / 2 ? b->max_len : INT32_MAX / 2;   // tiles count events in 32 bits
    s.pos = b->d_pos;
    s.key_off = b->d_key_off;
    s.bias = b->d_bias;
    s.hdr = a->hdr;
    s.n_heads = a->n_heads;
    s.group = a->n_heads / a->n_kv_heads;
    s.n_bounds = a->n_bounds;
    s.causal = a->causal;
    s.cells = a->cells;
    s.scale = a->scale;
    return s;
}

// Sequences short enough (and rows narrow enough) for the kernels whose waves
// work apart.  us, short / long form, forward and training step, 8192
// sequences of 1..100 events: 4 heads on 4 of 64 in bf16 329 / 450 and 1283 /
// 1746, of 32 217 / 236 and 895 / 1137, of 32 in fp32 416 / 473 and 1669 / 1660.
// 8 heads on 2 share keys by fours, which suits the long form's forward: bf16
// of 64 594 / 447 and 2370 / 2510, fp32 of 32 750 / 597 and 3084 / 2862.  Past
// 128 events a block's sequences become too unequal (512 of 1..203, fp32 of 32,
// both ways: 525 us in the long form, 1190 with this one up to 256).
constexpr int64_t SHORT = 128;
inline bool short_form(const rse_seqattn* a, int64_t max_len) {
    return max_len <= SHORT && a->dim * (a->dtype == RSE_F32 ? 4 : 2) <= 128;
}

// What a forward leaves for its backward: base-2 log-sums [n_heads][n_events]
// and, unless the sequences are short, the unrounded outputs
// [n_events][n_heads][dim].
struct Saved {
    float* lse2;
    float* out32;
    size_t bytes;
};
inline Saved saved_view(const rse_seqattn* a, int64_t n, int64_t max_len, void* base) {
    Carver c(base);
    Saved v;
    v.lse2 = c.take<float>((size_t)a->n_heads * n);
    v.out32 = c.take<float>(short_form(a, max_len) ? 0 : (size_t)n * a->n_heads * a->dim);
    v.bytes = c.size();
    return v;
}

// f(T(), integral_constant<dim>) for the handle's type and dim.
template <typename F>
inline int by_type(const rse_seqattn* a, F f) {
    if (a->dtype == RSE_F32) {
        if (a->dim == 32) return f(float(), std::integral_constant<int, 32>());
        if (a->dim == 64) return f(float(), std::integral_constant<int, 64>());
        return f(float(), std::integral_constant<int, 128>());
    }
    if (a->dim == 32) return f(uint16_t(), std::integral_constant<int, 32>());
    if (a->dim == 64) return f(uint16_t(), std::integral_constant<int, 64>());
    return f(uint16_t(), std::integral_constant<int, 128>());
}

}  // namespace rse_host
