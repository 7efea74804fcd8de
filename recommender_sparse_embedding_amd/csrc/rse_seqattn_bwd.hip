// rse_seqattn_bwd.hip -- backward of the attention over behaviour sequences:
// the probabilities are recomputed from q, k and the forward's log-sums, tile
// by tile, once with the queries as columns (dq, the bias gradient) and once
// with the keys as columns (dk, dv), so that every sum has one owner and a
// fixed order.
//
// bf16: p and ds enter their products as pairs of bf16 values (2^-16 of each is
// lost), so that the gradients are fp32 arithmetic rounded once.  With one
// value each dq and dk were half again as far off as that, for 1240 instead of
// 1280 us a training step on 8192 sequences of 1..100 events, 4 heads of 64,
// and 365 instead of 397 on 12 of up to 2048, 8 heads on 2.
#include "rse_seqmma.h"

using namespace rse;
using namespace rse_host;

namespace {

// A wave's bucket sums in LDS, [bucket][cols]: lane l adds in column l % cols
// by a plain read, addition and write, so every entry has a fixed order of
// additions.  (An LDS atomic addition of floats took 93 LDS cycles here, a
// read and a write together some ten.)  Four at a time: read together, added
// in order, a later one taking the earlier one's sum where both are in one
// bucket, and written in order.  With 32 columns the two halves of the wave
// take turns.
__device__ __forceinline__ void add_sixteen(float* mine, int cols, const int (&idx)[16], const f32x16& x) {
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
        float* p[4];
        float h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[i] = mine + idx[r + i] * cols;
            h[i] = *p[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int e = 0; e < i; ++e) h[i] = idx[r + e] == idx[r + i] ? h[e] : h[i];
            h[i] += x[r + i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) *p[i] = h[i];
    }
}
__device__ __forceinline__ void add_pairs(float* hist, int cols, const int (&idx)[16], const f32x16& x) {
    const int lane = lane_anew();
    float* mine = hist + (lane & (cols - 1));
    if (cols == WAVE) {
        add_sixteen(mine, WAVE, idx, x);
    } else {
        if (lane < 32) add_sixteen(mine, 32, idx, x);
        wave_lds_sync();
        if (lane >= 32) add_sixteen(mine, 32, idx, x);
    }
    wave_lds_sync();
}
// One lane's sum per column pair into one bucket.
__device__ __forceinline__ void add_bucket(float* hist, int cols, int bucket, float sum) {
    sum += other_half(sum);
    const int lane = lane_anew();
    if (lane < 32) hist[bucket * cols + lane] += sum;
    wave_lds_sync();
}
__device__ __forceinline__ void add_one(float* hist, int cols, int bucket, const f32x16& x) {
    float sum = x[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) sum += x[r];
    add_bucket(hist, cols, bucket, sum);
}

// A tile's ds into the bucket sums: up to SUMS buckets one by one in
// registers, else pair by pair.  (dq of 12 sequences of up to 2048 events: 195
// us with only single buckets in registers, 172 with 2, 156 with 3, 154 with 7.)
constexpr int SUMS = 7;

__device__ __forceinline__ void add_tile(float* hist, int cols, const TileBuckets<true>& tb, const int (&idx)[16], const f32x16& x) {
    if (tb.lo == tb.hi) {
        add_one(hist, cols, tb.lo, x);
    } else if (tb.hi - tb.lo < SUMS) {
#pragma unroll 1
        for (int bk = tb.lo; bk <= tb.hi; ++bk) {
            float sum = 0.f;
#pragma unroll
            for (int r = 0; r < 16; ++r) sum += idx[r] == bk ? x[r] : 0.f;
            add_bucket(hist, cols, bk, sum);
        }
    } else {
        add_pairs(hist, cols, idx, x);
    }
}

// A block's bucket sums of each head, over its WQ waves and their columns: 8
// lanes each, in a fixed order.
template <int WH, int WQ>
__device__ __forceinline__ void reduce_sums(const SeqArgs& a, int h0, int nb, int cols, const float* s_hist, float* part) {
    for (int x = threadIdx.x / 8; x < WH * nb; x += blockDim.x / 8) {
        const int hh = x / nb, bk = x % nb, eighth = threadIdx.x % 8;
        float sum = 0.f;
        for (int y = 0; y < WQ; ++y)
            for (int c = eighth; c < cols; c += 8) sum += s_hist[((y * WH + hh) * nb + bk) * cols + c];
        sum += __shfl_xor(sum, 1, 8);
        sum += __shfl_xor(sum, 2, 8);
        sum += __shfl_xor(sum, 4, 8);
        if (eighth == 0 && h0 + hh < a.n_heads) part[((int64_t)(h0 + hh) * nb + bk) * gridDim.x + blockIdx.x] = sum;
    }
}

// dq and the bias gradient, queries as columns: per tile of keys
// S^T = K Q^T and dP^T = V dO^T, ds = p (dp - delta), dQ^T += K^T dS^T.
// delta = sum_j p dp = dO . out, from the unrounded outputs.  ds of a tile in
// one bucket is summed in registers, else scattered into the wave's LDS
// columns of bucket sums.  A block stays with its heads and takes tiles of
// queries blockIdx.x, + gridDim.x, ...; its sums go to part.
// Registers are held to what lets DQ_WAVES (DKV_WAVES) waves share a SIMD.
template <typename T, int D>
constexpr int DQ_WAVES = D * sizeof(T) <= 128 ? 2 : 1;
template <typename T, int D>
constexpr int DKV_WAVES = D * sizeof(T) <= 128 ? 2 : 1;

template <typename T, int D, typename SH>
__global__ __launch_bounds__(SH::WAVES * 64) __attribute__((amdgpu_waves_per_eu(DQ_WAVES<T, D>))) void k_attn_dq(
    SeqArgs a, TileGrid grid, Rows<const T> q, Rows<const T> k, Rows<const T> v, const float* lse2, const float* out32,
    Rows<const T> dout, Rows<T> dq, float* delta, float* part, int cols) {
    using TL = Tile<T, D>;
    constexpr int CH = SH::CH, KT = SH::KT, NS = SH::NS, NB = SH::NB, NT = SH::NT, WH = SH::WH, WQ = SH::WQ, ND = D / 32;
    __shared__ u32x4 s_k[SH::TEAMS][NB][KT * CH], s_v[SH::TEAMS][NB][KT * CH];
    __shared__ u32x4 s_pairs[WQ][NS][WAVE];
    __shared__ KeySide<KT> s_side[SH::TEAMS][NB];
    __shared__ LdsBuckets s_buckets;
    __shared__ float s_bias[WH][RSE_SEQ_MAX_BOUNDARIES + 1];
    extern __shared__ float s_hist[];           // [waves][n_bounds + 1][cols]
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE), half = lane >> 5, wh = w % WH, wq = w / WH;
    const int team = w / SH::TEAM, t = threadIdx.x % NT;
    const int h0 = blockIdx.y * WH, nb = a.n_bounds + 1;
    const bool live = h0 + wh < a.n_heads;
    const int head = live ? h0 + wh : a.n_heads - 1, g = head / a.group;
    float* hist = s_hist + w * nb * cols;

    WaveBuckets wb;
    wb.load(a.hdr, a.bias + head * nb, a.n_bounds);
    s_buckets.load(a.hdr);
    if (wq == 0) {
        s_bias[wh][lane] = wb.bias[0];
        s_bias[wh][64 + lane] = wb.bias[1];
    }
    for (int x = threadIdx.x; x < SH::WAVES * nb * cols; x += SH::WAVES * WAVE) s_hist[x] = 0.f;
    const float c2 = fabsf(a.scale) * LOG2E;

    for (int64_t item = blockIdx.x; item < grid.items; item += gridDim.x) {
        int64_t s;
        int len, tile;
        if (!find_tile(a, grid, item, 32 * WQ, a.causal, s, len, tile, h0 == 0)) continue;
        const int q0 = tile * 32 * WQ, w0 = q0 + 32 * wq, my_q = w0 + (lane & 31), row = my_q < len ? my_q : len - 1;
        const int end = a.causal ? (q0 + 32 * WQ < len ? q0 + 32 * WQ : len) : len;
        const int my_end = w0 >= len ? 0 : (a.causal && w0 + 32 < end ? w0 + 32 : end);
        RowStage<T, D, NT, KT> st;
        KeySideStage side;
        st.load(k, g, v, g, s, 0, end, a.key_off, t);
        side.load(a, s, 0, end, KT, t);
        ColFrag<T, D> qf, df;
        qf.load(q.at(s + row, head), half);
        df.load(dout.at(s + row, head), half);
        const int32_t my_pos = a.pos[s + row];
        float L = lse2[(int64_t)head * a.n_events + s + row];
        if (my_q >= len || L == -INFINITY) L = INFINITY;        // p = 0
        float del = 0.f;
        {
            const float* o = out32 + ((s + row) * a.n_heads + head) * D;
#pragma unroll
            for (int x = 0; x < CH / 2; ++x)
#pragma unroll
                for (int e = 0; e < TL::EPC; e += 4) {
                    const f32x4 of = gload_f4(o + (2 * x + half) * TL::EPC + e);
                    const f32x4 d4 = chunk_f32<T>(df.v[x], e);
#pragma unroll
                    for (int i = 0; i < 4; ++i) del = __builtin_fmaf(of[i], d4[i], del);
                }
            del += other_half(del);
        }
        if (my_q < len && half == 0 && live) delta[(int64_t)head * a.n_events + s + my_q] = del;
        if (a.scale < 0.f) qf.negate();
        const int32_t q_lo = half_min(my_pos), q_hi = half_max(my_pos);
        f32x16 acc[ND] = {};
        __syncthreads();                        // the previous item's LDS is no longer read
        st.store(s_k[team][0], s_v[team][0], t);
        side.store(s_side[team][0], t);
        __syncthreads();
        for (int k0 = 0, b = 0; k0 < end; k0 += KT, b ^= NB - 1) {
            if (k0 + KT < end) {
                st.load(k, g, v, g, s, k0 + KT, end, a.key_off, t);
                side.load(a, s, k0 + KT, end, KT, t);
            }
            const KeySide<KT>& ks = s_side[team][b];
#pragma unroll 1
            for (int u = 0; u < NS; ++u) {
                const int k1 = k0 + 32 * u;
                if (k1 >= my_end) break;
                TileBuckets<true> tb;
                tb.set(wb, q_lo, q_hi, ks.range[u]);
                if (tb.many) {
                    if (SH::TEAM == 1 && WH > 1) __syncthreads();
                    tb.find_pairs(s_pairs[wq][u], wh, WH, s_buckets, a.n_bounds, a.cells, ks.pos + 32 * u, my_pos);
                    if (WH > 1) __syncthreads();
                    else wave_lds_sync();
                }
                f32x16 x = mma_rows<T, D>(s_k[team][b], 32 * u, qf, f32x16{});
                const f32x16 dp = mma_rows<T, D>(s_v[team][b], 32 * u, df, f32x16{});
                int idx[16];
                if (tb.lo == tb.hi) {
                    const float b0 = wb.value(tb.lo) - L;
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = __builtin_fmaf(x[r], c2, b0);
                } else {
                    tb.index(idx, wb, s_pairs[wq][u], ks.pos + 32 * u, my_pos);
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = __builtin_fmaf(x[r], c2, s_bias[wh][idx[r]] - L);
                }
                hide(x, ks.hidden[u], ks.mask + 32 * u);
                if (a.causal && k1 + 31 > w0) {
                    const int lim = my_q - k1 - 4 * half;
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = tile_row(r, 0) <= lim ? x[r] : -INFINITY;
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) x[r] = __builtin_amdgcn_exp2f(x[r]) * (dp[r] - del);
                add_tile(hist, cols, tb, idx, x);
                OverRows<T, D>::add(acc, s_k[team][b], 32 * u, x);
            }
            if (k0 + KT < end) {
                if (SH::TEAM == 1) wave_lds_sync();
                st.store(s_k[team][b ^ (NB - 1)], s_v[team][b ^ (NB - 1)], t);
                side.store(s_side[team][b ^ (NB - 1)], t);
                team_sync<SH::TEAM>();
            }
        }
        if (my_q < len && live) {
            T* dst = dq.at(s + my_q, head);
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) store_column(dst + 32 * dt, acc[dt], a.scale);
        }
    }
    __syncthreads();
    reduce_sums<WH, WQ>(a, h0, nb, cols, s_hist, part);
}

// The same for short sequences: a block goes through its sequences' tiles of
// queries, the next tile's first loads in flight meanwhile, and delta comes
// from the probabilities themselves: forward through the tiles of keys it is
// summed, then, backward, used.  The last tile of the way there is the first
// of the way back, so its probabilities are formed once.  Nothing but the
// log-sums is needed of the forward (its outputs in fp32 would be written and
// read: 0.8 of 2.6 GB a training step on 8192 sequences of 1..100 events).
template <typename T, int D, typename SH>
__global__ __launch_bounds__(SH::WAVES * 64) __attribute__((amdgpu_waves_per_eu(2))) void k_attn_dq_short(
    SeqArgs a, Rows<const T> q, Rows<const T> k, Rows<const T> v, const float* lse2, Rows<const T> dout, Rows<T> dq,
    float* delta, float* part, int cols, int split) {
    constexpr int CH = SH::CH, KT = SH::KT, NT = SH::NT, WH = SH::WH, ND = D / 32;
    static_assert(SH::TEAM == 1 && SH::WQ == 1 && KT == 32, "waves apart");
    __shared__ u32x4 s_k[WH][KT * CH], s_v[WH][KT * CH];
    __shared__ u32x4 s_pairs[2][WAVE];          // this tile's and the last one's
    __shared__ KeySide<KT> s_side[WH];
    __shared__ LdsBuckets s_buckets;
    __shared__ float s_bias[WH][RSE_SEQ_MAX_BOUNDARIES + 1];
    extern __shared__ float s_hist[];           // [waves][n_bounds + 1][cols]
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE), half = lane >> 5;
    const int h0 = blockIdx.y * WH, nb = a.n_bounds + 1;
    const bool live = h0 + w < a.n_heads;
    const int head = live ? h0 + w : a.n_heads - 1, g = head / a.group;
    float* hist = s_hist + w * nb * cols;
    SeqTiles at;
    at.begin(a, blockIdx.x, gridDim.x, split, h0 == 0);

    RowStage<T, D, NT, KT> st;
    KeySideStage side;
    ColFrag<T, D> qn, dn;
    int32_t pn = 0;
    float ln = 0.f;
    auto end_of = [&](const SeqTiles& x) { return a.causal && (x.tile + 1) * 32 < x.len ? (x.tile + 1) * 32 : x.len; };
    auto load_first = [&](const SeqTiles& x) {
        st.load(k, g, v, g, x.s, 0, end_of(x), a.key_off, lane);
        side.load(a, x.s, 0, end_of(x), KT, lane);
        const int i = x.tile * 32 + (lane & 31);
        const int64_t row = x.s + (i < x.len ? i : x.len - 1);
        qn.load(q.at(row, head), half);
        dn.load(dout.at(row, head), half);
        pn = a.pos[row];
        ln = lse2[(int64_t)head * a.n_events + row];
    };
    if (at.valid) load_first(at);
    WaveBuckets wb;
    wb.load(a.hdr, a.bias + head * nb, a.n_bounds);
    s_buckets.load(a.hdr);
    s_bias[w][lane] = wb.bias[0];
    s_bias[w][64 + lane] = wb.bias[1];
    for (int x = threadIdx.x; x < WH * nb * cols; x += WH * WAVE) s_hist[x] = 0.f;
    const float c2 = fabsf(a.scale) * LOG2E;
    int wp = 0;
    __syncthreads();

    while (at.valid) {
        const int64_t s = at.s;
        const int len = at.len, w0 = at.tile * 32, my_q = w0 + (lane & 31), end = end_of(at), nk = (end + 31) / 32;
        ColFrag<T, D> qf = qn, df = dn;
        if (a.scale < 0.f) qf.negate();
        const float L = my_q >= len || ln == -INFINITY ? INFINITY : ln;         // infinity: p = 0
        const int32_t my_pos = pn, q_lo = half_min(my_pos), q_hi = half_max(my_pos);
        f32x16 acc[ND] = {};
        float del = 0.f;
        for (int step = 0; step < 2 * nk - 1; ++step) {
            const int kt = step < nk ? step : 2 * nk - 2 - step, k1 = 32 * kt;
            st.store(s_k[w], s_v[w], lane);
            side.store(s_side[w], lane);
            wave_lds_sync();
            if (step + 1 < 2 * nk - 1) {
                const int to = 32 * (step + 1 < nk ? step + 1 : 2 * nk - 3 - step);
                st.load(k, g, v, g, s, to, end, a.key_off, lane);
                side.load(a, s, to, end, KT, lane);
            } else {
                at.advance(a);
                if (at.valid) load_first(at);
            }
            const KeySide<KT>& ks = s_side[w];
            TileBuckets<true> tb;
            tb.set(wb, q_lo, q_hi, ks.range[0]);
            f32x16 x = mma_rows<T, D>(s_k[w], 0, qf, f32x16{});
            f32x16 dp = mma_rows<T, D>(s_v[w], 0, df, f32x16{});
            if (tb.many) {
                wp ^= 1;
                tb.find_pairs(s_pairs[wp], w, WH, s_buckets, a.n_bounds, a.cells, ks.pos, my_pos);
                if (WH > 1) __syncthreads();
                else wave_lds_sync();
            }
            x = tb.logits(x, c2, -L, wb, s_pairs[wp], s_bias[w], ks.pos, my_pos);
            hide(x, ks.hidden[0], ks.mask);
            if (a.causal && k1 + 31 > w0) {
                const int lim = my_q - k1 - 4 * half;
#pragma unroll
                for (int r = 0; r < 16; ++r) x[r] = tile_row(r, 0) <= lim ? x[r] : -INFINITY;
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] = __builtin_amdgcn_exp2f(x[r]);
            if (step < nk) {
#pragma unroll
                for (int r = 0; r < 16; ++r) del = __builtin_fmaf(x[r], dp[r], del);
            }
            if (step == nk - 1) del += other_half(del);
            if (step >= nk - 1) {
#pragma unroll
                for (int r = 0; r < 16; ++r) x[r] *= dp[r] - del;
                if (tb.lo == tb.hi) {
                    add_one(hist, cols, tb.lo, x);
                } else {                        // (sums in registers, as add_tile's, took 771 us here for 566)
                    int idx[16];
                    tb.index(idx, wb, s_pairs[wp], ks.pos, my_pos);
                    add_pairs(hist, cols, idx, x);
                }
                OverRows<T, D>::add(acc, s_k[w], 0, x);
            }
            wave_lds_sync();
        }
        if (my_q < len && live) {
            if (half == 0) delta[(int64_t)head * a.n_events + s + my_q] = del;
            T* dst = dq.at(s + my_q, head);
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) store_column(dst + 32 * dt, acc[dt], a.scale);
        }
    }
    __syncthreads();
    reduce_sums<WH, 1>(a, h0, nb, cols, s_hist, part);
}

// The blocks' bucket sums, added in 64 bits in a fixed order: one block per
// head and bucket.
__global__ __launch_bounds__(256) void k_attn_dbias(const float* part, int blocks, float* dbias) {
    __shared__ double s[4];
    const float* p = part + (int64_t)blockIdx.x * blocks;
    double t = 0.0;
    for (int x = threadIdx.x; x < blocks; x += 256) t += p[x];
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) t += shfl_xor_f64(t, m);
    if (lane_id() == 0) s[threadIdx.x / WAVE] = t;
    __syncthreads();
    if (threadIdx.x == 0) dbias[blockIdx.x] = (float)(s[0] + s[1] + s[2] + s[3]);
}

// dk and dv, keys as columns: per tile of queries and head of the group
// S = Q K^T and dP = dO V^T, dV^T += dO^T P, dK^T += Q^T dS.  WQ waves take
// tiles of keys, WH waves key heads or (IN_GROUP) query heads of one key head,
// whose sums are then added over the waves in LDS; the buckets of a tile are
// looked up once for the heads of the group.
// (12 sequences of up to 2048 events, 8 heads on 2: 402 us with 4 tiles of
// keys a block and its heads in turn, which leaves 384 blocks.)
template <typename T, int D, typename SH, bool IN_GROUP>
__global__ __launch_bounds__(SH::WAVES * 64) __attribute__((amdgpu_waves_per_eu(DKV_WAVES<T, D>))) void k_attn_dkv(
    SeqArgs a, TileGrid grid, Rows<const T> q, Rows<const T> k, Rows<const T> v, const float* lse2, const float* delta,
    Rows<const T> dout, Rows<T> dk, Rows<T> dv, int split) {
    constexpr int CH = SH::CH, KT = SH::KT, NS = SH::NS, NB = SH::NB, NT = SH::NT, WH = SH::WH, WQ = SH::WQ, ND = D / 32,
                  NBP = RSE_SEQ_MAX_BOUNDARIES + 1;
    __shared__ u32x4 s_rows[2][SH::TEAMS][NB][KT * CH];
    auto& s_q = s_rows[0];
    auto& s_d = s_rows[1];
    constexpr bool BRIEF = SH::TEAM == 1;
    __shared__ u32x4 s_pairs[BRIEF ? 2 : WQ][NS][WAVE];      // (BRIEF: this tile's and the last one's)
    // (read by 16 bytes)
    alignas(16) __shared__ float s_lse[SH::TEAMS][NB][KT], s_del[SH::TEAMS][NB][KT];
    alignas(16) __shared__ int32_t s_pos[SH::TEAMS][NB][KT];
    __shared__ int32_t s_range[SH::TEAMS][NB][NS][2];
    __shared__ LdsBuckets s_buckets;
    __shared__ float s_bias[SH::TEAMS][NB][NBP];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE), half = lane >> 5, wh = w % WH, wq = w / WH;
    const int team = w / SH::TEAM, t = threadIdx.x % NT;
    const int n_kv = a.n_heads / a.group, gblocks = IN_GROUP ? n_kv : (n_kv + WH - 1) / WH,
              g0 = blockIdx.x % gblocks * (IN_GROUP ? 1 : WH), nb = a.n_bounds + 1;
    const bool live = IN_GROUP || g0 + wh < n_kv;
    const int g = IN_GROUP ? g0 : (live ? g0 + wh : n_kv - 1);
    const int turns = IN_GROUP ? a.group / WH : a.group;            // heads one after the other
    SeqTiles at;
    // split > 0: the block goes on through its sequences' tiles
    if (BRIEF && split) {
        at.begin(a, blockIdx.x / gblocks, gridDim.x / gblocks, split, false);
        if (!at.valid) return;
    } else if (!find_tile(a, grid, blockIdx.x / gblocks, 32 * WQ, false, at.s, at.len, at.tile, false)) {
        return;
    }

    RowStage<T, D, NT, KT> st;
    int32_t rp = 0;
    float rl = 0.f, rd = 0.f, rb[(NBP + NT - 1) / NT];
    bool rin = false;
    auto first_of = [&](const SeqTiles& x) { return a.causal ? x.tile * 32 * WQ / KT * KT : 0; };   // queries of a block's tile
    auto load = [&](const SeqTiles& x, int it) {
        const int h = g * a.group + (IN_GROUP ? it % turns * WH + wh : it % turns), i0 = first_of(x) + it / turns * KT;
        st.load(q, h, dout, h, x.s, i0, x.len, nullptr, t);
        if (t < KT) {
            const int kk = i0 + t;
            const int64_t j = x.s + (kk < x.len ? kk : x.len - 1);
            rp = a.pos[j];
            rl = lse2[(int64_t)h * a.n_events + j];
            rd = delta[(int64_t)h * a.n_events + j];
            rin = kk < x.len;
        }
        if (it == 0 || turns > 1)
#pragma unroll
            for (int i = 0; i * NT < NBP; ++i) rb[i] = i * NT + t < nb ? a.bias[h * nb + i * NT + t] : 0.f;
    };
    auto store = [&](int b) {
        st.store(s_q[team][b], s_d[team][b], t);
        if (t < WAVE) {
            const int32_t lo = half_min(rp), hi = half_max(rp);
            if (t < KT) {
                s_pos[team][b][t] = rp;
                s_lse[team][b][t] = !rin || rl == -INFINITY ? INFINITY : rl;    // infinity: p = 0
                s_del[team][b][t] = rin ? rd : 0.f;
                if ((t & 31) == 0) {
                    s_range[team][b][t / 32][0] = lo;
                    s_range[team][b][t / 32][1] = hi;
                }
            }
        }
#pragma unroll
        for (int i = 0; i * NT < NBP; ++i)
            if (i * NT + t < NBP) s_bias[team][b][i * NT + t] = bias2(rb[i]);
    };

    load(at, 0);
    s_buckets.load(a.hdr);
    WaveBuckets wb;
    wb.load(a.hdr, a.bias, a.n_bounds);
    const float c2 = fabsf(a.scale) * LOG2E;
    int wp = wq;
    __syncthreads();
    for (;;) {
    const int64_t s = at.s;
    const int len = at.len, w0 = at.tile * 32 * WQ + 32 * wq, my_k = w0 + (lane & 31), row = my_k < len ? my_k : len - 1;
    const int first = first_of(at), total = (len - first + KT - 1) / KT * turns;    // tiles of queries, each in all turns
    ColFrag<T, D> kf, vf;
    kf.load(k.at(s + row, g), half);
    vf.load(v.at(s + row, g), half);
    const int32_t off = a.key_off ? reinterpret_cast<const int32_t*>(a.key_off + s + row)[1] : 0;
    const int32_t my_pos = a.pos[s + row];
    const int32_t k_lo = half_min(my_pos), k_hi = half_max(my_pos);
    const bool seen = off >= 0;
    if (a.scale < 0.f) kf.negate();
    f32x16 ak[ND] = {}, av[ND] = {};
    for (int it = 0, b = 0; it < total; ++it, b ^= NB - 1) {
        const int i0 = first + it / turns * KT;
        store(b);
        team_sync<SH::TEAM>();
        if (it + 1 < total) {
            load(at, it + 1);
        } else if (BRIEF && split) {
            at.advance(a);
            if (at.valid) load(at, 0);
        }
        if (w0 < len) {
            wb.bias[0] = s_bias[team][b][lane];
            wb.bias[1] = s_bias[team][b][64 + lane];
#pragma unroll 1
            for (int u = 0; u < NS; ++u) {
                const int i1 = i0 + 32 * u;
                if (i1 >= len) break;
                if (a.causal && i1 + 31 < w0) continue;
                TileBuckets<false> tb;
                tb.set(wb, k_lo, k_hi, s_range[team][b][u]);
                f32x16 x = mma_rows<T, D>(s_q[team][b], 32 * u, kf, f32x16{});
                f32x16 dp = mma_rows<T, D>(s_d[team][b], 32 * u, vf, f32x16{});
                if (tb.many && it % turns == 0) {
                    if (BRIEF) wp ^= 1;
                    tb.find_pairs(s_pairs[wp][u], wh, WH, s_buckets, a.n_bounds, a.cells, s_pos[team][b] + 32 * u, my_pos);
                    if (WH > 1) __syncthreads();
                    else wave_lds_sync();
                }
                x = tb.logits(x, c2, 0.f, wb, s_pairs[wp][u], s_bias[team][b], s_pos[team][b] + 32 * u, my_pos);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 L = *reinterpret_cast<const f32x4*>(&s_lse[team][b][32 * u + 8 * j + 4 * half]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[4 * j + i] -= L[i];
                }
                if (a.causal && i1 < w0 + 31) {         // (after the log-sums: one of NaN goes no further than it is seen)
                    const int lim = my_k - i1 - 4 * half;
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = tile_row(r, 0) >= lim ? x[r] : -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 de = *reinterpret_cast<const f32x4*>(&s_del[team][b][32 * u + 8 * j + 4 * half]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[4 * j + i] = __builtin_amdgcn_exp2f(x[4 * j + i]);
                        dp[4 * j + i] = x[4 * j + i] * (dp[4 * j + i] - de[i]);
                    }
                }
                if constexpr (sizeof(T) == 4) {     // (one after the other: more spills at 128 elements, 64 of up to 333 671 us for 630)
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) {
                        OverRows<T, D>::add(av[dt], s_d[team][b], 32 * u, dt, x);
                        OverRows<T, D>::add(ak[dt], s_q[team][b], 32 * u, dt, dp);
                    }
                } else {
                    OverRows<T, D>::add(av, s_d[team][b], 32 * u, x);
                    OverRows<T, D>::add(ak, s_q[team][b], 32 * u, dp);
                }
            }
        }
        if (BRIEF) wave_lds_sync();             // read before the next tile is stored
    }
    bool more = false;
    if (BRIEF) more = split && at.valid;
    if (!IN_GROUP) {
        if (my_k < len && live) {
            T* pk = dk.at(s + my_k, g);
            T* pv = dv.at(s + my_k, g);
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) {
                if (!seen) ak[dt] = av[dt] = f32x16{};      // hidden: whatever the key held
                store_column(pk + 32 * dt, ak[dt], a.scale);
                store_column(pv + 32 * dt, av[dt], 1.f);
            }
        }
        if (!more) return;
        continue;
    }
    // wave w adds and stores the w-th quarter of each 32 elements
    f32x4* s_sum = reinterpret_cast<f32x4*>(s_rows);
    static_assert(!IN_GROUP || sizeof(s_rows) >= 4 * 4 * WAVE * 16, "room for the sums");
#pragma unroll
    for (int x = 0; x < 2 * ND; ++x) {
        const f32x16& mine = x < ND ? ak[x % ND] : av[x % ND];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            s_sum[(w * 4 + j) * WAVE + lane] = f32x4{mine[4 * j], mine[4 * j + 1], mine[4 * j + 2], mine[4 * j + 3]};
        __syncthreads();
        f32x4 sum = s_sum[w * WAVE + lane];
#pragma unroll
        for (int y = 1; y < 4; ++y) sum += s_sum[(y * 4 + w) * WAVE + lane];
        if (my_k < len) {
            if (x < ND) sum *= a.scale;
            if (!seen) sum = f32x4{0.f, 0.f, 0.f, 0.f};
            T* p = (x < ND ? dk.at(s + my_k, g) : dv.at(s + my_k, g)) + 32 * (x % ND) + 8 * w + 4 * half;
            store_four(p, sum);
        }
    }
    if (!more) return;
    __syncthreads();                            // the sums are read before the next tile is stored
    }
}

// ------------------------------------------------------------------ host --
// Blocks of k_attn_dq over all heads: enough to fill the GPU several times
// over; more would only add partial bucket sums.
constexpr int64_t DQ_BLOCKS = 2048;

struct BwdWs {
    float* delta;
    float* part;
    size_t bytes;
    int64_t blocks;              // of k_attn_dq, per heads side by side
    int split;
};

// The blocks of k_attn_dq, by the rules of the forward.
struct DqForm {
    int wh, wq;
};
DqForm dq_form(const rse_seqattn* a, int64_t max_len) {
    if (short_form(a, max_len)) return {a->n_heads > 1 ? 4 : 1, 1};
    if (a->n_heads / a->n_kv_heads % 4 == 0) return {4, 1};
    const bool apart = by_type(a, [](auto t, auto d) { return LONG_APART<decltype(t), decltype(d)::value>; });
    if (apart && a->n_heads > 2) return {4, 1};
    return {1, by_type(a, [](auto t, auto d) { return LONG_WAVES<decltype(t), decltype(d)::value>; })};
}

BwdWs bwd_ws(const rse_seqattn* a, int64_t n, int64_t batch, int64_t max_len, void* base) {
    BwdWs w;
    const DqForm f = dq_form(a, max_len);
    if (short_form(a, max_len)) {
        const ShortGrid g = short_grid(batch, (a->n_heads + f.wh - 1) / f.wh, max_len, f.wh);
        w.blocks = g.blocks;
        w.split = g.split;
    } else {
        w.blocks = tile_grid(n, batch, max_len, 32 * f.wq).items;
        const int64_t most = DQ_BLOCKS * f.wh / a->n_heads;
        if (w.blocks > most) w.blocks = most > 16 ? most : 16;
        w.split = 1;
    }
    Carver c(base);
    w.delta = c.take<float>((size_t)a->n_heads * n);
    w.part = c.take<float>((size_t)a->n_heads * w.blocks * (a->n_bounds + 1));
    w.bytes = c.size();
    return w;
}

template <typename T, int D, int TEAM, int WH, int WQ, int KTEAM, int KH, int KQ, bool IN_GROUP, bool brief>
int run_bwd(const SeqArgs& a, const rse_seq_rows* q, const rse_seq_rows* k, const rse_seq_rows* v, const Saved& sv,
            const rse_seq_rows* dout, const rse_seq_rows* dq, const rse_seq_rows* dk, const rse_seq_rows* dv,
            float* dbias, const BwdWs& w, hipStream_t s) {
    using QS = Shape<T, D, TEAM, WH, WQ>;
    using KS = Shape<T, D, KTEAM, KH, KQ>;
    const int nb = a.n_bounds + 1, n_kv = a.n_heads / a.group;
    const int cols = nb <= 32 ? 64 : 32;        // at most 32 KiB a block of 4 waves up to 64 buckets, 64 KiB past that
    const TileGrid tq = tile_grid(a.n_events, a.batch, a.max_len, 32 * WQ);
    const TileGrid tk = tile_grid(a.n_events, a.batch, a.max_len, 32 * KQ);
    const int64_t gblocks = IN_GROUP ? n_kv : (n_kv + KH - 1) / KH;
    const ShortGrid sg = short_grid(a.batch, gblocks, a.max_len, KS::WAVES);
    const int64_t blocks = gblocks * (brief ? sg.blocks : tk.items);
    if (!launch_holds(blocks, KS::WAVES * WAVE)) return RSE_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)w.blocks, (a.n_heads + WH - 1) / WH), block(QS::WAVES * WAVE);
    const size_t lds = QS::WAVES * nb * cols * sizeof(float);
    if constexpr (brief)
        hipLaunchKernelGGL((k_attn_dq_short<T, D, QS>), grid, block, lds, s, a, rows_view<const T>(q), rows_view<const T>(k),
                           rows_view<const T>(v), sv.lse2, rows_view<const T>(dout), rows_view<T>(dq), w.delta, w.part, cols,
                           w.split);
    else
        hipLaunchKernelGGL((k_attn_dq<T, D, QS>), grid, block, lds, s, a, tq, rows_view<const T>(q), rows_view<const T>(k),
                           rows_view<const T>(v), sv.lse2, sv.out32, rows_view<const T>(dout), rows_view<T>(dq), w.delta,
                           w.part, cols);
    int rc = launch_status();
    if (rc) return rc;
    hipLaunchKernelGGL(k_attn_dbias, dim3(a.n_heads * nb), dim3(256), 0, s, w.part, (int)w.blocks, dbias);
    hipLaunchKernelGGL((k_attn_dkv<T, D, KS, IN_GROUP>), dim3((unsigned)blocks), dim3(KS::WAVES * WAVE), 0, s, a, tk,
                       rows_view<const T>(q), rows_view<const T>(k), rows_view<const T>(v), sv.lse2, w.delta,
                       rows_view<const T>(dout), rows_view<T>(dk), rows_view<T>(dv), brief ? sg.split : 0);
    return launch_status();
}

}  // namespace

extern "C" {

int rse_seqattn_bwd_workspace_size(const rse_seqattn* attn, int64_t n_events, int64_t batch, int64_t max_len,
                                   size_t* bytes_out) {
    if (!attn || !bytes_out || n_events < 0 || batch < 0 || max_len < 0) return RSE_ERR_INVALID_ARG;
    *bytes_out = bwd_ws(attn, n_events, batch, max_len, nullptr).bytes;
    return RSE_OK;
}

int seq_attention_bwd(const rse_seqattn* attn, const rse_seq_batch* batch, const rse_seq_rows* q,
                      const rse_seq_rows* k, const rse_seq_rows* v, const void* d_saved, size_t saved_bytes,
                      const rse_seq_rows* dout, const rse_seq_rows* dq, const rse_seq_rows* dk,
                      const rse_seq_rows* dv, float* d_dbias, void* d_ws, size_t ws_bytes, void* stream) {
    int rc = batch_ok(attn, batch);
    if (rc) return rc;
    if (!d_dbias || !d_ws || reinterpret_cast<uintptr_t>(d_ws) % 256) return RSE_ERR_INVALID_ARG;
    const BwdWs w = bwd_ws(attn, batch->n_events, batch->batch, batch->max_len, d_ws);
    if (ws_bytes < w.bytes) return RSE_ERR_WORKSPACE;
    hipStream_t s = as_stream(stream);
    if (batch->n_events == 0) {
        hipLaunchKernelGGL(k_attn_dbias, dim3(attn->n_heads * (attn->n_bounds + 1)), dim3(256), 0, s, w.part, 0, d_dbias);
        return launch_status();
    }
    for (const rse_seq_rows* r : {q, k, v, dout})
        if (!rows_ok(r, attn->dtype)) return RSE_ERR_INVALID_ARG;
    for (const rse_seq_rows* r : {dq, dk, dv})
        if (!out_rows_ok(r, attn->dtype, batch->n_events, r == dq ? attn->n_heads : attn->n_kv_heads, attn->dim))
            return RSE_ERR_INVALID_ARG;
    if (!d_saved || reinterpret_cast<uintptr_t>(d_saved) % 256) return RSE_ERR_INVALID_ARG;
    const Saved sv = saved_view(attn, batch->n_events, batch->max_len, const_cast<void*>(d_saved));
    if (saved_bytes < sv.bytes) return RSE_ERR_WORKSPACE;
    const SeqArgs a = seq_args(attn, batch);
    return by_type(attn, [&](auto t, auto d) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        auto run = [&](auto team, auto wh, auto wq, auto kteam, auto kh, auto kq, auto in_group, auto brief) {
            return run_bwd<T, D, team.value, wh.value, wq.value, kteam.value, kh.value, kq.value, in_group.value, brief.value>(
                a, q, k, v, sv, dout, dq, dk, dv, d_dbias, w, s);
        };
        using I1 = std::integral_constant<int, 1>;
        using IL = std::integral_constant<int, LONG_WAVES<T, D>>;
        using I4 = std::integral_constant<int, 4>;
        std::true_type in_group, brief;
        std::false_type apart, full;
        const bool fours = a.group % 4 == 0;
        // (dq's team, heads, tiles; dkv's)
        if constexpr (HAS_SHORT<T, D>) {
            if (short_form(attn, batch->max_len)) {
                if (a.n_heads == 1) return run(I1(), I1(), I1(), I1(), I1(), I1(), apart, brief);
                if (fours) return run(I1(), I4(), I1(), I1(), I4(), I1(), in_group, brief);
                return run(I1(), I4(), I1(), I1(), I4(), I1(), apart, brief);
            }
        }
        if constexpr (sizeof(T) * D <= 256)
            if (fours) return run(I4(), I4(), I1(), I1(), I4(), I1(), in_group, full);
        if (fours) return run(I4(), I4(), I1(), IL(), I1(), IL(), apart, full);
        if constexpr (LONG_APART<T, D>)
            if (a.n_heads > 2) {
                if (attn->n_kv_heads > 2) return run(I1(), I4(), I1(), I1(), I4(), I1(), apart, full);
                return run(I1(), I4(), I1(), IL(), I1(), IL(), apart, full);
            }
        return run(IL(), I1(), IL(), IL(), I1(), IL(), apart, full);
    });
}

}  // extern "C"
