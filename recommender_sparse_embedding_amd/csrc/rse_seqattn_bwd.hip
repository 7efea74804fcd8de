// rse_seqattn_bwd.hip -- backward of the attention over behaviour sequences:
// the probabilities are recomputed from q, k and the forward's log-sums, tile
// by tile, once with the queries as columns (dq, the bias gradient) and once
// with the keys as columns (dk, dv), so that every sum has one owner and a
// fixed order.
#include "rse_seqmma.h"

using namespace rse;
using namespace rse_host;

namespace {

// Columns of a wave's bucket sums: the two halves of the wave add in turn to
// the same 32, so each entry is added to in program order.
constexpr int HC = 32;

__device__ __forceinline__ void lds_add(float* p, float x) {
    __builtin_amdgcn_ds_faddf((RSE_LDS float*)p, x, 0, 0, false);
}

// dq and the bias gradient, queries as columns: per tile of keys
// S^T = K Q^T and dP^T = V dO^T, ds = p (dp - delta), dQ^T += K^T dS^T.
// delta = sum_j p dp = dO . out, from the unrounded outputs.  ds of a tile in
// one bucket is summed in registers, else scattered into the wave's LDS
// columns of bucket sums.  A block stays with its head and takes tiles of
// queries blockIdx.x, + gridDim.x, ...; its sums go to part.
// Registers are held to what lets DQ_WAVES (DKV_WAVES) waves share a SIMD.
template <typename T, int D>
constexpr int DQ_WAVES = Shape<T, D>::RB <= 64 ? 3 : (Shape<T, D>::RB <= 256 ? 2 : 1);
template <typename T, int D>
constexpr int DKV_WAVES = Shape<T, D>::RB <= 64 ? 3 : (Shape<T, D>::RB <= 128 || sizeof(T) == 4 && D == 64 ? 2 : 1);

template <typename T, int D, int W, int KT>
__global__ __launch_bounds__(W * 64) __attribute__((amdgpu_waves_per_eu(DQ_WAVES<T, D>))) void k_attn_dq(SeqArgs a, TileGrid grid, Rows<const T> q, Rows<const T> k,
                                                    Rows<const T> v, const float* lse2, const float* out32,
                                                    Rows<const T> dout, Rows<T> dq, float* delta, float* part) {
    using TL = Tile<T, D>;
    constexpr int NT = W * 64, CH = TL::CH, NS = KT / 32, ND = D / 32;
    __shared__ u32x4 s_k[2][KT * CH], s_v[2][KT * CH];
    __shared__ KeySide<KT> s_side;
    __shared__ int32_t s_bounds[RSE_SEQ_MAX_BOUNDARIES + 1];
    __shared__ float s_bias[RSE_SEQ_MAX_BOUNDARIES + 1];
    __shared__ uint32_t s_cell[128];
    extern __shared__ float s_hist[];           // [W][n_bounds + 1][HC]
    const int lane = lane_id(), w = threadIdx.x / WAVE, half = lane >> 5;
    const int head = blockIdx.y, g = head / a.group, nb = a.n_bounds + 1;
    float* hist = s_hist + w * nb * HC + (lane & 31);

    WaveBuckets wb;
    wb.load(a.hdr, a.bias + head * nb, a.n_bounds, LOG2E);
    for (int t = threadIdx.x; t <= RSE_SEQ_MAX_BOUNDARIES; t += NT) {
        s_bounds[t] = a.hdr->bounds[t];
        s_cell[t] = reinterpret_cast<const uint32_t*>(a.hdr->cell)[t];
        s_bias[t] = t < nb ? a.bias[head * nb + t] * LOG2E : 0.f;
    }
    for (int t = threadIdx.x; t < W * nb * HC; t += NT) s_hist[t] = 0.f;
    const float c2 = fabsf(a.scale) * LOG2E;

    const LdsBuckets lb = {s_bounds, s_cell, a.cells != 0, a.n_bounds};
    for (int64_t item = blockIdx.x; item < grid.items; item += gridDim.x) {
        int64_t s;
        int len, tile;
        if (!find_tile(a, grid, item, 32 * W, a.causal, s, len, tile, head == 0)) continue;
        const int q0 = tile * 32 * W, w0 = q0 + 32 * w, my_q = w0 + (lane & 31), row = my_q < len ? my_q : len - 1;
        const int end = a.causal ? (q0 + 32 * W < len ? q0 + 32 * W : len) : len;
        const int my_end = w0 >= len ? 0 : (a.causal && w0 + 32 < end ? w0 + 32 : end);
        RowStage<T, D, NT, KT> st;
        KeySideStage side;
        st.load(k, g, v, g, s, 0, end, a.key_off);
        side.load(a, s, 0, end, KT);
        ColFrag<T, D> qf, df;
        qf.load(q.at(s + row, head), half);
        df.load(dout.at(s + row, head), half);
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
        float L = lse2[(int64_t)head * a.n_events + s + row];
        if (my_q >= len || L == -INFINITY) L = INFINITY;        // p = 0
        if (my_q < len && half == 0) delta[(int64_t)head * a.n_events + s + my_q] = del;
        if (a.scale < 0.f) qf.negate();
        const int32_t my_pos = a.pos[s + row];
        const int32_t q_lo = half_min(my_pos), q_hi = half_max(my_pos);
        f32x16 acc[ND] = {};
        __syncthreads();                        // the previous tile's LDS is no longer read
        st.store(s_k[0], s_v[0]);
        side.store(s_side, 0);
        __syncthreads();
        for (int k0 = 0, b = 0; k0 < end; k0 += KT, b ^= 1) {
            if (k0 + KT < end) {
                st.load(k, g, v, g, s, k0 + KT, end, a.key_off);
                side.load(a, s, k0 + KT, end, KT);
            }
#pragma unroll
            for (int u = 0; u < NS; ++u) {
                const int k1 = k0 + 32 * u;
                if (k1 >= my_end) continue;
                f32x16 x = mma_rows<T, D>(s_k[b], 32 * u, qf, f32x16{});
                const f32x16 dp = mma_rows<T, D>(s_v[b], 32 * u, df, f32x16{});
                TileBuckets<true> tb;
                tb.set(wb, q_lo, q_hi, s_side.range[b][u]);
                int idx[16];
                if (tb.lo == tb.hi) {
                    const float b0 = wb.value(tb.lo) - L;
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = __builtin_fmaf(x[r], c2, b0);
                } else {
                    tb.index(idx, wb, lb, s_side.pos[b] + 32 * u, my_pos);
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = __builtin_fmaf(x[r], c2, -L) + s_bias[idx[r]];
                }
                if (__builtin_amdgcn_readfirstlane((uint32_t)(s_side.hidden[b] >> (32 * u)))) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f32x4 mk = *reinterpret_cast<const f32x4*>(&s_side.mask[b][32 * u + 8 * j + 4 * half]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[4 * j + i] += mk[i];
                    }
                }
                if (a.causal && k1 + 31 > w0) {
                    const int lim = my_q - k1 - 4 * half;
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = tile_row(r, 0) <= lim ? x[r] : -INFINITY;
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) x[r] = __builtin_amdgcn_exp2f(x[r]) * (dp[r] - del);
                if (tb.lo == tb.hi) {
                    float sum = x[0];
#pragma unroll
                    for (int r = 1; r < 16; ++r) sum += x[r];
                    sum += other_half(sum);
                    if (half == 0) lds_add(hist + tb.lo * HC, sum);
                } else if (half == 0) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) lds_add(hist + idx[r] * HC, x[r]);
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r) lds_add(hist + idx[r] * HC, x[r]);
                }
                RowOperand<T> ds;
                ds.set(x);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) acc[dt] = mma_over_rows<D>(s_k[b], 32 * u, dt, ds, acc[dt]);
            }
            if (k0 + KT < end) {
                st.store(s_k[b ^ 1], s_v[b ^ 1]);
                side.store(s_side, b ^ 1);
                __syncthreads();
            }
        }
        if (my_q < len) {
            T* dst = dq.at(s + my_q, head);
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) store_column(dst + 32 * dt, acc[dt], a.scale);
        }
    }
    __syncthreads();
    for (int t = threadIdx.x; t < nb; t += NT) {
        float sum = 0.f;
        for (int x = 0; x < W; ++x)
            for (int c = 0; c < HC; ++c) sum += s_hist[(x * nb + t) * HC + ((c + t) & (HC - 1))];
        part[((int64_t)head * gridDim.x + blockIdx.x) * nb + t] = sum;
    }
}

// The blocks' bucket sums, added in 64 bits in a fixed order: one block per
// head, 8 threads per bucket.
__global__ __launch_bounds__(1024) void k_attn_dbias(const float* part, int blocks, int nb, float* dbias) {
    __shared__ double s[8][RSE_SEQ_MAX_BOUNDARIES + 1];
    const int h = blockIdx.x, b = threadIdx.x & 127, p = threadIdx.x >> 7;
    double t = 0.0;
    if (b < nb)
        for (int x = p; x < blocks; x += 8) t += part[((int64_t)h * blocks + x) * nb + b];
    s[p][b] = t;
    __syncthreads();
    if (p == 0 && b < nb) {
        for (int x = 1; x < 8; ++x) t += s[x][b];
        dbias[h * nb + b] = (float)t;
    }
}

// dk and dv, keys as columns: per tile of queries of each head of the group
// S = Q K^T and dP = dO V^T, dV^T += dO^T P, dK^T += Q^T dS.
template <typename T, int D, int W, int KT>
__global__ __launch_bounds__(W * 64) __attribute__((amdgpu_waves_per_eu(DKV_WAVES<T, D>))) void k_attn_dkv(SeqArgs a, TileGrid grid, Rows<const T> q, Rows<const T> k, Rows<const T> v,
                                                     const float* lse2, const float* delta, Rows<const T> dout,
                                                     Rows<T> dk, Rows<T> dv) {
    using TL = Tile<T, D>;
    constexpr int NT = W * 64, CH = TL::CH, NS = KT / 32, ND = D / 32, NBP = RSE_SEQ_MAX_BOUNDARIES + 1;
    __shared__ u32x4 s_q[2][KT * CH], s_d[2][KT * CH];
    __shared__ float s_lse[2][KT], s_del[2][KT];
    __shared__ int32_t s_pos[2][KT];
    __shared__ int32_t s_range[2][NS][2];
    __shared__ int32_t s_bounds[NBP];
    __shared__ float s_bias[2][NBP];
    __shared__ uint32_t s_cell[128];
    const int lane = lane_id(), w = threadIdx.x / WAVE, half = lane >> 5;
    const int n_kv = a.n_heads / a.group, g = blockIdx.x % n_kv, nb = a.n_bounds + 1;
    int64_t s;
    int len, tile;
    if (!find_tile(a, grid, blockIdx.x / n_kv, 32 * W, false, s, len, tile, false)) return;
    const int j0 = tile * 32 * W, w0 = j0 + 32 * w, my_k = w0 + (lane & 31), row = my_k < len ? my_k : len - 1;
    const bool seen = !(a.key_off && a.key_off[s + row] < 0);
    const int first = a.causal ? j0 / KT * KT : 0;                  // queries of the block: first .. len
    const int per_head = (len - first + KT - 1) / KT, total = per_head * a.group;

    for (int t = threadIdx.x; t < NBP; t += NT) {
        s_bounds[t] = a.hdr->bounds[t];
        s_cell[t] = reinterpret_cast<const uint32_t*>(a.hdr->cell)[t];
    }
    ColFrag<T, D> kf, vf;
    kf.load(k.at(s + row, g), half);
    vf.load(v.at(s + row, g), half);
    if (a.scale < 0.f) kf.negate();
    const float c2 = fabsf(a.scale) * LOG2E;
    const int32_t my_pos = a.pos[s + row];
    const int32_t k_lo = half_min(my_pos), k_hi = half_max(my_pos);
    const LdsBuckets lb = {s_bounds, s_cell, a.cells != 0, a.n_bounds};
    WaveBuckets wb;
    wb.load(a.hdr, a.bias, a.n_bounds, LOG2E);

    RowStage<T, D, NT, KT> st;
    int32_t rp = 0;
    float rl = 0.f, rd = 0.f, rb[NBP / NT + 1];
    auto load = [&](int it) {
        const int h = g * a.group + it / per_head, i0 = first + it % per_head * KT;
        st.load(q, h, dout, h, s, i0, len, nullptr);
        if (threadIdx.x < KT) {
            const int kk = i0 + (int)threadIdx.x;
            const int64_t j = s + (kk < len ? kk : len - 1);
            rp = a.pos[j];
            rl = lse2[(int64_t)h * a.n_events + j];
            rd = kk < len ? delta[(int64_t)h * a.n_events + j] : 0.f;
            if (kk >= len || rl == -INFINITY) rl = INFINITY;        // p = 0
        }
#pragma unroll
        for (int i = 0; i * NT < NBP; ++i) {
            const int t = i * NT + (int)threadIdx.x;
            rb[i] = t < nb ? a.bias[h * nb + t] * LOG2E : 0.f;
        }
    };
    auto store = [&](int b) {
        st.store(s_q[b], s_d[b]);
        if (w == 0) {
            const int32_t lo = half_min(rp), hi = half_max(rp);
            if (lane < KT) {
                s_pos[b][lane] = rp;
                s_lse[b][lane] = rl;
                s_del[b][lane] = rd;
                if ((lane & 31) == 0) {
                    s_range[b][lane / 32][0] = lo;
                    s_range[b][lane / 32][1] = hi;
                }
            }
        }
#pragma unroll
        for (int i = 0; i * NT < NBP; ++i) {
            const int t = i * NT + (int)threadIdx.x;
            if (t < NBP) s_bias[b][t] = rb[i];
        }
    };

    f32x16 ak[ND] = {}, av[ND] = {};
    load(0);
    store(0);
    __syncthreads();
    for (int it = 0, b = 0; it < total; ++it, b ^= 1) {
        const int i0 = first + it % per_head * KT;
        if (it + 1 < total) load(it + 1);
        if (w0 < len && (!a.causal || i0 + KT - 1 >= w0)) {
            wb.bias[0] = s_bias[b][lane];
            wb.bias[1] = s_bias[b][64 + lane];
#pragma unroll
            for (int u = 0; u < NS; ++u) {
                const int i1 = i0 + 32 * u;
                if (i1 >= len || (a.causal && i1 + 31 < w0)) continue;
                f32x16 x = mma_rows<T, D>(s_q[b], 32 * u, kf, f32x16{});
                f32x16 dp = mma_rows<T, D>(s_d[b], 32 * u, vf, f32x16{});
                TileBuckets<false> tb;
                tb.set(wb, k_lo, k_hi, s_range[b][u]);
                x = tb.logits(x, c2, 0.f, wb, lb, s_bias[b], s_pos[b] + 32 * u, my_pos);
                if (a.causal && i1 < w0 + 31) {
                    const int lim = my_k - i1 - 4 * half;
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = tile_row(r, 0) >= lim ? x[r] : -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 L = *reinterpret_cast<const f32x4*>(&s_lse[b][32 * u + 8 * j + 4 * half]);
                    const f32x4 de = *reinterpret_cast<const f32x4*>(&s_del[b][32 * u + 8 * j + 4 * half]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[4 * j + i] = __builtin_amdgcn_exp2f(x[4 * j + i] - L[i]);
                        dp[4 * j + i] = x[4 * j + i] * (dp[4 * j + i] - de[i]);
                    }
                }
                RowOperand<T> p, ds;
                p.set(x);
                ds.set(dp);
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) {
                    av[dt] = mma_over_rows<D>(s_d[b], 32 * u, dt, p, av[dt]);
                    ak[dt] = mma_over_rows<D>(s_q[b], 32 * u, dt, ds, ak[dt]);
                }
            }
        }
        if (it + 1 < total) {
            store(b ^ 1);
            __syncthreads();
        }
    }
    if (my_k < len) {
        T* pk = dk.at(s + my_k, g);
        T* pv = dv.at(s + my_k, g);
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) {
            if (!seen) ak[dt] = av[dt] = f32x16{};      // hidden: whatever the key held
            store_column(pk + 32 * dt, ak[dt], a.scale);
            store_column(pv + 32 * dt, av[dt], 1.f);
        }
    }
}

// ------------------------------------------------------------------ host --
// Blocks of k_attn_dq over all heads: enough to fill the GPU several times
// over; more would only add partial bucket sums.
constexpr int64_t DQ_BLOCKS = 4096;

struct BwdWs {
    float* delta;
    float* part;
    size_t bytes;
    int64_t blocks;              // of k_attn_dq, per head
};

// Events of a block's tile.
int tile_events(const rse_seqattn* a, int64_t max_len) {
    return by_type(a, [&](auto t, auto d) {
        using S = Shape<decltype(t), decltype(d)::value>;
        return 32 * (max_len <= SHORT ? S::W_SHORT : S::W_LONG);
    });
}

BwdWs bwd_ws(const rse_seqattn* a, int64_t n, int64_t batch, int64_t max_len, void* base) {
    BwdWs w;
    const int64_t most = DQ_BLOCKS / a->n_heads > 16 ? DQ_BLOCKS / a->n_heads : 16;
    w.blocks = tile_grid(n, batch, max_len, tile_events(a, max_len)).items;
    if (w.blocks > most) w.blocks = most;
    Carver c(base);
    w.delta = c.take<float>((size_t)a->n_heads * n);
    w.part = c.take<float>((size_t)a->n_heads * w.blocks * (a->n_bounds + 1));
    w.bytes = c.size();
    return w;
}

template <typename T, int D, int W, int KT>
int run_bwd(const SeqArgs& a, const rse_seq_rows* q, const rse_seq_rows* k, const rse_seq_rows* v, const Saved& sv,
              const rse_seq_rows* dout, const rse_seq_rows* dq, const rse_seq_rows* dk, const rse_seq_rows* dv,
              float* dbias, const BwdWs& w, hipStream_t s) {
    const int nb = a.n_bounds + 1;
    const TileGrid tg = tile_grid(a.n_events, a.batch, a.max_len, 32 * W);
    const int64_t dkv = tg.items * (a.n_heads / a.group);
    if (dkv > INT32_MAX) return RSE_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((k_attn_dq<T, D, W, KT>), dim3((unsigned)w.blocks, a.n_heads), dim3(W * WAVE),
                       W * nb * HC * sizeof(float), s, a, tg, rows_view<const T>(q), rows_view<const T>(k),
                       rows_view<const T>(v), sv.lse2, sv.out32, rows_view<const T>(dout), rows_view<T>(dq), w.delta, w.part);
    int rc = launch_status();
    if (rc) return rc;
    hipLaunchKernelGGL(k_attn_dbias, dim3(a.n_heads), dim3(1024), 0, s, w.part, (int)w.blocks, nb, dbias);
    hipLaunchKernelGGL((k_attn_dkv<T, D, W, KT>), dim3((unsigned)dkv), dim3(W * WAVE), 0, s, a, tg,
                       rows_view<const T>(q), rows_view<const T>(k), rows_view<const T>(v), sv.lse2, w.delta,
                       rows_view<const T>(dout), rows_view<T>(dk), rows_view<T>(dv));
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
        hipLaunchKernelGGL(k_attn_dbias, dim3(attn->n_heads), dim3(1024), 0, s, w.part, 0, attn->n_bounds + 1, d_dbias);
        return launch_status();
    }
    for (const rse_seq_rows* r : {q, k, v, dout, dq, dk, dv})
        if (!rows_ok(r, attn->dtype)) return RSE_ERR_INVALID_ARG;
    if (!d_saved || reinterpret_cast<uintptr_t>(d_saved) % 256) return RSE_ERR_INVALID_ARG;
    const Saved sv = saved_view(attn, batch->n_events, const_cast<void*>(d_saved));
    if (saved_bytes < sv.bytes) return RSE_ERR_WORKSPACE;
    const SeqArgs a = seq_args(attn, batch);
    return by_type(attn, [&](auto t, auto d) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        using S = Shape<T, D>;
        if (a.max_len <= SHORT)
            return run_bwd<T, D, S::W_SHORT, S::KT_SHORT>(a, q, k, v, sv, dout, dq, dk, dv, d_dbias, w, s);
        return run_bwd<T, D, S::W_LONG, S::KT_LONG>(a, q, k, v, sv, dout, dq, dk, dv, d_dbias, w, s);
    });
}

}  // extern "C"
