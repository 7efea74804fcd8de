// rse_seqattn_bwd.hip -- backward of the attention over behaviour sequences:
// the probabilities are recomputed from q, k and the forward's log-sums, tile
// by tile, once with the queries as columns (dq, the bias gradient) and once
// with the keys as columns (dk, dv), so that every sum has one owner and a
// fixed order.
#include "rse_seqmma.h"

using namespace rse;
using namespace rse_host;

namespace {

// Rows k0 .. k0 + KT - 1 of two tensors on their way to LDS: loaded into
// registers (thread t: chunk t % CH of rows t / CH, + NT / CH, ...), stored
// after the current tile's work.  Hidden rows and rows past the end are
// stored as zeros, whatever they hold.
template <typename T, int D, int NT, int KT>
struct RowStage {
    using TL = Tile<T, D>;
    static constexpr int CH = TL::CH, PER = KT * CH / NT, STEP = NT / CH;
    static_assert(KT * CH % NT == 0, "tile shape");
    u32x4 x[PER], y[PER];
    bool hid[PER];
    __device__ __forceinline__ void load(const Rows<const T>& X, int hx, const Rows<const T>& Y, int hy, int64_t s, int k0,
                                         int end, const int64_t* key_off) {
        const int row = threadIdx.x / CH, c = threadIdx.x % CH;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int kk = k0 + row + i * STEP;
            const int64_t j = s + (kk < end ? kk : end - 1);
            x[i] = gload_u4(X.at(j, hx) + c * TL::EPC);
            y[i] = gload_u4(Y.at(j, hy) + c * TL::EPC);
            hid[i] = kk >= end || (key_off && key_off[j] < 0);
        }
    }
    __device__ __forceinline__ void store(u32x4* sx, u32x4* sy) const {
        const int row = threadIdx.x / CH, c = threadIdx.x % CH;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = TL::chunk_at(row + i * STEP, c);
            sx[at] = hid[i] ? u32x4{0, 0, 0, 0} : x[i];
            sy[at] = hid[i] ? u32x4{0, 0, 0, 0} : y[i];
        }
    }
};

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
template <typename T, int D, int W, int KT>
__global__ __launch_bounds__(W * 64) void k_attn_dq(SeqArgs a, int64_t slots, Rows<const T> q, Rows<const T> k,
                                                    Rows<const T> v, const float* lse2, const float* out32,
                                                    Rows<const T> dout, Rows<T> dq, float* delta, float* part) {
    using TL = Tile<T, D>;
    constexpr int NT = W * 64, CH = TL::CH, NS = KT / 32, ND = D / 32;
    __shared__ u32x4 s_k[2][KT * CH], s_v[2][KT * CH];
    __shared__ float s_mask[2][KT];
    __shared__ int32_t s_pos[2][KT];
    __shared__ int32_t s_range[2][3];
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

    for (int64_t slot = blockIdx.x; slot < slots; slot += gridDim.x) {
        int64_t s;
        int len, tile;
        if (!find_tile(a, slot, 32 * W, s, len, tile, head == 0)) continue;
        const int q0 = tile * 32 * W, my_q = q0 + 32 * w + (lane & 31), row = my_q < len ? my_q : len - 1;
        const int end = a.causal ? (q0 + 32 * W < len ? q0 + 32 * W : len) : len;
        const int my_end = a.causal && q0 + 32 * w + 32 < end ? q0 + 32 * w + 32 : end;
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
        const int32_t q_lo = wave_min(my_pos), q_hi = wave_max(my_pos);

        RowStage<T, D, NT, KT> st;
        int32_t rp = 0;
        bool rs = false;
        auto load_side = [&](int k0) {
            if (threadIdx.x < KT) {
                const int kk = k0 + (int)threadIdx.x;
                const int64_t j = s + (kk < end ? kk : end - 1);
                rp = a.pos[j];
                rs = kk < end && !(a.key_off && a.key_off[j] < 0);
            }
        };
        auto store_side = [&](int b) {
            if (w == 0) {
                const bool mine = lane < KT;
                const int32_t lo = wave_min(mine ? rp : INT32_MAX), hi = wave_max(mine ? rp : INT32_MIN);
                const bool any = __ballot(mine && !rs) != 0;
                if (mine) {
                    s_mask[b][lane] = rs ? 0.f : -INFINITY;
                    s_pos[b][lane] = rp;
                }
                if (lane == 0) {
                    s_range[b][0] = lo;
                    s_range[b][1] = hi;
                    s_range[b][2] = any;
                }
            }
        };

        f32x16 acc[ND] = {};
        st.load(k, g, v, g, s, 0, end, a.key_off);
        load_side(0);
        __syncthreads();                        // the previous tile's LDS is no longer read
        st.store(s_k[0], s_v[0]);
        store_side(0);
        __syncthreads();
        for (int k0 = 0, b = 0; k0 < end; k0 += KT, b ^= 1) {
            if (k0 + KT < end) {
                st.load(k, g, v, g, s, k0 + KT, end, a.key_off);
                load_side(k0 + KT);
            }
            if (k0 < my_end) {
                const int lo = wb.bucket(seq_dist(q_lo, s_range[b][1])), hi = wb.bucket(seq_dist(q_hi, s_range[b][0]));
                const bool hidden = __builtin_amdgcn_readfirstlane(s_range[b][2]);
                const bool diagonal = a.causal && k0 + KT - 1 > q0 + 32 * w;
                float sum = 0.f;
#pragma unroll
                for (int u = 0; u < NS; ++u) {
                    if (k0 + 32 * u >= my_end) continue;
                    f32x16 x = mma_rows<T, D>(s_k[b], 32 * u, qf, f32x16{});
                    const f32x16 dp = mma_rows<T, D>(s_v[b], 32 * u, df, f32x16{});
                    int idx[16];
                    if (lo == hi) {
                        const float b0 = wb.value(lo);
#pragma unroll
                        for (int r = 0; r < 16; ++r) x[r] = __builtin_fmaf(x[r], c2, b0);
                    } else {
                        bucket_index<true>(idx, wb, lo, hi, s_pos[b] + 32 * u, my_pos, a.cells, s_cell, s_bounds);
#pragma unroll
                        for (int r = 0; r < 16; ++r) x[r] = __builtin_fmaf(x[r], c2, s_bias[idx[r]]);
                    }
                    if (hidden) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const f32x4 mk = *reinterpret_cast<const f32x4*>(&s_mask[b][32 * u + 8 * j + 4 * half]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[4 * j + i] += mk[i];
                        }
                    }
                    if (diagonal) {
                        const int lim = my_q - k0 - 32 * u - 4 * half;
#pragma unroll
                        for (int r = 0; r < 16; ++r) x[r] = tile_row(r, 0) <= lim ? x[r] : -INFINITY;
                    }
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = __builtin_amdgcn_exp2f(x[r] - L) * (dp[r] - del);
                    if (lo == hi) {
#pragma unroll
                        for (int r = 0; r < 16; ++r) sum += x[r];
                    } else {
                        if (half == 0) {
#pragma unroll
                            for (int r = 0; r < 16; ++r) lds_add(hist + idx[r] * HC, x[r]);
                        } else {
#pragma unroll
                            for (int r = 0; r < 16; ++r) lds_add(hist + idx[r] * HC, x[r]);
                        }
                    }
                    RowOperand<T> ds;
                    ds.set(x);
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) acc[dt] = mma_over_rows<D>(s_k[b], 32 * u, dt, ds, acc[dt]);
                }
                if (lo == hi) {
                    sum += other_half(sum);
                    if (half == 0) lds_add(hist + lo * HC, sum);
                }
            }
            if (k0 + KT < end) {
                st.store(s_k[b ^ 1], s_v[b ^ 1]);
                store_side(b ^ 1);
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
__global__ __launch_bounds__(W * 64) void k_attn_dkv(SeqArgs a, Rows<const T> q, Rows<const T> k, Rows<const T> v,
                                                     const float* lse2, const float* delta, Rows<const T> dout,
                                                     Rows<T> dk, Rows<T> dv) {
    using TL = Tile<T, D>;
    constexpr int NT = W * 64, CH = TL::CH, NS = KT / 32, ND = D / 32, NBP = RSE_SEQ_MAX_BOUNDARIES + 1;
    __shared__ u32x4 s_q[2][KT * CH], s_d[2][KT * CH];
    __shared__ float s_lse[2][KT], s_del[2][KT];
    __shared__ int32_t s_pos[2][KT];
    __shared__ int32_t s_range[2][2];
    __shared__ int32_t s_bounds[NBP];
    __shared__ float s_bias[2][NBP];
    __shared__ uint32_t s_cell[128];
    const int lane = lane_id(), w = threadIdx.x / WAVE, half = lane >> 5;
    const int g = blockIdx.y, nb = a.n_bounds + 1;
    int64_t s;
    int len, tile;
    if (!find_tile(a, blockIdx.x, 32 * W, s, len, tile, false)) return;
    const int j0 = tile * 32 * W, my_k = j0 + 32 * w + (lane & 31), row = my_k < len ? my_k : len - 1;
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
    const int32_t k_lo = wave_min(my_pos), k_hi = wave_max(my_pos);
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
            const bool mine = lane < KT;
            const int32_t lo = wave_min(mine ? rp : INT32_MAX), hi = wave_max(mine ? rp : INT32_MIN);
            if (mine) {
                s_pos[b][lane] = rp;
                s_lse[b][lane] = rl;
                s_del[b][lane] = rd;
            }
            if (lane == 0) {
                s_range[b][0] = lo;
                s_range[b][1] = hi;
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
        if (!a.causal || i0 + KT - 1 >= j0 + 32 * w) {
            wb.bias[0] = s_bias[b][lane];
            wb.bias[1] = s_bias[b][64 + lane];
            const int lo = wb.bucket(seq_dist(s_range[b][0], k_hi)), hi = wb.bucket(seq_dist(s_range[b][1], k_lo));
            const bool diagonal = a.causal && i0 < j0 + 32 * w + 31;
#pragma unroll
            for (int u = 0; u < NS; ++u) {
                if (i0 + 32 * u >= len || (a.causal && i0 + 32 * u + 31 < j0 + 32 * w)) continue;
                f32x16 x = mma_rows<T, D>(s_q[b], 32 * u, kf, f32x16{});
                f32x16 dp = mma_rows<T, D>(s_d[b], 32 * u, vf, f32x16{});
                if (lo == hi) {
                    const float b0 = wb.value(lo);
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = __builtin_fmaf(x[r], c2, b0);
                } else {
                    x = add_bias<false>(x, c2, wb, lo, hi, s_pos[b] + 32 * u, my_pos, a.cells, s_cell, s_bounds, s_bias[b]);
                }
                if (diagonal) {
                    const int lim = my_k - i0 - 32 * u - 4 * half;
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

int waves_for(int64_t max_len) { return max_len <= 128 ? 1 : 4; }

BwdWs bwd_ws(const rse_seqattn* a, int64_t n, int64_t batch, int64_t max_len, void* base) {
    BwdWs w;
    const int64_t most = DQ_BLOCKS / a->n_heads > 16 ? DQ_BLOCKS / a->n_heads : 16;
    w.blocks = tile_slots(n, batch, 32 * waves_for(max_len));
    if (w.blocks > most) w.blocks = most;
    Carver c(base);
    w.delta = c.take<float>((size_t)a->n_heads * n);
    w.part = c.take<float>((size_t)a->n_heads * w.blocks * (a->n_bounds + 1));
    w.bytes = c.size();
    return w;
}

template <typename T, int D, int W>
int run_bwd_w(const SeqArgs& a, const rse_seq_rows* q, const rse_seq_rows* k, const rse_seq_rows* v, const Saved& sv,
              const rse_seq_rows* dout, const rse_seq_rows* dq, const rse_seq_rows* dk, const rse_seq_rows* dv,
              float* dbias, const BwdWs& w, hipStream_t s) {
    constexpr int KT = W > 1 && D * sizeof(T) <= 256 ? 64 : 32;
    const int nb = a.n_bounds + 1;
    const int64_t slots = tile_slots(a.n_events, a.batch, 32 * W);
    if (slots > INT32_MAX) return RSE_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((k_attn_dq<T, D, W, KT>), dim3((unsigned)w.blocks, a.n_heads), dim3(W * WAVE),
                       W * nb * HC * sizeof(float), s, a, slots, rows_view<const T>(q), rows_view<const T>(k),
                       rows_view<const T>(v), sv.lse2, sv.out32, rows_view<const T>(dout), rows_view<T>(dq), w.delta, w.part);
    int rc = launch_status();
    if (rc) return rc;
    hipLaunchKernelGGL(k_attn_dbias, dim3(a.n_heads), dim3(1024), 0, s, w.part, (int)w.blocks, nb, dbias);
    hipLaunchKernelGGL((k_attn_dkv<T, D, W, KT>), dim3((unsigned)slots, a.n_heads / a.group), dim3(W * WAVE), 0, s, a,
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
        switch (waves_for(a.max_len)) {
            case 1: return run_bwd_w<T, D, 1>(a, q, k, v, sv, dout, dq, dk, dv, d_dbias, w, s);
            default: return run_bwd_w<T, D, 4>(a, q, k, v, sv, dout, dq, dk, dv, d_dbias, w, s);
        }
    });
}

}  // extern "C"
