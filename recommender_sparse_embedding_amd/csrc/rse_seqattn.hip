// rse_seqattn.hip -- attention over the events of each behaviour sequence of
// a jagged batch, with a learned bias by buckets of the events' distance:
// forward, and the backward that recomputes the probabilities.
#include <cmath>
#include <new>

#include "rse_seqmma.h"

using namespace rse;
using namespace rse_host;

namespace {

constexpr int AB = 256;                 // threads per block
constexpr int AW = AB / WAVE;

struct InitArgs {
    int32_t n_bounds;
    int32_t bounds[RSE_SEQ_MAX_BOUNDARIES + 1];
};

__global__ void k_attn_init(SeqHeader* h, InitArgs a) {
    if (threadIdx.x == 0) {
        h->status = 0;
        h->n_bounds = a.n_bounds;
    }
    if (threadIdx.x <= RSE_SEQ_MAX_BOUNDARIES) h->bounds[threadIdx.x] = a.bounds[threadIdx.x];
}

__global__ void k_attn_clear(SeqHeader* h) { h->status = 0; }

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m, WAVE);
    return x;
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) x = fmaxf(x, __shfl_xor(x, m, WAVE));
    return x;
}

// The sequence of event i, or false (status set) if its offsets are malformed.
__device__ __forceinline__ bool find_seq(const SeqArgs& a, int64_t i, int64_t& s, int64_t& e) {
    const int64_t b = wave_last_le(a.batch, [&](int64_t x) { return a.offsets[x]; }, i);
    s = a.offsets[b];
    e = a.offsets[b + 1];
    if (s < 0 || e > a.n_events || i < s || i >= e || e - s > a.max_len) {
        if (lane_id() == 0) set_status(&a.hdr->status, RSE_ERR_BAD_INPUT);
        return false;
    }
    return true;
}

template <typename T, int D>
__device__ __forceinline__ float dot_row(const float* x, const T* y) {
    float s = 0.f;
#pragma unroll 8
    for (int d = 0; d < D; ++d) s = __fmaf_rn(x[d], to_f32(y[d]), s);
    return s;
}

__device__ __forceinline__ bool visible(const SeqArgs& a, int64_t i, int64_t j) {
    return (!a.causal || j <= i) && (!a.key_off || a.key_off[j] >= 0);
}

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// More distinct buckets than this in a tile: looked up event by event.
constexpr int CHAIN = 6;

// Bias (base 2) of the lane's column for the 16 rows of a 32 x 32 tile that
// may span buckets lo .. hi, added to s times c.  row_pos: positions of the
// tile's rows in LDS.  A tile of few buckets compares each distance with the
// boundaries between them; with many, each distance is searched in the LDS
// copy of the boundaries.
// `column_first`: the column event is the query (distance = column - row).
template <bool column_first>
__device__ __forceinline__ f32x16 add_bias(f32x16 s, float c, const WaveBuckets& wb, int lo, int hi, const int32_t* row_pos,
                                           int32_t col_pos, const int32_t* s_bounds, const float* s_bias) {
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
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) b[r] = s_bias[seq_bucket(s_bounds, wb.n, dist[r])];
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = __builtin_fmaf(s[r], c, b[r]);
    return s;
}

// Forward.  A block of W waves takes 32 W queries of one sequence and head; a
// wave has 32 of them as columns.  Keys go by in tiles of KT, staged in LDS
// row-major (the next tile's loads are in flight meanwhile): S^T = K Q^T,
// online softmax down the registers of a lane (a row's maximum needs one
// exchange between the wave's halves, its sum none until the end), and
// O^T += V^T P^T with the same registers as operand.
template <typename T, int D, int W, int KT>
__global__ __launch_bounds__(W * 64) void k_attn_fwd(SeqArgs a, Rows<const T> q, Rows<const T> k, Rows<const T> v,
                                                     Rows<T> out, float* lse) {
    using TL = Tile<T, D>;
    constexpr int NT = W * 64, CH = TL::CH, PER = KT * CH / NT, NS = KT / 32, ND = D / 32;
    static_assert(KT * CH % NT == 0 && KT <= 64, "tile shape");
    __shared__ u32x4 s_k[2][KT * CH], s_v[2][KT * CH];
    __shared__ float s_mask[2][KT];
    __shared__ int32_t s_pos[2][KT];
    __shared__ int32_t s_range[2][3];           // lowest and highest position, any key hidden
    __shared__ int32_t s_bounds[RSE_SEQ_MAX_BOUNDARIES + 1];
    __shared__ float s_bias[RSE_SEQ_MAX_BOUNDARIES + 1];
    const int lane = lane_id(), w = threadIdx.x / WAVE, half = lane >> 5;
    const int head = blockIdx.y, g = head / a.group, nb = a.n_bounds + 1;
    int64_t s;
    int len, tile;
    if (!find_tile(a, blockIdx.x, 32 * W, s, len, tile, head == 0)) return;
    const int n_tiles = (len + 32 * W - 1) / (32 * W);
    if (a.causal) tile = n_tiles - 1 - tile;    // the longest first
    const int q0 = tile * 32 * W, my_q = q0 + 32 * w + (lane & 31), row = my_q < len ? my_q : len - 1;
    const int end = a.causal ? (q0 + 32 * W < len ? q0 + 32 * W : len) : len;      // keys of the block
    const int my_end = a.causal && q0 + 32 * w + 32 < end ? q0 + 32 * w + 32 : end;  // and of the wave

    WaveBuckets wb;
    wb.load(a.hdr, a.bias + head * nb, a.n_bounds, LOG2E);
    for (int t = threadIdx.x; t <= RSE_SEQ_MAX_BOUNDARIES; t += NT) {
        s_bounds[t] = a.hdr->bounds[t];
        s_bias[t] = t < nb ? a.bias[head * nb + t] * LOG2E : 0.f;
    }
    ColFrag<T, D> qf;
    qf.load(q.at(s + row, head), half);
    if (a.scale < 0.f) qf.negate();
    const float c2 = fabsf(a.scale) * LOG2E;
    const int32_t my_pos = a.pos[s + row];
    const int32_t q_lo = wave_min(my_pos), q_hi = wave_max(my_pos);

    // staging: thread t holds chunk t % CH of rows t / CH, + NT / CH, ...
    const int srow = threadIdx.x / CH, sch = threadIdx.x % CH;
    u32x4 rk[PER], rv[PER];
    int32_t rp = 0;
    bool rs = false;
    bool hid[PER];
    auto load_tile = [&](int k0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int kk = k0 + srow + i * (NT / CH);
            const int64_t j = s + (kk < end ? kk : end - 1);
            rk[i] = gload_u4(k.at(j, g) + sch * TL::EPC);
            rv[i] = gload_u4(v.at(j, g) + sch * TL::EPC);
            hid[i] = kk >= end || (a.key_off && a.key_off[j] < 0);
        }
        if (threadIdx.x < KT) {
            const int kk = k0 + (int)threadIdx.x;
            const int64_t j = s + (kk < end ? kk : end - 1);
            rp = a.pos[j];
            rs = kk < end && !(a.key_off && a.key_off[j] < 0);
        }
    };
    auto store_tile = [&](int b) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = TL::chunk_at(srow + i * (NT / CH), sch);
            s_k[b][at] = hid[i] ? u32x4{0, 0, 0, 0} : rk[i];
            s_v[b][at] = hid[i] ? u32x4{0, 0, 0, 0} : rv[i];
        }
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

    f32x16 o[ND] = {};
    float m = -INFINITY, l = 0.f;
    load_tile(0);
    store_tile(0);
    __syncthreads();
    for (int k0 = 0, b = 0; k0 < end; k0 += KT, b ^= 1) {
        if (k0 + KT < end) load_tile(k0 + KT);
        if (k0 < my_end) {
            f32x16 x[NS];
#pragma unroll
            for (int u = 0; u < NS; ++u) x[u] = mma_rows<T, D>(s_k[b], 32 * u, qf, f32x16{});
            const int lo = wb.bucket(seq_dist(q_lo, s_range[b][1])), hi = wb.bucket(seq_dist(q_hi, s_range[b][0]));
            const bool hidden = __builtin_amdgcn_readfirstlane(s_range[b][2]);
            const bool diagonal = a.causal && k0 + KT - 1 > q0 + 32 * w;
            float c = c2, bias = 0.f;           // p = exp2(x c + bias - m)
            if (lo == hi && !hidden && !diagonal) {
                bias = wb.value(lo);
            } else {
                c = 1.f;
#pragma unroll
                for (int u = 0; u < NS; ++u) {
                    x[u] = add_bias<true>(x[u], c2, wb, lo, hi, s_pos[b] + 32 * u, my_pos, s_bounds, s_bias);
                    if (hidden) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const f32x4 mk = *reinterpret_cast<const f32x4*>(&s_mask[b][32 * u + 8 * j + 4 * half]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[u][4 * j + i] += mk[i];
                        }
                    }
                    if (diagonal) {
                        const int lim = my_q - k0 - 32 * u - 4 * half;
#pragma unroll
                        for (int r = 0; r < 16; ++r) x[u][r] = tile_row(r, 0) <= lim ? x[u][r] : -INFINITY;
                    }
                }
            }
            float top = x[0][0];
#pragma unroll
            for (int u = 0; u < NS; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, x[u][r]);
            top = fmaxf(top, other_half(top));
            top = __builtin_fmaf(top, c, bias);
            // the reference of the exponents follows the maximum only when it
            // has grown by more than 8 (p up to 2^8, exact in a float), so
            // that most tiles leave the sums as they are
            if (__any(top > m + 8.f || (m == -INFINITY && top > -INFINITY))) {
                const float ref = fmaxf(m, top);
                const float r = ref == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - ref);
                m = ref;
                l *= r;
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) o[dt] *= r;
            }
            const float shift = m == -INFINITY ? 0.f : bias - m;
            RowOperand<T> p[NS];
#pragma unroll
            for (int u = 0; u < NS; ++u) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    x[u][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[u][r], c, shift));
                    l += x[u][r];
                }
                p[u].set(x[u]);
            }
#pragma unroll
            for (int u = 0; u < NS; ++u)
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) o[dt] = mma_over_rows<D>(s_v[b], 32 * u, dt, p[u], o[dt]);
        }
        if (k0 + KT < end) {
            store_tile(b ^ 1);
            __syncthreads();
        }
    }
    l += other_half(l);
    const float inv = l > 0.f ? 1.f / l : 0.f;
    if (my_q < len) {
        T* dst = out.at(s + my_q, head);
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) store_column(dst + 32 * dt, o[dt], inv);
        if (lse && half == 0) lse[(int64_t)head * a.n_events + s + my_q] = l > 0.f ? (m + log2f(l)) * LN2 : -INFINITY;
    }
}

// dq, delta and the bias gradient: one wave per event, all waves of a block
// for one head (blockIdx.y).  Each lane adds into its own LDS column of the
// bucket sums; the block's sums go to part[block][bucket].
template <typename T, int D>
__global__ __launch_bounds__(AB) void k_attn_dq(SeqArgs a, Rows<const T> q, Rows<const T> k, Rows<const T> v,
                                                const float* lse, Rows<const T> dout, Rows<T> dq, float* delta,
                                                float* part) {
    extern __shared__ float hist[];     // [n_bounds + 1][AB]
    __shared__ int32_t bounds[RSE_SEQ_MAX_BOUNDARIES + 1];
    __shared__ float sq[AW][D], sd[AW][D];
    const int nb = a.n_bounds + 1;
    for (int t = threadIdx.x; t <= RSE_SEQ_MAX_BOUNDARIES; t += AB) bounds[t] = a.hdr->bounds[t];
    for (int t = threadIdx.x; t < nb * AB; t += AB) hist[t] = 0.f;
    __syncthreads();
    constexpr int E = (D + WAVE - 1) / WAVE;
    const int lane = lane_id(), w = threadIdx.x / WAVE, h = blockIdx.y, g = h / a.group;
    const float* bias = a.bias + h * nb;
    for (int64_t i = (int64_t)blockIdx.x * AW + w; i < a.n_events; i += (int64_t)gridDim.x * AW) {
        int64_t s, e;
        if (!find_seq(a, i, s, e)) continue;
        for (int d = lane; d < D; d += WAVE) {
            sq[w][d] = to_f32(q.at(i, h)[d]);
            sd[w][d] = to_f32(dout.at(i, h)[d]);
        }
        wave_lds_sync();
        const float L = lse[(int64_t)h * a.n_events + i];
        const int64_t end = a.causal ? i + 1 : e;
        float sum = 0.f, acc[E] = {};
        for (int pass = 0; pass < 2; ++pass) {
            for (int64_t c = s; c < end; c += WAVE) {
                const int64_t j = c + lane;
                float p = 0.f, dp = 0.f;
                int b = 0;
                const bool on = j < end && visible(a, i, j);
                if (on) {
                    b = seq_bucket(bounds, a.n_bounds, seq_dist(a.pos[i], a.pos[j]));
                    p = expf(dot_row<T, D>(sq[w], k.at(j, g)) * a.scale + bias[b] - L);
                    dp = dot_row<T, D>(sd[w], v.at(j, g));
                }
                if (pass == 0) {
                    sum += on ? p * dp : 0.f;
                    continue;
                }
                const float ds = on ? p * (dp - sum) : 0.f;
                if (on) hist[b * AB + threadIdx.x] += ds;
                const unsigned long long used = __ballot(on);
                for (int t = 0; t < WAVE; ++t) {
                    if (!((used >> t) & 1)) continue;
                    const float dt = __shfl(ds, t, WAVE);
#pragma unroll
                    for (int u = 0; u < E; ++u)
                        if (u * WAVE + lane < D)
                            acc[u] = __fmaf_rn(dt, to_f32(k.at(c + t, g)[u * WAVE + lane]), acc[u]);
                }
            }
            if (pass == 0) sum = wave_sum(sum);
        }
#pragma unroll
        for (int u = 0; u < E; ++u)
            if (u * WAVE + lane < D) from_f32(dq.at(i, h)[u * WAVE + lane], acc[u] * a.scale);
        if (lane == 0) delta[(int64_t)h * a.n_events + i] = sum;
        wave_lds_sync();
    }
    __syncthreads();
    for (int b = threadIdx.x; b < nb; b += AB) {
        float t = 0.f;
        for (int x = 0; x < AB; ++x) t += hist[b * AB + x];
        part[((int64_t)h * gridDim.x + blockIdx.x) * nb + b] = t;
    }
}

__global__ void k_attn_dbias(const float* part, int blocks, int nb, float* dbias) {
    const int h = blockIdx.x;
    for (int b = threadIdx.x; b < nb; b += blockDim.x) {
        double t = 0.0;
        for (int x = 0; x < blocks; ++x) t += part[((int64_t)h * blocks + x) * nb + b];
        dbias[h * nb + b] = (float)t;
    }
}

// dk and dv: one wave per event and key/value head, 64 queries at a time.
template <typename T, int D>
__global__ __launch_bounds__(AB) void k_attn_dkv(SeqArgs a, Rows<const T> q, Rows<const T> k, Rows<const T> v,
                                                 const float* lse, const float* delta, Rows<const T> dout,
                                                 Rows<T> dk, Rows<T> dv) {
    __shared__ int32_t bounds[RSE_SEQ_MAX_BOUNDARIES + 1];
    __shared__ float sk[AW][D], sv[AW][D];
    for (int t = threadIdx.x; t <= RSE_SEQ_MAX_BOUNDARIES; t += AB) bounds[t] = a.hdr->bounds[t];
    __syncthreads();
    constexpr int E = (D + WAVE - 1) / WAVE;
    const int lane = lane_id(), w = threadIdx.x / WAVE, nkv = a.n_heads / a.group, nb = a.n_bounds + 1;
    const int64_t items = a.n_events * nkv;
    for (int64_t it = (int64_t)blockIdx.x * AW + w; it < items; it += (int64_t)gridDim.x * AW) {
        const int64_t j = it / nkv;
        const int g = (int)(it % nkv);
        int64_t s, e;
        if (!find_seq(a, j, s, e)) continue;
        const bool seen = !a.key_off || a.key_off[j] >= 0;
        for (int d = lane; d < D; d += WAVE) {
            sk[w][d] = to_f32(k.at(j, g)[d]);
            sv[w][d] = to_f32(v.at(j, g)[d]);
        }
        wave_lds_sync();
        float ak[E] = {}, av[E] = {};
        for (int h = g * a.group; seen && h < (g + 1) * a.group; ++h) {
            for (int64_t c = a.causal ? j : s; c < e; c += WAVE) {
                const int64_t i = c + lane;
                float p = 0.f, ds = 0.f;
                if (i < e) {
                    const int b = seq_bucket(bounds, a.n_bounds, seq_dist(a.pos[i], a.pos[j]));
                    p = expf(dot_row<T, D>(sk[w], q.at(i, h)) * a.scale + a.bias[h * nb + b] -
                             lse[(int64_t)h * a.n_events + i]);
                    ds = p * (dot_row<T, D>(sv[w], dout.at(i, h)) - delta[(int64_t)h * a.n_events + i]);
                }
                const int n = (int)(e - c < WAVE ? e - c : WAVE);
                for (int t = 0; t < n; ++t) {
                    const float pt = __shfl(p, t, WAVE), dt = __shfl(ds, t, WAVE);
#pragma unroll
                    for (int u = 0; u < E; ++u)
                        if (u * WAVE + lane < D) {
                            av[u] = __fmaf_rn(pt, to_f32(dout.at(c + t, h)[u * WAVE + lane]), av[u]);
                            ak[u] = __fmaf_rn(dt, to_f32(q.at(c + t, h)[u * WAVE + lane]), ak[u]);
                        }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < E; ++u)
            if (u * WAVE + lane < D) {
                from_f32(dk.at(j, g)[u * WAVE + lane], ak[u] * a.scale);
                from_f32(dv.at(j, g)[u * WAVE + lane], av[u]);
            }
        wave_lds_sync();
    }
}

// ------------------------------------------------------------------ host --
int batch_ok(const rse_seqattn* a, const rse_seq_batch* b) {
    if (!a || !b || !b->d_offsets || !b->d_bias) return RSE_ERR_INVALID_ARG;
    if (b->batch < 0 || b->n_events < 0 || b->max_len < 0) return RSE_ERR_INVALID_ARG;
    if (b->n_events > 0 && (!b->d_pos || b->batch == 0 || b->max_len == 0)) return RSE_ERR_INVALID_ARG;
    return RSE_OK;
}

SeqArgs seq_args(const rse_seqattn* a, const rse_seq_batch* b) {
    SeqArgs s;
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
    s.scale = a->scale;
    return s;
}

size_t saved_bytes_of(const rse_seqattn* a, int64_t n) { return (size_t)a->n_heads * (size_t)n * sizeof(float); }

constexpr int DQ_BLOCKS = 512;

struct BwdWs {
    float* delta;
    float* part;
    size_t bytes;
};
BwdWs bwd_ws(const rse_seqattn* a, int64_t n, void* base) {
    Carver c(base);
    BwdWs w;
    w.delta = c.take<float>((size_t)a->n_heads * n);
    w.part = c.take<float>((size_t)a->n_heads * DQ_BLOCKS * (a->n_bounds + 1));
    w.bytes = c.size();
    return w;
}

template <typename T, int D, int W>
int run_fwd_w(const SeqArgs& a, const rse_seq_rows* q, const rse_seq_rows* k, const rse_seq_rows* v,
              const rse_seq_rows* out, float* lse, hipStream_t s) {
    // keys of a tile: 64 where two buffers of them take at most 64 KiB and
    // there are several waves to stage them
    constexpr int KT = W > 1 && D * sizeof(T) <= 256 ? 64 : 32;
    const int64_t slots = tile_slots(a.n_events, a.batch, 32 * W);
    if (slots > INT32_MAX) return RSE_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((k_attn_fwd<T, D, W, KT>), dim3((unsigned)slots, a.n_heads), dim3(W * WAVE), 0, s, a,
                       rows_view<const T>(q), rows_view<const T>(k), rows_view<const T>(v), rows_view<T>(out), lse);
    return launch_status();
}

// Waves of a block: as many groups of 32 queries as a sequence can have, up to 4.
template <typename T, int D>
int run_fwd(const SeqArgs& a, const rse_seq_rows* q, const rse_seq_rows* k, const rse_seq_rows* v,
            const rse_seq_rows* out, float* lse, hipStream_t s) {
    if (a.max_len <= 32) return run_fwd_w<T, D, 1>(a, q, k, v, out, lse, s);
    if (a.max_len <= 64) return run_fwd_w<T, D, 2>(a, q, k, v, out, lse, s);
    return run_fwd_w<T, D, 4>(a, q, k, v, out, lse, s);
}

template <typename T, int D>
int run_bwd(const rse_seqattn* at, const SeqArgs& a, const rse_seq_rows* q, const rse_seq_rows* k,
            const rse_seq_rows* v, const float* lse, const rse_seq_rows* dout, const rse_seq_rows* dq,
            const rse_seq_rows* dk, const rse_seq_rows* dv, float* dbias, const BwdWs& w, hipStream_t s) {
    const int nb = a.n_bounds + 1;
    const int blocks = fill_blocks(a.n_events, AW, DQ_BLOCKS);
    hipLaunchKernelGGL((k_attn_dq<T, D>), dim3(blocks, a.n_heads), dim3(AB), nb * AB * sizeof(float), s, a,
                       rows_view<const T>(q), rows_view<const T>(k), rows_view<const T>(v), lse,
                       rows_view<const T>(dout), rows_view<T>(dq), w.delta, w.part);
    int rc = launch_status();
    if (rc) return rc;
    hipLaunchKernelGGL(k_attn_dbias, dim3(a.n_heads), dim3(128), 0, s, w.part, blocks, nb, dbias);
    hipLaunchKernelGGL((k_attn_dkv<T, D>), dim3(fill_blocks(a.n_events * at->n_kv_heads, AW, 1 << 16)), dim3(AB), 0, s,
                       a, rows_view<const T>(q), rows_view<const T>(k), rows_view<const T>(v), lse, w.delta,
                       rows_view<const T>(dout), rows_view<T>(dk), rows_view<T>(dv));
    return launch_status();
}

// Calls F.template operator()<T, D>() for the handle's type and dim.
template <typename F>
int by_type(const rse_seqattn* a, F f) {
    if (a->dtype == RSE_F32) {
        if (a->dim == 32) return f(float(), std::integral_constant<int, 32>());
        if (a->dim == 64) return f(float(), std::integral_constant<int, 64>());
        return f(float(), std::integral_constant<int, 128>());
    }
    if (a->dim == 32) return f(uint16_t(), std::integral_constant<int, 32>());
    if (a->dim == 64) return f(uint16_t(), std::integral_constant<int, 64>());
    return f(uint16_t(), std::integral_constant<int, 128>());
}

}  // namespace

extern "C" {

int rse_seqattn_mem_size(size_t* bytes_out) {
    if (!bytes_out) return RSE_ERR_INVALID_ARG;
    *bytes_out = sizeof(SeqHeader);
    return RSE_OK;
}

int rse_seqattn_create(rse_seqattn** out, void* d_mem, size_t mem_bytes, int32_t n_heads, int32_t n_kv_heads,
                       int32_t dim, int32_t dtype, int32_t causal, float scale, const int32_t* boundaries,
                       int32_t n_boundaries, void* stream) {
    if (!out || !d_mem || reinterpret_cast<uintptr_t>(d_mem) % 256) return RSE_ERR_INVALID_ARG;
    if (mem_bytes < sizeof(SeqHeader)) return RSE_ERR_WORKSPACE;
    if (n_heads < 1 || n_heads > RSE_SEQ_MAX_HEADS || n_kv_heads < 1 || n_heads % n_kv_heads) return RSE_ERR_INVALID_ARG;
    if (dtype != RSE_F32 && dtype != RSE_BF16) return RSE_ERR_INVALID_ARG;
    if (dim != 32 && dim != 64 && dim != 128) return RSE_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return RSE_ERR_INVALID_ARG;
    if (n_boundaries < 0 || n_boundaries > RSE_SEQ_MAX_BOUNDARIES || (n_boundaries > 0 && !boundaries))
        return RSE_ERR_INVALID_ARG;
    InitArgs a;
    a.n_bounds = n_boundaries;
    for (int i = 0; i <= RSE_SEQ_MAX_BOUNDARIES; ++i) {
        a.bounds[i] = i < n_boundaries ? boundaries[i] : INT32_MAX;
        if (i < n_boundaries && (a.bounds[i] == INT32_MIN || (i > 0 && a.bounds[i] < a.bounds[i - 1])))
            return RSE_ERR_INVALID_ARG;
    }
    rse_seqattn* h = new (std::nothrow) rse_seqattn();
    if (!h) return RSE_ERR_INVALID_ARG;
    h->n_heads = n_heads;
    h->n_kv_heads = n_kv_heads;
    h->dim = dim;
    h->dtype = dtype;
    h->causal = causal != 0;
    h->n_bounds = n_boundaries;
    h->scale = scale;
    h->hdr = static_cast<SeqHeader*>(d_mem);
    hipLaunchKernelGGL(k_attn_init, dim3(1), dim3(128), 0, as_stream(stream), h->hdr, a);
    const int rc = launch_status();
    if (rc) {
        delete h;
        return rc;
    }
    *out = h;
    return RSE_OK;
}

int rse_seqattn_destroy(rse_seqattn* attn) {
    delete attn;
    return RSE_OK;
}

int rse_seqattn_status(rse_seqattn* attn, int32_t* status_out, void* stream) {
    if (!attn || !status_out) return RSE_ERR_INVALID_ARG;
    int32_t st = 0;
    if (hipMemcpyAsync(&st, &attn->hdr->status, sizeof(st), hipMemcpyDeviceToHost, as_stream(stream)) != hipSuccess)
        return RSE_ERR_HIP;
    if (hipStreamSynchronize(as_stream(stream)) != hipSuccess) return RSE_ERR_HIP;
    *status_out = st;
    return RSE_OK;
}

int rse_seqattn_clear_status(rse_seqattn* attn, void* stream) {
    if (!attn) return RSE_ERR_INVALID_ARG;
    hipLaunchKernelGGL(k_attn_clear, dim3(1), dim3(1), 0, as_stream(stream), attn->hdr);
    return launch_status();
}

int rse_seqattn_saved_size(const rse_seqattn* attn, int64_t n_events, int64_t max_len, size_t* bytes_out) {
    if (!attn || !bytes_out || n_events < 0 || max_len < 0) return RSE_ERR_INVALID_ARG;
    *bytes_out = saved_bytes_of(attn, n_events);
    return RSE_OK;
}

int seq_attention_fwd(const rse_seqattn* attn, const rse_seq_batch* batch, const rse_seq_rows* q,
                      const rse_seq_rows* k, const rse_seq_rows* v, const rse_seq_rows* out, void* d_saved,
                      size_t saved_bytes, void* stream) {
    int rc = batch_ok(attn, batch);
    if (rc) return rc;
    if (batch->n_events == 0) return RSE_OK;
    if (!rows_ok(q, attn->dtype) || !rows_ok(k, attn->dtype) || !rows_ok(v, attn->dtype) || !rows_ok(out, attn->dtype))
        return RSE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(d_saved) % 256) return RSE_ERR_INVALID_ARG;
    if (d_saved && saved_bytes < saved_bytes_of(attn, batch->n_events)) return RSE_ERR_WORKSPACE;
    const SeqArgs a = seq_args(attn, batch);
    return by_type(attn, [&](auto t, auto d) {
        return run_fwd<decltype(t), decltype(d)::value>(a, q, k, v, out, static_cast<float*>(d_saved),
                                                        as_stream(stream));
    });
}

int rse_seqattn_bwd_workspace_size(const rse_seqattn* attn, int64_t n_events, int64_t batch, int64_t max_len,
                                   size_t* bytes_out) {
    if (!attn || !bytes_out || n_events < 0 || batch < 0 || max_len < 0) return RSE_ERR_INVALID_ARG;
    *bytes_out = bwd_ws(attn, n_events, nullptr).bytes;
    return RSE_OK;
}

int seq_attention_bwd(const rse_seqattn* attn, const rse_seq_batch* batch, const rse_seq_rows* q,
                      const rse_seq_rows* k, const rse_seq_rows* v, const void* d_saved, size_t saved_bytes,
                      const rse_seq_rows* dout, const rse_seq_rows* dq, const rse_seq_rows* dk,
                      const rse_seq_rows* dv, float* d_dbias, void* d_ws, size_t ws_bytes, void* stream) {
    int rc = batch_ok(attn, batch);
    if (rc) return rc;
    if (!d_dbias || !d_ws || reinterpret_cast<uintptr_t>(d_ws) % 256) return RSE_ERR_INVALID_ARG;
    const BwdWs w = bwd_ws(attn, batch->n_events, d_ws);
    if (ws_bytes < w.bytes) return RSE_ERR_WORKSPACE;
    hipStream_t s = as_stream(stream);
    if (batch->n_events == 0) {
        hipLaunchKernelGGL(k_attn_dbias, dim3(attn->n_heads), dim3(128), 0, s, w.part, 0, attn->n_bounds + 1, d_dbias);
        return launch_status();
    }
    for (const rse_seq_rows* r : {q, k, v, dout, dq, dk, dv})
        if (!rows_ok(r, attn->dtype)) return RSE_ERR_INVALID_ARG;
    if (!d_saved || reinterpret_cast<uintptr_t>(d_saved) % 256) return RSE_ERR_INVALID_ARG;
    if (saved_bytes < saved_bytes_of(attn, batch->n_events)) return RSE_ERR_WORKSPACE;
    const SeqArgs a = seq_args(attn, batch);
    return by_type(attn, [&](auto t, auto d) {
        return run_bwd<decltype(t), decltype(d)::value>(attn, a, q, k, v, static_cast<const float*>(d_saved), dout, dq,
                                                        dk, dv, d_dbias, w, s);
    });
}

}  // extern "C"
