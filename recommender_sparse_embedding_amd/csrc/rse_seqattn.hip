// rse_seqattn.hip -- attention over the events of each behaviour sequence of
// a jagged batch, with a learned bias by buckets of the events' distance:
// forward, and the backward that recomputes the probabilities.
#include <cmath>
#include <new>

#include "rse_seqmma.h"

using namespace rse;
using namespace rse_host;

namespace {

struct InitArgs {
    int32_t n_bounds;
    int32_t bounds[RSE_SEQ_MAX_BOUNDARIES + 1];
    uint8_t cell[512];
};

__global__ void k_attn_init(SeqHeader* h, InitArgs a) {
    if (threadIdx.x == 0) {
        h->status = 0;
        h->n_bounds = a.n_bounds;
    }
    if (threadIdx.x <= RSE_SEQ_MAX_BOUNDARIES) h->bounds[threadIdx.x] = a.bounds[threadIdx.x];
    for (int t = threadIdx.x; t < 512; t += blockDim.x) h->cell[t] = a.cell[t];
}

// Fills a.cell; true if no cell holds two boundaries past its first distance.
// A cell's distances are consecutive (the conversion to float is monotonic):
// its first is found by bisection.
bool fill_cells(InitArgs& a) {
    bool single = true;
    for (int sign = 0; sign < 2; ++sign)
        for (int c = 0; c < 256; ++c) {
            // smallest magnitude of code c or more, and of c + 1 or more
            int64_t at[2];
            for (int u = 0; u < 2; ++u) {
                int64_t lo = 0, hi = (1ll << 31) + 1;
                while (lo < hi) {
                    const int64_t mid = (lo + hi) / 2;
                    const int64_t d = sign ? -mid : (mid < INT32_MAX ? mid : INT32_MAX);
                    if (mid > (1ll << 31) || (seq_cell((int32_t)d) & 255) >= c + u) hi = mid;
                    else lo = mid + 1;
                }
                at[u] = lo;
            }
            const int64_t first = sign ? -(at[1] - 1) : at[0], last = sign ? -at[0] : at[1] - 1;
            int base = 0, inside = 0;
            for (int m = 0; m < a.n_bounds; ++m) {
                base += a.bounds[m] <= first;
                inside += a.bounds[m] > first && a.bounds[m] <= last;
            }
            a.cell[sign * 256 + c] = (uint8_t)base;
            if (inside > 1 && first <= last) single = false;
        }
    return single;
}

__global__ void k_attn_clear(SeqHeader* h) { h->status = 0; }

// Forward.  A block of W waves takes 32 W queries of one sequence and head; a
// wave has 32 of them as columns.  Keys go by in tiles of KT, staged in LDS
// row-major (the next tile's loads are in flight meanwhile): S^T = K Q^T,
// online softmax down the registers of a lane (a row's maximum needs one
// exchange between the wave's halves, its sum none until the end), and
// O^T += V^T P^T with the same registers as operand.
// SAVE: also leaves the log-sums and outputs for the backward, whose
// dO . out has to equal sum_j p dp to fp32 accuracy (the bias gradient sums
// differences from it): what bf16 rounds off the probabilities goes through
// a second product into those outputs.
template <typename T, int D, int W, int KT, bool SAVE>
__global__ __launch_bounds__(W * 64) void k_attn_fwd(SeqArgs a, Rows<const T> q, Rows<const T> k, Rows<const T> v,
                                                     Rows<T> out, float* lse2, float* out32) {
    using TL = Tile<T, D>;
    constexpr int NT = W * 64, CH = TL::CH, PER = KT * CH / NT, NS = KT / 32, ND = D / 32;
    static_assert(KT * CH % NT == 0 && KT <= 64, "tile shape");
    __shared__ u32x4 s_k[2][KT * CH], s_v[2][KT * CH];
    __shared__ float s_mask[2][KT];
    __shared__ int32_t s_pos[2][KT];
    __shared__ int32_t s_range[2][3];           // lowest and highest position, any key hidden
    __shared__ int32_t s_bounds[RSE_SEQ_MAX_BOUNDARIES + 1];
    __shared__ float s_bias[RSE_SEQ_MAX_BOUNDARIES + 1];
    __shared__ uint32_t s_cell[128];
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
        s_cell[t] = reinterpret_cast<const uint32_t*>(a.hdr->cell)[t];
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

    constexpr bool REST = SAVE && sizeof(T) == 2;
    f32x16 o[ND] = {}, rest[REST ? ND : 1] = {};
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
                    x[u] = add_bias<true>(x[u], c2, wb, lo, hi, s_pos[b] + 32 * u, my_pos, a.cells, s_cell,
                                          s_bounds, s_bias);
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
                if (REST)
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) rest[dt] *= r;
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
            if (REST)
#pragma unroll
                for (int u = 0; u < NS; ++u) {
                    RowOperand<T> lo;
                    lo.set_rest(x[u], p[u]);
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) rest[dt] = mma_over_rows<D>(s_v[b], 32 * u, dt, lo, rest[dt]);
                }
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
        if (SAVE) {
            if (half == 0) lse2[(int64_t)head * a.n_events + s + my_q] = l > 0.f ? m + log2f(l) : -INFINITY;
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) {
                if (REST) o[dt] += rest[dt];
                store_column(out32 + ((s + my_q) * a.n_heads + head) * D + 32 * dt, o[dt], inv);
            }
        }
    }
}

// ------------------------------------------------------------------ host --
template <typename T, int D, int W>
int run_fwd_w(const SeqArgs& a, const rse_seq_rows* q, const rse_seq_rows* k, const rse_seq_rows* v,
              const rse_seq_rows* out, const Saved& sv, hipStream_t s) {
    // keys of a tile: 64 where two buffers of them take at most 64 KiB and
    // there are several waves to stage them
    constexpr int KT = W > 1 && D * sizeof(T) <= 256 ? 64 : 32;
    const int64_t slots = tile_slots(a.n_events, a.batch, 32 * W);
    if (slots > INT32_MAX) return RSE_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)slots, a.n_heads), block(W * WAVE);
    if (sv.lse2)
        hipLaunchKernelGGL((k_attn_fwd<T, D, W, KT, true>), grid, block, 0, s, a, rows_view<const T>(q),
                           rows_view<const T>(k), rows_view<const T>(v), rows_view<T>(out), sv.lse2, sv.out32);
    else
        hipLaunchKernelGGL((k_attn_fwd<T, D, W, KT, false>), grid, block, 0, s, a, rows_view<const T>(q),
                           rows_view<const T>(k), rows_view<const T>(v), rows_view<T>(out), nullptr, nullptr);
    return launch_status();
}

// Waves of a block: as many groups of 32 queries as a sequence can have, up to 4.
template <typename T, int D>
int run_fwd(const SeqArgs& a, const rse_seq_rows* q, const rse_seq_rows* k, const rse_seq_rows* v,
            const rse_seq_rows* out, const Saved& sv, hipStream_t s) {
    if (a.max_len <= 128) return run_fwd_w<T, D, 1>(a, q, k, v, out, sv, s);
    return run_fwd_w<T, D, 4>(a, q, k, v, out, sv, s);
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
    h->cells = fill_cells(a);
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
    *bytes_out = saved_view(attn, n_events, nullptr).bytes;
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
    Saved sv = saved_view(attn, batch->n_events, d_saved);
    if (d_saved && saved_bytes < sv.bytes) return RSE_ERR_WORKSPACE;
    if (!d_saved) sv.lse2 = sv.out32 = nullptr;
    const SeqArgs a = seq_args(attn, batch);
    return by_type(attn, [&](auto t, auto d) {
        return run_fwd<decltype(t), decltype(d)::value>(a, q, k, v, out, sv, as_stream(stream));
    });
}

}  // extern "C"
