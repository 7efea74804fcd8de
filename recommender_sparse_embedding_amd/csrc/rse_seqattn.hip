// rse_seqattn.hip -- attention over the events of each behaviour sequence of
// a jagged batch, with a learned bias by buckets of the events' distance:
// handles and the forward.
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

// Forward.  A wave has 32 queries of one sequence and head as columns.  Keys
// go by in tiles staged in LDS row-major (the next tile's loads are in flight
// meanwhile), 32 at a time: S^T = K Q^T, online softmax down the registers of
// a lane (a row's maximum needs one exchange between the wave's halves, its
// sum none until the end), and O^T += V^T P^T with the same registers as
// operand.
//
// The logits are formed relative to a reference m of the row, in base 2:
// y = s c + (bias - m), p = exp2(y).  m follows the row's maximum only when
// that has grown by more than 8 (p up to 2^8, exact in a float), so most
// tiles need neither a second pass over y nor a rescaling of the sums.
//
// bf16: the probabilities enter V^T P^T as pairs of bf16 values (2^-16 of each
// is lost), so that out is fp32 arithmetic rounded once.  With one value each
// their rounding put as much into out again as its own: 0.0022 of its size
// against 0.0016, for 188 instead of 218 us on 16 histories of up to 4096
// events and 37 instead of 38 on 96 sessions of up to 333 (dim 128).
//
// SAVE: also leaves the log-sums for the backward, and SAVE_OUT the outputs:
// its dO . out has to equal sum_j p dp to fp32 accuracy (the bias gradient
// sums differences from it), so what the pairs leave of the probabilities goes
// through one more product into those outputs (three bf16 terms hold a float:
// the bias gradient is then as near to 64 bits as plain fp32 is, 3e-7 on 12
// sequences of up to 2048 events, 8 heads).
enum { SAVE_NONE = 0, SAVE = 1, SAVE_OUT = 2 };
//
// Short sequences: a block goes on through its sequences' tiles of queries,
// and the next tile's first loads are in flight during the last step of the
// current one.  (8192 sequences of 1..100 events, 4 heads of 64: 454 us with a
// block per tile, most of it waiting for the first loads of each.)
//
// Registers are held to what lets FWD_WAVES waves share a SIMD.
template <typename T, int D, int S>
constexpr int FWD_WAVES = D * sizeof(T) <= 64 ? 3 : (D * sizeof(T) == 128 || (D * sizeof(T) == 256 && !(S == SAVE_OUT && D == 128)) ? 2 : 1);

template <typename T, int D, typename SH, int S>
__global__ __launch_bounds__(SH::WAVES * 64) __attribute__((amdgpu_waves_per_eu(FWD_WAVES<T, D, S>))) void k_attn_fwd(
    SeqArgs a, TileGrid grid, Rows<const T> q, Rows<const T> k, Rows<const T> v, Rows<T> out, float* lse2, float* out32, int split) {
    constexpr int CH = SH::CH, KT = SH::KT, NS = SH::NS, NB = SH::NB, NT = SH::NT, WH = SH::WH, WQ = SH::WQ, ND = D / 32;
    constexpr bool REST = S == SAVE_OUT && sizeof(T) == 2, BRIEF = SH::TEAM == 1;
    __shared__ u32x4 s_k[SH::TEAMS][NB][KT * CH], s_v[SH::TEAMS][NB][KT * CH];
    __shared__ u32x4 s_pairs[BRIEF ? 2 : WQ][NS][WAVE];      // (BRIEF: this tile's and the last one's)
    __shared__ KeySide<KT> s_side[SH::TEAMS][NB];
    __shared__ LdsBuckets s_buckets;
    __shared__ float s_bias[WH][RSE_SEQ_MAX_BOUNDARIES + 1];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE), half = lane >> 5, wh = w % WH, wq = w / WH;
    const int team = w / SH::TEAM, t = threadIdx.x % NT;
    const int hblocks = (a.n_heads + WH - 1) / WH, h0 = blockIdx.x % hblocks * WH, nb = a.n_bounds + 1;
    const bool live = h0 + wh < a.n_heads;
    const int head = live ? h0 + wh : a.n_heads - 1, g = head / a.group;
    SeqTiles at;
    const bool on = BRIEF && split > 0;         // the block goes on through its sequences' tiles
    if (on) {
        at.begin(a, blockIdx.x / hblocks, gridDim.x / hblocks, split, h0 == 0);
        if (!at.valid) return;
    } else if (!find_tile(a, grid, blockIdx.x / hblocks, 32 * WQ, a.causal, at.s, at.len, at.tile, h0 == 0)) {
        return;
    }

    RowStage<T, D, NT, KT> st;
    KeySideStage side;
    ColFrag<T, D> qn;
    int32_t pn;
    // keys of a block's tile end here
    auto end_of = [&](const SeqTiles& x) {
        const int past = (x.tile + 1) * 32 * WQ;
        return a.causal && past < x.len ? past : x.len;
    };
    auto load_first = [&](const SeqTiles& x) {
        st.load(k, g, v, g, x.s, 0, end_of(x), a.key_off, t);
        side.load(a, x.s, 0, end_of(x), KT, t);
        const int i = x.tile * 32 * WQ + 32 * wq + (lane & 31);
        const int64_t row = x.s + (i < x.len ? i : x.len - 1);
        qn.load(q.at(row, head), half);
        pn = a.pos[row];
    };
    load_first(at);
    WaveBuckets wb;
    wb.load(a.hdr, a.bias + head * nb, a.n_bounds);
    s_buckets.load(a.hdr);
    if (wq == 0) {
        s_bias[wh][lane] = wb.bias[0];
        s_bias[wh][64 + lane] = wb.bias[1];
    }
    const float c2 = fabsf(a.scale) * LOG2E;
    int wp = wq;
    __syncthreads();
    for (;;) {
        const int64_t s = at.s;
        const int len = at.len, w0 = at.tile * 32 * WQ + 32 * wq, my_q = w0 + (lane & 31), end = end_of(at);
        const int my_end = w0 >= len ? 0 : (a.causal && w0 + 32 < end ? w0 + 32 : end);     // keys of the wave
        ColFrag<T, D> qf = qn;
        if (a.scale < 0.f) qf.negate();
        const int32_t my_pos = pn, q_lo = half_min(my_pos), q_hi = half_max(my_pos);
        f32x16 o[ND] = {}, rest[REST ? ND : 1] = {};
        float m = 0.f, l = 0.f;
        bool set = false;                       // m has been taken from a visible key
        for (int k0 = 0, b = 0; k0 < end; k0 += KT, b ^= NB - 1) {
            st.store(s_k[team][b], s_v[team][b], t);
            side.store(s_side[team][b], t);
            team_sync<SH::TEAM>();
            if (k0 + KT < end) {
                st.load(k, g, v, g, s, k0 + KT, end, a.key_off, t);
                side.load(a, s, k0 + KT, end, KT, t);
            } else if (on) {
                at.advance(a);
                if (at.valid) load_first(at);
            }
            const KeySide<KT>& ks = s_side[team][b];
#pragma unroll 1
            for (int u = 0; u < NS; ++u) {
                const int k1 = k0 + 32 * u;
                if (k1 >= my_end) break;
                TileBuckets<true> tb;
                tb.set(wb, q_lo, q_hi, ks.range[u]);
                f32x16 x = mma_rows<T, D>(s_k[team][b], 32 * u, qf, f32x16{});
                if (tb.many) {
                    // all waves of a column tile are here, and share the lookups
                    if (BRIEF) wp ^= 1;
                    tb.find_pairs(s_pairs[wp][u], wh, WH, s_buckets, a.n_bounds, a.cells, ks.pos + 32 * u, my_pos);
                    if (WH > 1) __syncthreads();
                    else wave_lds_sync();
                }
                x = tb.logits(x, c2, -m, wb, s_pairs[wp][u], s_bias[wh], ks.pos + 32 * u, my_pos);
                hide(x, ks.hidden[u], ks.mask + 32 * u);
                if (a.causal && k1 + 31 > w0) {
                    const int lim = my_q - k1 - 4 * half;
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[r] = tile_row(r, 0) <= lim ? x[r] : -INFINITY;
                }
                float top = x[0];
#pragma unroll
                for (int r = 1; r < 16; ++r) top = fmaxf(top, x[r]);
                top = fmaxf(top, other_half(top));
                const bool move = top > 8.f || (!set && top > -INFINITY);
                set |= top > -INFINITY;
                if (__any(move)) {
                    const float by = move ? top : 0.f, r = __builtin_amdgcn_exp2f(-by);
                    m += by;
                    // nothing summed yet: 0, also where exp2 overflows
                    l = l == 0.f ? 0.f : l * r;
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] -= by;
                    const float ro = r < INFINITY ? r : 0.f;
#pragma unroll
                    for (int dt = 0; dt < ND; ++dt) {
                        o[dt] *= ro;
                        if (REST) rest[dt] *= ro;
                    }
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) x[r] = __builtin_amdgcn_exp2f(x[r]);
                l += sum_registers(x);
                OverRows<T, D>::add(o, s_v[team][b], 32 * u, x);
                if constexpr (REST) OverRows<T, D, 1>::add(rest, s_v[team][b], 32 * u, x);
            }
            if (BRIEF) wave_lds_sync();         // read before the next tile is stored
        }
        l += other_half(l);
        // a score of NaN or +infinity has left l NaN, and o: both stay
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (my_q < len && live) {
            T* dst = out.at(s + my_q, head);
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) store_column(dst + 32 * dt, o[dt], inv);
            if (S != SAVE_NONE && half == 0)
                lse2[(int64_t)head * a.n_events + s + my_q] = l == 0.f ? -INFINITY : m + log2f(l);
            if (S == SAVE_OUT)
#pragma unroll
                for (int dt = 0; dt < ND; ++dt) {
                    if (REST) o[dt] += rest[dt];
                    store_column(out32 + ((s + my_q) * a.n_heads + head) * D + 32 * dt, o[dt], inv);
                }
        }
        if (!on || !at.valid) return;
    }
}

// ------------------------------------------------------------------ host --
// KEEP: what a forward before a backward leaves; SAVE is the short form.
template <typename T, int D, int TEAM, int WH, int WQ, int KEEP>
int run_fwd(const SeqArgs& a, const rse_seq_rows* q, const rse_seq_rows* k, const rse_seq_rows* v,
            const rse_seq_rows* out, const Saved& sv, hipStream_t s) {
    using SH = Shape<T, D, TEAM, WH, WQ>;
    const TileGrid tg = tile_grid(a.n_events, a.batch, a.max_len, 32 * WQ);
    const int64_t hblocks = (a.n_heads + WH - 1) / WH;
    ShortGrid sg = {0, 0};
    if (KEEP == SAVE) sg = short_grid(a.batch, hblocks, a.max_len, SH::WAVES);
    const int64_t blocks = hblocks * (KEEP == SAVE ? sg.blocks : tg.items);
    if (blocks > INT32_MAX) return RSE_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks), block(SH::WAVES * WAVE);
    if (sv.lse2)
        hipLaunchKernelGGL((k_attn_fwd<T, D, SH, KEEP>), grid, block, 0, s, a, tg, rows_view<const T>(q),
                           rows_view<const T>(k), rows_view<const T>(v), rows_view<T>(out), sv.lse2, sv.out32, sg.split);
    else
        hipLaunchKernelGGL((k_attn_fwd<T, D, SH, SAVE_NONE>), grid, block, 0, s, a, tg, rows_view<const T>(q),
                           rows_view<const T>(k), rows_view<const T>(v), rows_view<T>(out), nullptr, nullptr, sg.split);
    return launch_status();
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
    *bytes_out = saved_view(attn, n_events, max_len, nullptr).bytes;
    return RSE_OK;
}

int seq_attention_fwd(const rse_seqattn* attn, const rse_seq_batch* batch, const rse_seq_rows* q,
                      const rse_seq_rows* k, const rse_seq_rows* v, const rse_seq_rows* out, void* d_saved,
                      size_t saved_bytes, void* stream) {
    int rc = batch_ok(attn, batch);
    if (rc) return rc;
    if (batch->n_events == 0) return RSE_OK;
    if (!rows_ok(q, attn->dtype) || !rows_ok(k, attn->dtype) || !rows_ok(v, attn->dtype) ||
        !out_rows_ok(out, attn->dtype, batch->n_events, attn->n_heads, attn->dim))
        return RSE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(d_saved) % 256) return RSE_ERR_INVALID_ARG;
    Saved sv = saved_view(attn, batch->n_events, batch->max_len, d_saved);
    if (d_saved && saved_bytes < sv.bytes) return RSE_ERR_WORKSPACE;
    if (!d_saved) sv.lse2 = sv.out32 = nullptr;
    const SeqArgs a = seq_args(attn, batch);
    return by_type(attn, [&](auto t, auto d) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        const hipStream_t st = as_stream(stream);
        if constexpr (HAS_SHORT<T, D>)
            if (short_form(attn, batch->max_len)) {
                if (a.n_heads > 1) return run_fwd<T, D, 1, 4, 1, SAVE>(a, q, k, v, out, sv, st);
                return run_fwd<T, D, 1, 1, 1, SAVE>(a, q, k, v, out, sv, st);
            }
        if (a.group % 4 == 0) return run_fwd<T, D, 4, 4, 1, SAVE_OUT>(a, q, k, v, out, sv, st);
        if constexpr (LONG_APART<T, D>)
            if (a.n_heads > 2) return run_fwd<T, D, 1, 4, 1, SAVE_OUT>(a, q, k, v, out, sv, st);
        return run_fwd<T, D, LONG_WAVES<T, D>, 1, LONG_WAVES<T, D>, SAVE_OUT>(a, q, k, v, out, sv, st);
    });
}

}  // extern "C"
