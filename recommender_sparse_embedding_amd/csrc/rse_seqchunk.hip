// rse_seqchunk.hip -- attention of several new events of every user over the
// user's paged history and each other; their keys, values and times are stored
// in the same launch.
//
// Columns of a tile are pairs (new event, query head) of one key/value head, so
// that heads that share keys and a few events fill the 32 columns of the matrix
// products; rows are the keys.  Formulas and softmax are those of the forward
// (rse_seqattn.hip): S^T = K Q^T, online softmax down a lane's registers
// relative to a reference that follows the maximum when it has grown by 2^8,
// O^T += V^T P^T with the probabilities as pairs of bf16 values.
//
// A key is read from its page if it was cached before the call and from the
// call's arguments if it is new: no block waits for another's stores.
#include "rse_seqmma.h"

using namespace rse;
using namespace rse_host;

namespace {

constexpr int CW = 4;                   // waves of a block

// What the kernels know of the cache.
struct PageArgs {
    SeqCacheHeader* status;
    const int32_t* table;
    const int64_t* lens;
    int32_t* tp;
    int64_t max_pages, n_pages, max_len;
    int32_t shift;
};

// How the columns are laid out: a tile takes `events` new events of one user
// and `cols` query heads of one key/value head (events * cols <= 32); a key/value
// head has `blocks` such groups of query heads.
struct Columns {
    int cols, blocks, events;
};

// The slot of event e of user b, or -1 (status set) for a page out of the pool.
__device__ __forceinline__ int64_t slot_of(const PageArgs& p, int64_t page, int64_t e) {
    if (page < 0 || page >= p.n_pages) {
        set_status(&p.status->status, RSE_ERR_BAD_INPUT);
        return -1;
    }
    return (page << p.shift) + (e & ((1ll << p.shift) - 1));
}

// Events that user b has cached before its `count` new ones; -1: idle, or they
// do not fit (status set).
__device__ __forceinline__ int64_t cached_of(const PageArgs& p, int64_t b, int count) {
    const int64_t n = uniform(p.lens[b]);
    if (n < 0) return -1;
    if (n > p.max_len - count || (n + count - 1) >> p.shift >= p.max_pages) {
        set_status(&p.status->status, RSE_ERR_BAD_INPUT);
        return -1;
    }
    return n;
}

// A block's part of the work.
struct Work {
    int64_t b, s;                       // user, its first new event
    int count, tile;                    // new events, tile of them
    int split, g, h0, nc;               // part of the keys; key/value head, first query head, query heads
};
__device__ __forceinline__ bool find_work(const SeqArgs& a, const TileGrid& grid, const Columns& cl, int splits, int tq, int64_t x,
                                          Work& w) {
    w.split = (int)(x % splits);
    x /= splits;
    const int n_kv = a.n_heads / a.group, units = n_kv * cl.blocks, u = (int)(x % units);
    x /= units;
    w.g = u / cl.blocks;
    const int cb = u % cl.blocks;
    w.h0 = w.g * a.group + cb * cl.cols;
    w.nc = a.group - cb * cl.cols < cl.cols ? a.group - cb * cl.cols : cl.cols;
    return find_tile(a, grid, x, tq, false, w.b, w.s, w.count, w.tile, u == 0 && w.split == 0);
}

// The tile's new events into their pages, by the threads of the blocks that
// share them out by key/value head.
template <typename T, int D>
__device__ __forceinline__ void store_events(const SeqArgs& a, const PageArgs& p, const Work& w, int64_t had, int first, int last,
                                             const Rows<const T>& k, const Rows<const T>& v, T* kp, T* vp) {
    using TL = Tile<T, D>;
    const int64_t row_elems = (int64_t)(a.n_heads / a.group) * D;
    for (int t = threadIdx.x; t < (last - first) * TL::CH; t += CW * WAVE) {
        const int i = first + t / TL::CH, c = t % TL::CH;
        const int64_t e = had + i, slot = slot_of(p, p.table[w.b * p.max_pages + (e >> p.shift)], e);
        if (slot < 0) continue;
        const int64_t at = slot * row_elems + w.g * D + c * TL::EPC;
        gstore_u4(kp + at, gload_u4(k.at(w.s + i, w.g) + c * TL::EPC));
        gstore_u4(vp + at, gload_u4(v.at(w.s + i, w.g) + c * TL::EPC));
        if (w.g == 0 && c == 0) p.tp[slot] = a.pos[w.s + i];
    }
}

// The softmax of a lane's column over the tiles of keys that went by, and the
// sums of the values.
template <typename T, int D>
struct Online {
    f32x16 o[D / 32];
    float m, l;
    bool set;                           // m has been taken from a visible key
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt) o[dt] = f32x16{};
        m = l = 0.f;
        set = false;
    }
    // x: logits less m, -infinity where not visible
    __device__ __forceinline__ void add(f32x16& x, const u32x4* values, int r0) {
        float top = x[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) top = fmaxf(top, x[r]);
        top = fmaxf(top, other_half(top));
        const bool move = top > 8.f || (!set && top > -INFINITY);
        set |= top > -INFINITY;
        if (__any(move)) {
            const float by = move ? top : 0.f, r = __builtin_amdgcn_exp2f(-by);
            m += by;
            l = l == 0.f ? 0.f : l * r;         // nothing summed yet: 0, also where exp2 overflows
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] -= by;
            const float ro = r < INFINITY ? r : 0.f;
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) o[dt] *= ro;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = __builtin_amdgcn_exp2f(x[r]);
        l += sum_registers(x);
        OverRows<T, D>::add(o, values, r0, x);
    }
    // the reference as a part leaves it: what saw nothing weighs nothing
    __device__ __forceinline__ float reference() const { return l == 0.f ? -INFINITY : m; }
};

// Parts are joined relative to the largest reference M; a NaN stays.
__device__ __forceinline__ float part_weight(float m, float M) { return m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - M); }

// -infinity for keys after the lane's event (lim: the last of the tile's rows
// that it may see, less 4 half).
__device__ __forceinline__ void hide_after(f32x16& x, int lim) {
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r] = tile_row(r, 0) <= lim ? x[r] : -INFINITY;
}

// The table of biases of a block's heads, in base 2, a row a head.
__device__ __forceinline__ int bias_stride(int n_bounds) { return (n_bounds + 1) | 1; }
__device__ __forceinline__ void load_bias(float* s_bias, const SeqArgs& a, const Work& w) {
    const int nb = a.n_bounds + 1, st = bias_stride(a.n_bounds);
    for (int t = threadIdx.x; t < w.nc * nb; t += CW * WAVE) s_bias[t / nb * st + t % nb] = bias2(a.bias[(w.h0 + t / nb) * nb + t % nb]);
}

// What a column works on.
template <typename T, int D>
struct Column {
    ColFrag<T, D> q;
    int32_t pos, lo, hi;                // and the lowest and highest of the tile's columns
    int event, head;                    // of the user's new ones; of all heads
    bool live;
    __device__ __forceinline__ void load(const SeqArgs& a, const Columns& cl, const Work& w, int first, const Rows<const T>& rows) {
        const int c = lane_id() & 31;
        int i = first + c / w.nc, hh = c % w.nc;
        live = c < cl.events * w.nc && i < w.count;
        if (!live) {                            // a double of the first one
            i = first < w.count ? first : w.count - 1;
            hh = 0;
        }
        event = i;
        head = w.h0 + hh;
        q.load(rows.at(w.s + i, head), lane_id() >> 5);
        if (a.scale < 0.f) q.negate();
        pos = a.pos[w.s + i];
        lo = half_min(pos);
        hi = half_max(pos);
    }
};

// Few columns: all waves of a block have the same tile of columns and take
// tiles of 32 keys in turn, each from memory to its own registers and LDS, so
// that no wave waits for another; they are joined in LDS at the end.
template <typename T, int D>
constexpr int FEW_WAVES = D * sizeof(T) <= 128 ? 2 : 1;

template <typename T, int D>
__global__ __launch_bounds__(CW * 64) __attribute__((amdgpu_waves_per_eu(FEW_WAVES<T, D>))) void k_chunk_few(
    SeqArgs a, PageArgs p, TileGrid grid, Columns cl, Rows<const T> q, Rows<const T> k, Rows<const T> v, T* kp, T* vp, Rows<T> out,
    int splits, float* part_o, float* part_ml) {
    using TL = Tile<T, D>;
    constexpr int CH = TL::CH, ND = D / 32, NC = CH / 2;
    extern __shared__ float s_bias[];           // [cols][bias_stride]
    __shared__ u32x4 s_mem[CW * 32 * CH > CW * 32 * D / 4 ? CW * 32 * CH : CW * 32 * D / 4];    // tiles of V, then the waves' sums
    __shared__ LdsBuckets s_buckets;
    __shared__ u32x4 s_pairs[CW][WAVE];
    alignas(16) __shared__ int32_t s_pos[CW][32];       // (read by 16 bytes)
    __shared__ float s_ml[CW][2][32];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE), half = lane >> 5, col = lane & 31;
    Work wk;
    if (!find_work(a, grid, cl, splits, cl.events, blockIdx.x, wk)) return;
    u32x4* tile = s_mem + w * 32 * CH;
    const int first = wk.tile * cl.events, last = first + cl.events < wk.count ? first + cl.events : wk.count;
    const int64_t had = cached_of(p, wk.b, wk.count);
    load_bias(s_bias, a, wk);
    s_buckets.load(a.hdr);
    if (had >= 0 && wk.split == 0 && wk.h0 == wk.g * a.group) store_events<T, D>(a, p, wk, had, first, last, k, v, kp, vp);
    Column<T, D> c;
    c.load(a, cl, wk, first, q);
    LaneBuckets lb;
    lb.load(a.hdr, s_bias + (c.head - wk.h0) * bias_stride(a.n_bounds), a.n_bounds);
    __syncthreads();

    // keys that some column may see: 0 .. end - 1; the wave's tiles t0 + w, + CW, ...
    const int64_t end = had < 0 ? 0 : had + (a.causal ? last : wk.count);
    const int64_t nt = (end + 31) / 32, t0 = nt * wk.split / splits, t1 = nt * (wk.split + 1) / splits;
    const int64_t row_elems = (int64_t)(a.n_heads / a.group) * D;
    const float c2 = fabsf(a.scale) * LOG2E;
    auto page_of = [&](int64_t t) -> int64_t {
        const int64_t e = t * 32 + col;
        return t < t1 && e < had ? (int64_t)p.table[wk.b * p.max_pages + (e >> p.shift)] : 0;
    };
    u32x4 rk[NC], rv[NC];
    int32_t rp = 0;
    bool see = false;
    auto load_rows = [&](int64_t t, int64_t page) {
        const int64_t e = t * 32 + col;
        // a new event's rows, also (the last one's) for lanes past the end
        const int64_t i = wk.s + (e < had ? 0 : (e - had < wk.count ? e - had : wk.count - 1));
        const T *kr = k.at(i, wk.g), *vr = v.at(i, wk.g);
        const int32_t* at = a.pos + i;
        see = e < end;
        if (e < had) {
            const int64_t s = slot_of(p, page, e);
            see = s >= 0;
            if (see) {
                kr = kp + s * row_elems + wk.g * D;
                vr = vp + s * row_elems + wk.g * D;
                at = p.tp + s;
            }
        }
        rp = *at;
#pragma unroll
        for (int i2 = 0; i2 < NC; ++i2) {
            rk[i2] = gload_u4(kr + (2 * i2 + half) * TL::EPC);
            rv[i2] = gload_u4(vr + (2 * i2 + half) * TL::EPC);
        }
    };
    Online<T, D> sm;
    sm.clear();
    int64_t t = t0 + w;
    int64_t page = page_of(t);
    if (t < t1) load_rows(t, page);
    page = page_of(t + CW);
    for (; t < t1; t += CW) {
        f32x16 x = {};
#pragma unroll
        for (int i = 0; i < NC; ++i) x = mma_chunk<T>(rk[i], c.q.v[i], x);
#pragma unroll
        for (int i = 0; i < NC; ++i) tile[TL::chunk_at(col, 2 * i + half)] = see ? rv[i] : u32x4{0, 0, 0, 0};
        const uint32_t seen = (uint32_t)__ballot(see);
        s_pos[w][col] = rp;
        const int32_t range[2] = {half_min(rp), half_max(rp)};
        wave_lds_sync();
        if (t + CW < t1) load_rows(t + CW, page);
        page = page_of(t + 2 * CW);
        TileBuckets<true> tb;
        tb.set(lb, c.lo, c.hi, range);
        if (tb.many) {
            tb.find_pairs(s_pairs[w], 0, 1, s_buckets, a.n_bounds, a.cells, s_pos[w], c.pos);
            wave_lds_sync();
        }
        x = tb.logits(x, c2, -sm.m, lb, s_pairs[w], lb.bias, s_pos[w], c.pos);
        if (seen != ~0u) {
            const uint32_t bits = seen >> (4 * half);
#pragma unroll
            for (int r = 0; r < 16; ++r) x[r] = (bits >> tile_row(r, 0)) & 1 ? x[r] : -INFINITY;
        }
        if (a.causal && t * 32 + 31 > had + first) hide_after(x, (int)(had - t * 32) + c.event - 4 * half);
        sm.add(x, tile, 0);
        wave_lds_sync();                        // read before the next tile is stored
    }
    sm.l += other_half(sm.l);
    if (half == 0) {
        s_ml[w][0][col] = sm.reference();
        s_ml[w][1][col] = sm.l;
    }
    __syncthreads();                            // the V tiles are done with: their place takes the sums
    float* s_sum = reinterpret_cast<float*>(s_mem);
#pragma unroll
    for (int dt = 0; dt < ND; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<f32x4*>(s_sum + (w * 32 + col) * D + 32 * dt + 8 * j + 4 * half) =
                f32x4{sm.o[dt][4 * j], sm.o[dt][4 * j + 1], sm.o[dt][4 * j + 2], sm.o[dt][4 * j + 3]};
    __syncthreads();
    for (int y = threadIdx.x; y < (last - first) * wk.nc * D; y += CW * WAVE) {
        const int cc = y / D, d = y % D;
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int u = 0; u < CW; ++u) M = fmaxf(M, s_ml[u][0][cc]);
        for (int u = 0; u < CW; ++u) {
            const float r = part_weight(s_ml[u][0][cc], M);
            L = __builtin_fmaf(s_ml[u][1][cc], r, L);
            O = __builtin_fmaf(s_sum[(u * 32 + cc) * D + d], r, O);
        }
        const int64_t ev = wk.s + first + cc / wk.nc;
        const int head = wk.h0 + cc % wk.nc;
        if (splits == 1) {
            from_f32(out.at(ev, head)[d], L == 0.f ? 0.f : O / L);
        } else {
            const int64_t at = (ev * a.n_heads + head) * splits + wk.split;
            part_o[at * D + d] = O;
            if (d == 0) {
                part_ml[2 * at] = M;
                part_ml[2 * at + 1] = L;
            }
        }
    }
}

// Many columns: every wave has a tile of columns of its own, and the block
// stages tiles of KT keys for them in LDS, the next one's loads in flight
// meanwhile; slots are looked up two tiles ahead.
template <typename T, int D>
struct Many {
    static constexpr int RB = D * (int)sizeof(T), KT = RB <= 256 ? 64 : 32, NS = KT / 32;
    static constexpr int CH = Tile<T, D>::CH, NT = CW * WAVE, PER = KT * CH / NT, STEP = NT / CH;
    static constexpr int WAVES = RB <= 256 ? 2 : 1;         // that share a SIMD
};

template <typename T, int D>
__global__ __launch_bounds__(CW * 64) __attribute__((amdgpu_waves_per_eu(Many<T, D>::WAVES))) void k_chunk_many(
    SeqArgs a, PageArgs p, TileGrid grid, Columns cl, Rows<const T> q, Rows<const T> k, Rows<const T> v, T* kp, T* vp, Rows<T> out,
    int splits, float* part_o, float* part_ml) {
    using TL = Tile<T, D>;
    using MY = Many<T, D>;
    constexpr int CH = MY::CH, KT = MY::KT, NS = MY::NS, PER = MY::PER, STEP = MY::STEP, ND = D / 32;
    extern __shared__ float s_bias[];           // [cols][bias_stride]
    __shared__ u32x4 s_k[2][KT * CH], s_v[2][KT * CH];
    __shared__ KeySide<KT> s_side[2];
    __shared__ int64_t s_slot[2][KT];           // of a tile's keys: slot, -1: hidden, -2 - i: new event i
    __shared__ LdsBuckets s_buckets;
    __shared__ u32x4 s_pairs[CW][WAVE];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE), half = lane >> 5, t = threadIdx.x;
    Work wk;
    if (!find_work(a, grid, cl, splits, CW * cl.events, blockIdx.x, wk)) return;
    const int begin = wk.tile * CW * cl.events, past = begin + CW * cl.events < wk.count ? begin + CW * cl.events : wk.count;
    const int64_t had = cached_of(p, wk.b, wk.count);
    load_bias(s_bias, a, wk);
    s_buckets.load(a.hdr);
    if (had >= 0 && wk.split == 0 && wk.h0 == wk.g * a.group) store_events<T, D>(a, p, wk, had, begin, past, k, v, kp, vp);
    const int first = begin + w * cl.events;
    Column<T, D> c;
    c.load(a, cl, wk, first, q);
    LaneBuckets lb;
    lb.load(a.hdr, s_bias + (c.head - wk.h0) * bias_stride(a.n_bounds), a.n_bounds);

    // the block's tiles of keys, and the end of those that the wave's columns see
    const int64_t end = had < 0 ? 0 : had + (a.causal ? past : wk.count);
    const int64_t nt = (end + KT - 1) / KT, t0 = nt * wk.split / splits, t1 = nt * (wk.split + 1) / splits;
    const int my_last = first + cl.events < wk.count ? first + cl.events : wk.count;
    const int64_t my_end = had < 0 || first >= wk.count ? 0 : had + (a.causal ? my_last : wk.count);
    const int64_t row_elems = (int64_t)(a.n_heads / a.group) * D;
    const float c2 = fabsf(a.scale) * LOG2E;

    // thread t < KT: key t of a tile, its page one step before its slot
    int64_t page = 0, slot = -1;
    int32_t key_pos = 0;
    auto page_of = [&](int64_t tile) {
        const int64_t e = tile * KT + t;
        page = t < KT && tile < t1 && e < had ? (int64_t)p.table[wk.b * p.max_pages + (e >> p.shift)] : 0;
    };
    auto find_slot = [&](int64_t tile) {        // and the load of its time
        if (t >= KT) return;
        const int64_t e = tile * KT + t;
        slot = -1;
        const int32_t* at = a.pos + wk.s;
        if (tile < t1 && e < end) {
            if (e < had) {
                slot = slot_of(p, page, e);
                if (slot >= 0) at = p.tp + slot;
            } else {
                slot = -2 - (e - had);
                at += e - had;
            }
        }
        key_pos = *at;
        s_slot[tile & 1][t] = slot;
    };
    u32x4 x[PER], y[PER];
    uint32_t hid = 0;                           // bit i: the thread's row i is hidden
    auto load_rows = [&](int64_t tile) {
        const int row = t / CH, ch = t % CH;
        hid = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t s = s_slot[tile & 1][row + i * STEP];
            if (s == -1) hid |= 1u << i;
            const int64_t ev = wk.s + (s <= -2 ? -2 - s : 0);
            const T* kr = s >= 0 ? kp + s * row_elems + wk.g * D : k.at(ev, wk.g);
            const T* vr = s >= 0 ? vp + s * row_elems + wk.g * D : v.at(ev, wk.g);
            x[i] = gload_u4(kr + ch * TL::EPC);
            y[i] = gload_u4(vr + ch * TL::EPC);
        }
    };
    auto store_rows = [&](int b) {
        const int row = t / CH, ch = t % CH;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = TL::chunk_at(row + i * STEP, ch);
            const bool z = (hid >> i) & 1;
            s_k[b][at] = z ? u32x4{0, 0, 0, 0} : x[i];
            s_v[b][at] = z ? u32x4{0, 0, 0, 0} : y[i];
        }
    };
    auto store_side = [&](KeySide<KT>& ks) {    // of the key whose slot was found last
        if (t >= WAVE) return;
        const bool see = slot != -1;
        const int32_t lo = half_min(key_pos), hi = half_max(key_pos);
        const uint64_t hm = __ballot(t < KT && !see);
        if (t < KT) {
            ks.mask[t] = see ? 0.f : -INFINITY;
            ks.pos[t] = key_pos;
            if ((t & 31) == 0) {
                ks.range[t / 32][0] = lo;
                ks.range[t / 32][1] = hi;
                ks.hidden[t / 32] = (uint32_t)(hm >> t);
            }
        }
    };
    Online<T, D> sm;
    sm.clear();
    if (t0 < t1) {
        page_of(t0);
        find_slot(t0);
        page_of(t0 + 1);
    }
    __syncthreads();
    if (t0 < t1) load_rows(t0);
    for (int64_t tile = t0; tile < t1; ++tile) {
        const int b = (int)(tile - t0) & 1;
        store_rows(b);
        store_side(s_side[b]);
        find_slot(tile + 1);
        __syncthreads();
        page_of(tile + 2);
        if (tile + 1 < t1) load_rows(tile + 1);
        const KeySide<KT>& ks = s_side[b];
#pragma unroll 1
        for (int u = 0; u < NS; ++u) {
            const int64_t k1 = tile * KT + 32 * u;
            if (k1 >= my_end) break;
            TileBuckets<true> tb;
            tb.set(lb, c.lo, c.hi, ks.range[u]);
            f32x16 z = mma_rows<T, D>(s_k[b], 32 * u, c.q, f32x16{});
            if (tb.many) {
                tb.find_pairs(s_pairs[w], 0, 1, s_buckets, a.n_bounds, a.cells, ks.pos + 32 * u, c.pos);
                wave_lds_sync();
            }
            z = tb.logits(z, c2, -sm.m, lb, s_pairs[w], lb.bias, ks.pos + 32 * u, c.pos);
            hide(z, ks.hidden[u], ks.mask + 32 * u);
            if (a.causal && k1 + 31 > had + first) hide_after(z, (int)(had - k1) + c.event - 4 * half);
            sm.add(z, s_v[b], 32 * u);
        }
    }
    sm.l += other_half(sm.l);
    if (!c.live) return;
    const int64_t ev = wk.s + c.event;
    if (splits == 1) {
        const float inv = sm.l == 0.f ? 0.f : 1.f / sm.l;
        T* dst = out.at(ev, c.head);
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) store_column(dst + 32 * dt, sm.o[dt], inv);
    } else {
        const int64_t at = (ev * a.n_heads + c.head) * splits + wk.split;
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) store_column(part_o + at * D + 32 * dt, sm.o[dt], 1.f);
        if (half == 0) {
            part_ml[2 * at] = sm.reference();
            part_ml[2 * at + 1] = sm.l;
        }
    }
}

// Joins the parts: a block for the columns of one tile, D / 4 threads a column.
constexpr int JT = 256;
template <typename T, int D>
__global__ __launch_bounds__(JT) void k_chunk_join(SeqArgs a, TileGrid grid, Columns cl, int tq, int splits, const float* part_o,
                                                   const float* part_ml, Rows<T> out) {
    constexpr int LR = D / 4;
    Work wk;
    if (!find_work(a, grid, cl, 1, tq, blockIdx.x, wk)) return;
    const int first = wk.tile * tq, last = first + tq < wk.count ? first + tq : wk.count;
    for (int c = threadIdx.x / LR; c < (last - first) * wk.nc; c += JT / LR) {
        const int64_t ev = wk.s + first + c / wk.nc;
        const int head = wk.h0 + c % wk.nc, d = 4 * (threadIdx.x % LR);
        const int64_t at = (ev * a.n_heads + head) * splits;
        float M = -INFINITY, L = 0.f;
        for (int s = 0; s < splits; ++s) M = fmaxf(M, part_ml[2 * (at + s)]);
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            const float r = part_weight(part_ml[2 * (at + s)], M);
            L = __builtin_fmaf(part_ml[2 * (at + s) + 1], r, L);
            const f32x4 x = gload_f4(part_o + (at + s) * D + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(x[i], r, o[i]);
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= inv;
        store_four(out.at(ev, head) + d, o);
    }
}

// ------------------------------------------------------------------ host --
// Blocks in all where histories are long enough, and the parts of one: of 256
// keys at least, at most 64.
constexpr int64_t CHUNK_BLOCKS = 1024;

struct ChunkPlan {
    Columns cl;
    bool few;
    int tq, splits;
    TileGrid grid;
    int64_t units;              // blocks of one part
};
ChunkPlan chunk_plan(const rse_seqattn* at, int64_t n_events, int64_t batch, int64_t max_new, int64_t max_len) {
    ChunkPlan p;
    const int group = at->n_heads / at->n_kv_heads;
    p.cl.cols = group < 32 ? group : 32;
    p.cl.blocks = (group + p.cl.cols - 1) / p.cl.cols;
    p.cl.events = 32 / p.cl.cols;
    p.few = max_new <= p.cl.events;
    p.tq = p.few ? p.cl.events : CW * p.cl.events;
    p.grid = tile_grid(n_events, batch, max_new, p.tq);
    p.units = p.grid.items * at->n_kv_heads * p.cl.blocks;
    int64_t s = p.units > 0 ? (CHUNK_BLOCKS + p.units - 1) / p.units : 1;
    const int64_t most = max_len / 256;
    if (s > most) s = most;
    p.splits = (int)(s < 1 ? 1 : (s > 64 ? 64 : s));
    return p;
}

struct ChunkWs {
    float* o;
    float* ml;
    size_t bytes;
};
ChunkWs chunk_ws(const rse_seqattn* at, int64_t n_events, const ChunkPlan& p, void* base) {
    Carver c(base);
    const size_t n = p.splits > 1 ? (size_t)n_events * at->n_heads * p.splits : 0;
    ChunkWs w;
    w.o = c.take<float>(n * at->dim);
    w.ml = c.take<float>(2 * n);
    w.bytes = c.size();
    return w;
}

template <typename T, int D>
int run_chunk(const rse_seqcache* c, const SeqArgs& a, const PageArgs& pg, const ChunkPlan& p, const ChunkWs& ws,
              const rse_seq_rows* q, const rse_seq_rows* k, const rse_seq_rows* v, const rse_seq_rows* out, hipStream_t s) {
    if (p.units * p.splits > INT32_MAX) return RSE_ERR_UNSUPPORTED;
    const size_t lds = (size_t)p.cl.cols * ((a.n_bounds + 1) | 1) * sizeof(float);
    const dim3 grid((unsigned)(p.units * p.splits)), block(CW * WAVE);
    const auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, lds, s, a, pg, p.grid, p.cl, rows_view<const T>(q), rows_view<const T>(k),
                           rows_view<const T>(v), static_cast<T*>(c->k), static_cast<T*>(c->v), rows_view<T>(out), p.splits, ws.o,
                           ws.ml);
    };
    if (p.few) run(k_chunk_few<T, D>);
    else run(k_chunk_many<T, D>);
    if (p.splits > 1)
        hipLaunchKernelGGL((k_chunk_join<T, D>), dim3((unsigned)p.units), dim3(JT), 0, s, a, p.grid, p.cl, p.tq, p.splits, ws.o,
                           ws.ml, rows_view<T>(out));
    return launch_status();
}

}  // namespace

extern "C" {

int rse_seqattn_chunk_workspace_size(const rse_seqattn* attn, int64_t n_events, int64_t batch, int64_t max_new, int64_t max_len,
                                     size_t* bytes_out) {
    if (!attn || !bytes_out || n_events < 0 || batch < 0 || max_new < 0 || max_len < 0) return RSE_ERR_INVALID_ARG;
    *bytes_out = n_events ? chunk_ws(attn, n_events, chunk_plan(attn, n_events, batch, max_new, max_len), nullptr).bytes : 0;
    return RSE_OK;
}

int seq_attention_chunk(const rse_seqattn* attn, rse_seqcache* cache, const rse_seq_batch* batch, const rse_seq_rows* q,
                        const rse_seq_rows* k, const rse_seq_rows* v, const int32_t* d_page_table, int32_t max_pages,
                        const int64_t* d_lens, int64_t max_len, const rse_seq_rows* out, void* d_ws, size_t ws_bytes,
                        void* stream) {
    int rc = batch_ok(attn, batch);
    if (rc) return rc;
    if (!cache || max_pages < 0 || max_len < 0 || batch->d_key_off) return RSE_ERR_INVALID_ARG;
    if (attn->dim != cache->dim || attn->dtype != cache->dtype || attn->n_kv_heads != cache->n_kv_heads)
        return RSE_ERR_INVALID_ARG;
    if (batch->n_events == 0) return RSE_OK;
    if (!d_lens || (max_pages > 0 && !d_page_table)) return RSE_ERR_INVALID_ARG;
    for (const rse_seq_rows* r : {q, k, v})
        if (!rows_ok(r, attn->dtype)) return RSE_ERR_INVALID_ARG;
    if (!out_rows_ok(out, attn->dtype, batch->n_events, attn->n_heads, attn->dim)) return RSE_ERR_INVALID_ARG;
    const ChunkPlan plan = chunk_plan(attn, batch->n_events, batch->batch, batch->max_len, max_len);
    const ChunkWs ws = chunk_ws(attn, batch->n_events, plan, d_ws);
    if (ws_bytes < ws.bytes) return RSE_ERR_WORKSPACE;
    if (ws.bytes && (!d_ws || reinterpret_cast<uintptr_t>(d_ws) % 256)) return RSE_ERR_INVALID_ARG;
    const SeqArgs a = seq_args(attn, batch);
    PageArgs p;
    p.status = cache->hdr;
    p.table = d_page_table;
    p.lens = d_lens;
    p.tp = cache->pos;
    p.max_pages = max_pages;
    p.n_pages = cache->n_pages;
    p.max_len = max_len;
    p.shift = cache->page_shift;
    return by_type(attn, [&](auto t, auto d) {
        return run_chunk<decltype(t), decltype(d)::value>(cache, a, p, plan, ws, q, k, v, out, as_stream(stream));
    });
}

}  // extern "C"
