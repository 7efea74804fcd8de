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

// What a block works on: the keys of a part, if the keys are split, with a tile
// of columns.
struct Work {
    int64_t b, s;                       // user, its first new event
    int64_t had;                        // events cached; -1: they do not fit
    int count, tile;                    // new events, tile of them
    int g, h0, nc;                      // key/value head, first query head, query heads
    int split, parts, tiles;            // part of the keys, of how many; the user's tiles
    int per;                            // tiles of keys of a part
    int number;                         // of all parts' results; those of a tile stand `tiles` apart
    __device__ __forceinline__ void heads(const SeqArgs& a, const Columns& cl, uint32_t u) {
        g = (int)(u / (uint32_t)cl.blocks);
        const int cb = (int)(u % (uint32_t)cl.blocks);
        h0 = g * a.group + cb * cl.cols;
        nc = a.group - cb * cl.cols < cl.cols ? a.group - cb * cl.cols : cl.cols;
    }
};

// The keys split: k_chunk_plan leaves an entry for every block.
struct alignas(16) Item {
    int64_t s, had;
    int32_t b, count, tile, unit;       // b = -1: idle
    int32_t split, parts, tiles, per;
    int32_t number, pad[3];
};

// The blocks of a launch: groups of query heads of all key/value heads
// (fastest) by tiles of new events (TileGrid's items), or the entries of `list`.
struct Layout {
    uint32_t units, items, per_seq;
    const Item* list;
};

// What is wrong with a user's events and what they take: its new events'
// count, or 0, and the number cached, or -1 where they do not fit.
__device__ __forceinline__ int user_events(const SeqArgs& a, const PageArgs& p, int64_t s, int64_t e, int64_t& had, bool tell) {
    if (s < 0 || e < s || e > a.n_events || e - s > a.max_len) {
        if (tell) set_status(&a.hdr->status, RSE_ERR_BAD_INPUT);
        return 0;
    }
    const int count = (int)(e - s);
    if (had < 0) {
        had = -1;
    } else if (count > 0 && (had > p.max_len - count || (had + count - 1) >> p.shift >= p.max_pages)) {
        if (tell) set_status(&p.status->status, RSE_ERR_BAD_INPUT);
        had = -1;
    }
    return count;
}

// (The block numbers fit 32 bits, as 64-bit divisions took a third of a small
// call, and the lengths are loaded beside the offsets.)  False if the block has no tile.
__device__ __forceinline__ bool find_work(const SeqArgs& a, const PageArgs& p, const Columns& cl, const Layout& lo, int tq, Work& w) {
    if (lo.list) {
        const Item& i = lo.list[blockIdx.x];
        w.b = uniform(i.b);
        if (w.b < 0) return false;
        w.s = uniform(i.s);
        w.had = uniform(i.had);
        w.count = uniform(i.count);
        w.tile = uniform(i.tile);
        w.split = uniform(i.split);
        w.parts = uniform(i.parts);
        w.tiles = uniform(i.tiles);
        w.per = uniform(i.per);
        w.number = uniform(i.number);
        w.heads(a, cl, (uint32_t)uniform(i.unit));
        return true;
    }
    const uint32_t item = blockIdx.x / lo.units, u = blockIdx.x - item * lo.units;
    // every call checks the offsets once (there are no fewer items than users);
    // what is loaded for it arrives with what the block itself needs
    const int64_t i = (int64_t)item * blockDim.x + threadIdx.x;
    const bool check = u == 0 && i < a.batch;
    int64_t x = 0, y = 0;
    if (check) {
        x = a.offsets[i];
        y = a.offsets[i + 1];
    }
    int64_t t = 0;
    if (lo.per_seq) {
        const uint32_t n = (uint32_t)a.batch, first = item / n;
        w.b = item - first * n;
        t = first;
    } else {
        w.b = wave_last_le(a.batch, [&](int64_t x) { return a.offsets[x] / tq + x; }, (int64_t)item);
    }
    const int64_t s = a.offsets[w.b], e = a.offsets[w.b + 1], n = p.lens[w.b];
    w.s = uniform(s);
    const int64_t end = uniform(e);
    w.had = uniform(n);
    if (check && (x > y || (i == 0 && x != 0) || (i == a.batch - 1 && y != a.n_events)))
        set_status(&a.hdr->status, RSE_ERR_BAD_INPUT);
    w.count = user_events(a, p, w.s, end, w.had, lane_id() == 0);
    if (w.count <= 0) return false;             // (past this s is an event's number, and the products do not overflow)
    if (!lo.per_seq) t = (int64_t)item - (w.s / tq + w.b);
    if (t < 0 || t * tq >= w.count) return false;
    w.tile = (int)t;
    w.split = 0;
    w.parts = 1;
    w.heads(a, cl, u);
    return true;
}

// The parts of the keys, by what the lengths on the device are: parts of
// nearly equal length, as few tiles each as make about `want` parts of them all
// (what the card runs at a time), but at least `least`, and a user's equal.
// (Parts of max_len / 32 keys, with lengths up to it: 304 us for 205, 8 users of
// up to 32768 events.)  One block; the lists of a user's units, parts and tiles, tiles
// fastest, are dealt out so that an XCD gets neighbours, which read the same keys.
constexpr int PLAN_THREADS = 1024, PLAN_USERS = 2048;
__device__ __forceinline__ int32_t wave_total(int32_t x) {
    x += row_ror<8>(x);
    x += row_ror<4>(x);
    x += row_ror<2>(x);
    x += row_ror<1>(x);
    const u32x2 r = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
    const uint32_t y = r.x + r.y;
    const u32x2 h = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return (int32_t)(h.x + h.y);
}
__device__ __forceinline__ int parts_of(int n, int per) { return n <= per ? 1 : (int)(((uint32_t)n + (uint32_t)per - 1) / (uint32_t)per); }
__global__ __launch_bounds__(PLAN_THREADS) void k_chunk_plan(SeqArgs a, PageArgs p, int units, int tq, int kt, int least, int want,
                                                             int bound, Item* list) {
    constexpr int NW = PLAN_THREADS / WAVE, EACH = PLAN_USERS / PLAN_THREADS;
    __shared__ float s_work[NW];
    __shared__ int32_t s_sum[2][NW], s_first[PLAN_USERS];
    const int t = threadIdx.x, lane = lane_id(), w = t / WAVE;
    int turn = 0;
    auto total = [&](int32_t x) {
        x = wave_total(x);
        if (lane == 0) s_sum[turn][w] = x;
        __syncthreads();
        x = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) x += s_sum[turn][i];
        turn ^= 1;
        return x;
    };
    int n[EACH], blocks[EACH];                  // tiles of keys; blocks of a part, above `bound` if not possible
    float work = 0.f;
    int whole = 0;
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
        const int64_t b = (int64_t)t * EACH + u;
        n[u] = blocks[u] = 0;
        if (b < a.batch) {
            const int64_t s = a.offsets[b], e = a.offsets[b + 1];
            int64_t had = p.lens[b];
            if (s > e || (b == 0 && s != 0) || (b == a.batch - 1 && e != a.n_events)) set_status(&a.hdr->status, RSE_ERR_BAD_INPUT);
            const int count = user_events(a, p, s, e, had, true);
            const int64_t x = (int64_t)units * ((count + (int64_t)tq - 1) / tq);
            blocks[u] = x > bound ? bound + 1 : (int)x;
            n[u] = (int)(had < 0 || !count ? 0 : (had + count + kt - 1) / kt);
        }
        work += (float)n[u] * (float)blocks[u];
        whole += blocks[u];
    }
#pragma unroll
    for (int m = 1; m < WAVE; m *= 2) work += __shfl_xor(work, m);
    if (lane == 0) s_work[w] = work;
    whole = total(whole);
    work = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) work += s_work[i];
    int items = 0, per = 1, mine = 0;
    // (only offsets that descend, of overlapping ranges, make more: status is set, and
    // all are left out; those of a batch make at most bound - want)
    if (whole <= bound) {
        // the least length that makes no more than `most` parts is from `per` to high
        const int most = want > whole + want / 2 ? want : whole + want / 2;
        int high = (int)(work * (1.f + 1e-5f) / (float)(most - whole)) + 1;
        per = (int)(work / (float)most);
        per = per < least ? least : per;
        while (per < high) {
            const int mid = (per + high) / 2;
            mine = 0;
#pragma unroll
            for (int u = 0; u < EACH; ++u) mine += blocks[u] * parts_of(n[u], mid);
            if (total(mine) <= most) high = mid;
            else per = mid + 1;
        }
        mine = 0;
#pragma unroll
        for (int u = 0; u < EACH; ++u) mine += blocks[u] * parts_of(n[u], per);
        items = total(mine);
        if (items > bound) items = 0;
    }
    // where the users begin
    int sum = mine;
#pragma unroll
    for (int m = 1; m < WAVE; m *= 2) {
        const int x = __shfl_up(sum, m);
        if (lane >= m) sum += x;
    }
    if (lane == WAVE - 1) s_sum[turn][w] = sum;
    __syncthreads();
    for (int i = 0; i < w; ++i) sum += s_sum[turn][i];
    int first = sum - mine;
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
        s_first[t * EACH + u] = first;
        first += blocks[u] * parts_of(n[u], per);
    }
    __syncthreads();
    const int row = (items + 7) / 8;
    for (int x = t; x < bound; x += PLAN_THREADS) {
        const int at = (x & 7) * row + (x >> 3);
        Item it = {};
        it.b = -1;
        if (x >> 3 < row && at < items) {
            int b = 0;                          // the last user that begins at or before `at`
            for (int step = PLAN_USERS / 2; step > 0; step /= 2)
                if (b + step < a.batch && s_first[b + step] <= at) b += step;
            it.s = a.offsets[b];
            it.had = p.lens[b];
            it.b = b;
            it.count = user_events(a, p, it.s, a.offsets[b + 1], it.had, false);
            it.tiles = (int)((it.count + (int64_t)tq - 1) / tq);
            const int keys = it.had < 0 ? 0 : (int)((it.had + it.count + kt - 1) / kt);
            it.parts = parts_of(keys, per);
            it.per = (keys + it.parts - 1) / it.parts;
            const int i = at - s_first[b];
            it.tile = i % it.tiles;
            it.split = i / it.tiles % it.parts;
            it.unit = i / it.tiles / it.parts;
            it.number = at;
        }
        list[x] = it;
    }
}

// The tile's new events into their pages, by the block of the key/value head's
// first query heads and first part.
template <typename T, int D>
__device__ __forceinline__ void store_events(const SeqArgs& a, const PageArgs& p, const Work& w, int first, int last,
                                             const Rows<const T>& k, const Rows<const T>& v, T* kp, T* vp) {
    using TL = Tile<T, D>;
    if (w.had < 0 || w.split != 0 || w.h0 != w.g * a.group) return;
    const int64_t row_elems = (int64_t)(a.n_heads / a.group) * D;
    for (int t = threadIdx.x; t < (last - first) * TL::CH; t += blockDim.x) {
        const int i = first + t / TL::CH, c = t % TL::CH;
        const int64_t e = w.had + i, page = p.table[w.b * p.max_pages + (e >> p.shift)];
        const u32x4 kr = gload_u4(k.at(w.s + i, w.g) + c * TL::EPC), vr = gload_u4(v.at(w.s + i, w.g) + c * TL::EPC);
        const int32_t at = a.pos[w.s + i];
        __builtin_amdgcn_sched_barrier(0);      // one latency, not three
        const int64_t slot = slot_of(p, page, e), to = slot * row_elems + w.g * D + c * TL::EPC;
        if (slot < 0) continue;
        gstore_u4(kp + to, kr);
        gstore_u4(vp + to, vr);
        if (w.g == 0 && c == 0) p.tp[slot] = at;
    }
}

// The operands of 16 rows of values and the probabilities of them: registers
// 8 i .. 8 i + 7 of a lane (rows 16 i and on).  bf16: the probabilities as pairs
// of values, the second the rounded remainder of the first.
template <typename T, int D>
struct Step;
template <int D>
struct Step<uint16_t, D> {
    static constexpr int MMA = D / 16, READS = D / 16;
    u32x4 v[D / 32], p[2];
    __device__ __forceinline__ void load(const u32x4* tile, int r0) {
        const int lane = lane_id(), h = lane >> 5, i = lane & 15;
        const char* base = reinterpret_cast<const char*>(tile);
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt) {
            const int c = 4 * dt + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);       // (as in OverRows)
            s16x4 x[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int row = r0 + 8 * u + 4 * h + (i >> 2);
                x[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (RSE_LDS s16x4*)(base + Tile<uint16_t, D>::chunk_at(row, c) * 16 + (i & 1) * 8));
            }
            v[dt].xy = __builtin_bit_cast(u32x2, x[0]);
            v[dt].zw = __builtin_bit_cast(u32x2, x[1]);
        }
    }
    __device__ __forceinline__ void take(const float (&x)[8]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            p[0][j] = pack_bf16(x[2 * j], x[2 * j + 1]);
            p[1][j] = pack_bf16(x[2 * j] - __uint_as_float(p[0][j] << 16), x[2 * j + 1] - __uint_as_float(p[0][j] & 0xFFFF0000u));
        }
    }
    __device__ __forceinline__ void add(f32x16 (&o)[D / 32]) const {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt)
                o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v[dt]), __builtin_bit_cast(bf16x8, p[t]),
                                                                o[dt], 0, 0, 0);
    }
};
template <int D>
struct Step<float, D> {
    static constexpr int MMA = D / 4, READS = D / 4;
    float v[D / 32][8], p[8];
    __device__ __forceinline__ void load(const u32x4* tile, int r0) {
        const int lane = lane_id(), h = lane >> 5;
        const float* f = reinterpret_cast<const float*>(tile);
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int row = r0 + tile_row(r, h), d = 32 * dt + (lane & 31);
                v[dt][r] = f[Tile<float, D>::chunk_at(row, d >> 2) * 4 + (d & 3)];
            }
    }
    __device__ __forceinline__ void take(const float (&x)[8]) {
#pragma unroll
        for (int r = 0; r < 8; ++r) p[r] = x[r];
    }
    __device__ __forceinline__ void add(f32x16 (&o)[D / 32]) const {
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) o[dt] = __builtin_amdgcn_mfma_f32_32x32x2f32(v[dt][r], p[r], o[dt], 0, 0, 0);
    }
};

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
    // x: logits less m of 32 N keys, -infinity where not visible
    template <int N>
    __device__ __forceinline__ void add(f32x16 (&x)[N], const u32x4* values) {
        float top = x[0][0];
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, x[u][r]);
        top = fmaxf(top, other_half(top));
        const bool move = top > 8.f || (!set && top > -INFINITY);
        set |= top > -INFINITY;
        if (__any(move)) {
            const float by = move ? top : 0.f, r = __builtin_amdgcn_exp2f(-by);
            m += by;
            l = l == 0.f ? 0.f : l * r;         // nothing summed yet: 0, also where exp2 overflows
#pragma unroll
            for (int u = 0; u < N; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) x[u][i] -= by;
            const float ro = r < INFINITY ? r : 0.f;
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) o[dt] *= ro;
        }
        // a step's products run while the next one's operands are formed (in the
        // order that the compiler chose each pair of products waited for its own read)
        Step<T, D> step[2];
        auto form = [&](int i) {
            float e[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) e[r] = __builtin_amdgcn_exp2f(x[i / 2][8 * (i % 2) + r]);
            l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
            step[i % 2].take(e);
        };
        step[0].load(values, 0);
        form(0);
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            if (i + 1 < 2 * N) step[(i + 1) % 2].load(values, 16 * (i + 1));
            step[i % 2].add(o);
            if (i + 1 < 2 * N) {
                form(i + 1);
                __builtin_amdgcn_sched_group_barrier(0x100, Step<T, D>::READS, 0);
#pragma unroll
                for (int j = 0; j < Step<T, D>::MMA; ++j) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
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
// The block's bias and buckets, loaded well before they go to LDS.
struct Early {
    float bias;
    int32_t bound;
    uint32_t cell;
    __device__ __forceinline__ void load(const SeqArgs& a, const Work& w) {
        const int t = threadIdx.x;
        bias = t < w.nc * (a.n_bounds + 1) ? a.bias[w.h0 * (a.n_bounds + 1) + t] : 0.f;
        bound = t <= RSE_SEQ_MAX_BOUNDARIES ? a.hdr->bounds[t] : 0;
        cell = t <= RSE_SEQ_MAX_BOUNDARIES ? reinterpret_cast<const uint32_t*>(a.hdr->cell)[t] : 0;
    }
    __device__ __forceinline__ void put(const SeqArgs& a, const Work& w, float* s_bias, LdsBuckets& buckets) const {
        const int nb = a.n_bounds + 1, st = bias_stride(a.n_bounds), t = threadIdx.x;
        if (t < w.nc * nb) s_bias[t / nb * st + t % nb] = bias2(bias);
        for (int i = t + (int)blockDim.x; i < w.nc * nb; i += blockDim.x)
            s_bias[i / nb * st + i % nb] = bias2(a.bias[w.h0 * nb + i]);
        if (t <= RSE_SEQ_MAX_BOUNDARIES) {
            buckets.bounds[t] = bound;
            buckets.cell[t] = cell;
        }
    }
};

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
    }
    __device__ __forceinline__ void loaded() {
        lo = half_min(pos);
        hi = half_max(pos);
    }
};

// Few columns: all waves of a block have the same tile of columns and take
// tiles of 32 keys in turn, each from memory to its own registers and LDS, so
// that no wave waits for another; they are joined in LDS at the end.
// Bound by latency: a tile's rows are on their way while the last one's are
// used, and what a tile waits is covered by the other waves of its SIMD.  Three, of
// rows up to 128 bytes, though that spills some registers: 35.0 us for 42.2 with two on
// 256 users of up to 1024 events and 16 new ones (1.9 TB/s; the longest users'
// chains of nine tiles a wave end last).
template <typename T, int D, int CW>
__global__ __launch_bounds__(CW * 64) __attribute__((amdgpu_waves_per_eu(CW == 8 ? 2 : D * sizeof(T) <= 128 ? 3 : 1))) void k_chunk_few(
    SeqArgs a, PageArgs p, Layout lo, Columns cl, Rows<const T> q, Rows<const T> k, Rows<const T> v, T* kp, T* vp, Rows<T> out,
    float* part_o, float* part_ml) {
    using TL = Tile<T, D>;
    constexpr int CH = TL::CH, ND = D / 32, NC = CH / 2;
    extern __shared__ float s_bias[];           // [cols][bias_stride]
    constexpr int SR = D + 4;                   // a column's sums: columns 16 bytes of banks apart
    __shared__ u32x4 s_mem[CW * 32 * CH > CW * 32 * SR / 4 ? CW * 32 * CH : CW * 32 * SR / 4];  // tiles of V, then the waves' sums
    __shared__ LdsBuckets s_buckets;
    __shared__ u32x4 s_pairs[CW][WAVE];
    alignas(16) __shared__ int32_t s_pos[CW][32];       // (read by 16 bytes)
    __shared__ float s_ml[CW][2][32];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE), half = lane >> 5, col = lane & 31;
    auto page_of = [&](int64_t b, int64_t t) -> int32_t {
        const int64_t i = (t * 32 + col) >> p.shift;
        return i < p.max_pages ? p.table[b * p.max_pages + i] : 0;
    };
    // Each load of a call waits some 2000 cycles, the first tiles' pages not for
    // the lengths where the user is known without them.
    const bool known = !lo.list && lo.per_seq;
    int32_t pages[2];
    if (known) {
        const uint32_t b = blockIdx.x / lo.units % (uint32_t)a.batch;
        pages[0] = page_of(b, w);
        pages[1] = page_of(b, w + CW);
    }
    Work wk;
    if (!find_work(a, p, cl, lo, cl.events, wk)) return;
    u32x4* tile = s_mem + w * 32 * CH;
    const int first = wk.tile * cl.events, last = first + cl.events < wk.count ? first + cl.events : wk.count;
    const int64_t had = wk.had;
    // keys that some column may see: 0 .. end - 1; the wave's tiles t0 + w, + CW, ...
    const int64_t end = had < 0 ? 0 : had + (a.causal ? last : wk.count);
    int64_t t0 = 0, t1 = (end + 31) / 32;
    if (wk.parts > 1) {
        t0 = (int64_t)wk.split * wk.per;
        t1 = t0 + wk.per < t1 ? t0 + wk.per : t1;
        if (t0 >= t1) return;                   // (the join knows)
    }
    const int64_t row_elems = (int64_t)(a.n_heads / a.group) * D;
    const float c2 = fabsf(a.scale) * LOG2E;
    u32x4 rk[NC], rv[NC];
    int32_t rp = 0;
    bool see = false;
    auto load_rows = [&](int64_t t, int32_t page) {
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
    // what the rows wait for comes first, and what else the block needs before them
    int64_t t = t0 + w;
    if (!known) {
        pages[0] = page_of(wk.b, t);
        pages[1] = page_of(wk.b, t + CW);
    }
    Early early;
    early.load(a, wk);
    Column<T, D> c;
    c.load(a, cl, wk, first, q);
    LaneBuckets lb;
    lb.load(a.hdr, s_bias + (c.head - wk.h0) * bias_stride(a.n_bounds), a.n_bounds);
    if (t < t1) load_rows(t, pages[0]);
    int32_t page = pages[1];
    early.put(a, wk, s_bias, s_buckets);
    c.loaded();
    store_events<T, D>(a, p, wk, first, last, k, v, kp, vp);
    Online<T, D> sm;
    sm.clear();
    __syncthreads();
    for (; t < t1; t += CW) {
        f32x16 xs[1] = {};
        f32x16& x = xs[0];
#pragma unroll
        for (int i = 0; i < NC; ++i) x = mma_chunk<T>(rk[i], c.q.v[i], x);
#pragma unroll
        for (int i = 0; i < NC; ++i) tile[TL::chunk_at(col, 2 * i + half)] = see ? rv[i] : u32x4{0, 0, 0, 0};
        const uint32_t seen = (uint32_t)__ballot(see);
        s_pos[w][col] = rp;
        const int32_t range[2] = {half_min(rp), half_max(rp)};
        wave_lds_sync();
        if (t + CW < t1) load_rows(t + CW, page);
        page = page_of(wk.b, t + 2 * CW);
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
        sm.add(xs, tile);
        wave_lds_sync();                        // read before the next tile is stored
    }
    sm.l += other_half(sm.l);
    if (half == 0) {
        s_ml[w][0][col] = sm.reference();
        s_ml[w][1][col] = sm.l;
    }
    __syncthreads();                            // the V tiles are done with: their place takes the sums
    float* s_sum = reinterpret_cast<float*>(s_mem);
    if (c.live) {
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4*>(s_sum + (w * 32 + col) * SR + 32 * dt + 8 * j + 4 * half) =
                    f32x4{sm.o[dt][4 * j], sm.o[dt][4 * j + 1], sm.o[dt][4 * j + 2], sm.o[dt][4 * j + 3]};
    }
    __syncthreads();
    for (int y = threadIdx.x; y < (last - first) * wk.nc * D; y += CW * WAVE) {
        const int cc = y / D, d = y % D;
        float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
        for (int u = 0; u < CW; ++u) M = fmaxf(M, s_ml[u][0][cc]);
#pragma unroll
        for (int u = 0; u < CW; ++u) {
            const float r = part_weight(s_ml[u][0][cc], M);
            L = __builtin_fmaf(s_ml[u][1][cc], r, L);
            O = __builtin_fmaf(s_sum[(u * 32 + cc) * SR + d], r, O);
        }
        const int64_t ev = wk.s + first + cc / wk.nc;
        const int head = wk.h0 + cc % wk.nc;
        if (wk.parts == 1) {
            from_f32(out.at(ev, head)[d], L == 0.f ? 0.f : O / L);
        } else {
            const int64_t at = (int64_t)wk.number * 32 + cc;
            part_o[at * D + d] = O;
            if (d == 0) {
                part_ml[2 * at] = M;
                part_ml[2 * at + 1] = L;
            }
        }
    }
}

// Many columns: every wave has a tile of columns of its own, and the block
// brings tiles of KT keys to LDS for them, NST - 1 tiles ahead and without
// registers in between (with the next tile's rows in registers, and those spilled:
// 350 us for 192 on 8 users of up to 32768 events and 128 new ones, bf16 rows of 128).
// 64 keys at a time in bf16 (32: 207 us there): one maximum and one question whether it
// has moved, and one for the bias, for twice the products.  In fp32 32 (64: 180 us
// for 139 on 24 users of up to 2048 events and 512 new ones, rows of 64).
// Dims of 32 leave registers for three waves a SIMD: 95 users of up to 53 events and
// 292 new ones, 32 heads on 4, bf16 121 us for 95; where histories are long no faster.
// In general two waves share a SIMD, and their products and vector operations take turns
// more than they overlap: 25 % of the cycles are products in bf16, 36 % in fp32.
template <typename T, int D>
struct Many {
    static constexpr int RB = D * (int)sizeof(T), KT = sizeof(T) == 2 ? 64 : 32;
    static constexpr int NST = KT * RB <= 8192 ? 4 : sizeof(T) == 2 ? 2 : 3;       // (40 to 105 KiB: two blocks a CU, one of rows of 512 bytes)
    static constexpr int CH = Tile<T, D>::CH, NT = CW * WAVE, PER = KT * CH / NT;
    static constexpr int WAVES = D == 32 ? 3 : RB <= 256 ? 2 : 1;       // that share a SIMD
    static constexpr int PAGES = 512;                       // of the table in LDS at a time
};

// What rows past the end and of pages out of the pool are read from.
__device__ u32x4 g_no_row[32];

template <typename T, int D>
__global__ __launch_bounds__(CW * 64) __attribute__((amdgpu_waves_per_eu(Many<T, D>::WAVES))) void k_chunk_many(
    SeqArgs a, PageArgs p, Layout lo, Columns cl, Rows<const T> q, Rows<const T> k, Rows<const T> v, T* kp, T* vp, Rows<T> out,
    float* part_o, float* part_ml) {
    using TL = Tile<T, D>;
    using MY = Many<T, D>;
    constexpr int CH = MY::CH, KT = MY::KT, PER = MY::PER, NST = MY::NST, ND = D / 32, SENT = 2 * PER + 1;
    extern __shared__ float s_bias[];           // [cols][bias_stride]
    __shared__ u32x4 s_k[NST][KT * CH], s_v[NST][KT * CH];
    alignas(16) __shared__ int32_t s_pos[CW][NST][KT];      // (read by 16 bytes; each wave brings its own)
    __shared__ int32_t s_page[MY::PAGES];       // -1: out of the pool
    __shared__ uint64_t s_seen[CW][NST];        // bit per key that may be seen
    __shared__ LdsBuckets s_buckets;
    __shared__ u32x4 s_pairs[CW][WAVE];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE), half = lane >> 5, t = threadIdx.x;
    Work wk;
    if (!find_work(a, p, cl, lo, CW * cl.events, wk)) return;
    const int begin = wk.tile * CW * cl.events, past = begin + CW * cl.events < wk.count ? begin + CW * cl.events : wk.count;
    const int64_t had = wk.had;
    // keys that some column of the block may see: 0 .. end - 1; its tiles of KT: t0 .. t1 - 1
    const int64_t end = had < 0 ? 0 : had + (a.causal ? past : wk.count);
    int64_t t0 = 0, t1 = (end + KT - 1) / KT;
    if (wk.parts > 1) {
        t0 = (int64_t)wk.split * wk.per;
        t1 = t0 + wk.per < t1 ? t0 + wk.per : t1;
        if (t0 >= t1) return;                   // (the join knows)
    }
    Early early;
    early.load(a, wk);
    const int first = begin + w * cl.events;
    Column<T, D> c;
    c.load(a, cl, wk, first, q);
    LaneBuckets lb;
    lb.load(a.hdr, s_bias + (c.head - wk.h0) * bias_stride(a.n_bounds), a.n_bounds);
    early.put(a, wk, s_bias, s_buckets);
    c.loaded();
    store_events<T, D>(a, p, wk, begin, past, k, v, kp, vp);
    const int64_t row_elems = (int64_t)(a.n_heads / a.group) * D;
    const float c2 = fabsf(a.scale) * LOG2E;

    // the part of the page table for keys from `from` on; all threads come here
    int64_t window = 0, window_end = 0;         // keys
    auto load_pages = [&](int64_t from) {
        __syncthreads();                        // the last part has been used
        window = from >> p.shift << p.shift;
        window_end = window + ((int64_t)MY::PAGES << p.shift);
        for (int i = t; i < MY::PAGES; i += MY::NT) {
            const int64_t e = window + ((int64_t)i << p.shift);
            int32_t page = 0;
            if (e < had && e < t1 * KT) {
                page = p.table[wk.b * p.max_pages + (e >> p.shift)];
                if (page < 0 || page >= p.n_pages) {
                    set_status(&p.status->status, RSE_ERR_BAD_INPUT);
                    page = -1;
                }
            }
            s_page[i] = page;
        }
        __syncthreads();
    };
    // where the thread's piece of a tile is; those of its other pieces are NT / CH rows
    // apart, with the swizzle's term for the eighth row in odd ones of rows of 512 bytes
    constexpr int ROWS = MY::NT / CH;
    const uint32_t off_at = (uint32_t)(t / CH * (int)row_elems + ((t % CH) ^ TL::swz(t / CH)) * TL::EPC) * (uint32_t)sizeof(T);
    const bool in_page = p.shift >= (KT == 64 ? 6 : 5);         // a tile lies in one page
    auto send = [&](int64_t tile, int st) {
        if (tile * KT >= window_end) load_pages(tile * KT);
        const int64_t k0 = tile * KT;
        if (in_page && k0 + KT <= had) {
            const int64_t page = uniform((int64_t)s_page[(k0 - window) >> p.shift]);
            if (page >= 0) {
                const int64_t first_slot = (page << p.shift) + (k0 & ((1ll << p.shift) - 1));
                const T *kt = kp + first_slot * row_elems + wk.g * D, *vt = vp + first_slot * row_elems + wk.g * D;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const uint32_t off = off_at ^ (uint32_t)(TL::swz(i * ROWS) * 16);
                    to_lds(kt + i * ROWS * row_elems, off, &s_k[st][i * MY::NT + w * WAVE]);
                    to_lds(vt + i * ROWS * row_elems, off, &s_v[st][i * MY::NT + w * WAVE]);
                }
                if (lane < KT) to_lds4(p.tp + first_slot, 4 * lane, s_pos[w][st]);
                if (lane == 0) s_seen[w][st] = KT == 64 ? ~0ull : 0xFFFFFFFFull;
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = i * MY::NT + t, row = at / CH, off = ((at % CH) ^ TL::swz(row)) * TL::EPC;
            const int64_t e = k0 + row;
            const T *kr = reinterpret_cast<const T*>(g_no_row), *vr = kr;
            if (e < had) {
                const int64_t page = s_page[(e - window) >> p.shift];
                if (page >= 0) {
                    const int64_t s = ((page << p.shift) + (e & ((1ll << p.shift) - 1))) * row_elems + wk.g * D;
                    kr = kp + s;
                    vr = vp + s;
                }
            } else if (e < end) {
                kr = k.at(wk.s + (e - had), wk.g);
                vr = v.at(wk.s + (e - had), wk.g);
            }
            to_lds(kr + off, &s_k[st][i * MY::NT + w * WAVE]);
            to_lds(vr + off, &s_v[st][i * MY::NT + w * WAVE]);
        }
        const int64_t e = k0 + lane;
        const int32_t* at = a.pos + wk.s;
        bool see = lane < KT && e < end;
        if (see && e < had) {
            const int64_t page = s_page[(e - window) >> p.shift];
            see = page >= 0;
            if (see) at = p.tp + (page << p.shift) + (e & ((1ll << p.shift) - 1));
        } else if (see) {
            at += e - had;
        }
        if (lane < KT) to_lds4(at, s_pos[w][st]);
        const uint64_t seen = __ballot(see);
        if (lane == 0) s_seen[w][st] = seen;
    };
    Online<T, D> sm;
    sm.clear();
    if (t0 < t1) load_pages(t0 * KT);
    else __syncthreads();
#pragma unroll 1
    for (int i = 0; i < NST - 1; ++i)
        if (t0 + i < t1) send(t0 + i, i);
    none_left();
    int st = 0;
    auto next = [&](int64_t tile) {
        // the tiles behind this one stay in flight
        if (tile + NST - 2 < t1) loads_left<(NST - 2) * SENT>();
        else loads_left<0>();
        lds_barrier();                          // the tile has landed; all are done with the last one's place
        if (tile + NST - 1 < t1) send(tile + NST - 1, st == 0 ? NST - 1 : st - 1);
    };
    if (first >= wk.count) {                    // a wave without columns (a condition in the loop below had the sums
        for (int64_t tile = t0; tile < t1; ++tile) {        // copied from registers to registers, and spilled)
            next(tile);
            st = st == NST - 1 ? 0 : st + 1;
        }
        return;
    }
    for (int64_t tile = t0; tile < t1; ++tile) {
        next(tile);
        const int64_t k0 = tile * KT;
        const int32_t* pos = s_pos[w][st];
        u32x4 rows[KT / 32][CH / 2];            // all on their way before the first is waited for
        const int32_t rp = pos[lane % KT];
#pragma unroll
        for (int u = 0; u < KT / 32; ++u)
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) rows[u][i] = s_k[st][TL::chunk_at(32 * u + (lane & 31), 2 * i + half)];
        __builtin_amdgcn_sched_barrier(0);
        const int32_t low = half_min(rp), high = half_max(rp);
        const int32_t l0 = __builtin_amdgcn_readlane(low, 0), l1 = __builtin_amdgcn_readlane(low, 32);
        const int32_t h0 = __builtin_amdgcn_readlane(high, 0), h1 = __builtin_amdgcn_readlane(high, 32);
        const int32_t range[2] = {l0 < l1 ? l0 : l1, h0 > h1 ? h0 : h1};
        TileBuckets<true> tb;
        tb.set(lb, c.lo, c.hi, range);
        f32x16 z[KT / 32];
#pragma unroll
        for (int u = 0; u < KT / 32; ++u) {
            z[u] = f32x16{};
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) z[u] = mma_chunk<T>(rows[u][i], c.q.v[i], z[u]);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < KT / 32; ++u) {
            if (tb.many) {
                tb.find_pairs(s_pairs[w], 0, 1, s_buckets, a.n_bounds, a.cells, pos + 32 * u, c.pos);
                wave_lds_sync();
            }
            z[u] = tb.logits(z[u], c2, -sm.m, lb, s_pairs[w], lb.bias, pos + 32 * u, c.pos);
            if (tb.many) wave_lds_sync();       // read before the next are written
        }
        const uint64_t seen = s_seen[w][st];
        const uint32_t seen_lo = __builtin_amdgcn_readfirstlane((uint32_t)seen), seen_hi = __builtin_amdgcn_readfirstlane((uint32_t)(seen >> 32));
        if ((KT == 64 ? seen_lo & seen_hi : seen_lo) != ~0u) {
#pragma unroll
            for (int u = 0; u < KT / 32; ++u) {
                const uint32_t bits = (u ? seen_hi : seen_lo) >> (4 * half);
#pragma unroll
                for (int r = 0; r < 16; ++r) z[u][r] = (bits >> tile_row(r, 0)) & 1 ? z[u][r] : -INFINITY;
            }
        }
        if (a.causal && k0 + KT - 1 > had + first) {
#pragma unroll
            for (int u = 0; u < KT / 32; ++u) hide_after(z[u], (int)(had - k0) - 32 * u + c.event - 4 * half);
        }
        sm.add(z, s_v[st]);
        st = st == NST - 1 ? 0 : st + 1;
    }
    sm.l += other_half(sm.l);
    if (!c.live) return;
    const int64_t ev = wk.s + c.event;
    if (wk.parts == 1) {
        const float inv = sm.l == 0.f ? 0.f : 1.f / sm.l;
        T* dst = out.at(ev, c.head);
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) store_column(dst + 32 * dt, sm.o[dt], inv);
    } else {
        const int64_t at = ((int64_t)wk.number * CW + w) * 32 + (lane & 31);
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) store_column(part_o + at * D + 32 * dt, sm.o[dt], 1.f);
        if (half == 0) {
            part_ml[2 * at] = sm.reference();
            part_ml[2 * at + 1] = sm.l;
        }
    }
}

// Joins the parts: blocks (x, y) take the columns of a tile, D / 4 threads a
// column.  kt, waves: of the kernel that left the parts.
constexpr int JT = 256;
template <typename T, int D>
__global__ __launch_bounds__(JT) void k_chunk_join(SeqArgs a, PageArgs p, Layout lo, Columns cl, int kt, int waves, const float* part_o,
                                                   const float* part_ml, Rows<T> out) {
    constexpr int LR = D / 4;
    Work wk;
    if (!find_work(a, p, cl, lo, waves * cl.events, wk)) return;
    if (wk.split != 0 || wk.parts == 1) return;
    const int col = (int)blockIdx.y * (JT / LR) + threadIdx.x / LR, d = 4 * (threadIdx.x % LR), in = col & 31;
    const int begin = wk.tile * waves * cl.events, past = begin + waves * cl.events < wk.count ? begin + waves * cl.events : wk.count;
    const int event = begin + (col >> 5) * cl.events + in / wk.nc, head = wk.h0 + in % wk.nc;
    if (in >= cl.events * wk.nc || event >= wk.count) return;
    // parts with keys that some of the tile's columns see
    const int64_t end = wk.had + (a.causal ? past : wk.count);
    const int parts = (int)(((end + kt - 1) / kt + wk.per - 1) / wk.per);
    const int64_t at = (int64_t)wk.number * 32 * waves + col, step = (int64_t)wk.tiles * 32 * waves;
    float M = -INFINITY, L = 0.f;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) M = fmaxf(M, part_ml[2 * (at + s * step)]);
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
        const float r = part_weight(part_ml[2 * (at + s * step)], M);
        L = __builtin_fmaf(part_ml[2 * (at + s * step) + 1], r, L);
        const f32x4 x = gload_f4(part_o + (at + s * step) * D + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(x[i], r, o[i]);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= inv;
    store_four(out.at(wk.s + event, head) + d, o);
}

// ------------------------------------------------------------------ host --
// Blocks that run at a time, 2 a CU (1 with rows of 512 bytes; 3 of few columns
// with rows up to 128).  Parts for twice as many: 199 us for 192, and the join 16 for
// 11 (8 users of up to 32768 events).
constexpr int ROOM = 512;
// The few-columns kernel takes tiles of columns apart up to this many of a user:
// the waves of a block share none of the loads, but wait for none of each other
// (256 users of up to 1024 events, two tiles: 35 us for 62 with the other kernel).
constexpr int FEW_TILES = 2;
// Blocks up to which each has 8 waves (one user of 300 events: 11.0 us for 12.2);
// with more, blocks of 4 overlap one's ends with the other's loop (256 users: 35 us for 58).
constexpr int FEW_BLOCKS = 256;

struct ChunkPlan {
    Columns cl;
    bool few;
    int tq, kt;
    TileGrid grid;
    int64_t units;
    int want, least;                    // want > 0: the keys are split
    int64_t whole() const { return grid.items * units; }
    int64_t blocks() const { return whole() + want; }
};
ChunkPlan chunk_plan(const rse_seqattn* at, int64_t n_events, int64_t batch, int64_t max_new, int64_t max_len) {
    ChunkPlan p;
    const int group = at->n_heads / at->n_kv_heads, row = at->dim * (at->dtype == RSE_BF16 ? 2 : 4);
    p.cl.cols = group < 32 ? group : 32;
    p.cl.blocks = (group + p.cl.cols - 1) / p.cl.cols;
    p.cl.events = 32 / p.cl.cols;
    p.few = max_new <= FEW_TILES * p.cl.events;
    p.tq = p.few ? p.cl.events : CW * p.cl.events;
    p.kt = p.few || at->dtype == RSE_F32 ? 32 : 64;
    p.grid = tile_grid(n_events, batch, max_new, p.tq);
    p.units = (int64_t)at->n_kv_heads * p.cl.blocks;
    p.least = 256 / p.kt;
    // Not for short histories, nor where there are blocks enough; few columns
    // with blocks for the CUs only where histories are long, as the plan and the join take
    // 17 us.  Whole / in parts, 256 users of up to 1024, 4096, 8192 events (1024 blocks,
    // bf16 rows of 64): 36 / 51, 102 / 95, 213 / 165; 128 of up to 4096 in fp32 (512): 170 / 152.
    const int64_t from = p.few && p.whole() >= ROOM ? 4096 : 512;
    if (max_len >= from && p.whole() < PLAN_USERS) p.want = p.few && row <= 128 ? 3 * ROOM / 2 : row > 256 ? ROOM / 2 : ROOM;
    else p.want = 0;
    return p;
}

struct ChunkWs {
    float* o;
    float* ml;
    Item* list;
    size_t bytes;
};
ChunkWs chunk_ws(const rse_seqattn* at, const ChunkPlan& p, void* base) {
    Carver c(base);
    const size_t n = p.want ? (size_t)p.blocks() * 32 * (p.few ? 1 : CW) : 0;
    ChunkWs w;
    w.o = c.take<float>(n * at->dim);
    w.ml = c.take<float>(2 * n);
    w.list = c.take<Item>(p.want ? (size_t)p.blocks() : 0);
    w.bytes = c.size();
    return w;
}

template <typename T, int D>
int run_chunk(const rse_seqcache* c, const SeqArgs& a, const PageArgs& pg, const ChunkPlan& p, const ChunkWs& ws,
              const rse_seq_rows* q, const rse_seq_rows* k, const rse_seq_rows* v, const rse_seq_rows* out, hipStream_t s) {
    if (!launch_holds(p.blocks(), CW * WAVE)) return RSE_ERR_UNSUPPORTED;
    const size_t lds = (size_t)p.cl.cols * ((a.n_bounds + 1) | 1) * sizeof(float);
    const Layout lo = {(uint32_t)p.units, (uint32_t)p.grid.items, (uint32_t)p.grid.per_seq, p.want ? ws.list : nullptr};
    const dim3 grid((unsigned)p.blocks());
    if (p.want)
        hipLaunchKernelGGL(k_chunk_plan, dim3(1), dim3(PLAN_THREADS), 0, s, a, pg, (int)p.units, p.tq, p.kt, p.least, p.want,
                           (int)p.blocks(), ws.list);
    const auto run = [&](auto kernel, int waves) {
        hipLaunchKernelGGL(kernel, grid, dim3(waves * WAVE), lds, s, a, pg, lo, p.cl, rows_view<const T>(q), rows_view<const T>(k),
                           rows_view<const T>(v), static_cast<T*>(c->k), static_cast<T*>(c->v), rows_view<T>(out), ws.o, ws.ml);
    };
    if (p.few) {
        if constexpr (D * sizeof(T) <= 128) {
            if (p.blocks() <= FEW_BLOCKS) run(k_chunk_few<T, D, 8>, 8);
            else run(k_chunk_few<T, D, 4>, 4);
        } else {
            run(k_chunk_few<T, D, 4>, 4);
        }
    } else run(k_chunk_many<T, D>, CW);
    if (p.want) {
        const int waves = p.few ? 1 : CW;
        hipLaunchKernelGGL((k_chunk_join<T, D>), dim3(grid.x, (unsigned)(waves * 32 * (D / 4) / JT)), dim3(JT), 0, s, a, pg, lo, p.cl,
                           p.kt, waves, ws.o, ws.ml, rows_view<T>(out));
    }
    return launch_status();
}

}  // namespace

extern "C" {

int rse_seqattn_chunk_workspace_size(const rse_seqattn* attn, int64_t n_events, int64_t batch, int64_t max_new, int64_t max_len,
                                     size_t* bytes_out) {
    if (!attn || !bytes_out || n_events < 0 || batch < 0 || max_new < 0 || max_len < 0) return RSE_ERR_INVALID_ARG;
    *bytes_out = n_events ? chunk_ws(attn, chunk_plan(attn, n_events, batch, max_new, max_len), nullptr).bytes : 0;
    return RSE_OK;
}

int seq_attention_chunk(const rse_seqattn* attn, rse_seqcache* cache, const rse_seq_batch* batch, const rse_seq_rows* q,
                        const rse_seq_rows* k, const rse_seq_rows* v, const int32_t* d_page_table, int32_t max_pages,
                        const int64_t* d_lens, int64_t max_len, const rse_seq_rows* out, void* d_ws, size_t ws_bytes,
                        void* stream) {
    int rc = batch_ok(attn, batch);
    if (rc) return rc;
    if (!cache || max_pages < 0 || max_len < 0 || batch->d_key_off) return RSE_ERR_INVALID_ARG;
    // users, and tiles of keys, are counted in 32 bits
    const int64_t most = INT64_C(1) << 35;
    if (batch->batch > INT32_MAX || (max_len > most && (int64_t)max_pages << cache->page_shift > most)) return RSE_ERR_UNSUPPORTED;
    if (attn->dim != cache->dim || attn->dtype != cache->dtype || attn->n_kv_heads != cache->n_kv_heads)
        return RSE_ERR_INVALID_ARG;
    if (batch->n_events == 0) return RSE_OK;
    if (!d_lens || (max_pages > 0 && !d_page_table)) return RSE_ERR_INVALID_ARG;
    for (const rse_seq_rows* r : {q, k, v})
        if (!rows_ok(r, attn->dtype)) return RSE_ERR_INVALID_ARG;
    if (!out_rows_ok(out, attn->dtype, batch->n_events, attn->n_heads, attn->dim)) return RSE_ERR_INVALID_ARG;
    const ChunkPlan plan = chunk_plan(attn, batch->n_events, batch->batch, batch->max_len, max_len);
    const ChunkWs ws = chunk_ws(attn, plan, d_ws);
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
    p.shift = cache->page_shift;
    p.max_len = max_len;
    return by_type(attn, [&](auto t, auto d) {
        return run_chunk<decltype(t), decltype(d)::value>(cache, a, p, plan, ws, q, k, v, out, as_stream(stream));
    });
}

}  // extern "C"
