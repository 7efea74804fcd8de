// rse_seqcache.hip -- the paged history cache of the sequence attention:
// page tables and slots from lengths, rows written into pages, and the
// attention of one new event per user over its cached history.
#include <new>

#include "rse_seqmma.h"

using namespace rse;
using namespace rse_host;

namespace {

constexpr int CB = 256;                 // threads per block

__global__ void k_cache_clear(SeqCacheHeader* h) { h->status = 0; }

// What the scan leaves for the kernels that fill the tables.
struct AssignWs {
    int64_t ok;
    int64_t pad[31];
    int64_t page_at[1];          // [batch] free-list position of each user's first new page
};

__device__ __forceinline__ int64_t pages_of(int64_t n, int shift) { return (n + (1ll << shift) - 1) >> shift; }

// The sum over the wave's lanes up to and with this one.
__device__ __forceinline__ int64_t wave_scan(int64_t x) {
#pragma unroll
    for (int m = 1; m < WAVE; m <<= 1) {
        const int64_t y = __shfl_up(x, m, WAVE);
        if (lane_id() >= m) x += y;
    }
    return x;
}

// One block: running sums of the counts and of the pages they need, SCAN_PER
// users a thread (4096 users: 16 us with one a thread and a scan through LDS, 9
// us so).
constexpr int SCAN_PER = 4;

__global__ __launch_bounds__(1024) void k_assign_scan(SeqCacheHeader* h, const int64_t* counts, const int64_t* lens,
                                                      int64_t batch, int shift, int64_t max_pages, int64_t n_free,
                                                      int64_t n_events, int64_t* offsets, int64_t* taken, AssignWs* ws) {
    __shared__ int64_t s_n[16], s_p[16];
    const int t = threadIdx.x, w = t / WAVE;
    int64_t base_n = 0, base_p = 0;
    bool bad = false;
    for (int64_t c = 0; c < batch; c += 1024 * SCAN_PER) {
        const int64_t b = c + t * SCAN_PER;
        int64_t len[SCAN_PER], cnt[SCAN_PER], n = 0, p = 0;
#pragma unroll
        for (int u = 0; u < SCAN_PER; ++u) {
            len[u] = b + u < batch ? lens[b + u] : 0;
            cnt[u] = b + u < batch ? counts[b + u] : 0;
        }
#pragma unroll
        for (int u = 0; u < SCAN_PER; ++u) {
            const int64_t room = max_pages << shift;
            if (len[u] < 0 || cnt[u] < 0 || len[u] > room || cnt[u] > room - len[u]) {
                bad = true;
                len[u] = cnt[u] = 0;
            }
            n += cnt[u];
            p += pages_of(len[u] + cnt[u], shift) - pages_of(len[u], shift);
        }
        const int64_t in_n = wave_scan(n), in_p = wave_scan(p);
        __syncthreads();                        // s_n, s_p of the last turn are no longer read
        if (lane_id() == WAVE - 1) {
            s_n[w] = in_n;
            s_p[w] = in_p;
        }
        __syncthreads();
        int64_t at_n = base_n + in_n - n, at_p = base_p + in_p - p;
        for (int x = 0; x < 16; ++x) {
            if (x < w) {
                at_n += s_n[x];
                at_p += s_p[x];
            }
            base_n += s_n[x];
            base_p += s_p[x];
        }
#pragma unroll
        for (int u = 0; u < SCAN_PER; ++u) {
            if (b + u < batch) {
                offsets[b + u] = at_n;
                ws->page_at[b + u] = at_p;
            }
            at_n += cnt[u];
            at_p += pages_of(len[u] + cnt[u], shift) - pages_of(len[u], shift);
        }
    }
    bad = __syncthreads_or(bad);
    if (t == 0) {
        offsets[batch] = base_n;
        int code = 0;
        if (bad || base_n != n_events) code = RSE_ERR_BAD_INPUT;
        else if (base_p > n_free) code = RSE_ERR_NEED_GROW;
        if (code) set_status(&h->status, code);
        ws->ok = code == 0;
        *taken = code ? 0 : base_p;
    }
}

// Slots, one event a thread, and the page table: the event that begins a page
// enters it.  The events of a wave mostly belong to one or two users: one
// search by the whole wave, then a step or two, or a search of the lane's own.
// An event on a page outside the pool gets no slot, and the page no entry.
__global__ __launch_bounds__(CB) void k_assign_slots(SeqCacheHeader* h, int64_t n_pages, const int64_t* lens, const int64_t* offsets, int64_t batch,
                                                     int shift, int32_t* table, int64_t max_pages,
                                                     const int32_t* free_pages, int64_t n_events, int64_t* slots,
                                                     const AssignWs* ws) {
    const bool ok = ws->ok != 0;
    for (int64_t i0 = (int64_t)blockIdx.x * CB; i0 < n_events; i0 += (int64_t)gridDim.x * CB) {
        const int64_t i = i0 + threadIdx.x, first = uniform(i0 + (int64_t)(threadIdx.x & ~(WAVE - 1)));
        if (!ok) {
            if (i < n_events) slots[i] = -1;
            continue;
        }
        int64_t b = wave_last_le(batch, [&](int64_t x) { return offsets[x]; }, first < n_events ? first : n_events - 1);
        if (i >= n_events) continue;
        for (int u = 0; u < 2 && b + 1 < batch && offsets[b + 1] <= i; ++u) ++b;
        if (b + 1 < batch && offsets[b + 1] <= i) {
            int64_t hi = batch - 1;
            while (b < hi) {
                const int64_t mid = (b + hi + 1) / 2;
                if (offsets[mid] <= i) b = mid;
                else hi = mid - 1;
            }
        }
        const int64_t len = lens[b], e = len + i - offsets[b], p = e >> shift, held = pages_of(len, shift);
        const int64_t in = e & ((1ll << shift) - 1);
        const int32_t page = p < held ? table[b * max_pages + p] : free_pages[ws->page_at[b] + p - held];
        if (page < 0 || page >= n_pages) {
            set_status(&h->status, RSE_ERR_BAD_INPUT);
            slots[i] = -1;
            continue;
        }
        if (in == 0) table[b * max_pages + p] = page;
        slots[i] = ((int64_t)page << shift) + in;
    }
}

// One 16-byte piece of a row per thread.
__global__ __launch_bounds__(CB) void k_cache_write(SeqCacheHeader* h, const int64_t* slots, int64_t n, Rows<const char> k,
                                                    Rows<const char> v, const int32_t* pos, char* kp, char* vp,
                                                    int32_t* tp, int64_t n_slots, int n_kv, int head_bytes) {
    const int pieces = head_bytes / 16, per = n_kv * pieces;
    const int64_t row = (int64_t)n_kv * head_bytes;
    for (int64_t x = (int64_t)blockIdx.x * CB + threadIdx.x; x < n * per; x += (int64_t)gridDim.x * CB) {
        const int64_t i = x / per;
        const int r = (int)(x - i * per), g = r / pieces, c = r - g * pieces;
        const int64_t s = slots[i];
        if (s < 0) continue;
        if (s >= n_slots) {
            set_status(&h->status, RSE_ERR_BAD_INPUT);
            continue;
        }
        gstore_u4(kp + s * row + (int64_t)r * 16, gload_u4(k.at(i, g) + c * 16));
        gstore_u4(vp + s * row + (int64_t)r * 16, gload_u4(v.at(i, g) + c * 16));
        if (r == 0) tp[s] = pos[i];
    }
}

struct StepArgs {
    SeqHeader* hdr;
    SeqCacheHeader* status;
    const int32_t* table;
    int64_t max_pages, n_pages, max_len;
    const int64_t* lens;
    const int32_t* pos;
    const float* bias;
    int32_t* tp;
    int32_t shift, n_heads, group, n_bounds;
    int64_t batch;
    float scale;
};

// The slot of event e of user b, or -1 (status set) for a page out of the pool.
__device__ __forceinline__ int64_t slot_of(const StepArgs& a, int64_t b, int64_t e) {
    const int64_t page = a.table[b * a.max_pages + (e >> a.shift)];
    if (page < 0 || page >= a.n_pages) {
        set_status(&a.status->status, RSE_ERR_BAD_INPUT);
        return -1;
    }
    return (page << a.shift) + (e & ((1ll << a.shift) - 1));
}

__device__ __forceinline__ bool step_ok(const StepArgs& a, int64_t n) {
    if (n < 0) return false;
    if (n >= a.max_len || (n >> a.shift) >= a.max_pages) {
        set_status(&a.status->status, RSE_ERR_BAD_INPUT);
        return false;
    }
    return true;
}

// A row's result from its sums.  Nothing seen: 0.  A score of NaN or +infinity
// has left l NaN, and stays.
__device__ __forceinline__ float over(float o, float l) { return l == 0.f ? 0.f : o / l; }

// One new event per user.  A block of SW waves takes the heads that share one
// key/value head (at most 32, as columns; column c is head h0 + c) and one of
// `splits` equal parts of a user's tiles of 32 events; its waves take tiles in
// turn, each from memory to its own registers and LDS, so that no wave waits
// for another: K rows are read as matrix operands straight from the page, V
// rows pass through the wave's LDS tile.  The waves' softmax sums are joined
// in LDS at the end; with more than one part, k_step_join joins the parts.
// The new event's own key and value are read from the call's arguments (no
// other block waits for the store that the first part makes).  bf16: the
// probabilities enter their product as pairs of bf16 values (2^-16 of each is
// lost), so that out is fp32 arithmetic rounded once.
constexpr int SW = 4;

// Registers are held to what lets STEP_WAVES waves share a SIMD.
template <typename T, int D>
constexpr int STEP_WAVES = D * sizeof(T) <= 128 ? 3 : (D * sizeof(T) == 256 ? 2 : 1);

template <typename T, int D>
__global__ __launch_bounds__(SW * 64) __attribute__((amdgpu_waves_per_eu(STEP_WAVES<T, D>))) void k_step(StepArgs a, Rows<const T> q, Rows<const T> k, Rows<const T> v, T* kp,
                                                  T* vp, Rows<T> out, int splits, int cols, float* part_o, float* part_ml) {
    using TL = Tile<T, D>;
    constexpr int CH = TL::CH, ND = D / 32, NC = CH / 2;
    extern __shared__ u32x4 s_mem[];            // SW tiles of V, then the waves' sums; s_bias [nb][cols]
    __shared__ int32_t s_bounds[RSE_SEQ_MAX_BOUNDARIES + 1];
    alignas(16) __shared__ int32_t s_idx[SW][32];       // (read by 16 bytes)
    __shared__ float s_ml[SW][2][32];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE), half = lane >> 5, col = lane & 31;
    const int n_kv = a.n_heads / a.group, nb = a.n_bounds + 1, blocks = (a.group + cols - 1) / cols;
    int64_t x = blockIdx.x;
    const int split = (int)(x % splits);
    x /= splits;
    const int cb = (int)(x % blocks);
    x /= blocks;
    const int g = (int)(x % n_kv);
    const int64_t b = x / n_kv;
    const int h0 = g * a.group + cb * cols, nc = a.group - cb * cols < cols ? a.group - cb * cols : cols;
    const int head = h0 + (col < nc ? col : nc - 1);
    u32x4* tile = s_mem + w * 32 * CH;
    const int tiles_bytes = SW * 32 * CH * 16, sums_bytes = SW * cols * D * 4;
    float* s_sum = reinterpret_cast<float*>(s_mem);
    float* s_bias = reinterpret_cast<float*>(reinterpret_cast<char*>(s_mem) + (tiles_bytes > sums_bytes ? tiles_bytes : sums_bytes));

    for (int t = threadIdx.x; t <= RSE_SEQ_MAX_BOUNDARIES; t += SW * 64) s_bounds[t] = a.hdr->bounds[t];
    for (int t = threadIdx.x; t < nb * cols; t += SW * 64) {
        const int c = t % cols;
        s_bias[t] = bias2(a.bias[(h0 + (c < nc ? c : nc - 1)) * nb + t / cols]);
    }
    int64_t n = uniform(a.lens[b]);
    if (!step_ok(a, n)) n = -1;
    const int64_t nt = (n + 32) / 32, t0 = nt * split / splits, t1 = nt * (split + 1) / splits;
    const int32_t my_pos = a.pos[b];
    const int64_t row_elems = (int64_t)n_kv * D;
    if (n >= 0 && split == 0 && cb == 0 && w == 0) {                // the new event into its page
        const int64_t s = slot_of(a, b, n);
        if (s >= 0) {
            const int c = lane < CH ? lane : 0;
            const u32x4 kv = gload_u4(k.at(b, g) + c * TL::EPC), vv = gload_u4(v.at(b, g) + c * TL::EPC);
            if (lane < CH) {
                gstore_u4(kp + s * row_elems + g * D + c * TL::EPC, kv);
                gstore_u4(vp + s * row_elems + g * D + c * TL::EPC, vv);
            }
            if (g == 0 && lane == 0) a.tp[s] = my_pos;
        }
    }
    __syncthreads();

    ColFrag<T, D> qf;
    qf.load(q.at(b, head), half);
    if (a.scale < 0.f) qf.negate();
    const float c2 = fabsf(a.scale) * LOG2E;

    // the lane's event of a tile: its page, then its rows and time
    auto page_of = [&](int64_t t) -> int64_t {
        const int64_t e = t * 32 + col;
        return t < t1 && e < n ? (int64_t)a.table[b * a.max_pages + (e >> a.shift)] : 0;
    };
    u32x4 rk[NC], rv[NC];
    int32_t rp = 0;
    bool see = false;
    auto load_rows = [&](int64_t t, int64_t page) {
        const int64_t e = t * 32 + col;
        const T *kr = k.at(b, g), *vr = v.at(b, g);     // the new event's, also for lanes that may not look
        rp = my_pos;
        see = e <= n;
        if (e < n) {
            if (page < 0 || page >= a.n_pages) {
                set_status(&a.status->status, RSE_ERR_BAD_INPUT);
                see = false;
            } else {
                const int64_t s = (page << a.shift) + (e & ((1ll << a.shift) - 1));
                kr = kp + s * row_elems + g * D;
                vr = vp + s * row_elems + g * D;
                rp = a.tp[s];
            }
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            rk[i] = gload_u4(kr + (2 * i + half) * TL::EPC);
            rv[i] = gload_u4(vr + (2 * i + half) * TL::EPC);
        }
    };

    f32x16 o[ND] = {};
    float m = -INFINITY, l = 0.f;
    int64_t t = t0 + w;
    int64_t page = page_of(t);
    if (t < t1) load_rows(t, page);
    page = page_of(t + SW);
    for (; t < t1; t += SW) {
        f32x16 s = {};
#pragma unroll
        for (int i = 0; i < NC; ++i) s = mma_chunk<T>(rk[i], qf.v[i], s);
#pragma unroll
        for (int i = 0; i < NC; ++i) tile[TL::chunk_at(col, 2 * i + half)] = see ? rv[i] : u32x4{0, 0, 0, 0};
        const bool hidden = __ballot(!see) != 0;
        const uint32_t seen = (uint32_t)__ballot(see);
        // the 32 events' buckets; all in one is the common case far back
        const int idx = seq_bucket(s_bounds, a.n_bounds, seq_dist(my_pos, rp));
        const int lo = __builtin_amdgcn_readfirstlane(idx);
        const bool one = __all(idx == lo);
        s_idx[w][col] = idx * cols;
        wave_lds_sync();
        if (t + SW < t1) load_rows(t + SW, page);
        page = page_of(t + 2 * SW);
        const int cc = col < nc ? col : nc - 1;
        if (one) {
            const float b0 = s_bias[lo * cols + cc];
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = __builtin_fmaf(s[r], c2, b0);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const i32x4 at = *reinterpret_cast<const i32x4*>(&s_idx[w][8 * j + 4 * half]);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[4 * j + i] = __builtin_fmaf(s[4 * j + i], c2, s_bias[at[i] + cc]);
            }
        }
        if (hidden) {
            const uint32_t bits = seen >> (4 * half);
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = (bits >> tile_row(r, 0)) & 1 ? s[r] : -INFINITY;
        }
        float top = s[0];
#pragma unroll
        for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
        top = fmaxf(top, other_half(top));
        const float ref = fmaxf(m, top);
        if (__any(ref > m)) {
            const float r = ref == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - ref);
            m = ref;
            l *= r;
#pragma unroll
            for (int dt = 0; dt < ND; ++dt) o[dt] *= r;
        }
        const float shift = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(s[r] - shift);
        l += sum_registers(s);
        OverRows<T, D>::add(o, tile, 0, s);
        wave_lds_sync();
    }
    l += other_half(l);
    if (half == 0) {
        s_ml[w][0][col] = m;
        s_ml[w][1][col] = l;
    }
    __syncthreads();                            // the V tiles are done with: their place takes the sums
    if (col < nc) {
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4*>(s_sum + (w * cols + col) * D + 32 * dt + 8 * j + 4 * half) =
                    f32x4{o[dt][4 * j], o[dt][4 * j + 1], o[dt][4 * j + 2], o[dt][4 * j + 3]};
    }
    __syncthreads();
    for (int y = threadIdx.x; y < nc * D; y += SW * 64) {
        const int c = y / D, d = y % D;
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int u = 0; u < SW; ++u) M = fmaxf(M, s_ml[u][0][c]);
        for (int u = 0; u < SW; ++u) {
            const float r = M == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(s_ml[u][0][c] - M);
            L = __builtin_fmaf(s_ml[u][1][c], r, L);
            O = __builtin_fmaf(s_sum[(u * cols + c) * D + d], r, O);
        }
        if (splits == 1) {
            from_f32(out.at(b, h0 + c)[d], over(O, L));
        } else {
            const int64_t at = (b * a.n_heads + h0 + c) * splits + split;
            part_o[at * D + d] = O;
            if (d == 0) {
                part_ml[2 * at] = M;
                part_ml[2 * at + 1] = L;
            }
        }
    }
}

// Sum over the LR lanes that share a row, in every one of them.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
    return x + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(x), CTRL, 0xF, 0xF, false));
}
template <int LR>
__device__ __forceinline__ float row_sum(float x) {
    x = dpp_add<0xB1>(x);                       // the other of a pair, the other pair of four,
    x = dpp_add<0x4E>(x);
    x = dpp_add<0x141>(x);                      // 8 mirrored, 16 mirrored
    if (LR >= 16) x = dpp_add<0x140>(x);
    if (LR >= 32) x += __shfl_xor(x, 16, WAVE);
    return x;
}

// The same in fp32 for few heads a key/value head.  Products of tiles would
// fill as few of the matrix cores' 32 columns, at 64 cycles for two of the
// summed elements; here LR = D / 4 lanes hold a row in 16-byte pieces, a wave
// FEW_LOADS loads of 64 / LR rows, and each lane multiplies its piece for all
// NH heads.  Each group of LR lanes keeps the softmax of the rows that it
// took; they are joined at the end.
constexpr int FEW_LOADS = 8;

template <int D, int NH>
__global__ __launch_bounds__(SW * 64) void k_step_few(StepArgs a, Rows<const float> q, Rows<const float> k,
                                                      Rows<const float> v, float* kp, float* vp, Rows<float> out,
                                                      int splits, float* part_o, float* part_ml) {
    constexpr int LR = D / 4, RG = WAVE / LR, NI = FEW_LOADS, TE = NI * RG;
    extern __shared__ float s_few[];            // bias in base 2 [nb][NH]
    __shared__ int32_t s_bounds[RSE_SEQ_MAX_BOUNDARIES + 1];
    __shared__ float s_ml[SW][2][NH];
    alignas(16) __shared__ float s_sum[SW][NH][D];      // (written by 16 bytes)
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE), piece = lane % LR, row = lane / LR;
    const int n_kv = a.n_heads / a.group, nb = a.n_bounds + 1, nc = a.group;
    int64_t x = blockIdx.x;
    const int split = (int)(x % splits);
    x /= splits;
    const int g = (int)(x % n_kv);
    const int64_t b = x / n_kv;
    const int h0 = g * nc;

    for (int t = threadIdx.x; t <= RSE_SEQ_MAX_BOUNDARIES; t += SW * 64) s_bounds[t] = a.hdr->bounds[t];
    for (int t = threadIdx.x; t < nb * NH; t += SW * 64) {
        const int c = t % NH;
        s_few[t] = bias2(a.bias[(h0 + (c < nc ? c : nc - 1)) * nb + t / NH]);
    }
    int64_t n = uniform(a.lens[b]);
    if (!step_ok(a, n)) n = -1;
    const int64_t nt = (n + TE) / TE, t0 = nt * split / splits, t1 = nt * (split + 1) / splits;
    const int32_t my_pos = a.pos[b];
    const int64_t row_elems = (int64_t)n_kv * D;
    const float *k_new = k.at(b, g) + piece * 4, *v_new = v.at(b, g) + piece * 4;
    if (n >= 0 && split == 0 && w == 0) {                           // the new event into its page
        const int64_t s = slot_of(a, b, n);
        if (s >= 0 && lane < LR) {
            gstore_u4(kp + s * row_elems + g * D + piece * 4, gload_u4(k_new));
            gstore_u4(vp + s * row_elems + g * D + piece * 4, gload_u4(v_new));
            if (g == 0 && lane == 0) a.tp[s] = my_pos;
        }
    }
    f32x4 qf[NH];
#pragma unroll
    for (int c = 0; c < NH; ++c)
        qf[c] = __builtin_bit_cast(f32x4, gload_u4(q.at(b, h0 + (c < nc ? c : nc - 1)) + piece * 4));
    const float c2 = a.scale * LOG2E;
    __syncthreads();

    // lane j < TE looks event j of a tile up: its page two tiles ahead, its
    // slot (-1: the new event's rows, also for lanes that may not look) and
    // time one ahead
    auto page_of = [&](int64_t t) -> int64_t {
        const int64_t e = t * TE + lane;
        return t < t1 && lane < TE && e < n ? (int64_t)a.table[b * a.max_pages + (e >> a.shift)] : 0;
    };
    int64_t slot = -1;
    int32_t rp = my_pos;
    bool see = false;
    auto look = [&](int64_t t, int64_t page) {
        const int64_t e = t * TE + lane;
        slot = -1;
        rp = my_pos;
        see = lane < TE && e <= n;
        if (t < t1 && lane < TE && e < n) {
            if (page < 0 || page >= a.n_pages) {
                set_status(&a.status->status, RSE_ERR_BAD_INPUT);
                see = false;
            } else {
                slot = (page << a.shift) + (e & ((1ll << a.shift) - 1));
                rp = a.tp[slot];
            }
        }
    };
    // a tile's rows, from each lane's piece of the pool
    const int64_t mine = (int64_t)g * D + piece * 4;
    auto load = [&](u32x4 (&r)[NI], const float* pool, const float* fresh, int64_t sl) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int64_t at = __shfl(sl, i * RG + row, WAVE);
            r[i] = gload_u4(at < 0 ? fresh : pool + at * row_elems + mine);
        }
    };

    f32x4 o[NH] = {};
    float m[NH], l[NH];
#pragma unroll
    for (int c = 0; c < NH; ++c) {
        m[c] = -INFINITY;
        l[c] = 0.f;
    }
    u32x4 rk[NI], rv[NI];
    int64_t t = t0 + w;
    if (t < t1) {
        look(t, page_of(t));
        load(rk, kp, k_new, slot);
    }
    int64_t page = page_of(t + SW);
    for (; t < t1; t += SW) {
        load(rv, vp, v_new, slot);
        const uint64_t seen = __ballot(see);
        const int idx = seq_bucket(s_bounds, a.n_bounds, seq_dist(my_pos, rp));
        const int lo = __builtin_amdgcn_readfirstlane(idx);
        const bool one = __all(idx == lo || lane >= TE);
        float s[NI][NH];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const f32x4 kk = __builtin_bit_cast(f32x4, rk[i]);
#pragma unroll
            for (int c = 0; c < NH; ++c) {
                float d = kk[0] * qf[c][0];
#pragma unroll
                for (int u = 1; u < 4; ++u) d = __builtin_fmaf(kk[u], qf[c][u], d);
                s[i][c] = row_sum<LR>(d);
            }
        }
        look(t + SW, page);
        page = page_of(t + 2 * SW);
        if (t + SW < t1) load(rk, kp, k_new, slot);
        if (one) {
#pragma unroll
            for (int c = 0; c < NH; ++c) {
                const float b0 = s_few[lo * NH + c];
#pragma unroll
                for (int i = 0; i < NI; ++i) s[i][c] = __builtin_fmaf(s[i][c], c2, b0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const float* bias = s_few + __shfl(idx, i * RG + row, WAVE) * NH;
#pragma unroll
                for (int c = 0; c < NH; ++c) s[i][c] = __builtin_fmaf(s[i][c], c2, bias[c]);
            }
        }
        if (seen != (TE == WAVE ? ~0ull : (1ull << (TE % WAVE)) - 1)) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const bool here = (seen >> (i * RG + row)) & 1;
                if (!here) rv[i] = u32x4{0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < NH; ++c) s[i][c] = here ? s[i][c] : -INFINITY;
            }
        }
#pragma unroll
        for (int c = 0; c < NH; ++c) {
            float top = s[0][c];
#pragma unroll
            for (int i = 1; i < NI; ++i) top = fmaxf(top, s[i][c]);
            const float ref = fmaxf(m[c], top);
            if (__any(ref > m[c])) {
                const float r = ref == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m[c] - ref);
                m[c] = ref;
                l[c] *= r;
                o[c] *= r;
            }
            const float shift = m[c] == -INFINITY ? 0.f : m[c];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const float p = __builtin_amdgcn_exp2f(s[i][c] - shift);
                const f32x4 vv = __builtin_bit_cast(f32x4, rv[i]);
                l[c] += p;
#pragma unroll
                for (int u = 0; u < 4; ++u) o[c][u] = __builtin_fmaf(p, vv[u], o[c][u]);
            }
        }
    }
    // the wave's groups of lanes, then its waves, then (k_step_join) the parts
#pragma unroll
    for (int c = 0; c < NH; ++c) {
        float M = m[c];
#pragma unroll
        for (int u = LR; u < WAVE; u *= 2) M = fmaxf(M, __shfl_xor(M, u, WAVE));
        const float r = M == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[c] - M);
        l[c] *= r;
        o[c] *= r;
#pragma unroll
        for (int u = LR; u < WAVE; u *= 2) {
            l[c] += __shfl_xor(l[c], u, WAVE);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[c][e] += __shfl_xor(o[c][e], u, WAVE);
        }
        if (lane < LR) *reinterpret_cast<f32x4*>(&s_sum[w][c][piece * 4]) = o[c];
        if (lane == 0) {
            s_ml[w][0][c] = M;
            s_ml[w][1][c] = l[c];
        }
    }
    __syncthreads();
    for (int y = threadIdx.x; y < nc * D; y += SW * 64) {
        const int c = y / D, d = y % D;
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int u = 0; u < SW; ++u) M = fmaxf(M, s_ml[u][0][c]);
        for (int u = 0; u < SW; ++u) {
            const float r = M == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(s_ml[u][0][c] - M);
            L = __builtin_fmaf(s_ml[u][1][c], r, L);
            O = __builtin_fmaf(s_sum[u][c][d], r, O);
        }
        if (splits == 1) {
            out.at(b, h0 + c)[d] = over(O, L);
        } else {
            const int64_t at = (b * a.n_heads + h0 + c) * splits + split;
            part_o[at * D + d] = O;
            if (d == 0) {
                part_ml[2 * at] = M;
                part_ml[2 * at + 1] = L;
            }
        }
    }
}

// Joins a head's parts: one block per user and head, CB / D groups of threads
// taking parts in turn, their sums added in order.
template <typename T, int D>
__global__ __launch_bounds__(CB) void k_step_join(const float* part_o, const float* part_ml, int n_heads, int splits,
                                                  Rows<T> out) {
    constexpr int G = CB / D;
    __shared__ float s_r[64], s_o[G][D];
    __shared__ float s_l;
    const int lane = lane_id(), d = threadIdx.x % D, grp = threadIdx.x / D;
    const int64_t at = blockIdx.x;
    float o = 0.f, v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {               // the first loads fly while the weights are formed
        const int s = grp + i * G;
        v[i] = s < splits ? part_o[(at * splits + s) * D + d] : 0.f;
    }
    if (threadIdx.x < WAVE) {
        const float m = lane < splits ? part_ml[2 * (at * splits + lane)] : -INFINITY;
        const float l = lane < splits ? part_ml[2 * (at * splits + lane) + 1] : 0.f;
        float M = m;
        for (int s = 32; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor(M, s, WAVE));
        const float r = M == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - M);
        float L = r * l;
        for (int s = 32; s > 0; s >>= 1) L += __shfl_xor(L, s, WAVE);
        s_r[lane] = r;
        if (lane == 0) s_l = L;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (grp + i * G < splits) o = __builtin_fmaf(s_r[grp + i * G], v[i], o);
#pragma unroll 4
    for (int s = grp + 4 * G; s < splits; s += G) o = __builtin_fmaf(s_r[s], part_o[(at * splits + s) * D + d], o);
    s_o[grp][d] = o;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
        for (int x = 1; x < G; ++x) o += s_o[x][d];
        from_f32(out.at(at / n_heads, at % n_heads)[d], over(o, s_l));
    }
}

// Parts of a history: 1024 blocks in all where histories are long enough (4 a
// CU, of which registers let 1 to 3 be there at once; 2048 and 4096 were no
// faster), a part of 256 events at least (two tiles a wave of k_step; of
// k_step_few one at 32 elements a head, else two or four), and at most the 64
// parts that k_step_join reads: one user on one key head keeps 64 CUs busy.
constexpr int64_t STEP_BLOCKS = 1024;

// fp32 heads a key/value head that k_step_few takes.  128 users of up to 2048
// events, one head to a key/value head, 4 of them, 64 (128) elements: 95 ->
// 50 us (232 -> 107), 4.9 TB/s; 4 heads to the only one: 37 -> 28 (80 -> 43);
// 8 heads: 38 -> 58 (82 -> 93), its registers leaving one wave a SIMD.  In
// bf16 a product of tiles takes an eighth of the time and is no bound.
constexpr int FEW_HEADS = 4;

struct StepPlan {
    int cols, blocks, splits;
};
StepPlan step_plan(const rse_seqattn* at, int64_t batch, int64_t max_len) {
    StepPlan p;
    const int group = at->n_heads / at->n_kv_heads;
    p.cols = group < 32 ? group : 32;
    p.blocks = (group + p.cols - 1) / p.cols;
    const int64_t units = batch * at->n_kv_heads * p.blocks;
    int64_t s = units > 0 ? (STEP_BLOCKS + units - 1) / units : 1;
    const int64_t most = max_len / (32 * SW * 2);
    if (s > most) s = most;
    p.splits = (int)(s < 1 ? 1 : (s > 64 ? 64 : s));
    return p;
}

struct StepWs {
    float* o;
    float* ml;
    size_t bytes;
};
StepWs step_ws(const rse_seqattn* at, int64_t batch, const StepPlan& p, void* base) {
    Carver c(base);
    const size_t n = p.splits > 1 ? (size_t)batch * at->n_heads * p.splits : 0;
    StepWs w;
    w.o = c.take<float>(n * at->dim);
    w.ml = c.take<float>(2 * n);
    w.bytes = c.size();
    return w;
}

template <typename T, int D>
int run_step(const rse_seqattn* at, const rse_seqcache* c, const StepArgs& a, const StepPlan& p, const StepWs& ws,
             const rse_seq_rows* q, const rse_seq_rows* k, const rse_seq_rows* v, const rse_seq_rows* out, hipStream_t s) {
    const size_t tiles = SW * 32 * D * sizeof(T), sums = (size_t)SW * p.cols * D * sizeof(float);
    const size_t lds = (tiles > sums ? tiles : sums) + (size_t)(a.n_bounds + 1) * p.cols * sizeof(float);
    const int64_t grid = a.batch * at->n_kv_heads * p.blocks * p.splits;
    if (grid > INT32_MAX) return RSE_ERR_UNSUPPORTED;
    const int few = std::is_same_v<T, float> && p.cols <= FEW_HEADS ? p.cols : 0;
    if constexpr (std::is_same_v<T, float>) {
        const auto run = [&](auto kernel, int heads) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(SW * WAVE), (a.n_bounds + 1) * heads * sizeof(float),
                               s, a, rows_view<const T>(q), rows_view<const T>(k), rows_view<const T>(v),
                               static_cast<T*>(c->k), static_cast<T*>(c->v), rows_view<T>(out), p.splits, ws.o, ws.ml);
        };
        if (few == 1) run(k_step_few<D, 1>, 1);
        if (few == 2) run(k_step_few<D, 2>, 2);
        if (few > 2) run(k_step_few<D, 4>, 4);
    }
    if (!few) {
        hipLaunchKernelGGL((k_step<T, D>), dim3((unsigned)grid), dim3(SW * WAVE), lds, s, a, rows_view<const T>(q),
                           rows_view<const T>(k), rows_view<const T>(v), static_cast<T*>(c->k), static_cast<T*>(c->v),
                           rows_view<T>(out), p.splits, p.cols, ws.o, ws.ml);
    }
    if (p.splits > 1) {
        hipLaunchKernelGGL((k_step_join<T, D>), dim3((unsigned)(a.batch * a.n_heads)), dim3(CB), 0, s, ws.o, ws.ml,
                           a.n_heads, p.splits, rows_view<T>(out));
    }
    return launch_status();
}

}  // namespace

extern "C" {

int rse_seqcache_meta_size(size_t* bytes_out) {
    if (!bytes_out) return RSE_ERR_INVALID_ARG;
    *bytes_out = sizeof(SeqCacheHeader);
    return RSE_OK;
}

int rse_seqcache_create(rse_seqcache** out, void* d_meta, size_t meta_bytes, void* d_k, void* d_v, int32_t* d_pos,
                        int64_t n_pages, int32_t page_size, int32_t n_kv_heads, int32_t dim, int32_t dtype,
                        void* stream) {
    if (!out || !d_meta || !d_k || !d_v || !d_pos) return RSE_ERR_INVALID_ARG;
    for (const void* p : {(const void*)d_k, (const void*)d_v, (const void*)d_pos})
        if (reinterpret_cast<uintptr_t>(p) % 16) return RSE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(d_meta) % 256) return RSE_ERR_INVALID_ARG;
    if (meta_bytes < sizeof(SeqCacheHeader)) return RSE_ERR_WORKSPACE;
    if (dtype != RSE_F32 && dtype != RSE_BF16) return RSE_ERR_INVALID_ARG;
    if (dim != 32 && dim != 64 && dim != 128) return RSE_ERR_UNSUPPORTED;
    if (n_kv_heads < 1 || n_kv_heads > RSE_SEQ_MAX_HEADS) return RSE_ERR_INVALID_ARG;
    if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1))) return RSE_ERR_UNSUPPORTED;
    if (n_pages < 1 || n_pages > INT32_MAX || n_pages * page_size > 1ll << 40) return RSE_ERR_INVALID_ARG;
    rse_seqcache* c = new (std::nothrow) rse_seqcache();
    if (!c) return RSE_ERR_INVALID_ARG;
    c->hdr = static_cast<SeqCacheHeader*>(d_meta);
    c->k = d_k;
    c->v = d_v;
    c->pos = d_pos;
    c->n_pages = n_pages;
    c->page_size = page_size;
    c->page_shift = __builtin_ctz(page_size);
    c->n_kv_heads = n_kv_heads;
    c->dim = dim;
    c->dtype = dtype;
    hipLaunchKernelGGL(k_cache_clear, dim3(1), dim3(1), 0, as_stream(stream), c->hdr);
    const int rc = launch_status();
    if (rc) {
        delete c;
        return rc;
    }
    *out = c;
    return RSE_OK;
}

int rse_seqcache_destroy(rse_seqcache* cache) {
    delete cache;
    return RSE_OK;
}

int rse_seqcache_status(rse_seqcache* cache, int32_t* status_out, void* stream) {
    if (!cache || !status_out) return RSE_ERR_INVALID_ARG;
    int32_t st = 0;
    if (hipMemcpyAsync(&st, &cache->hdr->status, sizeof(st), hipMemcpyDeviceToHost, as_stream(stream)) != hipSuccess)
        return RSE_ERR_HIP;
    if (hipStreamSynchronize(as_stream(stream)) != hipSuccess) return RSE_ERR_HIP;
    *status_out = st;
    return RSE_OK;
}

int rse_seqcache_clear_status(rse_seqcache* cache, void* stream) {
    if (!cache) return RSE_ERR_INVALID_ARG;
    hipLaunchKernelGGL(k_cache_clear, dim3(1), dim3(1), 0, as_stream(stream), cache->hdr);
    return launch_status();
}

int rse_seqcache_assign_workspace_size(int64_t batch, size_t* bytes_out) {
    if (!bytes_out || batch < 0) return RSE_ERR_INVALID_ARG;
    *bytes_out = align_up(sizeof(AssignWs) + (size_t)batch * sizeof(int64_t), 256);
    return RSE_OK;
}

int seq_cache_assign(rse_seqcache* cache, const int64_t* d_counts, const int64_t* d_lens, int64_t batch,
                     int32_t* d_page_table, int32_t max_pages, const int32_t* d_free, int64_t n_free,
                     int64_t n_events, int64_t* d_slots, int64_t* d_offsets, int64_t* d_taken, void* d_ws,
                     size_t ws_bytes, void* stream) {
    if (!cache || batch < 0 || max_pages < 0 || n_free < 0 || n_events < 0 || !d_offsets || !d_taken || !d_ws)
        return RSE_ERR_INVALID_ARG;
    if (batch > 0 && (!d_counts || !d_lens || (max_pages > 0 && !d_page_table))) return RSE_ERR_INVALID_ARG;
    if ((n_free > 0 && !d_free) || (n_events > 0 && !d_slots) || (n_events > 0 && batch == 0)) return RSE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(d_ws) % 256) return RSE_ERR_INVALID_ARG;
    size_t need = 0;
    rse_seqcache_assign_workspace_size(batch, &need);
    if (ws_bytes < need) return RSE_ERR_WORKSPACE;
    AssignWs* ws = static_cast<AssignWs*>(d_ws);
    hipStream_t s = as_stream(stream);
    const int shift = cache->page_shift;
    hipLaunchKernelGGL(k_assign_scan, dim3(1), dim3(1024), 0, s, cache->hdr, d_counts, d_lens, batch, shift,
                       (int64_t)max_pages, n_free, n_events, d_offsets, d_taken, ws);
    if (n_events > 0)
        hipLaunchKernelGGL(k_assign_slots, dim3(fill_blocks(n_events, CB, 4096)), dim3(CB), 0, s, cache->hdr,
                           cache->n_pages, d_lens, d_offsets, batch, shift, d_page_table, (int64_t)max_pages, d_free, n_events, d_slots, ws);
    return launch_status();
}

int seq_cache_write(rse_seqcache* cache, const int64_t* d_slots, int64_t n_events, const rse_seq_rows* k,
                    const rse_seq_rows* v, const int32_t* d_pos, void* stream) {
    if (!cache || n_events < 0) return RSE_ERR_INVALID_ARG;
    if (n_events == 0) return RSE_OK;
    if (!d_slots || !d_pos || !rows_ok(k, cache->dtype) || !rows_ok(v, cache->dtype)) return RSE_ERR_INVALID_ARG;
    const int e = cache->dtype == RSE_F32 ? 4 : 2, head_bytes = cache->dim * e;
    const Rows<const char> kr = {static_cast<const char*>(k->data), k->row_stride * e, k->head_stride * e};
    const Rows<const char> vr = {static_cast<const char*>(v->data), v->row_stride * e, v->head_stride * e};
    const int64_t items = n_events * cache->n_kv_heads * (head_bytes / 16);
    hipLaunchKernelGGL(k_cache_write, dim3(fill_blocks(items, CB, 16384)), dim3(CB), 0, as_stream(stream), cache->hdr,
                       d_slots, n_events, kr, vr, d_pos, static_cast<char*>(cache->k), static_cast<char*>(cache->v),
                       cache->pos, cache->n_pages << cache->page_shift, cache->n_kv_heads, head_bytes);
    return launch_status();
}

int rse_seqattn_step_workspace_size(const rse_seqattn* attn, int64_t batch, int64_t max_len, size_t* bytes_out) {
    if (!attn || !bytes_out || batch < 0 || max_len < 0) return RSE_ERR_INVALID_ARG;
    *bytes_out = step_ws(attn, batch, step_plan(attn, batch, max_len), nullptr).bytes;
    return RSE_OK;
}

int seq_attention_step(const rse_seqattn* attn, rse_seqcache* cache, const rse_seq_rows* q, const rse_seq_rows* k,
                       const rse_seq_rows* v, const int32_t* d_pos, const float* d_bias,
                       const int32_t* d_page_table, int32_t max_pages, const int64_t* d_lens, int64_t batch,
                       int64_t max_len, const rse_seq_rows* out, void* d_ws, size_t ws_bytes, void* stream) {
    if (!attn || !cache || batch < 0 || batch > INT32_MAX / RSE_SEQ_MAX_HEADS || max_len < 0 || max_pages < 0)
        return RSE_ERR_INVALID_ARG;
    if (attn->dim != cache->dim || attn->dtype != cache->dtype || attn->n_kv_heads != cache->n_kv_heads)
        return RSE_ERR_INVALID_ARG;
    if (batch == 0) return RSE_OK;
    if (!d_pos || !d_bias || !d_page_table || !d_lens) return RSE_ERR_INVALID_ARG;
    for (const rse_seq_rows* r : {q, k, v})
        if (!rows_ok(r, attn->dtype)) return RSE_ERR_INVALID_ARG;
    if (!out_rows_ok(out, attn->dtype, batch, attn->n_heads, attn->dim)) return RSE_ERR_INVALID_ARG;
    const StepPlan plan = step_plan(attn, batch, max_len);
    const StepWs ws = step_ws(attn, batch, plan, d_ws);
    if (ws_bytes < ws.bytes) return RSE_ERR_WORKSPACE;
    if (ws.bytes && (!d_ws || reinterpret_cast<uintptr_t>(d_ws) % 256)) return RSE_ERR_INVALID_ARG;
    StepArgs a;
    a.hdr = attn->hdr;
    a.status = cache->hdr;
    a.table = d_page_table;
    a.max_pages = max_pages;
    a.n_pages = cache->n_pages;
    a.max_len = max_len;
    a.lens = d_lens;
    a.pos = d_pos;
    a.bias = d_bias;
    a.tp = cache->pos;
    a.shift = cache->page_shift;
    a.n_heads = attn->n_heads;
    a.group = attn->n_heads / attn->n_kv_heads;
    a.n_bounds = attn->n_bounds;
    a.batch = batch;
    a.scale = attn->scale;
    hipStream_t s = as_stream(stream);
    return by_type(attn, [&](auto t, auto d) {
        return run_step<decltype(t), decltype(d)::value>(attn, cache, a, plan, ws, q, k, v, out, s);
    });
}

}  // extern "C"
