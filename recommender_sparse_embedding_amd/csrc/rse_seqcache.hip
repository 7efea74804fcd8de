// rse_seqcache.hip -- the paged history cache of the sequence attention:
// page tables and slots from lengths, rows written into pages, and the
// attention of one new event per user over its cached history.
#include <new>

#include "rse_seq.h"

using namespace rse;
using namespace rse_host;

namespace {

constexpr int CB = 256;                 // threads per block
constexpr int CW = CB / WAVE;

__global__ void k_cache_clear(SeqCacheHeader* h) { h->status = 0; }

// What the scan leaves for the kernels that fill the tables.
struct AssignWs {
    int64_t ok;
    int64_t pad[31];
    int64_t page_at[1];          // [batch] free-list position of each user's first new page
};

__device__ __forceinline__ int64_t pages_of(int64_t n, int shift) { return (n + (1ll << shift) - 1) >> shift; }

// One block: running sums of the counts and of the pages they need.
__global__ __launch_bounds__(1024) void k_assign_scan(SeqCacheHeader* h, const int64_t* counts, const int64_t* lens,
                                                      int64_t batch, int shift, int64_t max_pages, int64_t n_free,
                                                      int64_t n_events, int64_t* offsets, int64_t* taken, AssignWs* ws) {
    __shared__ int64_t s_n[1024], s_p[1024];
    __shared__ int s_bad;
    const int t = threadIdx.x;
    if (t == 0) s_bad = 0;
    int64_t base_n = 0, base_p = 0;
    bool bad = false;
    for (int64_t c = 0; c < batch; c += 1024) {
        const int64_t b = c + t;
        int64_t n = 0, p = 0;
        if (b < batch) {
            const int64_t len = lens[b], cnt = counts[b];
            if (len < 0 || cnt < 0 || len > (max_pages << shift) || cnt > (max_pages << shift) - len) bad = true;
            else {
                n = cnt;
                p = pages_of(len + cnt, shift) - pages_of(len, shift);
            }
        }
        s_n[t] = n;
        s_p[t] = p;
        __syncthreads();
        for (int d = 1; d < 1024; d <<= 1) {
            const int64_t xn = t >= d ? s_n[t - d] : 0, xp = t >= d ? s_p[t - d] : 0;
            __syncthreads();
            s_n[t] += xn;
            s_p[t] += xp;
            __syncthreads();
        }
        if (b < batch) {
            offsets[b] = base_n + s_n[t] - n;
            ws->page_at[b] = base_p + s_p[t] - p;
        }
        base_n += s_n[1023];
        base_p += s_p[1023];
        __syncthreads();
    }
    if (bad) s_bad = 1;
    __syncthreads();
    if (t == 0) {
        offsets[batch] = base_n;
        int code = 0;
        if (s_bad || base_n != n_events) code = RSE_ERR_BAD_INPUT;
        else if (base_p > n_free) code = RSE_ERR_NEED_GROW;
        if (code) set_status(&h->status, code);
        ws->ok = code == 0;
        *taken = code ? 0 : base_p;
    }
}

__global__ __launch_bounds__(CB) void k_assign_pages(const int64_t* counts, const int64_t* lens, int64_t batch,
                                                     int shift, int32_t* table, int64_t max_pages,
                                                     const int32_t* free_pages, const AssignWs* ws) {
    if (!ws->ok) return;
    const int lane = lane_id();
    for (int64_t b = (int64_t)blockIdx.x * CW + threadIdx.x / WAVE; b < batch; b += (int64_t)gridDim.x * CW) {
        const int64_t first = pages_of(lens[b], shift), n = pages_of(lens[b] + counts[b], shift) - first;
        for (int64_t p = lane; p < n; p += WAVE) table[b * max_pages + first + p] = free_pages[ws->page_at[b] + p];
    }
}

__global__ __launch_bounds__(CB) void k_assign_slots(const int64_t* lens, const int64_t* offsets, int64_t batch,
                                                     int shift, const int32_t* table, int64_t max_pages,
                                                     int64_t n_events, int64_t* slots, const AssignWs* ws) {
    const bool ok = ws->ok != 0;
    for (int64_t i = (int64_t)blockIdx.x * CB + threadIdx.x; i < n_events; i += (int64_t)gridDim.x * CB) {
        if (!ok) {
            slots[i] = -1;
            continue;
        }
        int64_t lo = 0, hi = batch - 1;      // the last user whose first event is <= i
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if (offsets[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        const int64_t e = lens[lo] + i - offsets[lo];
        slots[i] = ((int64_t)table[lo * max_pages + (e >> shift)] << shift) + (e & ((1ll << shift) - 1));
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

template <typename T>
__global__ __launch_bounds__(CB) void k_step_append(StepArgs a, Rows<const T> k, Rows<const T> v, T* kp, T* vp, int n_kv,
                                                    int dim) {
    const int64_t b = blockIdx.x, n = a.lens[b];
    if (!step_ok(a, n)) return;
    const int64_t s = slot_of(a, b, n);
    if (s < 0) return;
    for (int x = threadIdx.x; x < n_kv * dim; x += CB) {
        kp[s * n_kv * dim + x] = k.at(b, x / dim)[x % dim];
        vp[s * n_kv * dim + x] = v.at(b, x / dim)[x % dim];
    }
    if (threadIdx.x == 0) a.tp[s] = a.pos[b];
}

// One wave per user and query head, 64 events at a time.
template <typename T, int D>
__global__ __launch_bounds__(CB) void k_step(StepArgs a, Rows<const T> q, const T* kp, const T* vp, Rows<T> out) {
    __shared__ int32_t bounds[RSE_SEQ_MAX_BOUNDARIES + 1];
    __shared__ float sq[CW][D];
    for (int t = threadIdx.x; t <= RSE_SEQ_MAX_BOUNDARIES; t += CB) bounds[t] = a.hdr->bounds[t];
    __syncthreads();
    constexpr int E = (D + WAVE - 1) / WAVE;
    const int lane = lane_id(), w = threadIdx.x / WAVE, n_kv = a.n_heads / a.group;
    const int64_t it = (int64_t)blockIdx.x * CW + w;
    if (it >= a.batch * a.n_heads) return;
    const int64_t b = it / a.n_heads;
    const int h = (int)(it % a.n_heads), g = h / a.group;
    const int64_t n = a.lens[b];
    float m = -INFINITY, l = 0.f, acc[E] = {};
    if (step_ok(a, n)) {
        for (int d = lane; d < D; d += WAVE) sq[w][d] = to_f32(q.at(b, h)[d]);
        wave_lds_sync();
        for (int64_t c = 0; c <= n; c += WAVE) {
            const int64_t e = c + lane;
            float x = -INFINITY;
            const int64_t s = e <= n ? slot_of(a, b, e) : -1;
            if (s >= 0) {
                const T* row = kp + (s * n_kv + g) * D;
                float dot = 0.f;
                for (int d = 0; d < D; ++d) dot = __fmaf_rn(sq[w][d], to_f32(row[d]), dot);
                x = dot * a.scale +
                    a.bias[h * (a.n_bounds + 1) + seq_bucket(bounds, a.n_bounds, seq_dist(a.pos[b], a.tp[s]))];
            }
            float top = x;
            for (int k = 32; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor(top, k, WAVE));
            top = fmaxf(top, m);
            if (top == -INFINITY) continue;
            const float p = expf(x - top), r = expf(m - top);
            float sum = p;
            for (int k = 32; k > 0; k >>= 1) sum += __shfl_xor(sum, k, WAVE);
            l = l * r + sum;
            m = top;
#pragma unroll
            for (int u = 0; u < E; ++u) acc[u] *= r;
            for (int t = 0; t < WAVE; ++t) {
                const int64_t st = __shfl(s, t, WAVE);
                if (st < 0) continue;
                const float pt = __shfl(p, t, WAVE);
#pragma unroll
                for (int u = 0; u < E; ++u)
                    if (u * WAVE + lane < D)
                        acc[u] = __fmaf_rn(pt, to_f32(vp[(st * n_kv + g) * D + u * WAVE + lane]), acc[u]);
            }
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int u = 0; u < E; ++u)
        if (u * WAVE + lane < D) from_f32(out.at(b, h)[u * WAVE + lane], acc[u] * inv);
}

template <typename T, int D>
int run_step(const rse_seqcache* c, const StepArgs& a, const rse_seq_rows* q, const rse_seq_rows* k,
             const rse_seq_rows* v, const rse_seq_rows* out, hipStream_t s) {
    T* kp = static_cast<T*>(c->k);
    T* vp = static_cast<T*>(c->v);
    hipLaunchKernelGGL(k_step_append<T>, dim3((unsigned)a.batch), dim3(CB), 0, s, a, rows_view<const T>(k),
                       rows_view<const T>(v), kp, vp, c->n_kv_heads, c->dim);
    hipLaunchKernelGGL((k_step<T, D>), dim3((unsigned)((a.batch * a.n_heads + CW - 1) / CW)), dim3(CB), 0, s, a,
                       rows_view<const T>(q), kp, vp, rows_view<T>(out));
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
    if (n_pages < 1 || n_pages > INT32_MAX) return RSE_ERR_INVALID_ARG;
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
    if (batch > 0)
        hipLaunchKernelGGL(k_assign_pages, dim3(fill_blocks(batch, CW, 2048)), dim3(CB), 0, s, d_counts, d_lens, batch,
                           shift, d_page_table, (int64_t)max_pages, d_free, ws);
    if (n_events > 0)
        hipLaunchKernelGGL(k_assign_slots, dim3(fill_blocks(n_events, CB, 2048)), dim3(CB), 0, s, d_lens, d_offsets,
                           batch, shift, d_page_table, (int64_t)max_pages, n_events, d_slots, ws);
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
    *bytes_out = 256;
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
    if (!d_pos || !d_bias || !d_page_table || !d_lens || !d_ws) return RSE_ERR_INVALID_ARG;
    for (const rse_seq_rows* r : {q, k, v, out})
        if (!rows_ok(r, attn->dtype)) return RSE_ERR_INVALID_ARG;
    size_t need = 0;
    rse_seqattn_step_workspace_size(attn, batch, max_len, &need);
    if (ws_bytes < need) return RSE_ERR_WORKSPACE;
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
    const bool f = attn->dtype == RSE_F32;
    switch (attn->dim) {
        case 32: return f ? run_step<float, 32>(cache, a, q, k, v, out, s) : run_step<uint16_t, 32>(cache, a, q, k, v, out, s);
        case 64: return f ? run_step<float, 64>(cache, a, q, k, v, out, s) : run_step<uint16_t, 64>(cache, a, q, k, v, out, s);
        default: return f ? run_step<float, 128>(cache, a, q, k, v, out, s) : run_step<uint16_t, 128>(cache, a, q, k, v, out, s);
    }
}

}  // extern "C"
