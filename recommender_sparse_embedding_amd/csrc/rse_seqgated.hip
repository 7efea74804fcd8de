// rse_seqgated.hip -- the gated feed-forward's two projections, activation and
// product in one kernel, and their backward.
//
//   out = act(g) u,  g = x Wg^T,  u = x Wu^T
//   dg = dout u act'(g),  du = dout act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// All five are tiled matrix products on the matrix cores with fp32 sums.  The
// backward forms g and u anew (4 dim operations a hidden element) instead of
// reading them back in fp32 (8 bytes, and 8 to write): 0.9 ps against 3.3 ps at
// dim 256.  dg and du pass through the workspace in the rows' type.
#include "rse_seqmma.h"

using namespace rse;
using namespace rse_host;

namespace {

constexpr int GT = 256;                 // threads of a block: 4 waves, 2 by 2
constexpr int TILE = 128;               // rows and columns of a block's tile
constexpr int KB = 128;                 // bytes of the contraction a step: 64 bf16, 32 fp32
constexpr int KCH = KB / 16;

template <typename T>
struct Mat {
    T* p;
    int64_t stride;
    __device__ __forceinline__ T* row(int64_t i) const { return p + i * stride; }
};

template <typename T>
constexpr int EPC = 16 / (int)sizeof(T);
template <typename T>
constexpr int KT = KB / (int)sizeof(T);

// ------------------------------------------------------------- operands --
// A block's operand of TILE rows (of the result) by KT<T> of the contraction,
// on its way from memory through registers to LDS, and read from there as
// matrix operands: 16 bytes a lane, of row `lane % 32` the elements
// 8 s' + 4 (lane / 32) .. of step s in fp32, 16 s + 8 (lane / 32) .. in bf16.
// Pieces past an end are zeros.
constexpr int PER = TILE * KCH / GT;

// Rows of the result are rows in memory: the contraction is contiguous.
template <typename T, typename F>
struct AlongRows {
    using TL = Tile<T, KT<T>>;
    F row_at;                           // pointer of tile row r, or null past the end
    int64_t k_end;
    u32x4 x[PER];
    uint32_t in;
    __device__ __forceinline__ void load(int64_t k0) {
        in = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = i * GT + threadIdx.x, r = t / KCH, c = t % KCH;
            const T* p = row_at(r);
            const int64_t k = k0 + c * EPC<T>;
            const bool ok = p && k < k_end;
            x[i] = u32x4{0, 0, 0, 0};
            if (ok) x[i] = gload_u4(p + k);
        }
    }
    __device__ __forceinline__ void store(u32x4* lds) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = i * GT + threadIdx.x;
            lds[TL::chunk_at(t / KCH, t % KCH)] = x[i];
        }
    }
    static __device__ __forceinline__ u32x4 frag(const u32x4* lds, int r0, int s) {
        const int lane = lane_id();
        return lds[TL::chunk_at(r0 + (lane & 31), 2 * s + (lane >> 5))];
    }
};

// Rows of the result are columns in memory: one row in memory a step of the
// contraction.
template <typename T, typename F>
struct AcrossRows {
    using TL = Tile<T, TILE>;
    F k_row;                            // pointer of the row of contraction index k
    int64_t k_end;
    int cols;                           // of the tile, that exist
    u32x4 x[PER];
    __device__ __forceinline__ void load(int64_t k0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = i * GT + threadIdx.x, c = t % TL::CH;
            const int64_t k = k0 + t / TL::CH;
            x[i] = u32x4{0, 0, 0, 0};
            if (k < k_end && c * EPC<T> < cols) x[i] = gload_u4(k_row(k) + c * EPC<T>);
        }
    }
    __device__ __forceinline__ void store(u32x4* lds) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = i * GT + threadIdx.x;
            lds[TL::chunk_at(t / TL::CH, t % TL::CH)] = x[i];
        }
    }
    static __device__ __forceinline__ u32x4 frag(const u32x4* lds, int r0, int s) {
        const int lane = lane_id(), h = lane >> 5;
        u32x4 a;
        if constexpr (sizeof(T) == 4) {
            const float* f = reinterpret_cast<const float*>(lds);
            const int c = r0 + (lane & 31);
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = __float_as_uint(f[TL::chunk_at(8 * s + 4 * h + e, c >> 2) * 4 + (c & 3)]);
        } else {
            // four rows of a column at a time by the transposing read (see OverRows)
            const int i = lane & 15, c = r0 / 8 + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
            s16x4 p[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int row = 16 * s + 8 * h + 4 * u + (i >> 2);
                const char* at = reinterpret_cast<const char*>(lds) + TL::chunk_at(row, c) * 16 + (i & 1) * 8;
                p[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((RSE_LDS s16x4*)at);
            }
            a.xy = __builtin_bit_cast(u32x2, p[0]);
            a.zw = __builtin_bit_cast(u32x2, p[1]);
        }
        return a;
    }
};

// acc[j][i] += P rows p0 + p_step j .. times Q rows q0 + 32 i .., over the
// contraction from k0 to k1.  Two buffers in LDS: the next step's pieces fly
// while the current one is multiplied.
template <typename T, typename P, typename Q>
__device__ __forceinline__ void multiply(P& p, Q& q, int64_t k0, int64_t k1, int p0, int p_step, int q0, f32x16 (&acc)[2][2],
                                         u32x4 (*lds)[2][TILE * KCH]) {
    if (k0 >= k1) return;
    p.load(k0);
    q.load(k0);
    for (int b = 0; k0 < k1; k0 += KT<T>, b ^= 1) {
        p.store(lds[b][0]);
        q.store(lds[b][1]);
        __syncthreads();
        if (k0 + KT<T> < k1) {
            p.load(k0 + KT<T>);
            q.load(k0 + KT<T>);
        }
#pragma unroll
        for (int s = 0; s < KCH / 2; ++s) {
            u32x4 a[2], c[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) a[j] = P::frag(lds[b][0], p0 + j * p_step, s);
#pragma unroll
            for (int i = 0; i < 2; ++i) c[i] = Q::frag(lds[b][1], q0 + 32 * i, s);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) acc[j][i] = mma_chunk<T>(a[j], c[i], acc[j][i]);
        }
    }
}

// Elements of the lane's row from registers, 16 bytes a store: acc's register
// r is element tile_row(r, half) of p[0 .. 31]; pieces at `left` and on do not exist.
__device__ __forceinline__ void put_column(float* p, const f32x16& acc, int64_t left) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (8 * j + 4 * h < left) gstore_f4(p + 8 * j + 4 * h, f32x4{acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]});
}
__device__ __forceinline__ void put_column(uint16_t* p, const f32x16& acc, int64_t left) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        u32x4 o;                                // (the exchange of store_column)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x2 s = __builtin_amdgcn_permlane32_swap(pack_bf16(acc[4 * j + 2 * i], acc[4 * j + 2 * i + 1]),
                                                             pack_bf16(acc[4 * j + 4 + 2 * i], acc[4 * j + 5 + 2 * i]), false, false);
            o[i] = s.x;
            o[2 + i] = s.y;
        }
        if (8 * (j + h) < left) gstore_u4(p + 8 * (j + h), o);
    }
}
// The same elements read; 0 past the end (and where the row does not exist).
__device__ __forceinline__ void get_column(const float* p, f32x16& x, int64_t left) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (8 * j + 4 * h < left) v = gload_f4(p + 8 * j + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * j + i] = v[i];
    }
}
__device__ __forceinline__ void get_column(const uint16_t* p, f32x16& x, int64_t left) {
    const int h = lane_id() >> 5;
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        u32x4 o = {0, 0, 0, 0};
        if (8 * (j + h) < left) o = gload_u4(p + 8 * (j + h));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x2 s = __builtin_amdgcn_permlane32_swap(o[i], o[2 + i], false, false);
            x[4 * j + 2 * i] = __uint_as_float(s.x << 16);
            x[4 * j + 2 * i + 1] = __uint_as_float(s.x & 0xFFFF0000u);
            x[4 * j + 4 + 2 * i] = __uint_as_float(s.y << 16);
            x[4 * j + 5 + 2 * i] = __uint_as_float(s.y & 0xFFFF0000u);
        }
    }
}

// act(g) and act'(g).
__device__ __forceinline__ void activate(int act, float g, float& a, float& da) {
    if (act == RSE_GELU) {
        const float cdf = 0.5f * erfcf(g * -0.70710678118654752f);
        a = g * cdf;
        da = __builtin_fmaf(g * 0.39894228040143268f, __builtin_amdgcn_exp2f(g * g * (-0.5f * LOG2E)), cdf);
    } else {
        const float s = 1.f / (1.f + __builtin_amdgcn_exp2f(-LOG2E * g)), t = s - s * s;
        a = act == RSE_SILU ? g * s : s;
        da = act == RSE_SILU ? __builtin_fmaf(g, t, s) : t;
    }
}

// Block x's tile of a grid of `total`: blocks of one XCD (x % 8) take
// consecutive ones, so that what they share stays in its L2.
__device__ __forceinline__ int64_t xcd_tile(int64_t x, int64_t total) {
    const int64_t per = total / 8, rest = total % 8, xcd = x % 8;
    return xcd * per + (xcd < rest ? xcd : rest) + x / 8;
}

struct GatedArgs {
    int64_t n;
    int32_t dim, hidden, act;
};

// out (BWD: dg beside du) of TILE rows by TILE / 2 hidden elements: the tile's
// P rows are TILE / 2 rows of Wg, then the same ones of Wu, and a wave's
// accumulators hold g and u of the same elements.
template <typename T, bool BWD>
__global__ __launch_bounds__(GT) void k_gated(GatedArgs a, Mat<const T> x, Mat<const T> wg, Mat<const T> wu,
                                              Mat<const T> dout, Mat<T> out) {
    constexpr int HT = TILE / 2;
    __shared__ u32x4 lds[2][2][TILE * KCH];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE);
    const int64_t ht = (a.hidden + HT - 1) / HT, tile = xcd_tile(blockIdx.x, gridDim.x);
    const int64_t r0 = tile / ht * TILE;
    const int h0 = (int)(tile % ht) * HT;
    auto w_row = [&](int r) -> const T* {
        const int h = h0 + r % HT;
        return h < a.hidden ? (r < HT ? wg.row(h) : wu.row(h)) : nullptr;
    };
    auto x_row = [&](int r) -> const T* { return r0 + r < a.n ? x.row(r0 + r) : nullptr; };
    AlongRows<T, decltype(w_row)> p = {w_row, a.dim};
    AlongRows<T, decltype(x_row)> q = {x_row, a.dim};
    f32x16 acc[2][2] = {};
    const int hw = 32 * (w & 1), qw = 64 * (w >> 1);
    multiply<T>(p, q, 0, a.dim, hw, HT, qw, acc, lds);
    const int64_t left = a.hidden - h0 - hw;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t r = r0 + qw + 32 * i + (lane & 31);
        f32x16 &g = acc[0][i], &u = acc[1][i];
        if constexpr (BWD) {
            f32x16 d;
            get_column(dout.row(r < a.n ? r : a.n - 1) + h0 + hw, d, left);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float f, df;
                activate(a.act, g[e], f, df);
                g[e] = d[e] * u[e] * df;
                u[e] = d[e] * f;
            }
            const int64_t there = r < a.n ? left : 0;
            put_column(out.row(r < a.n ? r : 0) + h0 + hw, g, there);
            put_column(out.row(r < a.n ? r : 0) + a.hidden + h0 + hw, u, there);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float f, df;
                activate(a.act, g[e], f, df);
                g[e] = f * u[e];
            }
            put_column(out.row(r < a.n ? r : 0) + h0 + hw, g, r < a.n ? left : 0);
        }
    }
}

// dx = [dg du] [Wg; Wu].
template <typename T>
__global__ __launch_bounds__(GT) void k_gated_dx(GatedArgs a, Mat<const T> d, Mat<const T> wg, Mat<const T> wu, Mat<T> dx) {
    __shared__ u32x4 lds[2][2][TILE * KCH];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE);
    const int64_t ct = (a.dim + TILE - 1) / TILE, tile = xcd_tile(blockIdx.x, gridDim.x);
    const int64_t r0 = tile / ct * TILE;
    const int c0 = (int)(tile % ct) * TILE;
    auto w_row = [&](int64_t k) -> const T* { return (k < a.hidden ? wg.row(k) : wu.row(k - a.hidden)) + c0; };
    auto d_row = [&](int r) -> const T* { return r0 + r < a.n ? d.row(r0 + r) : nullptr; };
    AcrossRows<T, decltype(w_row)> p = {w_row, 2ll * a.hidden, a.dim - c0};
    AlongRows<T, decltype(d_row)> q = {d_row, 2ll * a.hidden};
    f32x16 acc[2][2] = {};
    const int pw = 64 * (w & 1), qw = 64 * (w >> 1);
    multiply<T>(p, q, 0, 2ll * a.hidden, pw, 32, qw, acc, lds);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t r = r0 + qw + 32 * i + (lane & 31);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = c0 + pw + 32 * j;
            put_column(dx.row(r < a.n ? r : 0) + c, acc[j][i], r < a.n ? a.dim - c : 0);
        }
    }
}

// Part s of [dWg; dWu] = [dg du]^T x: the rows from s `rows` on.
template <typename T>
__global__ __launch_bounds__(GT) void k_gated_dw(GatedArgs a, Mat<const T> d, Mat<const T> x, int64_t rows, float* part) {
    __shared__ u32x4 lds[2][2][TILE * KCH];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE);
    const int64_t ct = (a.dim + TILE - 1) / TILE, ht = (2ll * a.hidden + TILE - 1) / TILE;
    int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
    const int c0 = (int)(tile % ct) * TILE;
    tile /= ct;
    const int h0 = (int)(tile % ht) * TILE;
    const int64_t s = tile / ht, k0 = s * rows, k1 = k0 + rows < a.n ? k0 + rows : a.n;
    auto x_row = [&](int64_t k) -> const T* { return x.row(k) + c0; };
    auto d_row = [&](int64_t k) -> const T* { return d.row(k) + h0; };
    AcrossRows<T, decltype(x_row)> p = {x_row, k1, a.dim - c0};
    AcrossRows<T, decltype(d_row)> q = {d_row, k1, 2 * a.hidden - h0};
    f32x16 acc[2][2] = {};
    const int pw = 64 * (w & 1), qw = 64 * (w >> 1);
    multiply<T>(p, q, k0, k1, pw, 32, qw, acc, lds);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t h = h0 + qw + 32 * i + (lane & 31);
        const bool in = h < 2ll * a.hidden;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = c0 + pw + 32 * j;
            put_column(part + ((s * 2 * a.hidden + (in ? h : 0)) * a.dim + c), acc[j][i], in ? a.dim - c : 0);
        }
    }
}

// The parts added, rounded once: four elements a thread.
template <typename T>
__global__ __launch_bounds__(GT) void k_gated_dw_join(GatedArgs a, const float* part, int splits, Mat<T> dwg, Mat<T> dwu) {
    const int64_t size = 2ll * a.hidden * a.dim;
    for (int64_t t = 4 * ((int64_t)blockIdx.x * GT + threadIdx.x); t < size; t += 4ll * GT * gridDim.x) {
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int s = 0; s < splits; ++s) o += gload_f4(part + s * size + t);
        const int64_t h = t / a.dim;
        const int c = (int)(t - h * a.dim);
        store_four((h < a.hidden ? dwg.row(h) : dwu.row(h - a.hidden)) + c, o);
    }
}

// ------------------------------------------------------------------ host --
bool mat_ok(const rse_seq_mat* m, int32_t dtype) {
    return m && m->data && reinterpret_cast<uintptr_t>(m->data) % 16 == 0 && m->stride % (dtype == RSE_F32 ? 4 : 8) == 0;
}
bool out_mat_ok(const rse_seq_mat* m, int32_t dtype, int64_t n, int64_t width) {
    return mat_ok(m, dtype) && (n <= 1 || m->stride >= width || -m->stride >= width);
}
template <typename T>
Mat<T> view(const rse_seq_mat* m) {
    return {static_cast<T*>(m->data), m->stride};
}

int gated_args(int64_t n, int32_t dim, int32_t hidden, int32_t dtype) {
    if (n < 0 || dim < 1 || hidden < 1 || (dtype != RSE_F32 && dtype != RSE_BF16)) return RSE_ERR_INVALID_ARG;
    const int per16 = dtype == RSE_F32 ? 4 : 8;
    if (dim % per16 || hidden % per16 || dim > RSE_SEQ_MAX_GATED || hidden > RSE_SEQ_MAX_GATED) return RSE_ERR_UNSUPPORTED;
    return RSE_OK;
}

// Parts of the events for dW: 512 blocks in all (two a CU), parts of whole
// steps, 512 events at least.
struct DwPlan {
    int splits;
    int64_t rows;
};
DwPlan dw_plan(int64_t n, int32_t dim, int32_t hidden) {
    const int64_t tiles = (int64_t)((dim + TILE - 1) / TILE) * ((2ll * hidden + TILE - 1) / TILE);
    int64_t s = (512 + tiles - 1) / tiles;
    const int64_t most = (n + 511) / 512;
    if (s > most) s = most;
    if (s < 1) s = 1;
    DwPlan p;
    p.rows = ((n + s - 1) / s + 63) / 64 * 64;
    p.splits = (int)(p.rows > 0 ? (n + p.rows - 1) / p.rows : 0);
    return p;
}

struct GatedWs {
    void* d;
    float* part;
    size_t bytes;
};
GatedWs gated_ws(int64_t n, int32_t dim, int32_t hidden, int32_t dtype, void* base) {
    Carver c(base);
    const size_t e = dtype == RSE_F32 ? 4 : 2;
    GatedWs w;
    w.d = c.take<char>((size_t)n * 2 * hidden * e);
    w.part = c.take<float>((size_t)dw_plan(n, dim, hidden).splits * 2 * hidden * dim);
    w.bytes = c.size();
    return w;
}

template <typename F>
int by_dtype(int32_t dtype, F f) {
    return dtype == RSE_F32 ? f(float()) : f(uint16_t());
}

}  // namespace

extern "C" {

int seq_gated_linear_fwd(const rse_seq_mat* x, const rse_seq_mat* w_gate, const rse_seq_mat* w_up, int64_t n, int32_t dim,
                         int32_t hidden, int32_t dtype, int32_t act, const rse_seq_mat* out, void* stream) {
    int rc = gated_args(n, dim, hidden, dtype);
    if (rc) return rc;
    if (act < RSE_SIGMOID || act > RSE_GELU || !mat_ok(w_gate, dtype) || !mat_ok(w_up, dtype)) return RSE_ERR_INVALID_ARG;
    if (n == 0) return RSE_OK;
    if (!mat_ok(x, dtype) || !out_mat_ok(out, dtype, n, hidden)) return RSE_ERR_INVALID_ARG;
    const int64_t blocks = (n + TILE - 1) / TILE * ((hidden + TILE / 2 - 1) / (TILE / 2));
    if (blocks > INT32_MAX) return RSE_ERR_UNSUPPORTED;
    const GatedArgs a = {n, dim, hidden, act};
    return by_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        hipLaunchKernelGGL((k_gated<T, false>), dim3((unsigned)blocks), dim3(GT), 0, as_stream(stream), a, view<const T>(x),
                           view<const T>(w_gate), view<const T>(w_up), Mat<const T>{nullptr, 0}, view<T>(out));
        return launch_status();
    });
}

int rse_seq_gated_linear_bwd_workspace_size(int64_t n, int32_t dim, int32_t hidden, int32_t dtype, size_t* bytes_out) {
    int rc = gated_args(n, dim, hidden, dtype);
    if (rc) return rc;
    if (!bytes_out) return RSE_ERR_INVALID_ARG;
    *bytes_out = gated_ws(n, dim, hidden, dtype, nullptr).bytes;
    return RSE_OK;
}

int seq_gated_linear_bwd(const rse_seq_mat* x, const rse_seq_mat* w_gate, const rse_seq_mat* w_up, const rse_seq_mat* dout,
                         int64_t n, int32_t dim, int32_t hidden, int32_t dtype, int32_t act, const rse_seq_mat* dx,
                         const rse_seq_mat* dw_gate, const rse_seq_mat* dw_up, void* d_ws, size_t ws_bytes, void* stream) {
    int rc = gated_args(n, dim, hidden, dtype);
    if (rc) return rc;
    if (act < RSE_SIGMOID || act > RSE_GELU || !mat_ok(w_gate, dtype) || !mat_ok(w_up, dtype) ||
        !out_mat_ok(dw_gate, dtype, hidden, dim) || !out_mat_ok(dw_up, dtype, hidden, dim))
        return RSE_ERR_INVALID_ARG;
    if (n > 0 && (!mat_ok(x, dtype) || !mat_ok(dout, dtype) || !out_mat_ok(dx, dtype, n, dim))) return RSE_ERR_INVALID_ARG;
    const GatedWs ws = gated_ws(n, dim, hidden, dtype, d_ws);
    if (ws_bytes < ws.bytes) return RSE_ERR_WORKSPACE;
    if (ws.bytes && (!d_ws || reinterpret_cast<uintptr_t>(d_ws) % 256)) return RSE_ERR_INVALID_ARG;
    const DwPlan dp = dw_plan(n, dim, hidden);
    const int64_t rt = (n + TILE - 1) / TILE, ct = (dim + TILE - 1) / TILE;
    const int64_t in_blocks = rt * ((hidden + TILE / 2 - 1) / (TILE / 2)), dx_blocks = rt * ct;
    const int64_t dw_blocks = dp.splits * ct * ((2ll * hidden + TILE - 1) / TILE);
    if (in_blocks > INT32_MAX || dw_blocks > INT32_MAX) return RSE_ERR_UNSUPPORTED;
    const GatedArgs a = {n, dim, hidden, act};
    hipStream_t s = as_stream(stream);
    return by_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const Mat<T> d = {static_cast<T*>(ws.d), 2ll * hidden};
        const Mat<const T> dc = {d.p, d.stride};
        if (n > 0) {
            hipLaunchKernelGGL((k_gated<T, true>), dim3((unsigned)in_blocks), dim3(GT), 0, s, a, view<const T>(x),
                               view<const T>(w_gate), view<const T>(w_up), view<const T>(dout), d);
            hipLaunchKernelGGL((k_gated_dx<T>), dim3((unsigned)dx_blocks), dim3(GT), 0, s, a, dc, view<const T>(w_gate),
                               view<const T>(w_up), view<T>(dx));
            hipLaunchKernelGGL((k_gated_dw<T>), dim3((unsigned)dw_blocks), dim3(GT), 0, s, a, dc, view<const T>(x), dp.rows,
                               ws.part);
        }
        hipLaunchKernelGGL((k_gated_dw_join<T>), dim3(fill_blocks(2ll * hidden * dim, 4 * GT, 4096)), dim3(GT), 0, s, a, ws.part,
                           dp.splits, view<T>(dw_gate), view<T>(dw_up));
        return launch_status();
    });
}

}  // extern "C"
