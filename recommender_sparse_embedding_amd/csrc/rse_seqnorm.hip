// rse_seqnorm.hip -- layer norm of event rows, with the residual stream on the
// way, and its backward with the sums over the rows.
//
// Bound by memory: forward x (and the residual) in, y (and the sum) out;
// backward x, dy (and the stream's gradient) in, dx out: 5.5 and 5.1 TB/s on
// 413696 rows of 256 in bf16.  A row stays in the registers of the G lanes that
// share it (V pieces of 16 bytes a lane), so its mean, the sum of squares about
// that mean and the result are one reading.
#include "rse_seqmma.h"

using namespace rse;
using namespace rse_host;

namespace {

constexpr int NB = 256;                 // threads of a block

// Rows as the kernels see them.
template <typename T>
struct Mat {
    T* p;
    int64_t stride;
    __device__ __forceinline__ T* row(int64_t i) const { return p + i * stride; }
};

// 16 bytes at any element's address (the memory pipeline takes them unaligned).
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));

// The EPC elements of a 16-byte piece as fp32.
template <typename T>
struct Piece {
    static constexpr int EPC = 16 / (int)sizeof(T);
    static __device__ __forceinline__ void widen(float (&x)[EPC], u32x4 v) {
#pragma unroll
        for (int e = 0; e < EPC; e += 4) {
            const f32x4 f = chunk_f32<T>(v, e);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[e + i] = f[i];
        }
    }
    static __device__ __forceinline__ u32x4 narrow(const float (&x)[EPC]) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) v[i] = __float_as_uint(x[i]);
            else v[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        }
        return v;
    }
    // Piece c of a row of dim elements, on its way: of a row that ends inside the
    // piece its last 16 bytes, which `settle` moves to their places (element by
    // element such a row's loads waited for one another: 132 us for 66 on 100003
    // rows of 321).
    static __device__ __forceinline__ u32x4 load(const T* row, int c, int dim) {
        if (dim >= EPC) return *(const RSE_GLOBAL u32x4_at2*)(row + (c * EPC < dim - EPC ? c * EPC : dim - EPC));
        u32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < EPC; ++e)
            if (e < dim) {
                const T x = *(const RSE_GLOBAL T*)(row + e);
                if constexpr (sizeof(T) == 4) v[e] = __float_as_uint(x);
                else v[e / 2] |= (uint32_t)x << (16 * (e & 1));
            }
        return v;
    }
    static __device__ __forceinline__ u32x4 settle(u32x4 v, int c, int dim) {
        if (dim % EPC == 0 || dim < EPC) return v;
        int by = c * EPC - (dim - EPC);         // elements
        by = by > 0 ? by : 0;
        if (sizeof(T) == 2) {
            if (by & 1) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
            by >>= 1;
        }
        if (by & 1) v = u32x4{v[1], v[2], v[3], 0};
        if (by & 2) v = u32x4{v[2], v[3], 0, 0};
        return v;
    }
    static __device__ __forceinline__ void store(T* row, int c, int dim, u32x4 v) {
        T* p = row + c * EPC;
        if ((c + 1) * EPC <= dim) {
            *(RSE_GLOBAL u32x4_at2*)p = v;
            return;
        }
#pragma unroll
        for (int e = 0; e < EPC; ++e)
            if (c * EPC + e < dim) {
                T x;
                if constexpr (sizeof(T) == 4) x = __uint_as_float(v[e]);
                else x = (T)(v[e / 2] >> (16 * (e & 1)));
                *(RSE_GLOBAL T*)(p + e) = x;
            }
    }
    // Elements of a vector of weights, `other` where there is none and past the end.
    static __device__ __forceinline__ void weights(float (&x)[EPC], const float* w, int c, int dim, float other) {
#pragma unroll
        for (int e = 0; e < EPC; ++e) x[e] = w && c * EPC + e < dim ? w[c * EPC + e] : other;
    }
};

// The sums of two values over the G lanes that share a row, in each of them.
template <int G>
__device__ __forceinline__ void row_sums(float& a, float& b, float (*s)[2]) {
#pragma unroll
    for (int m = 1; m < (G < WAVE ? G : WAVE); m <<= 1) {
        a += __shfl_xor(a, m, WAVE);
        b += __shfl_xor(b, m, WAVE);
    }
    if constexpr (G > WAVE) {
        const int w = threadIdx.x / WAVE;
        __syncthreads();                // the last sums have been read
        if (lane_id() == 0) {
            s[w][0] = a;
            s[w][1] = b;
        }
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < G / WAVE; ++i) {
            a += s[i][0];
            b += s[i][1];
        }
    }
}

template <typename T, int G, int V>
__global__ __launch_bounds__(NB) void k_norm_fwd(Mat<const T> x, Mat<const T> res, Mat<T> sum, const float* weight,
                                                 const float* bias, float eps, int64_t n, int dim, Mat<T> y, float* stats) {
    using P = Piece<T>;
    constexpr int EPC = P::EPC, RB = NB / G;
    __shared__ float s_sum[NB / WAVE][2];
    const int g = threadIdx.x % G;
    const float inv = 1.f / (float)dim;
    float w[V][EPC], bb[V][EPC];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        P::weights(w[v], weight, v * G + g, dim, 1.f);
        P::weights(bb[v], bias, v * G + g, dim, 0.f);
    }
    // (of a block's rows, all take part in the barriers of row_sums)
    for (int64_t r0 = (int64_t)blockIdx.x * RB; r0 < n; r0 += (int64_t)gridDim.x * RB) {
        const int64_t r = r0 + threadIdx.x / G;
        const bool live = r < n;
        u32x4 raw[V], more[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            raw[v] = more[v] = u32x4{0, 0, 0, 0};
            const int c = v * G + g;
            if (live && c * EPC < dim) {
                raw[v] = P::load(x.row(r), c, dim);
                if (res.p) more[v] = P::load(res.row(r), c, dim);
            }
        }
        float f[V][EPC];
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P::widen(f[v], P::settle(raw[v], v * G + g, dim));
            if (res.p) {
                float o[EPC];
                P::widen(o, P::settle(more[v], v * G + g, dim));
#pragma unroll
                for (int e = 0; e < EPC; ++e) f[v][e] += o[e];
                const u32x4 st = P::narrow(f[v]);           // the stream as it is stored is what is normalised
                P::widen(f[v], st);
                const int c = v * G + g;
                if (live && c * EPC < dim) P::store(sum.row(r), c, dim, st);
            }
#pragma unroll
            for (int e = 0; e < EPC; ++e) a += f[v][e];
        }
        row_sums<G>(a, b, s_sum);
        const float mean = a * inv;
        a = b = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                f[v][e] = (v * G + g) * EPC + e < dim ? f[v][e] - mean : 0.f;
                a = __builtin_fmaf(f[v][e], f[v][e], a);
            }
        row_sums<G>(a, b, s_sum);
        const float rs = 1.f / sqrtf(a * inv + eps);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * G + g;
            if (live && c * EPC < dim) {
#pragma unroll
                for (int e = 0; e < EPC; ++e) f[v][e] = __builtin_fmaf(f[v][e] * rs, w[v][e], bb[v][e]);
                P::store(y.row(r), c, dim, P::narrow(f[v]));
            }
        }
        if (stats && live && g == 0) {
            stats[2 * r] = mean;
            stats[2 * r + 1] = rs;
        }
    }
}

// dx, and of a block's rows the sums of dy xh and dy (part: [blocks][2][dim],
// added by k_norm_join).
template <typename T, int G, int V>
__global__ __launch_bounds__(NB) void k_norm_bwd(Mat<const T> x, Mat<const T> dy, const float* weight, const float* stats,
                                                 Mat<const T> dsum, int64_t n, int dim, Mat<T> dx, float* part) {
    using P = Piece<T>;
    constexpr int EPC = P::EPC, RB = NB / G;
    __shared__ float s_sum[NB / WAVE][2];
    const int g = threadIdx.x % G;
    const float inv = 1.f / (float)dim;
    float w[V][EPC], dw[V][EPC], db[V][EPC];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        P::weights(w[v], weight, v * G + g, dim, 1.f);
#pragma unroll
        for (int e = 0; e < EPC; ++e) dw[v][e] = db[v][e] = 0.f;
    }
    for (int64_t r0 = (int64_t)blockIdx.x * RB; r0 < n; r0 += (int64_t)gridDim.x * RB) {
        const int64_t r = r0 + threadIdx.x / G;
        const bool live = r < n;
        u32x4 xr[V], yr[V], sr[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            xr[v] = yr[v] = sr[v] = u32x4{0, 0, 0, 0};
            const int c = v * G + g;
            if (live && c * EPC < dim) {
                xr[v] = P::load(x.row(r), c, dim);
                yr[v] = P::load(dy.row(r), c, dim);
                if (dsum.p) sr[v] = P::load(dsum.row(r), c, dim);
            }
        }
        const float mean = live ? stats[2 * r] : 0.f, rs = live ? stats[2 * r + 1] : 0.f;
        float a = 0.f, b = 0.f, xh[V][EPC], dn[V][EPC];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P::widen(xh[v], P::settle(xr[v], v * G + g, dim));
            P::widen(dn[v], P::settle(yr[v], v * G + g, dim));
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                xh[v][e] = live && (v * G + g) * EPC + e < dim ? (xh[v][e] - mean) * rs : 0.f;
                dw[v][e] = __builtin_fmaf(dn[v][e], xh[v][e], dw[v][e]);
                db[v][e] += dn[v][e];
                dn[v][e] *= w[v][e];
                a += dn[v][e];
                b = __builtin_fmaf(dn[v][e], xh[v][e], b);
            }
        }
        row_sums<G>(a, b, s_sum);
        a *= inv;
        b *= inv;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * G + g;
            if (live && c * EPC < dim) {
                float o[EPC];
                P::widen(o, P::settle(sr[v], c, dim));
#pragma unroll
                for (int e = 0; e < EPC; ++e) {
                    const float d = (dn[v][e] - a - xh[v][e] * b) * rs;
                    o[e] = dsum.p ? o[e] + d : d;
                }
                P::store(dx.row(r), c, dim, P::narrow(o));
            }
        }
    }
    if (!part) return;
    // a wave's groups of lanes by shuffles, then the waves one after the other (all
    // groups one after the other took 38 us for 13 on 183672 rows of 32, 64 groups a
    // block; side by side in LDS they would leave room for two blocks a CU at rows of 4 KB)
    extern __shared__ float s_part[];           // [2][V * G * EPC], of rows that fit a wave
    constexpr int W = V * G * EPC, TURNS = G < NB ? NB / (G < WAVE ? WAVE : G) : 1;
    float* mine = part + (int64_t)blockIdx.x * 2 * dim;
#pragma unroll
    for (int m = G; m < WAVE; m <<= 1)
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                dw[v][e] += __shfl_xor(dw[v][e], m, WAVE);
                db[v][e] += __shfl_xor(db[v][e], m, WAVE);
            }
    const bool first = G >= WAVE || lane_id() < G;
    const int q = G < NB ? threadIdx.x / (G < WAVE ? WAVE : G) : 0;
    for (int turn = 0; turn < TURNS; ++turn) {
        if (q == turn && first)
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < EPC; ++e) {
                    const int d = (v * G + g) * EPC + e;
                    if constexpr (TURNS > 1) {
                        if (turn > 0) {
                            dw[v][e] += s_part[d];
                            db[v][e] += s_part[W + d];
                        }
                        s_part[d] = dw[v][e];
                        s_part[W + d] = db[v][e];
                    }
                    if (turn == TURNS - 1 && d < dim) {
                        mine[d] = dw[v][e];
                        mine[dim + d] = db[v][e];
                    }
                }
        if constexpr (TURNS > 1) __syncthreads();
    }
}

// Columns of part [parts][2 dim] added up: 16 columns a block, 16 threads a
// column, each a strided run of the parts.
constexpr int JC = 16, JR = NB / JC;
__global__ __launch_bounds__(NB) void k_norm_join(const float* part, int64_t parts, int dim, float* dw, float* db) {
    __shared__ float s[JR][JC];
    const int c = threadIdx.x % JC, q = threadIdx.x / JC;
    const int64_t t = (int64_t)blockIdx.x * JC + c;
    float a = 0.f;
    if (t < 2 * dim)
#pragma unroll 8
        for (int64_t i = q; i < parts; i += JR) a += part[i * 2 * dim + t];
    s[q][c] = a;
    __syncthreads();
    if (q == 0 && t < 2 * dim) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < JR; ++i) a += s[i][c];
        if (t < dim) {
            if (dw) dw[t] = a;
        } else if (db) {
            db[t - dim] = a;
        }
    }
}

// ------------------------------------------------------------------ host --
bool mat_ok(const rse_seq_mat* m, int32_t dtype) {
    return m && m->data && reinterpret_cast<uintptr_t>(m->data) % (dtype == RSE_F32 ? 4 : 2) == 0;
}
bool out_mat_ok(const rse_seq_mat* m, int32_t dtype, int64_t n, int32_t dim) {
    return mat_ok(m, dtype) && (n <= 1 || m->stride >= dim || -m->stride >= dim);
}
template <typename T>
Mat<T> view(const rse_seq_mat* m) {
    return m ? Mat<T>{static_cast<T*>(m->data), m->stride} : Mat<T>{nullptr, 0};
}

// f(T(), integral_constant<G>, integral_constant<V>): the fewest lanes (4 to
// a wave) that hold a row in one piece each, then more pieces, then a block; the
// backward, whose sums of four pieces a lane would leave two waves a SIMD, goes from
// two pieces to a block.  us, four pieces a lane of one wave / a block: forward of 133333
// rows of 1500 in bf16 200 / 258, of 97656 of 2048 171 / 189; backward 482 / 325 and
// 332 / 240.
template <bool BWD, typename T, typename F>
int by_pieces(int32_t dim, F f) {
    constexpr int EPC = 16 / (int)sizeof(T);
    const int pieces = (dim + EPC - 1) / EPC;
    const auto go = [&](auto g, auto v) { return f(T(), g, v); };
#define RSE_C(x) std::integral_constant<int, x>()
    if (pieces <= 4) return go(RSE_C(4), RSE_C(1));
    if (pieces <= 8) return go(RSE_C(8), RSE_C(1));
    if (pieces <= 16) return go(RSE_C(16), RSE_C(1));
    if (pieces <= 32) return go(RSE_C(32), RSE_C(1));
    if (pieces <= 64) return go(RSE_C(64), RSE_C(1));
    if (pieces <= 128) return go(RSE_C(64), RSE_C(2));
    if (pieces <= 256) return go(RSE_C(BWD ? 256 : 64), RSE_C(BWD ? 1 : 4));
    if (pieces <= 512) return go(RSE_C(256), RSE_C(2));
    if (pieces <= 1024) return go(RSE_C(256), RSE_C(4));
    return go(RSE_C(256), RSE_C(8));
#undef RSE_C
}
template <bool BWD, typename F>
int by_norm(int32_t dtype, int32_t dim, F f) {
    return dtype == RSE_F32 ? by_pieces<BWD, float>(dim, f) : by_pieces<BWD, uint16_t>(dim, f);
}

int norm_args(int64_t n, int32_t dim, int32_t dtype) {
    if (n < 0 || dim < 1 || (dtype != RSE_F32 && dtype != RSE_BF16)) return RSE_ERR_INVALID_ARG;
    return dim > RSE_SEQ_MAX_NORM_DIM ? RSE_ERR_UNSUPPORTED : RSE_OK;
}

// Blocks that go through the rows, their weights in registers (a block for
// every few rows, which loaded them each time, took 383 us for 153 on 413696 rows
// of 256).  us, forward with 1024 / 1536 / 2048, backward with 512 / 768 / 1024
// blocks: 413696 rows of 256 bf16 153 / 164 / 172 and 172 / 166 / 174, 24571 of
// 2048 fp32 72 / 74 / 83 and 133 / 119 / 127, 100003 of 321 bf16 67 / 63 / 73 and
// 139 / 73 / 65.  A block of the backward leaves sums of two rows' length.
constexpr int FWD_BLOCKS = 1024;
constexpr int64_t BWD_BLOCKS = 768;
template <int G>
int64_t bwd_blocks(int64_t n) {
    const int64_t b = (n + NB / G - 1) / (NB / G);
    return b < BWD_BLOCKS ? b : BWD_BLOCKS;
}

}  // namespace

extern "C" {

int seq_layer_norm_fwd(const rse_seq_mat* x, const rse_seq_mat* residual, const rse_seq_mat* sum, const float* d_weight,
                       const float* d_bias, float eps, int64_t n, int32_t dim, int32_t dtype, const rse_seq_mat* y,
                       float* d_stats, void* stream) {
    int rc = norm_args(n, dim, dtype);
    if (rc) return rc;
    if (!(eps >= 0.f) || !residual != !sum) return RSE_ERR_INVALID_ARG;
    if (n == 0) return RSE_OK;
    if (!mat_ok(x, dtype) || !out_mat_ok(y, dtype, n, dim)) return RSE_ERR_INVALID_ARG;
    if (residual && (!mat_ok(residual, dtype) || !out_mat_ok(sum, dtype, n, dim))) return RSE_ERR_INVALID_ARG;
    return by_norm<false>(dtype, dim, [&](auto t, auto g, auto v) {
        using T = decltype(t);
        constexpr int G = decltype(g)::value, V = decltype(v)::value;
        hipLaunchKernelGGL((k_norm_fwd<T, G, V>), dim3(fill_blocks(n, NB / G, FWD_BLOCKS)), dim3(NB), 0, as_stream(stream),
                           view<const T>(x), view<const T>(residual), view<T>(sum), d_weight, d_bias, eps, n, dim,
                           view<T>(y), d_stats);
        return launch_status();
    });
}

int rse_seq_layer_norm_bwd_workspace_size(int64_t n, int32_t dim, int32_t dtype, size_t* bytes_out) {
    int rc = norm_args(n, dim, dtype);
    if (rc) return rc;
    if (!bytes_out) return RSE_ERR_INVALID_ARG;
    return by_norm<true>(dtype, dim, [&](auto, auto g, auto) {
        *bytes_out = align_up((size_t)bwd_blocks<decltype(g)::value>(n) * 2 * dim * sizeof(float), 256);
        return RSE_OK;
    });
}

int seq_layer_norm_bwd(const rse_seq_mat* x, const rse_seq_mat* dy, const float* d_weight, const float* d_stats,
                       const rse_seq_mat* dsum, int64_t n, int32_t dim, int32_t dtype, const rse_seq_mat* dx,
                       float* d_dweight, float* d_dbias, void* d_ws, size_t ws_bytes, void* stream) {
    int rc = norm_args(n, dim, dtype);
    if (rc) return rc;
    if (n > 0 && (!mat_ok(x, dtype) || !mat_ok(dy, dtype) || !d_stats || !out_mat_ok(dx, dtype, n, dim) ||
                  (dsum && !mat_ok(dsum, dtype))))
        return RSE_ERR_INVALID_ARG;
    size_t need = 0;
    rse_seq_layer_norm_bwd_workspace_size(n, dim, dtype, &need);
    const bool sums = d_dweight || d_dbias;
    if (sums && n > 0 && ws_bytes < need) return RSE_ERR_WORKSPACE;
    if (sums && n > 0 && (!d_ws || reinterpret_cast<uintptr_t>(d_ws) % 256)) return RSE_ERR_INVALID_ARG;
    return by_norm<true>(dtype, dim, [&](auto t, auto g, auto v) {
        using T = decltype(t);
        constexpr int G = decltype(g)::value, V = decltype(v)::value;
        constexpr size_t lds = G < NB ? (size_t)2 * V * G * Piece<T>::EPC * sizeof(float) : 0;
        const int64_t blocks = bwd_blocks<G>(n);
        float* part = sums ? static_cast<float*>(d_ws) : nullptr;
        if (n > 0)
            hipLaunchKernelGGL((k_norm_bwd<T, G, V>), dim3((unsigned)blocks), dim3(NB), part ? lds : 0, as_stream(stream),
                               view<const T>(x), view<const T>(dy), d_weight, d_stats, view<const T>(dsum), n, dim,
                               view<T>(dx), part);
        if (sums)
            hipLaunchKernelGGL(k_norm_join, dim3((2 * dim + JC - 1) / JC), dim3(NB), 0, as_stream(stream), part, blocks, dim,
                               d_dweight, d_dbias);
        return launch_status();
    });
}

}  // extern "C"
