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
// dim 256, and as dear from a dim of some 1100 on.  dg and du pass through the
// workspace in the rows' type: in bf16 they are rounded once and enter the products
// that follow as single values, as plain bf16 products would take them (gradients
// 0.0023 from the float64 ones in relative 2-norm; 0.0017, which is the rounding of
// the gradients themselves, with both in fp32).  As pairs of values they would be
// that near too, and have the products of dx and dW done twice and twice the
// bytes of dg and du: some 950 us and more beside 2540, 413696 rows of 256 by 1024.
#include "rse_seqmma.h"

#include <tuple>

using namespace rse;
using namespace rse_host;

namespace {

constexpr int JT = 256;                 // threads of a block that adds parts up
constexpr int KB = 64;                  // bytes of the contraction a step: 32 bf16, 16 fp32
constexpr int KCH = KB / 16;
constexpr int NBUF = 3;                 // steps in LDS: one multiplied, two on their way

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

// A block's tile of the result: WQ by WP waves with MQ by MP tiles of 32 by 32
// each; Q rows are the lanes' side, P rows the registers'.
template <int MQ_, int MP_, int WQ_, int WP_>
struct Block {
    static constexpr int MQ = MQ_, MP = MP_, WQ = WQ_, WP = WP_, TQ = 32 * MQ * WQ, TP = 32 * MP * WP;
    static constexpr int GT = WQ * WP * WAVE;           // threads
};

// ------------------------------------------------------------- operands --
// A block's operand of R rows (of the result) by KT<T> of the contraction, on
// its way from memory to LDS, and read from there as matrix operands: 16 bytes a
// lane, of row `lane % 32` the elements 8 s' + 4 (lane / 32) .. of step s in
// fp32, 16 s + 8 (lane / 32) .. in bf16.  Thread t of GT moves the pieces that stand at
// t, t + GT, ... in LDS.  Rows of the result past the end are doubles of an existing one
// (their results are not stored); of a last, partial step the pieces past the
// end are zeros, written through registers.

// Rows of the result are rows in memory: the contraction is contiguous.
template <typename T, int R, int GT>
struct AlongRows {
    using TL = Tile<T, KT<T>>;
    static constexpr int PER = R * KCH / GT;
    static_assert(PER * GT == R * KCH, "a piece for every thread");
    const T* p[PER];
    int64_t k_end;
    template <typename F>
    __device__ __forceinline__ void begin(F row_at, int64_t end) {
        k_end = end;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = i * GT + threadIdx.x % GT, r = t / KCH;
            p[i] = row_at(r) + ((t % KCH) ^ TL::swz(r)) * EPC<T>;
        }
    }
    __device__ __forceinline__ void issue(int64_t k0, bool, u32x4* lds, int w) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) to_lds(p[i] + k0, lds + i * GT + w * WAVE);
    }
    __device__ __forceinline__ void partial(int64_t k0, u32x4* lds) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = i * GT + threadIdx.x % GT;
            const int64_t k = k0 + ((t % KCH) ^ TL::swz(t / KCH)) * EPC<T>;
            u32x4 x = {0, 0, 0, 0};
            if (k < k_end) x = gload_u4(p[i] + k0);
            lds[t] = x;
        }
    }
    static __device__ __forceinline__ u32x4 frag(const u32x4* lds, int r0, int s) {
        const int lane = lane_id();
        return lds[TL::chunk_at(r0 + (lane & 31), 2 * s + (lane >> 5))];
    }
};

// Rows of the result are columns in memory: one row in memory a step of the
// contraction.  F: pointer of the row of contraction index k.
template <typename T, int R, int GT, typename F>
struct AcrossRows {
    using TL = Tile<T, R>;
    static constexpr int PER = R * KCH / GT;
    static_assert(PER * GT == R * KCH, "a piece for every thread");
    F k_row;
    int64_t k_end;
    int cols;                           // of the tile, that exist
    __device__ __forceinline__ const T* at(int64_t k0, int i) const {
        const int t = i * GT + threadIdx.x % GT, r = t / TL::CH, c = ((t % TL::CH) ^ TL::swz(r)) * EPC<T>;
        return k_row(k0 + r) + (c < cols ? c : 0);
    }
    __device__ __forceinline__ void issue(int64_t k0, bool, u32x4* lds, int w) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) to_lds(at(k0, i), lds + i * GT + w * WAVE);
    }
    __device__ __forceinline__ void partial(int64_t k0, u32x4* lds) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = i * GT + threadIdx.x % GT;
            u32x4 x = {0, 0, 0, 0};
            if (k0 + t / TL::CH < k_end) x = gload_u4(at(k0, i));
            lds[t] = x;
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

// The same of a first matrix and, from contraction index `turn` on, of a second
// one.  Steps are sent in order: a step's rows are the last one's, KT further,
// but for the first step and the two around the turn (addresses formed anew every
// step: 575 us for 540 in k_gated_dx of 413696 rows of 256 by 1024; without a
// second matrix k_gated_dw is the faster the other way, 477 for 517).
template <typename T, int R, int GT>
struct StackedRows {
    using TL = Tile<T, R>;
    static constexpr int PER = R * KCH / GT;
    static_assert(PER * GT == R * KCH, "a piece for every thread");
    Mat<const T> m, m2;
    int64_t turn, k_end;
    const T* p[PER];                    // of the step sent last
    int c[PER];
    __device__ __forceinline__ const T* row(int64_t k) const {
        const bool first = k < turn;
        const int64_t i = first ? k : k - turn;
        const uint64_t base = first ? reinterpret_cast<uint64_t>(m.p) : reinterpret_cast<uint64_t>(m2.p);
        return reinterpret_cast<const T*>(base) + i * (first ? m.stride : m2.stride);
    }
    // cols: of the tile, that exist
    __device__ __forceinline__ void begin(Mat<const T> a, Mat<const T> b, int64_t at, int64_t end, int cols) {
        m = a;
        m2 = b;
        turn = at;
        k_end = end;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = i * GT + threadIdx.x % GT, x = ((t % TL::CH) ^ TL::swz(t / TL::CH)) * EPC<T>;
            c[i] = x < cols ? x : 0;
            p[i] = nullptr;
        }
    }
    __device__ __forceinline__ void issue(int64_t k0, bool first, u32x4* lds, int w) {
        const bool anew = first || (k0 + KT<T> > turn && k0 < turn + KT<T>);
        const int64_t ahead = KT<T> * (k0 < turn ? m.stride : m2.stride);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (anew) p[i] = row(k0 + (i * GT + (int)threadIdx.x % GT) / TL::CH) + c[i];
            else p[i] += ahead;
            to_lds(p[i], lds + i * GT + w * WAVE);
        }
    }
    __device__ __forceinline__ void partial(int64_t k0, u32x4* lds) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = i * GT + threadIdx.x % GT;
            const int64_t k = k0 + t / TL::CH;
            u32x4 x = {0, 0, 0, 0};
            if (k < k_end) x = gload_u4(row(k) + c[i]);
            lds[t] = x;
        }
    }
    static __device__ __forceinline__ u32x4 frag(const u32x4* lds, int r0, int s) {
        return AcrossRows<T, R, GT, int>::frag(lds, r0, s);
    }
};

// acc[j][i] += P rows p0(j) .. times Q rows q0 + 32 i .., over the contraction
// from k0 to k1.  One barrier a step: past it, the step's pieces have landed and
// all waves are done with the buffer that the step after next is sent to.  turns > 0:
// that many barriers, for more groups of waves that have other parts of the contraction.
template <typename T, typename B, typename P, typename Q, typename P0>
__device__ __forceinline__ void multiply(P& p, Q& q, int64_t k0, int64_t k1, P0 p0, int q0, f32x16 (&acc)[B::MP][B::MQ],
                                         u32x4* lds, int w, int turns = 0) {
    constexpr int SIZE = (B::TP + B::TQ) * KCH;
    const int steps = (int)((k1 - k0 + KT<T> - 1) / KT<T>), full = (int)((k1 - k0) / KT<T>);
    auto send = [&](int i, int b) {
        u32x4* to = lds + b * SIZE;
        if (i < full) {
            p.issue(k0 + (int64_t)i * KT<T>, i == 0, to, w);
            q.issue(k0 + (int64_t)i * KT<T>, i == 0, to + B::TP * KCH, w);
        } else if (i < steps) {
            p.partial(k0 + (int64_t)i * KT<T>, to);
            q.partial(k0 + (int64_t)i * KT<T>, to + B::TP * KCH);
        }
    };
    send(0, 0);
    send(1, 1);
    int b = 0, i = 0;
    do {
        if (i + 1 < full) loads_left<P::PER + Q::PER>();
        else loads_left<0>();
        lds_barrier();
        send(i + 2, b == 0 ? 2 : b - 1);
        const u32x4 *lp = lds + b * SIZE, *lq = lp + B::TP * KCH;
        if (turns == 0 || i < steps)
#pragma unroll
        for (int s = 0; s < KCH / 2; ++s) {
            u32x4 a[B::MP], c[B::MQ];
#pragma unroll
            for (int j = 0; j < B::MP; ++j) a[j] = P::frag(lp, p0(j), s);
#pragma unroll
            for (int u = 0; u < B::MQ; ++u) c[u] = Q::frag(lq, q0 + 32 * u, s);
#pragma unroll
            for (int j = 0; j < B::MP; ++j)
#pragma unroll
                for (int u = 0; u < B::MQ; ++u) acc[j][u] = mma_chunk<T>(a[j], c[u], acc[j][u]);
        }
        b = b == 2 ? 0 : b + 1;
    } while (++i < (turns ? turns : steps));
}

// A 32 by 32 tile of a lane's row as 16-byte pieces: piece(j) gives elements
// EPC (2 j + half) .. of the 32 along the registers.
template <typename T>
struct Pieces {
    static constexpr int N = sizeof(T);         // pieces a lane: 4 of fp32, 2 of bf16
    u32x4 v[N];
    __device__ __forceinline__ explicit Pieces(const f32x16& acc) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e / 4][e % 4] = __float_as_uint(acc[e]);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)         // (the exchange of store_column)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const u32x2 s = __builtin_amdgcn_permlane32_swap(pack_bf16(acc[8 * j + 2 * i], acc[8 * j + 2 * i + 1]),
                                                                     pack_bf16(acc[8 * j + 4 + 2 * i], acc[8 * j + 5 + 2 * i]), false, false);
                    v[j][i] = s.x;
                    v[j][2 + i] = s.y;
                }
        }
    }
};
// Straight to a row of memory; elements at `left` and on do not exist.
template <typename T>
__device__ __forceinline__ void put_column(T* p, const f32x16& acc, int64_t left) {
    const Pieces<T> x(acc);
    const int h = lane_id() >> 5;
#pragma unroll
    for (int j = 0; j < Pieces<T>::N; ++j)
        if (EPC<T> * (2 * j + h) < left) gstore_u4(p + EPC<T> * (2 * j + h), x.v[j]);
}
// To row `row`, columns c0 .. of a tile of W columns in LDS.
template <typename T, int W>
__device__ __forceinline__ void put_lds(u32x4* lds, int row, int c0, const f32x16& acc) {
    const Pieces<T> x(acc);
    const int h = lane_id() >> 5;
#pragma unroll
    for (int j = 0; j < Pieces<T>::N; ++j) lds[Tile<T, W>::chunk_at(row, c0 / EPC<T> + 2 * j + h)] = x.v[j];
}
// A tile of R rows by W columns from LDS to memory, whole lines of a row by
// neighbouring lanes; `rows` and `cols` exist.
template <typename T, int R, int W, int GT>
__device__ __forceinline__ void rows_to_memory(const u32x4* lds, const Mat<T>& out, int64_t r0, int64_t c0, int64_t rows, int64_t cols) {
    constexpr int CH = Tile<T, W>::CH;
#pragma unroll
    for (int i = 0; i < R * CH / GT; ++i) {
        const int t = i * GT + threadIdx.x, r = t / CH, c = t % CH;
        if (r < rows && c * EPC<T> < cols) gstore_u4(out.row(r0 + r) + c0 + c * EPC<T>, lds[Tile<T, W>::chunk_at(r, c)]);
    }
}

// The same elements read, as they stand in memory (0 past the end), and widened.
template <typename T>
struct RawColumn {
    u32x4 v[2 * (int)sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p, int64_t left) {
        const int h = lane_id() >> 5;
        constexpr int N = 2 * (int)sizeof(T) / 2, E = EPC<T>;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            v[j] = u32x4{0, 0, 0, 0};
            if (E * (2 * j + h) < left) v[j] = gload_u4(p + E * (2 * j + h));
        }
    }
    __device__ __forceinline__ f32x16 widen() const {
        f32x16 x;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(v[e / 4][e % 4]);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const u32x2 s = __builtin_amdgcn_permlane32_swap(v[j][i], v[j][2 + i], false, false);
                    x[8 * j + 2 * i] = __uint_as_float(s.x << 16);
                    x[8 * j + 2 * i + 1] = __uint_as_float(s.x & 0xFFFF0000u);
                    x[8 * j + 4 + 2 * i] = __uint_as_float(s.y << 16);
                    x[8 * j + 5 + 2 * i] = __uint_as_float(s.y & 0xFFFF0000u);
                }
        }
        return x;
    }
};

// e^(c x) for c x <= 0, by the hardware's exponential (base 2, one unit in the
// last place), c given in base 2 as the sum of two floats.  The exponent y is some
// 2^7 at most where the result is not 0, so its own rounding would be up to 2^7 units
// of the result: EXACT takes what it lost, and `rest` of x, back in.
template <bool EXACT>
__device__ __forceinline__ float exp_of(float x, float rest, float c, float c_lo) {
    const float y = x * c, e = __builtin_amdgcn_exp2f(y);
    if (!EXACT) return e;
    const float left = __builtin_fmaf(x, c, -y) + __builtin_fmaf(x, c_lo, rest * c);
    return __builtin_fmaf(e, left * 0.69314718f, e);
}

// act(g) and act'(g), by the hardware's exponential and reciprocal.  EXACT, in
// fp32: within 21 (GELU; 14 sigmoid', 10 the others) units of 2^-24 of themselves,
// of sums the terms.  Else exponents are one rounded product, which puts some 10^-6
// of themselves into results at |g| = 5 (GELU) or 20 (the others), small against the
// 2^-8 of a bf16 one, and SiLU' = s + g s (1 - s) takes 1 - s as it is.  us, one way
// and the other: training on 413696 rows of 256 by 1024 in bf16 2527, 2604 exact; on
// 20011 of 128 by 512 in fp32 232, 238 exact.
//  Sigmoids by e^-|g|, so that s (1 - s) is right at both ends.
//  GELU: Phi(-x) = e^(-x^2 / 2) R(x) for x >= 0, R / t a polynomial in
// t = 1 / (1 + 0.32 x) fitted to erfcx (3e-8 relative), and the exponential serves
// the derivative too.
template <int ACT, bool EXACT>
__device__ __forceinline__ void activate(float g, float& a, float& da) {
    constexpr float LOG2E_LO = 1.925963033500e-8f;      // log2(e) - LOG2E
    float x = fabsf(g);
    if (ACT == RSE_GELU) {
        if (EXACT) x = x > 20.f ? 20.f : x;             // e^-200 is 0 (and the square finite; NaN stays)
        const float q = EXACT ? x * x : g * g, e = exp_of<EXACT>(q, EXACT ? __builtin_fmaf(x, x, -q) : 0.f, -0.5f * LOG2E, -0.5f * LOG2E_LO);
        const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(x, 0.32f, 1.f));
        float r = -0.021151972926650987f;
        r = __builtin_fmaf(r, t, 0.09575628588024625f);
        r = __builtin_fmaf(r, t, -0.1474010975314183f);
        r = __builtin_fmaf(r, t, 0.06607995419458114f);
        r = __builtin_fmaf(r, t, -0.009860294843239454f);
        r = __builtin_fmaf(r, t, 0.058840354541432945f);
        r = __builtin_fmaf(r, t, 0.0877871262999502f);
        r = __builtin_fmaf(r, t, 0.11462742044437546f);
        r = __builtin_fmaf(r, t, 0.1276606749658141f);
        r = __builtin_fmaf(r, t, 0.12766153278717118f);
        r *= t * e;                             // Phi(-x)
        const float cdf = g < 0.f ? r : 1.f - r;
        a = g * cdf;
        da = __builtin_fmaf(g * 0.39894228040143268f, e, cdf);
    } else if (EXACT || ACT == RSE_SIGMOID) {
        x = x > 128.f ? 128.f : x;                      // e^-128 is 0 (NaN stays)
        const float e = exp_of<EXACT>(x, 0.f, -LOG2E, -LOG2E_LO), r = __builtin_amdgcn_rcpf(1.f + e);
        const float s = g < 0.f ? e * r : r, t = e * r * r;
        a = ACT == RSE_SILU ? g * s : s;
        da = ACT == RSE_SILU ? __builtin_fmaf(g, t, s) : t;
    } else {
        const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-LOG2E * g));
        a = g * s;
        da = __builtin_fmaf(g, __builtin_fmaf(-s, s, s), s);
    }
}

// Block x's tile of a grid of `total`: blocks of one XCD (x % 8) take
// consecutive ones, so that what they share stays in its L2.
__device__ __forceinline__ uint32_t xcd_tile(uint32_t x, uint32_t total) {
    const uint32_t per = total / 8, rest = total % 8, xcd = x % 8;
    return xcd * per + (xcd < rest ? xcd : rest) + x / 8;
}

struct GatedArgs {
    int64_t n;
    int32_t dim, hidden;
};

// Shapes, by the type's rate on the matrix cores.  bf16: a step of two blocks, which
// share a CU, is 1024 cycles of products, 1152 of LDS reads and writes, 768 of the
// vector memory path.  fp32 is 16 times as long in its products, and small tiles
// fill the GPU more evenly.
template <typename T>
using InBlock = std::conditional_t<sizeof(T) == 2, Block<2, 4, 2, 2>, Block<1, 2, 2, 2>>;
// bf16, where the large tiles would not give every CU one: 256 rows of 512 by
// 1536 11.7 us for 6.8, 2048 rows (192 large tiles) 13.5 for 13.1; 4096 rows (384) 20.0 for 23.0.
using FewBlock = Block<1, 2, 2, 2>;
// bf16, where the large tiles' columns past the end cost more than the 15 % that
// narrower ones do: forward of 100000 rows of 256 by 184 41.0 us for 32.7, backward 59.3 for
// 45.8; by 64 25.7 for 18.1.
using InNarrow = Block<2, 2, 2, 2>;
// fp32, whose products bound a CU: a wave a tile, and four of them a part of the
// contraction each.  us, tiles of 64 by 64 / so: 46 rows of 792 by 320 32.5 / 12.6, 1011 of
// 1496 by 304 59.8 / 34.1, 256 of 256 by 512 12.2 / 6.3.  (bf16, which waits for its loads
// instead: 64 rows of 512 by 1536 6.5 / 5.6, but 1024 of 256 by 512 4.6 / 5.6.)
using GroupBlock = Block<1, 2, 1, 1>;
constexpr int GROUPS = 4;
constexpr int CUS = 256;
// Waves that share a SIMD, by registers and by LDS, and blocks on the GPU at once.
template <typename B>
constexpr int BY_LDS = 160 * 1024 / (NBUF * (B::TP + B::TQ) * KB) * B::GT / (4 * WAVE);
template <typename B>
constexpr int SHARE = B::MQ * B::MP >= 8 ? 2 : BY_LDS<B> < 4 ? BY_LDS<B> : 4;
template <typename B>
constexpr int AT_ONCE = CUS * SHARE<B> * 4 * WAVE / B::GT;

// Of dx and dW, whose P side is dim: shapes of a type, widest first, with the
// time of a column of theirs relative to the first's; and a small one for where tiles
// are few (see dx_plan, dw_plan).  us, dx of 100000 rows with 512 hidden elements,
// bf16 of 256 / 128 / 64 columns: dim 32 67 / 46 / 33, 64 75 / 51 / 36, 128 74 / 55 /
// 58, 320 136 / 117 / 120; fp32 of 64 / 32: dim 32 164 / 102, 144 401 / 363.
using OutFew = Block<1, 1, 2, 2>;
template <typename T>
struct Out;
template <>
struct Out<uint16_t> {
    using Shapes = std::tuple<Block<2, 4, 2, 2>, Block<2, 2, 2, 2>, Block<2, 2, 4, 1>>;
    static constexpr double COST[] = {1.0, 1.15, 1.4};
};
template <>
struct Out<float> {
    using Shapes = std::tuple<Block<1, 1, 2, 2>, Block<1, 1, 2, 1>>;
    static constexpr double COST[] = {1.0, 1.1};
};

// out (BWD: dg beside du) of TQ rows by TP / 2 hidden elements: the tile's P
// rows are TP / 2 rows of Wg, then the same ones of Wu, and a wave's
// accumulators hold g and u of the same elements.  WK groups of waves have a part
// of the contraction each.
template <typename T, typename B, int WK, int ACT, bool BWD>
__global__ __launch_bounds__((WK * B::GT)) __attribute__((amdgpu_waves_per_eu(WK > 1 ? 2 : SHARE<B>))) void k_gated(
    GatedArgs a, Mat<const T> x, Mat<const T> wg, Mat<const T> wu, Mat<const T> dout, Mat<T> out) {
    constexpr int HT = B::TP / 2, MH = B::MP / 2;
    constexpr int BUF = NBUF * (B::TP + B::TQ) * KCH;
    __shared__ u32x4 lds[WK * BUF];
    const int lane = lane_id(), group = uniform((int)threadIdx.x / B::GT), w = uniform((int)threadIdx.x % B::GT / WAVE);
    const uint32_t ht = (a.hidden + HT - 1) / HT, tile = xcd_tile(blockIdx.x, gridDim.x);
    const int64_t r0 = (int64_t)(tile / ht) * B::TQ;
    const int h0 = (int)(tile % ht) * HT;
    AlongRows<T, B::TP, B::GT> p;
    p.begin([&](int r) {
        const int h = h0 + r % HT;
        return (r < HT ? wg : wu).row(h < a.hidden ? h : a.hidden - 1);
    }, a.dim);
    AlongRows<T, B::TQ, B::GT> q;
    q.begin([&](int r) { return x.row(r0 + r < a.n ? r0 + r : a.n - 1); }, a.dim);
    f32x16 acc[B::MP][B::MQ] = {};
    const int hw = 32 * MH * (w % B::WP), qw = 32 * B::MQ * (w / B::WP);
    RawColumn<T> d[BWD ? MH : 1][B::MQ];
    if (BWD && group == 0)                      // on its way while the projections are formed
#pragma unroll
        for (int i = 0; i < B::MQ; ++i) {
            const int64_t r = r0 + qw + 32 * i + (lane & 31);
#pragma unroll
            for (int j = 0; j < MH; ++j) {
                const int h = h0 + hw + 32 * j;
                d[j][i].load(dout.row(r < a.n ? r : 0) + h, r < a.n ? a.hidden - h : 0);
            }
        }
    const auto p_row = [&](int j) { return hw + (j < MH ? 32 * j : HT + 32 * (j - MH)); };
    if constexpr (WK == 1) {
        multiply<T, B>(p, q, 0, a.dim, p_row, qw, acc, lds, w);
    } else {
        const int turns = ((a.dim + KT<T> - 1) / KT<T> + WK - 1) / WK, k0 = group * turns * KT<T>, k1 = k0 + turns * KT<T>;
        multiply<T, B>(p, q, k0, k1 < a.dim ? k1 : (k0 < a.dim ? a.dim : k0), p_row, qw, acc, lds + group * BUF, w, turns);
        constexpr int NW = B::GT / WAVE, PART = B::MP * B::MQ * 4 * WAVE;       // a wave's sums
        static_assert((WK - 1) * NW * PART <= WK * BUF, "sums in LDS");
        lds_barrier();                          // all waves are done with the operands
        if (group > 0) {
#pragma unroll
            for (int t = 0; t < B::MP * B::MQ * 4; ++t) {
                const f32x16& x = acc[t / 4 / B::MQ][t / 4 % B::MQ];
                const int e = 4 * (t % 4);
                lds[((group - 1) * NW + w) * PART + t * WAVE + lane] =
                    __builtin_bit_cast(u32x4, f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]});
            }
        }
        lds_barrier();
        if (group > 0) return;
        for (int o = 0; o < WK - 1; ++o)
#pragma unroll
            for (int t = 0; t < B::MP * B::MQ * 4; ++t) {
                const f32x4 y = __builtin_bit_cast(f32x4, lds[(o * NW + w) * PART + t * WAVE + lane]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t / 4 / B::MQ][t / 4 % B::MQ][4 * (t % 4) + e] += y[e];
            }
    }
    // by way of LDS, so that a store instruction writes whole lines (32 bytes of
    // 32 rows each ran at 2.8 TB/s)
    constexpr int SIZE = B::TQ * HT / EPC<T>;
    static_assert((BWD ? 2 : 1) * SIZE <= WK * BUF, "tiles of results in LDS");
    lds_barrier();                              // all waves are done with the operands
#pragma unroll
    for (int i = 0; i < B::MQ; ++i) {
        const int r = qw + 32 * i + (lane & 31);
#pragma unroll
        for (int j = 0; j < MH; ++j) {
            f32x16 &g = acc[j][i], &u = acc[j + MH][i];
            if constexpr (BWD) {
                const f32x16 up = d[j][i].widen();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float f, df;
                    activate<ACT, sizeof(T) == 4>(g[e], f, df);
                    g[e] = up[e] * u[e] * df;
                    u[e] = up[e] * f;
                }
                put_lds<T, HT>(lds, r, hw + 32 * j, g);
                put_lds<T, HT>(lds + SIZE, r, hw + 32 * j, u);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float f, df;
                    activate<ACT, sizeof(T) == 4>(g[e], f, df);
                    g[e] = f * u[e];
                }
                put_lds<T, HT>(lds, r, hw + 32 * j, g);
            }
        }
    }
    lds_barrier();
    rows_to_memory<T, B::TQ, HT, B::GT>(lds, out, r0, h0, a.n - r0, a.hidden - h0);
    if constexpr (BWD) rows_to_memory<T, B::TQ, HT, B::GT>(lds + SIZE, out, r0, a.hidden + h0, a.n - r0, a.hidden - h0);
}

// dx = [dg du] [Wg; Wu]; where part is given, of part s of the contraction, the
// indexes from s `len` on.
template <typename T, typename B>
__global__ __launch_bounds__(B::GT) __attribute__((amdgpu_waves_per_eu(SHARE<B>))) void k_gated_dx(GatedArgs a, Mat<const T> d,
                                                                                                Mat<const T> wg, Mat<const T> wu,
                                                                                                Mat<T> dx, int64_t len, float* part) {
    __shared__ u32x4 lds[NBUF * (B::TP + B::TQ) * KCH];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE);
    const uint32_t ct = (a.dim + B::TP - 1) / B::TP, rt = (uint32_t)((a.n + B::TQ - 1) / B::TQ);
    uint32_t tile = xcd_tile(blockIdx.x, gridDim.x);
    const int c0 = (int)(tile % ct) * B::TP;
    tile /= ct;
    const int64_t r0 = (int64_t)(tile % rt) * B::TQ, s = tile / rt, k0 = s * len;
    const int64_t k_end = k0 + len < 2ll * a.hidden ? k0 + len : 2ll * a.hidden;
    StackedRows<T, B::TP, B::GT> p;
    p.begin({wg.p + c0, wg.stride}, {wu.p + c0, wu.stride}, a.hidden, k_end, a.dim - c0);
    AlongRows<T, B::TQ, B::GT> q;
    q.begin([&](int r) { return d.row(r0 + r < a.n ? r0 + r : a.n - 1); }, k_end);
    f32x16 acc[B::MP][B::MQ] = {};
    const int pw = 32 * B::MP * (w % B::WP), qw = 32 * B::MQ * (w / B::WP);
    multiply<T, B>(p, q, k0, k_end, [&](int j) { return pw + 32 * j; }, qw, acc, lds, w);
#pragma unroll
    for (int i = 0; i < B::MQ; ++i) {
        const int64_t r = r0 + qw + 32 * i + (lane & 31), at = r < a.n ? r : 0;
#pragma unroll
        for (int j = 0; j < B::MP; ++j) {
            const int c = c0 + pw + 32 * j, cols = r < a.n ? a.dim - c : 0;
            if (part) put_column(part + (s * a.n + at) * a.dim + c, acc[j][i], cols);
            else put_column(dx.row(at) + c, acc[j][i], cols);
        }
    }
}

// Part s of [dWg; dWu] = [dg du]^T x: the rows from s `rows` on.
template <typename T, typename B>
__global__ __launch_bounds__(B::GT) __attribute__((amdgpu_waves_per_eu(SHARE<B>))) void k_gated_dw(GatedArgs a, Mat<const T> d,
                                                                                                Mat<const T> x, int64_t rows,
                                                                                                float* part) {
    __shared__ u32x4 lds[NBUF * (B::TP + B::TQ) * KCH];
    const int lane = lane_id(), w = uniform((int)threadIdx.x / WAVE);
    const uint32_t ct = (a.dim + B::TP - 1) / B::TP, ht = (2u * a.hidden + B::TQ - 1) / B::TQ;
    uint32_t tile = xcd_tile(blockIdx.x, gridDim.x);
    const int c0 = (int)(tile % ct) * B::TP;
    tile /= ct;
    const int h0 = (int)(tile % ht) * B::TQ;
    const int64_t s = tile / ht, k0 = s * rows, k1 = k0 + rows < a.n ? k0 + rows : a.n;
    auto x_row = [&](int64_t k) -> const T* { return x.row(k) + c0; };
    auto d_row = [&](int64_t k) -> const T* { return d.row(k) + h0; };
    AcrossRows<T, B::TP, B::GT, decltype(x_row)> p = {x_row, k1, a.dim - c0};
    AcrossRows<T, B::TQ, B::GT, decltype(d_row)> q = {d_row, k1, 2 * a.hidden - h0};
    f32x16 acc[B::MP][B::MQ] = {};
    const int pw = 32 * B::MP * (w % B::WP), qw = 32 * B::MQ * (w / B::WP);
    multiply<T, B>(p, q, k0, k1, [&](int j) { return pw + 32 * j; }, qw, acc, lds, w);
#pragma unroll
    for (int i = 0; i < B::MQ; ++i) {
        const int64_t h = h0 + qw + 32 * i + (lane & 31);
        const bool in = h < 2ll * a.hidden;
#pragma unroll
        for (int j = 0; j < B::MP; ++j) {
            const int c = c0 + pw + 32 * j;
            put_column(part + ((s * 2 * a.hidden + (in ? h : 0)) * a.dim + c), acc[j][i], in ? a.dim - c : 0);
        }
    }
}

// The parts [splits][rows][dim] added, rounded once: four elements a thread.
// Rows from `turn` on go to the second matrix.
template <typename T>
__global__ __launch_bounds__(JT) void k_gated_join(const float* part, int splits, int64_t rows, int64_t turn, int32_t dim, Mat<T> m,
                                                   Mat<T> m2) {
    const int64_t size = rows * dim;
    for (int64_t t = 4 * ((int64_t)blockIdx.x * JT + threadIdx.x); t < size; t += 4ll * JT * gridDim.x) {
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int s = 0; s < splits; ++s) o += gload_f4(part + s * size + t);
        const int64_t r = t / dim;
        const int c = (int)(t - r * dim);
        store_four((r < turn ? m.row(r) : m2.row(r - turn)) + c, o);
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

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
template <typename B>
int64_t tiles(int64_t q, int64_t p) { return up(q, B::TQ) * up(p, B::TP); }

// How dx and dW are formed: by which of the type's shapes or, where its tiles
// are too few for the CUs, by the small one, and in how many parts of the contraction.
struct Plan {
    int shape;                          // -1: the small one
    int splits;
    int64_t len;                        // of a part
};
// f(the shape)
template <typename T, int I = 0, typename F>
int64_t by_shape(int shape, F f) {
    using S = typename Out<T>::Shapes;
    if (shape < 0) return f(OutFew());
    if constexpr (I + 1 < (int)std::tuple_size_v<S>)
        if (shape > I) return by_shape<T, I + 1>(shape, f);
    return f(std::tuple_element_t<I, S>());
}
template <typename T>
int64_t tiles_of(int shape, int64_t q, int64_t p) {
    return by_shape<T>(shape, [&](auto b) { return tiles<decltype(b)>(q, p); });
}
// the shape that takes the least for its columns, those past dim included
template <typename T>
int shape_for(int32_t dim) {
    int best = 0;
    double least = 0;
    for (int i = 0; i < (int)std::tuple_size_v<typename Out<T>::Shapes>; ++i) {
        const double cost = Out<T>::COST[i] * by_shape<T>(i, [&](auto b) { return up(dim, decltype(b)::TP) * decltype(b)::TP; });
        if (i == 0 || cost < least) {
            least = cost;
            best = i;
        }
    }
    return best;
}

// dx: parts where the small tiles are few too, of eight steps at least, for two
// blocks a CU (four: no faster).  3196 rows of 80 by 648 in fp32 42 us whole and 22
// with the join; in bf16 500 of 256 by 1024 41 with large tiles and 8, 3196 of 512 by
// 1368 56 and 32.
template <typename T>
Plan dx_plan(int64_t n, int32_t dim, int32_t hidden) {
    Plan p = {shape_for<T>(dim), 1, 2ll * hidden};
    if (tiles_of<T>(p.shape, n, dim) >= CUS) return p;
    p.shape = -1;
    const int64_t blocks = tiles<OutFew>(n, dim), steps = up(2ll * hidden, KT<T>);
    int64_t s = blocks > 0 ? 2 * CUS / blocks : 1;
    if (s > steps / 8) s = steps / 8;
    if (s > 1) {
        p.len = up(steps, s) * KT<T>;
        p.splits = (int)up(2ll * hidden, p.len);
    }
    return p;
}

// dW: parts of the events, of whole steps and 128 events at least: as many as
// make the rounds of blocks (AT_ONCE) shortest, the time to add a part
// up taken as that of an event for 24000 elements (413696 rows of 256 by 1024 in
// 32 parts 14 us beside 459, 24571 of 1024 by 2736 in 5 22 beside 306).
template <typename T>
Plan dw_plan(int64_t n, int32_t dim, int32_t hidden) {
    const int64_t most = up(n, 128) < 64 ? up(n, 128) : 64;
    Plan p = {shape_for<T>(dim), 1, 0};
    if (tiles_of<T>(p.shape, 2ll * hidden, dim) * most < CUS) p.shape = -1;
    const int64_t t = tiles_of<T>(p.shape, 2ll * hidden, dim);
    const int64_t at_once = by_shape<T>(p.shape, [](auto b) -> int64_t { return AT_ONCE<decltype(b)>; });
    double best = 0;
    for (int64_t c = 1; c <= most; ++c) {
        const double cost = (double)up(t * c, at_once) * ((double)n / c) + c * (2.0 * hidden * dim / 24000);
        if (c == 1 || cost < best) {
            best = cost;
            p.splits = (int)c;
        }
    }
    p.len = up(up(n, p.splits), 64) * 64;
    p.splits = (int)(n > 0 ? up(n, p.len) : 0);
    return p;
}

// whether a launch holds the plan's blocks
template <typename T>
bool plan_held(const Plan& p, int64_t q, int64_t c) {
    return by_shape<T>(p.shape, [&](auto b) { return (int64_t)launch_holds(p.splits * tiles<decltype(b)>(q, c), decltype(b)::GT); });
}

struct GatedWs {
    void* d;
    float *dw, *dx;                     // parts
    size_t bytes;
};
template <typename T>
GatedWs gated_ws(int64_t n, int32_t dim, int32_t hidden, void* base) {
    Carver c(base);
    const Plan x = dx_plan<T>(n, dim, hidden);
    GatedWs w;
    w.d = c.take<T>((size_t)n * 2 * hidden);
    w.dw = c.take<float>((size_t)dw_plan<T>(n, dim, hidden).splits * 2 * hidden * dim);
    w.dx = c.take<float>(x.splits > 1 ? (size_t)x.splits * n * dim : 0);
    w.bytes = c.size();
    return w;
}
GatedWs gated_ws(int64_t n, int32_t dim, int32_t hidden, int32_t dtype, void* base) {
    return dtype == RSE_F32 ? gated_ws<float>(n, dim, hidden, base) : gated_ws<uint16_t>(n, dim, hidden, base);
}

// f(block shape, integral_constant<groups of waves>, blocks) of the projections
template <typename T, typename F>
int by_blocks(int64_t n, int32_t dim, int32_t hidden, F f) {
    const auto blocks = [&](auto b) { return up(n, decltype(b)::TQ) * up(hidden, decltype(b)::TP / 2); };
    using One = std::integral_constant<int, 1>;
    if constexpr (sizeof(T) == 2)
        if (blocks(InBlock<T>()) >= CUS && up(hidden, 64) * 64 * 1.15 < up(hidden, 128) * 128) return f(InNarrow(), One(), blocks(InNarrow()));
    if (blocks(InBlock<T>()) < CUS) {
        if constexpr (sizeof(T) == 2) return f(FewBlock(), One(), blocks(FewBlock()));
        else if (up(dim, KT<T>) >= GROUPS) return f(GroupBlock(), std::integral_constant<int, GROUPS>(), blocks(GroupBlock()));
    }
    return f(InBlock<T>(), One(), blocks(InBlock<T>()));
}

// f(T(), integral_constant<act>)
template <typename F>
int by_kind(int32_t dtype, int32_t act, F f) {
    const auto go = [&](auto a) { return dtype == RSE_F32 ? f(float(), a) : f(uint16_t(), a); };
    if (act == RSE_SIGMOID) return go(std::integral_constant<int, RSE_SIGMOID>());
    if (act == RSE_SILU) return go(std::integral_constant<int, RSE_SILU>());
    return go(std::integral_constant<int, RSE_GELU>());
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
    const GatedArgs a = {n, dim, hidden};
    return by_kind(dtype, act, [&](auto t, auto ac) -> int {
        using T = decltype(t);
        constexpr int ACT = decltype(ac)::value;
        return by_blocks<T>(n, dim, hidden, [&](auto b, auto g, int64_t blocks) -> int {
            using B = decltype(b);
            constexpr int WK = decltype(g)::value;
            if (!launch_holds(blocks, WK * B::GT)) return RSE_ERR_UNSUPPORTED;
            hipLaunchKernelGGL((k_gated<T, B, WK, ACT, false>), dim3((unsigned)blocks), dim3(WK * B::GT), 0, as_stream(stream), a,
                               view<const T>(x), view<const T>(w_gate), view<const T>(w_up), Mat<const T>{nullptr, 0}, view<T>(out));
            return launch_status();
        });
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
    const GatedArgs a = {n, dim, hidden};
    hipStream_t s = as_stream(stream);
    return by_kind(dtype, act, [&](auto t, auto ac) -> int {
        using T = decltype(t);
        constexpr int ACT = decltype(ac)::value;
        const Plan x_plan = dx_plan<T>(n, dim, hidden), w_plan = dw_plan<T>(n, dim, hidden);
        const Mat<T> d = {static_cast<T*>(ws.d), 2ll * hidden};
        const Mat<const T> dc = {d.p, d.stride};
        if (n > 0) {
            int err = by_blocks<T>(n, dim, hidden, [&](auto b, auto g, int64_t blocks) -> int {
                using B = decltype(b);
                constexpr int WK = decltype(g)::value;
                if (!launch_holds(blocks, WK * B::GT) || !plan_held<T>(x_plan, n, dim) || !plan_held<T>(w_plan, 2ll * hidden, dim))
                    return RSE_ERR_UNSUPPORTED;
                hipLaunchKernelGGL((k_gated<T, B, WK, ACT, true>), dim3((unsigned)blocks), dim3(WK * B::GT), 0, s, a, view<const T>(x),
                                   view<const T>(w_gate), view<const T>(w_up), view<const T>(dout), d);
                return launch_status();
            });
            if (err) return err;
            by_shape<T>(w_plan.shape, [&](auto b) -> int64_t {
                using B = decltype(b);
                hipLaunchKernelGGL((k_gated_dw<T, B>), dim3((unsigned)(w_plan.splits * tiles<B>(2ll * hidden, dim))), dim3(B::GT), 0, s,
                                   a, dc, view<const T>(x), w_plan.len, ws.dw);
                return 0;
            });
            // (after dW, which reads x: dx may be x)
            by_shape<T>(x_plan.shape, [&](auto b) -> int64_t {
                using B = decltype(b);
                hipLaunchKernelGGL((k_gated_dx<T, B>), dim3((unsigned)(x_plan.splits * tiles<B>(n, dim))), dim3(B::GT), 0, s, a, dc,
                                   view<const T>(w_gate), view<const T>(w_up), view<T>(dx), x_plan.len,
                                   x_plan.splits > 1 ? ws.dx : nullptr);
                return 0;
            });
            if (x_plan.splits > 1)
                hipLaunchKernelGGL((k_gated_join<T>), dim3(fill_blocks(n * dim, 4 * JT, 4096)), dim3(JT), 0, s, ws.dx, x_plan.splits, n,
                                   n, dim, view<T>(dx), view<T>(dx));
        }
        hipLaunchKernelGGL((k_gated_join<T>), dim3(fill_blocks(2ll * hidden * dim, 4 * JT, 4096)), dim3(JT), 0, s, ws.dw, w_plan.splits,
                           2ll * hidden, (int64_t)hidden, dim, view<T>(dw_gate), view<T>(dw_up));
        return launch_status();
    });
}

}  // extern "C"
