// ffn.h -- the gated feed-forward block (gfx950): the products of its forward and
// its backward.
//
//   p = x W_in^T [n][2F] (the gate's F columns, then the other projection's)
//   a = act(p_g) p_u,  y = a W_out^T
//   da = gy W_out,  dp_g = da p_u act'(p_g),  dp_u = da act(p_g)
//   dx = dp W_in,  dW_in = dp^T x,  dW_out = gy^T a
//
// Six products by the tiles of tiles.h.  A tile of the first has rows of the
// gate and of the other projection in turn, 32 of each, so that both halves of
// a value of `a` meet in one thread: p leaves the registers only where the
// caller keeps it for the backward.  The backward's first product makes da, and
// dp and a from it and p, in the tile that holds da.  Matrix instructions and the
// power that they take bound the large sizes (8192 x 4096 x 16384 bf16: p and a in
// 1.96 ms, 1120 TFLOP/s with 1.3 GB written, y in 0.91, dp and a in 1.17, the three
// gradients in 4.0, 1370 TFLOP/s; the clock is at 1.5 to 1.8 GHz meanwhile).
//
// bf16 and fp16: a and dp are rounded to the inputs' type, half a step each,
// because the products that take them have operands of 16 bits; two terms of
// them, which they have where they are few (two_terms), double two thirds of the
// products.  Both are made from p in fp32, in the backward too: rounded to 16 bits
// there, p alone would add as much to the gradients' error (bf16: 3.5e-3 of their
// size, 2.3e-3 so).
//
// fp32: every operand is split into three bf16 terms (24 bits, the range of
// fp32), and the six products of terms above 2^-25 are added up: the rounding of
// fp32 products, at 1 / 6 of the bf16 rate, where the fp32 matrix instructions
// have 1 / 16 of it.
#pragma once

#include "tiles.h"

#include <utility>

namespace ttemb {

namespace {

constexpr int64_t kPad = 64;       // summed values of packed rows are padded to this
constexpr int64_t kSplit = 512;    // least summed values of a split
constexpr int kPacks = 6;          // copies that one launch makes, at most

template <class T>
struct FfnTerms {
    typedef T type;
    static constexpr int planes = 1;
};
template <>
struct FfnTerms<float> {
    typedef bf16 type;
    static constexpr int planes = 3;
};

// ------------------------------------------------------------- activations

// The values of the activation at z, and its slopes.  gelu's tanh form is z times
// the sigmoid of twice the argument, 2 sqrt(2 / pi) (z + 0.044715 z^3).  NEAR: for
// results that are rounded to 16 bits, with the hardware's exponential and
// reciprocal (off by some 2^-22 of the value), and the normal distribution's integral
// below -|z| as exp(-z^2 / 2) t P(t), t = 1 / (1 + 0.36 |z|).  P is the polynomial of
// degree 6 whose largest relative error for |z| up to 14 is least (8.5e-7 by linear
// programming; in fp32 2.1e-6 up to 6, 7.6e-6 up to 13), so the small values of the
// negative tail keep their bits, too.
template <bool NEAR>
__device__ __forceinline__ void activations(int act, const float (&z)[8], float (&value)[8], float (&slope)[8])
{
    // z times the sigmoid of x, dx the slope of x.  (What vanishes at the sigmoid's ends is
    // multiplied first: value times dx passes fp32 from z = 1.2e13 on in gelu's tanh form.)
    auto of_sigmoid = [&](int i, float x, float dx) {
        if constexpr (NEAR) {
            const float sg = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * x));
            value[i] = z[i] * sg;
            slope[i] = fmaf(value[i] * (1.f - sg), dx, sg);
        } else {
            const float e = expf(-fabsf(x)), r = 1.f / (1.f + e);
            const float sg = x < 0.f ? e * r : r, other = x < 0.f ? r : e * r; // sigmoid of x and of -x
            value[i] = z[i] * sg;
            slope[i] = fmaf(value[i] * other, dx, sg);
        }
    };
    if (act == TT_EMB_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) of_sigmoid(i, z[i], 1.f);
    } else if (act == TT_EMB_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float zz = fminf(z[i] * z[i], 1e30f); // (dx stays finite)
            of_sigmoid(i, z[i] * fmaf(0.0713548163f, zz, 1.59576912f), fmaf(0.214064449f, zz, 1.59576912f));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float c, e;
            if constexpr (NEAR) {
                e = __builtin_amdgcn_exp2f(-0.72134752f * z[i] * z[i]);
                const float t = __builtin_amdgcn_rcpf(fmaf(0.36f, fabsf(z[i]), 1.f));
                float q = fmaf(t, 0.0470081363f, -0.179592664f);
                q = fmaf(t, q, 0.180713044f);
                q = fmaf(t, q, 0.0267167525f);
                q = fmaf(t, q, 0.139659190f);
                q = fmaf(t, q, 0.141782891f);
                q = fmaf(t, q, 0.143712360f) * t * e;
                c = z[i] < 0.f ? q : 1.f - q;
            } else {
                e = expf(-0.5f * z[i] * z[i]);
                c = 0.5f * erfcf(-0.70710678f * z[i]); // (1 + erf would lose the small values)
            }
            value[i] = z[i] * c;
            slope[i] = fmaf(z[i], 0.39894228f * e, c);
        }
    }
}

// ------------------------------------------------------------------ copies

// A matrix as planes of 16-bit terms whose rows of `ld` columns are zero past
// the source's.  pair > 0: the source has 2 x pair rows, and 32 of the first
// half and 32 of the second follow each other; rows past them are zeros.  No
// source: zeros.
struct Pack {
    const void *src;
    int64_t ld_src, rows, cols;
    short *dst;
    int64_t width, ld, plane, pair; // width: columns that are written
};
struct Packs {
    Pack job[kPacks];
    int first[kPacks + 1]; // first block of each
};

template <class T>
__global__ __launch_bounds__(256) void k_ffn_pack(Packs p)
{
    typedef typename FfnTerms<T>::type E;
    constexpr int PL = FfnTerms<T>::planes;
    int k = 0;
    while (k + 1 < kPacks && (int)blockIdx.x >= p.first[k + 1]) ++k;
    const Pack &j = p.job[k];
    const int64_t chunks = j.width / 8, all = j.rows * chunks, step = (int64_t)(p.first[k + 1] - p.first[k]) * 256;
    for (int64_t c = (int64_t)((int)blockIdx.x - p.first[k]) * 256 + threadIdx.x; c < all; c += step) {
        const int64_t q = c / chunks, col = (c - q * chunks) * 8;
        int64_t r = q;
        bool in = true;
        if (j.pair) {
            const int64_t f = q / 64 * 32 + q % 32;
            in = f < j.pair;
            r = in ? f + (q & 32 ? j.pair : 0) : 0;
        }
        const int64_t left = in ? j.cols - col : 0;
        float x[8];
        load_part<T, 8>(static_cast<const T *>(j.src) + r * j.ld_src + (left > 0 ? col : 0),
                        (int)(left < 0 ? 0 : left < 8 ? left : 8), x);
        s16x8 w[PL];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            short s[PL];
            split_terms<E, PL>(x[i], s);
#pragma unroll
            for (int t = 0; t < PL; ++t) w[t][i] = s[t];
        }
#pragma unroll
        for (int t = 0; t < PL; ++t) *reinterpret_cast<s16x8 *>(j.dst + t * j.plane + q * j.ld + col) = w[t];
    }
}

// ---------------------------------------------------------------- products

// What a product's tiles become: a (and p), dp and a, or rows of an output (or
// of a partial sum of it, where `sum` is set).
enum { FFN_IN, FFN_MID, FFN_OUT };

struct FfnOut {
    int64_t rows, cols; // of the output
    void *out;
    int64_t ld_out;
    float *sum; // [splits][rows][cols]
    int splits;
    int64_t split_k;
    int64_t F;
    int act;
    float *pre; // [rows][2F]
    int64_t ld_pre;
    short *mid; // planes of [rows][ld_mid]
    int64_t ld_mid, plane_mid;
    short *dpre; // planes of [rows][ld_dpre]
    int64_t ld_dpre, plane_dpre;
    bool two_mid, two_dpre; // a, dp have two terms (16-bit types)
    bool two;               // an operand has: the latter half of the parts are the second's
};

// Rows of both projections as they lie in memory, 32 of the one and 32 of the
// other in turn: one load of a wave group fills 32 rows of a stage of 64 values.
template <int R>
struct PairLoader {
    typedef TileLds<false, R, 64> L;
    static constexpr int N = L::vecs;
    const short *gate, *up;
    int at, all, todo; // as in TileLoader, going round
    unsigned bytes;
    int off, step, to;

    __device__ __forceinline__ PairLoader(const Operand &a, int64_t F, int64_t r0, int stages, int first)
    {
        const int ld = (int)a.ld;
        const int64_t f0 = r0 / 2;
        const int rows = (int)(F - f0 < R / 2 ? F - f0 : R / 2);
        gate = a.p + f0 * a.ld + first * 64;
        up = gate + F * a.ld;
        at = first;
        all = stages;
        todo = rows > 0 ? stages : 0;
        bytes = (unsigned)((rows - 1) * ld + (int)a.cols) * 2 - first * 128;
        const int t = threadIdx.x, row = t / 8;
        off = (row * ld + ((t % 8) ^ L::turn(row)) * 8) * 2;
        step = 32 * ld * 2;
        to = __builtin_amdgcn_readfirstlane(t >> 6) * 1024;
    }
    __device__ __forceinline__ void load(char *lds)
    {
        const unsigned now = todo > 0 ? bytes : 0;
        const __amdgpu_buffer_rsrc_t g =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<short *>(gate), 0, now, 0x00027000);
        const __amdgpu_buffer_rsrc_t u = __builtin_amdgcn_make_buffer_rsrc(const_cast<short *>(up), 0, now, 0x00027000);
#pragma unroll
        for (int i = 0; i < N; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(i & 1 ? u : g, (lds_void)(lds + i * 4096 + to), 16, off,
                                                     i / 2 * step, 0, 0);
        gate += 64;
        up += 64;
        bytes -= 128;
        --todo;
        if (++at == all) {
            at = 0;
            gate -= all * 64;
            up -= all * 64;
            bytes += all * 128;
        }
    }
};

// Eight values of a row as they leave.
template <class T, int PL>
__device__ __forceinline__ void store_terms(short *p, int64_t plane, int left, const float (&x)[8])
{
    typedef typename FfnTerms<T>::type E;
    short w[PL][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        short s[PL];
        split_terms<E, PL>(x[i], s);
#pragma unroll
        for (int q = 0; q < PL; ++q) w[q][i] = s[q];
        // what rounds to infinity stays that
        if (PL == 2 && !(fabsf((float)__builtin_bit_cast(E, w[0][i])) < INFINITY)) w[1][i] = 0;
    }
#pragma unroll
    for (int q = 0; q < PL; ++q) {
        if (left >= 8) {
            typedef s16x8 __attribute__((aligned(2))) any8;
            s16x8 v;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = w[q][i];
            *reinterpret_cast<any8 *>(p + q * plane) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) p[q * plane + i] = w[q][i];
        }
    }
}

template <class T, int PL>
__device__ __forceinline__ void store_terms(short *p, int64_t plane, int left, const float (&x)[8], bool two)
{
    if (PL == 1 && two) store_terms<T, 2>(p, plane, left, x);
    else store_terms<T, PL>(p, plane, left, x);
}

// f for each of the numbers, as constants.
template <class F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>()), ...);
}

// Shapes of a product's tiles, (64 NI) x (64 NJ).  BIG ones read each operand
// least often.  Of SMALL ones a compute unit holds two, which hide each other's
// loads, starts and ends; of DEEP and SLIM ones, for grids that leave it no second,
// one with more loads in flight.  Three terms take three times the LDS (and no DEEP
// ones, which measured as SMALL ones do).
enum { BIG, SMALL, DEEP, SLIM };
template <int PL, int SHAPE>
struct FfnShape {
    static constexpr bool ahead = SHAPE == DEEP || SHAPE == SLIM;
    static constexpr int NI = SHAPE == BIG ? 4 : 2, NJ = PL > 1 ? NI / 2 : SHAPE == SLIM ? 1 : NI;
    static constexpr int TM = 64 * NI, TN = 64 * NJ;
};
inline int64_t tile_m(int shape) { return shape == BIG ? 256 : 128; }
inline int64_t tile_n(int PL, int shape) { return PL > 1 || shape == SLIM ? tile_m(shape) / 2 : tile_m(shape); }

// LDS of a product's tiles.  A tile leaves through LDS in fp32, in parts of 64
// rows and BP blocks of 32 columns of each half (as many as leave room for two
// blocks of small tiles on a compute unit).
template <int PL, bool XT, bool YT, int SHAPE>
struct FfnLds : FfnShape<PL, SHAPE> {
    typedef FfnShape<PL, SHAPE> S;
    typedef Stages<PL, XT, S::ahead> Stage;
    static constexpr int BK = Stage::values, NB = Stage::buffers;
    static constexpr int stage = PL * (TileLds<XT, S::TM, BK>::bytes + TileLds<YT, S::TN, BK>::bytes);
    static constexpr int BP = NB == 4 && SHAPE == SMALL ? 1 : 2, PW = 32 * BP, P = 2 * PW * 4 + 16, part = 64 * P;
    static constexpr int first = part > stage ? part : stage, more = NB == 4 ? stage : 16; // of two buffers each
};

// Which of the eight XCDs takes which tiles of a small grid: ranges of the tiles
// along m (p of them) and n (q) and of the sum's splits (r), p q r = 8, so that an
// XCD's L2 reads few rows of both operands.
struct XcdParts {
    int p, q, r; // their logarithms
};
__device__ __forceinline__ bool xcd_tile(const XcdParts &x, unsigned block, int mt, int nt, int splits, int64_t &m,
                                         int64_t &n, int &split)
{
    const int xcd = block & 7, local = (int)(block >> 3);
    const int ri = xcd & ((1 << x.r) - 1), qi = xcd >> x.r & ((1 << x.q) - 1), pi = xcd >> (x.r + x.q);
    const int m0 = pi * mt >> x.p, n0 = qi * nt >> x.q, s0 = ri * splits >> x.r;
    const int dm = ((pi + 1) * mt >> x.p) - m0, dn = ((qi + 1) * nt >> x.q) - n0, ds = ((ri + 1) * splits >> x.r) - s0;
    if (local >= dm * dn * ds) return false;
    const int row = (int)((unsigned)local / (unsigned)dm), part = (int)((unsigned)row / (unsigned)dn);
    m = m0 + local - row * dm;
    n = n0 + row - part * dn;
    split = s0 + part;
    return true;
}
inline XcdParts xcd_parts(int64_t mt, int64_t nt, int64_t splits, unsigned &grid)
{
    XcdParts best{0, 0, 3};
    int64_t cost = -1;
    for (int p = 0; p <= 3; ++p)
        for (int q = 0; p + q <= 3; ++q) {
            const int r = 3 - p - q;
            auto share = [](int64_t of, int log) { return (of + (1 << log) - 1) >> log; };
            const int64_t dm = share(mt, p), dn = share(nt, q), ds = share(splits, r);
            // the longest XCD's work, then the operands' rows that it reads
            const int64_t c = (dm * dn * ds + 3) / 4 * 4096 + (dm + dn) * ds;
            if (cost >= 0 && c >= cost) continue;
            cost = c;
            best = {p, q, r};
            grid = (unsigned)(8 * dm * dn * ds);
        }
    return best;
}

// A tile of one product: M outputs (along X's rows or columns) in each of N rows,
// K summed values, mt x nt tiles taken by `grid` blocks.  PAIRED: X is W_in as it
// lies in memory.
struct FfnJob {
    Operand X, Y;
    int64_t K, mt, nt;
    unsigned grid;
    XcdParts xcds;
    FfnOut o;
};
template <class T, bool XT, bool YT, int OUT, bool PAIRED, int SHAPE>
__device__ __forceinline__ void ffn_tile(const FfnJob &job, unsigned block, char *lds0, char *lds1, char *lds2,
                                         char *lds3)
{
    typedef typename FfnTerms<T>::type E;
    constexpr int PL = FfnTerms<T>::planes;
    typedef FfnLds<PL, XT, YT, SHAPE> Lds;
    constexpr int NI = Lds::NI, NJ = Lds::NJ, TM = Lds::TM, TN = Lds::TN, BK = Lds::BK;
    constexpr int BP = Lds::BP, PM = NI / BP, PW = Lds::PW, P = Lds::P;
    Operand X = job.X, Y = job.Y;
    const FfnOut &o = job.o;
    int64_t mi, ni, K = job.K;
    int sp;
    if (in_patches(job.mt, job.nt)) {
        if (!tile_of(block, job.grid, job.mt, job.nt, 1, mi, ni, sp)) return;
    } else if (!xcd_tile(job.xcds, block, (int)job.mt, (int)job.nt, OUT == FFN_OUT ? o.splits : 1, mi, ni, sp)) {
        return;
    }
    float *sum = nullptr;
    if (OUT == FFN_OUT && o.sum) { // this split's part of the sum
        const int parts = o.two ? o.splits / 2 : o.splits, second = sp >= parts;
        const int64_t k0 = (sp - second * parts) * o.split_k;
        auto from = [&](Operand &a, bool turned) {
            a.p += (turned ? k0 * a.ld : k0) + second * a.plane;
            (turned ? a.rows : a.cols) -= k0;
        };
        from(X, XT);
        from(Y, YT);
        K = K - k0 < o.split_k ? K - k0 : o.split_k;
        sum = o.sum + sp * o.rows * o.cols;
    }
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave & 1, wn = wave >> 1;
    const int64_t m0 = mi * TM, n0 = ni * TN;
    f32x16 acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    // eight values of a row per thread at a time; FFN_IN: of both projections
    constexpr int ROWV = (OUT == FFN_IN ? PW : 2 * PW) / 8, ITEMS = 64 * ROWV / 256, PARTS = NJ * PM;
    auto row_at = [&](int j, int k) {
        const int r = (tid + k * 256) / ROWV;
        return n0 + (r >> 5) * (TN / 2) + j * 32 + (r & 31);
    };
    auto col_at = [&](int h, int k) { // (of the output; FFN_IN: of a)
        const int at = (tid + k * 256) % ROWV * 8;
        if constexpr (OUT == FFN_IN) return m0 / 2 + at / 32 * (TM / 4) + h * 32 + at % 32;
        else return m0 + at / PW * (TM / 2) + h * PW + at % PW;
    };
    // p of a part, asked for while the part before is worked on
    float pre[OUT == FFN_MID ? ITEMS : 1][2][8];
    auto load_pre = [&](int part) {
        if constexpr (OUT == FFN_MID) {
            const int j = part / PM, h = part % PM;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int64_t i = row_at(j, k), m = col_at(h, k);
                // (from the last row and columns where there is none)
                const float *from = o.pre + (i < o.rows ? i : o.rows - 1) * o.ld_pre;
                const int left = m >= o.F ? 0 : o.F - m < 8 ? (int)(o.F - m) : 8;
                if (o.F >= 8) {
                    const int64_t c = left == 8 ? m : o.F - 8; // the last eight, moved into place when they are used
                    load_vec<float, 8>(from + c, pre[k][0]);
                    load_vec<float, 8>(from + o.F + c, pre[k][1]);
                } else {
                    load_part<float, 8>(from + (left ? m : 0), left, pre[k][0]);
                    load_part<float, 8>(from + o.F + (left ? m : 0), left, pre[k][1]);
                }
            }
        }
    };
    load_pre(0); // (there long before the products are)
    {
        const int stages = (int)(K / BK);
        // Tiles begin at different places of the sum where rows lie along it: rows a
        // multiple of a KB apart meet in few channels of the L2 (8192 x 4096 x 16384:
        // p and a 2.06 -> 1.94 ms, y 1.09 -> 0.98).  Small grids gain nothing.
        constexpr bool ROT = !YT && SHAPE == BIG;
        const int first = ROT ? (int)((8 * mi + ni) & 31) % stages : 0;
        TileLoader<YT, TN, BK, PL, ROT> y(Y, n0, stages, first);
        if constexpr (PAIRED) {
            PairLoader<TM> x(X, o.F, m0, stages, first);
            multiply<E, PL, XT, YT, Lds::ahead>(x, y, stages, lds0, lds1, lds2, lds3, acc);
        } else {
            TileLoader<XT, TM, BK, PL, ROT> x(X, m0, stages, first);
            multiply<E, PL, XT, YT, Lds::ahead>(x, y, stages, lds0, lds1, lds2, lds3, acc);
        }
    }
    __syncthreads();
    // One body for all parts, so that it stays in the instruction cache (unrolled,
    // dp and a in BIG tiles were 150 KB of code); only the registers that leave
    // have to be named.
#pragma clang loop unroll(disable)
    for (int p = 0; p < PARTS; ++p) {
        char *part = p & 1 ? lds1 : lds0; // one is written while the last is read
        each_of(std::make_integer_sequence<int, PARTS>(), [&](auto which) {
            constexpr int c = decltype(which)::value, j = c / PM, h = c % PM;
            if (p != c) return;
#pragma unroll
            for (int b = 0; b < BP; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16 &v = acc[h * BP + b][j];
                    const int col = wm * PW + b * 32 + 8 * q + 4 * (lane >> 5);
                    *reinterpret_cast<float4 *>(part + (wn * 32 + (lane & 31)) * P + col * 4) =
                        make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                }
        });
        float here[OUT == FFN_MID ? ITEMS : 1][2][8];
        if constexpr (OUT == FFN_MID) {
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    here[k][0][e] = pre[k][0][e];
                    here[k][1][e] = pre[k][1][e];
                }
            if (p + 1 < PARTS) load_pre(p + 1);
        }
        __syncthreads();
        const int j = p / PM, h = p % PM;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int c = tid + k * 256, at = c % ROWV * 8;
            const char *from = part + c / ROWV * P;
            const int64_t i = row_at(j, k), m = col_at(h, k);
            if constexpr (OUT == FFN_IN) {
                float g[8], u[8], a[8], slope[8];
                const char *gate = from + (at / 32 * PW + at % 32) * 4;
                load_vec<float, 8>(reinterpret_cast<const float *>(gate), g);
                load_vec<float, 8>(reinterpret_cast<const float *>(gate + 128), u);
                activations<PL == 1>(o.act, g, a, slope);
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = m + e < o.F ? a[e] * u[e] : 0.f;
                if (i >= o.rows || m >= o.ld_mid) continue;
                store_terms<T, PL>(o.mid + i * o.ld_mid + m, o.plane_mid, 8, a, SHAPE != BIG && o.two_mid);
                if (o.pre && m < o.F) {
                    float *to = o.pre + i * o.ld_pre + m;
                    const int left = (int)(o.F - m < 8 ? o.F - m : 8);
                    store_part<float, 8>(to, left, g);
                    store_part<float, 8>(to + o.F, left, u);
                }
            } else {
                const int left = (int)(o.cols - m < 8 ? o.cols - m : 8);
                float x[8];
                load_vec<float, 8>(reinterpret_cast<const float *>(from + at * 4), x);
                if constexpr (OUT == FFN_MID) {
                    float g[8], u[8], a[8], slope[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        g[e] = here[k][0][e];
                        u[e] = here[k][1][e];
                    }
                    if (left > 0 && left < 8 && o.F >= 8) { // the last columns, from the last eight values
                        for (int shift = left; shift < 8; ++shift) {
#pragma unroll
                            for (int e = 0; e < 7; ++e) {
                                g[e] = g[e + 1];
                                u[e] = u[e + 1];
                            }
                        }
                    }
                    activations<PL == 1>(o.act, g, a, slope);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        g[e] = x[e] * u[e] * slope[e];
                        slope[e] = a[e] * u[e];
                        u[e] = x[e] * a[e];
                    }
                    if (i >= o.rows || left <= 0) continue;
                    store_terms<T, PL>(o.mid + i * o.ld_mid + m, o.plane_mid, left, slope, SHAPE != BIG && o.two_mid);
                    short *d = o.dpre + i * o.ld_dpre + m;
                    store_terms<T, PL>(d, o.plane_dpre, left, g, SHAPE != BIG && o.two_dpre);
                    store_terms<T, PL>(d + o.F, o.plane_dpre, left, u, SHAPE != BIG && o.two_dpre);
                } else {
                    if (i >= o.rows || left <= 0) continue;
                    if (sum) store_part<float, 8>(sum + i * o.cols + m, left, x);
                    else store_part<T, 8>(static_cast<T *>(o.out) + i * o.ld_out + m, left, x);
                }
            }
        }
    }
}

template <class T, bool XT, bool YT, int OUT, bool PAIRED, int SHAPE>
__global__ __launch_bounds__(256, 1) void k_ffn(FfnJob job)
{
    typedef FfnLds<FfnTerms<T>::planes, XT, YT, SHAPE> Lds;
    __shared__ __align__(16) char lds0[Lds::first];
    __shared__ __align__(16) char lds1[Lds::first];
    __shared__ __align__(16) char lds2[Lds::more];
    __shared__ __align__(16) char lds3[Lds::more];
    ffn_tile<T, XT, YT, OUT, PAIRED, SHAPE>(job, blockIdx.x, lds0, lds1, lds2, lds3);
}

// Outputs from their splits' sums.
struct Join {
    const float *sum;
    int splits;
    int64_t rows, cols;
    void *out;
    int64_t ld;
};
struct Joins {
    Join job[3];
    int first[4]; // first block of each
};
template <class T>
__global__ __launch_bounds__(256) void k_ffn_join(Joins p)
{
    const int k = (int)blockIdx.x < p.first[1] ? 0 : (int)blockIdx.x < p.first[2] ? 1 : 2;
    const Join &j = p.job[k];
    const int64_t chunks = (j.cols + 3) / 4, all = j.rows * chunks, step = (int64_t)(p.first[k + 1] - p.first[k]) * 256;
    for (int64_t c = (int64_t)((int)blockIdx.x - p.first[k]) * 256 + threadIdx.x; c < all; c += step) {
        const int64_t i = c / chunks, m = (c - i * chunks) * 4;
        const int left = (int)(j.cols - m < 4 ? j.cols - m : 4);
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int q = 0; q < j.splits; ++q) {
            float y[4];
            load_part<float, 4>(j.sum + ((int64_t)q * j.rows + i) * j.cols + m, left, y);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] += y[r];
        }
        store_part<T, 4>(static_cast<T *>(j.out) + i * j.ld + m, left, x);
    }
}

// ------------------------------------------------------------ host: plans

unsigned blocks_for(int64_t threads)
{
    const int64_t b = (threads + 255) / 256;
    return (unsigned)(b < 16384 ? b : 16384);
}

// A product's sizes: M outputs in each of N rows, K summed values in `splits`
// parts of `each`; two: each part is there for both terms of an operand.
struct FfnSize {
    int64_t M, N, K;
    bool two;
    int splits;
    int64_t each;

    size_t bytes() const { return splits > 1 ? round256((size_t)splits * M * N * sizeof(float)) : 0; }
};
inline int64_t tiles_of(const FfnSize &z, int PL, int shape)
{
    const int64_t TM = tile_m(shape), TN = tile_n(PL, shape);
    return ((z.M + TM - 1) / TM) * ((z.N + TN - 1) / TN);
}

// The shape of the tiles of a launch of products, and how often each product's
// sum is split (may_split).
//
// 16 bits: BIG for two rounds of the compute units (2048 x 1024 x 4096, one round,
// p and a: 53 us, 47 in SMALL ones), else SMALL where some units get two of them
// (777 x 1024 x 2688, all outputs of the backward: 34 us, 46 in DEEP ones), else
// DEEP (300 x 4096 x 1000, p and a: 28 us, 43 in SMALL ones), or SLIM where there
// are units for them, too (21 us; 128 x 1024 x 4096: 9.5, 12.8 in DEEP ones).  fp32,
// whose products are six times as long: BIG for one round, counting the splits of a
// long sum (2048 x 2048 x 4096, y: 188 us, 240 in SMALL ones; 777 x 1024 x 2688: 47
// and 41), else SMALL.
//
// Sums are split so that the units have equal work, one block each (of the
// backward's SMALL tiles two), but not below kSplit values, a quarter of them for
// fp32: joining the parts is a launch, 4 us or more.
int ffn_shape(FfnSize *z, int count, int PL, bool may_split)
{
    int64_t big = 0, small = 0, slim = 0, work = 0;
    for (int i = 0; i < count; ++i) {
        const int64_t parts = may_split && PL > 1 ? (z[i].K < 1024 ? 1 : z[i].K < 4096 ? z[i].K / 1024 : 4) : 1;
        big += tiles_of(z[i], PL, BIG) * parts;
        small += tiles_of(z[i], PL, SMALL);
        slim += tiles_of(z[i], PL, SLIM);
    }
    const int shape = big >= (PL > 1 ? kCUs : 2 * kCUs) ? BIG
                      : PL > 1 || small > kCUs          ? SMALL
                                                        : slim > kCUs ? DEEP : SLIM;
    for (int i = 0; i < count; ++i) work += tiles_of(z[i], PL, shape) * z[i].K;
    const int64_t blocks = shape == SMALL && count > 1 ? 2 * kCUs : kCUs, least = PL > 1 ? kSplit / 4 : kSplit;
    for (int i = 0; i < count; ++i) {
        int64_t s = may_split ? (z[i].K * blocks + work - 1) / work : 1;
        if (z[i].two) s /= 2;
        if (s > z[i].K / least) s = z[i].K / least;
        if (s < 1) s = 1;
        z[i].each = up((z[i].K + s - 1) / s, kPad);
        z[i].splits = (int)((z[i].K + z[i].each - 1) / z[i].each) * (z[i].two ? 2 : 1);
    }
    return shape;
}
struct FfnSplit {
    int parts;
    int64_t each;
};

// Forward products of few rows take kernels of their own: 16-bit rows up to 16
// (4096 x 16384: 1 row 72 us, 16 rows 90, 17 rows 124 and by tiles 106), fp32 rows
// up to 128, whose tiles take a split copy of the weights (4 rows 147 us).
inline bool few_rows(int64_t n, bool fp32) { return n <= (fp32 ? 128 : 16); }
// Parts of a sum of K values that leave through `rows` columns: a block for each
// compute unit, of 256 summed values at least.
FfnSplit few_split(int64_t rows, int64_t K)
{
    const int64_t blocks = (rows + 15) / 16;
    int64_t s = kCUs / blocks;
    if (s > K / 256) s = K / 256;
    if (s < 1) s = 1;
    const int64_t each = up((K + s - 1) / s, 128);
    return {(int)((K + each - 1) / each), each};
}
size_t few_bytes(int64_t n, int64_t rows, int64_t K)
{
    const FfnSplit s = few_split(rows, K);
    return s.parts > 1 ? round256((size_t)s.parts * n * rows * sizeof(float)) : 0;
}

// Whether an operand serves as it lies in memory: 16-bit rows at multiples of 16
// bytes (further apart they would pass the 31 bits of a tile's loads) and of whole
// pieces of 16 bytes, or where they lie along the sum of whole steps: a piece that
// the last row's end cuts would be read past it.
bool lies_well(const void *p, int64_t ld)
{
    return ld % 8 == 0 && ld <= (1 << 20) && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}
// Which operands are copied.
struct FfnCopies {
    bool x, w_in, w_out, gy;
};
FfnCopies ffn_copies(bool fp32, bool grad, int64_t n, int64_t D, int64_t F, bool x, bool w_in, bool w_out, bool gy)
{
    const bool d = D % kPad == 0, f = F % kPad == 0;
    if (!grad && few_rows(n, fp32)) return {false, false, false, false};
    if (fp32) return {true, true, true, true};
    if (grad) return {!x || D % 8, !w_in || D % 8, !w_out || F % 8, !gy || !d}; // only gy lies along a sum
    return {!x || !d, !w_in || !d, !w_out || !f, false};
}

// Products that take a or dp of 16-bit inputs in two terms, 16 bits or more.  One term's
// roundings bring the outputs' error to 1.41 times their own rounding where both are
// many; few of either do not average out: of 400 draws of y the largest were 1.6 times
// with 2^11 outputs or values of a, 1.8 with 742 and 266 (14 x 53 x 19), 3.4 with 16 outputs
// of 16384 values.  So the fewer of the two decides, for each product by itself: a second
// term doubles the product and adds the join of its parts, 0 to 6 us of a call where
// the outputs are few, 14 us of 24 if the 1.2 million outputs of w_in's gradient at
// 4 x 300 x 2000 had it too, 21 of 27 at 64 x 2048 x 1024.
//
// outputs: grids in patches are not split, so a product with two terms has few tiles.
// n F and n: the tiles that store two terms are not BIG ones (never 512 of those).
bool two_terms(int64_t n, int64_t F, int64_t outputs)
{
    const int64_t values = n * F;
    return (values < outputs ? values : outputs) <= 1 << 11 && outputs <= 1 << 22 && values <= 1 << 20 && n <= 1 << 16;
}
// The sums of y, and of the gradients of x, w_in and w_out.
FfnSize y_size(int64_t n, int64_t D, int64_t F, int PL, int *shape = nullptr)
{
    FfnSize z{D, n, up(F, kPad), PL == 1 && two_terms(n, F, n * D)};
    const int s = ffn_shape(&z, 1, PL, true);
    if (shape) *shape = s;
    return z;
}
int grad_sizes(FfnSize *z, int64_t n, int64_t D, int64_t F, int PL)
{
    z[0] = {D, n, up(2 * F, kPad), PL == 1 && two_terms(n, F, n * D)};
    z[1] = {D, 2 * F, up(n, kPad), PL == 1 && two_terms(n, F, 2 * F * D)};
    z[2] = {F, D, up(n, kPad), PL == 1 && two_terms(n, F, F * D)};
    return ffn_shape(z, 3, PL, true);
}

struct FfnPlan {
    short *x, *w_in, *w_out, *gy, *mid, *dpre;
    float *sum;
    int64_t Dp, Fp, Pp; // padded columns of x and gy, of a, of dp
    int64_t ldD, ldF, ldP;
    bool two_mid, two_dpre;
    size_t bytes;
};
// Distance of rows of so many columns: an odd number of cache lines where it would
// be a multiple of 1 KB, at which a tile's rows meet in few channels of the L2
// (8192 x 4096 x 16384, rows of a 32 KB apart: y in 997 us, 902 with one line more).
inline int64_t apart(int64_t cols) { return cols % 512 ? cols : cols + 64; }

FfnPlan plan_ffn(int64_t n, int64_t D, int64_t F, int PL, bool grad, const FfnCopies &c, char *base)
{
    size_t off = TT_EMB_STATUS_BYTES;
    auto take = [&](int64_t rows, int64_t cols, int planes) {
        char *r = base ? base + off : nullptr;
        off += round256((size_t)planes * rows * cols * 2);
        return reinterpret_cast<short *>(r);
    };
    FfnPlan p{};
    if (n < 1) n = 1; // no rows: the least workspace
    p.Dp = up(D, kPad);
    p.Fp = up(F, kPad);
    p.Pp = up(2 * F, kPad);
    p.ldD = apart(p.Dp);
    p.ldF = apart(p.Fp);
    p.ldP = apart(p.Pp);
    if (c.x) p.x = take(n, p.ldD, PL);
    if (c.w_in) p.w_in = take(grad ? 2 * F : 2 * up(F, 32), p.ldD, PL);
    if (c.w_out) p.w_out = take(D, p.ldF, PL);
    if (c.gy) p.gy = take(n, p.ldD, PL);
    size_t sums;
    if (grad) {
        FfnSize z[3];
        grad_sizes(z, n, D, F, PL);
        p.two_dpre = z[0].two || z[1].two;
        p.two_mid = z[2].two;
        sums = z[0].bytes() + z[1].bytes() + z[2].bytes();
    } else if (few_rows(n, PL > 1)) {
        p.two_mid = PL == 1 && two_terms(n, F, n * D);
        sums = few_bytes(n, D, F);
    } else {
        const FfnSize z = y_size(n, D, F, PL);
        p.two_mid = z.two;
        sums = z.bytes();
    }
    p.mid = take(n, p.ldF, p.two_mid ? 2 : PL);
    if (grad) p.dpre = take(n, p.ldP, p.two_dpre ? 2 : PL);
    p.sum = reinterpret_cast<float *>(base ? base + off : nullptr);
    off += sums;
    p.bytes = off;
    return p;
}
FfnCopies copies_of(const FfnArgs &a, int dtype, bool grad)
{
    return ffn_copies(dtype == TT_EMB_DTYPE_FLOAT, grad, a.n, a.D, a.F, lies_well(a.x, a.ld_x),
                      lies_well(a.w_in, a.ld_in), lies_well(a.w_out, a.ld_out), lies_well(a.gy, a.ld_gy));
}

// ---------------------------------------------------------- host: launches

template <class T>
struct Packing {
    Packs p{};
    int n = 0;

    // The operand that a copy (where there is one) or the matrix itself makes.
    Operand operator()(const void *src, int64_t ld, int64_t rows, int64_t cols, short *dst, int64_t width, int64_t pair)
    {
        if (!dst) return Operand{static_cast<const short *>(src), ld, 0, rows, cols};
        const int64_t to = pair ? 2 * up(pair, 32) : rows, ldp = apart(width);
        add(Pack{src, ld, to, cols, dst, width, ldp, to * ldp, pair});
        return Operand{dst, ldp, FfnTerms<T>::planes > 1 ? to * ldp : 0, to, width};
    }
    void add(const Pack &job)
    {
        p.job[n] = job;
        p.first[n + 1] = p.first[n] + (int)blocks_for(job.rows * (job.width / 8));
        ++n;
    }
    void run(hipStream_t s)
    {
        if (!n) return;
        for (int k = n; k < kPacks; ++k) p.first[k + 1] = p.first[k];
        hipLaunchKernelGGL(k_ffn_pack<T>, dim3((unsigned)p.first[n]), dim3(256), 0, s, p);
    }
};

FfnJob job_of(const Operand &x, const Operand &y, const FfnSize &z, int PL, int shape, const FfnOut &o)
{
    const int64_t TM = tile_m(shape), TN = tile_n(PL, shape);
    const int64_t mt = (z.M + TM - 1) / TM, nt = (z.N + TN - 1) / TN;
    FfnJob job{x, y, z.K, mt, nt, 0, {}, o};
    if (in_patches(mt, nt)) job.grid = tile_grid(mt, nt, 1);
    else job.xcds = xcd_parts(mt, nt, z.splits, job.grid);
    return job;
}

template <class T, bool XT, bool YT, int OUT, bool PAIRED>
void launch(const FfnJob &job, int shape, hipStream_t s)
{
    auto run = [&](auto c) {
        hipLaunchKernelGGL((k_ffn<T, XT, YT, OUT, PAIRED, decltype(c)::value>), dim3(job.grid), dim3(256), 0, s, job);
    };
    if (shape == BIG) run(std::integral_constant<int, BIG>());
    if (shape == SMALL) run(std::integral_constant<int, SMALL>());
    if constexpr (FfnTerms<T>::planes == 1) {
        if (shape == DEEP) run(std::integral_constant<int, DEEP>());
        if (shape == SLIM) run(std::integral_constant<int, SLIM>());
    }
}

template <class T, bool XT, bool YT, int OUT, bool PAIRED>
void product(const Operand &x, const Operand &y, int64_t M, int64_t N, int64_t K, const FfnOut &o, hipStream_t s)
{
    constexpr int PL = FfnTerms<T>::planes;
    FfnSize z{M, N, K};
    const int shape = ffn_shape(&z, 1, PL, false);
    launch<T, XT, YT, OUT, PAIRED>(job_of(x, y, z, PL, shape, o), shape, s);
}

// Outputs [N][M] of T: each job takes what it needs of the room for partial sums.
template <class T>
struct Outputs {
    float *sum;
    Joins joins{};
    int n = 0;

    FfnJob operator()(const Operand &x, const Operand &y, const FfnSize &z, int shape, void *out, int64_t ld)
    {
        FfnOut o{};
        o.rows = z.N;
        o.cols = z.M;
        o.out = out;
        o.ld_out = ld;
        o.splits = z.splits;
        if (z.splits > 1) {
            o.sum = sum;
            o.split_k = z.each;
            o.two = z.two; // (operands without a second term have a plane of 0)
            sum += z.bytes() / sizeof(float);
            joins.job[n] = Join{o.sum, z.splits, z.N, z.M, out, ld};
            joins.first[n + 1] = joins.first[n] + (int)blocks_for(z.N * ((z.M + 3) / 4));
            ++n;
        }
        return job_of(x, y, z, FfnTerms<T>::planes, shape, o);
    }
    void join(hipStream_t s)
    {
        if (!n) return;
        for (int k = n; k < 3; ++k) joins.first[k + 1] = joins.first[k];
        hipLaunchKernelGGL(k_ffn_join<T>, dim3((unsigned)joins.first[n]), dim3(256), 0, s, joins);
    }
};

} // namespace

} // namespace ttemb
