// ffn.hip -- the gated feed-forward block, forward and backward (gfx950).
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
// dp and a from it and p, in the tile that holds da.  Matrix instructions bound
// the large sizes.
//
// bf16 and fp16: a and dp are rounded to the inputs' type, half a step each,
// because the products that take them have operands of 16 bits; two terms of
// them would double two thirds of the products.  Both are made from p before its
// rounding in the forward, after it in the backward.
//
// fp32: every operand is split into three bf16 terms (24 bits, the range of
// fp32), and the six products of terms above 2^-25 are added up: the rounding of
// fp32 products, at 1 / 6 of the bf16 rate, where the fp32 matrix instructions
// have 1 / 16 of it.
#include "tiles.h"

#include <utility>

namespace ttemb {

namespace {

constexpr int64_t kPad = 64;       // summed values of packed rows are padded to this
constexpr int64_t kSplit = 512;    // least summed values of a split
constexpr int kPacks = 5;          // copies that one launch makes, at most

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
// reciprocal (off by some 2^-22 of the value) and, for the normal distribution's
// integral, formula 7.1.26 of Abramowitz and Stegun (off by 1.5e-7).
template <bool NEAR>
__device__ __forceinline__ void activations(int act, const float (&z)[8], float (&value)[8], float (&slope)[8])
{
    if (act == TT_EMB_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float c, e;
            if constexpr (NEAR) {
                e = __builtin_amdgcn_exp2f(-0.72134752f * z[i] * z[i]);
                const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f * 0.70710678f, fabsf(z[i]), 1.f));
                float q = fmaf(t, 1.061405429f, -1.453152027f);
                q = fmaf(t, q, 1.421413741f);
                q = fmaf(t, q, -0.284496736f);
                q = fmaf(t, q, 0.254829592f) * t * 0.5f * e;
                c = z[i] < 0.f ? q : 1.f - q;
            } else {
                e = expf(-0.5f * z[i] * z[i]);
                c = 0.5f * erfcf(-0.70710678f * z[i]); // (1 + erf would lose the small values)
            }
            value[i] = z[i] * c;
            slope[i] = fmaf(z[i], 0.39894228f * e, c);
        }
        return;
    }
    const float cube = act == TT_EMB_ACT_GELU_TANH ? 0.044715f : 0.f, by = cube ? 1.59576912f : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float zz = cube * z[i] * z[i], x = by * fmaf(zz, z[i], z[i]), dx = by * fmaf(3.f, zz, 1.f);
        const float e = NEAR ? __builtin_amdgcn_exp2f(-1.44269504f * fabsf(x)) : expf(-fabsf(x));
        const float r = NEAR ? __builtin_amdgcn_rcpf(1.f + e) : 1.f / (1.f + e);
        const float sg = x < 0.f ? e * r : r, other = x < 0.f ? r : e * r; // sigmoid of x and of -x
        value[i] = z[i] * sg;
        slope[i] = fmaf(z[i] * dx, sg * other, sg);
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

// f for each of the numbers, as constants: a long loop's body may be left as a
// loop, whose registers would then be memory.
template <class F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>()), ...);
}

// LDS of a product's tiles.  A tile leaves through LDS in fp32, in parts of 64
// rows and BP blocks of 32 columns of each half (as many as leave room for two
// blocks of small tiles on a compute unit).
template <int PL, bool XT, bool YT, int NI, int NJ>
struct FfnLds {
    static constexpr int TM = 64 * NI, TN = 64 * NJ, BK = Stages<PL, XT>::values, NB = Stages<PL, XT>::buffers;
    static constexpr int stage = PL * (TileLds<XT, TM, BK>::bytes + TileLds<YT, TN, BK>::bytes);
    static constexpr int BP = NB == 4 && NI == 2 ? 1 : 2, PW = 32 * BP, P = 2 * PW * 4 + 16, part = 64 * P;
    static constexpr int first = part > stage ? part : stage, more = NB == 4 ? stage : 16; // of two buffers each
};

// Which of the eight XCDs takes which tiles of a small grid: ranges of the tiles
// along m (p of them) and n (q) and of the sum's splits (r), p q r = 8, so that an
// XCD's L2 reads few rows of both operands.
struct XcdParts {
    int p, q, r;
};
__device__ __forceinline__ bool xcd_tile(const XcdParts &x, unsigned block, int mt, int nt, int splits, int64_t &m,
                                         int64_t &n, int &split)
{
    const int xcd = block & 7, local = (int)(block >> 3);
    const int ri = xcd % x.r, qi = xcd / x.r % x.q, pi = xcd / (x.r * x.q);
    const int m0 = pi * mt / x.p, n0 = qi * nt / x.q, s0 = ri * splits / x.r;
    const int dm = (pi + 1) * mt / x.p - m0, dn = (qi + 1) * nt / x.q - n0, ds = (ri + 1) * splits / x.r - s0;
    if (local >= dm * dn * ds) return false;
    m = m0 + local % dm;
    n = n0 + local / dm % dn;
    split = s0 + local / (dm * dn);
    return true;
}
inline XcdParts xcd_parts(int64_t mt, int64_t nt, int64_t splits, unsigned &grid)
{
    XcdParts best{1, 1, 8};
    int64_t cost = -1;
    for (int p = 1; p <= 8; p *= 2)
        for (int q = 1; p * q <= 8; q *= 2) {
            const int r = 8 / (p * q);
            const int64_t dm = (mt + p - 1) / p, dn = (nt + q - 1) / q, ds = (splits + r - 1) / r;
            // the longest XCD's work, then the operands' rows that it reads
            const int64_t c = (dm * dn * ds * 8 + 31) / 32 * 4096 + (dm + dn) * ds;
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
template <class T, bool XT, bool YT, int OUT, bool PAIRED, int NI, int NJ>
__device__ __forceinline__ void ffn_tile(const FfnJob &job, unsigned block, char *lds0, char *lds1, char *lds2,
                                         char *lds3)
{
    typedef typename FfnTerms<T>::type E;
    constexpr int PL = FfnTerms<T>::planes;
    typedef FfnLds<PL, XT, YT, NI, NJ> Lds;
    constexpr int TM = Lds::TM, TN = Lds::TN, BK = Lds::BK, BP = Lds::BP, PM = NI / BP, PW = Lds::PW, P = Lds::P;
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
        const int64_t k0 = sp * o.split_k;
        if (k0 >= K) return;
        auto from = [&](Operand &a, bool turned) {
            a.p += turned ? k0 * a.ld : k0;
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
    // p of the next part is on its way while this part is worked on
    float pre[OUT == FFN_MID ? 2 : 1][OUT == FFN_MID ? ITEMS : 1][2][8];
    auto load_pre = [&](auto which) {
        constexpr int part = decltype(which)::value;
        if constexpr (OUT == FFN_MID && part < PARTS) {
            const int j = part / PM, h = part % PM;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int64_t i = row_at(j, k), m = col_at(h, k);
                // (from the last row and columns where there is none)
                const float *from = o.pre + (i < o.rows ? i : o.rows - 1) * o.ld_pre;
                const int left = m >= o.F ? 0 : o.F - m < 8 ? (int)(o.F - m) : 8;
                if (o.F >= 8) {
                    const int64_t c = left == 8 ? m : o.F - 8; // the last eight, moved into place when they are used
                    load_vec<float, 8>(from + c, pre[part & 1][k][0]);
                    load_vec<float, 8>(from + o.F + c, pre[part & 1][k][1]);
                } else {
                    load_part<float, 8>(from + (left ? m : 0), left, pre[part & 1][k][0]);
                    load_part<float, 8>(from + o.F + (left ? m : 0), left, pre[part & 1][k][1]);
                }
            }
        }
    };
    load_pre(std::integral_constant<int, 0>()); // (there long before the products are)
    {
        const int stages = (int)(K / BK);
        // Tiles begin at different places of the sum where rows lie along it: rows a
        // multiple of a KB apart meet in few channels of the L2 (8192 x 4096 x 16384:
        // p and a 2.06 -> 1.94 ms, y 1.09 -> 0.98).  Small grids gain nothing.
        constexpr bool ROT = !YT && NI == 4;
        const int first = ROT ? (int)((8 * mi + ni) & 31) % stages : 0;
        TileLoader<YT, TN, BK, PL, ROT> y(Y, n0, stages, first);
        if constexpr (PAIRED) {
            PairLoader<TM> x(X, o.F, m0, stages, first);
            multiply<E, PL, XT, YT>(x, y, stages, lds0, lds1, lds2, lds3, acc);
        } else {
            TileLoader<XT, TM, BK, PL, ROT> x(X, m0, stages, first);
            multiply<E, PL, XT, YT>(x, y, stages, lds0, lds1, lds2, lds3, acc);
        }
    }
    __syncthreads();
    each_of(std::make_integer_sequence<int, PARTS>(), [&](auto which) {
        constexpr int p = decltype(which)::value, j = p / PM, h = p % PM;
        char *part = p & 1 ? lds1 : lds0; // one is written while the last is read
        if (h == 0) keep_columns(acc, j);
        load_pre(std::integral_constant<int, p + 1>());
#pragma unroll
        for (int b = 0; b < BP; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x16 &v = acc[h * BP + b][j];
                const int col = wm * PW + b * 32 + 8 * q + 4 * (lane >> 5);
                *reinterpret_cast<float4 *>(part + (wn * 32 + (lane & 31)) * P + col * 4) =
                    make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            }
        __syncthreads();
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
                store_terms<T, PL>(o.mid + i * o.ld_mid + m, o.plane_mid, 8, a);
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
                        g[e] = pre[p & 1][k][0][e];
                        u[e] = pre[p & 1][k][1][e];
                    }
                    if (left > 0 && left < 8 && o.F >= 8) { // the last columns, from the last eight values
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            g[e] = 0.f;
                            u[e] = 0.f;
#pragma unroll
                            for (int q = e + 1; q < 8; ++q)
                                if (q - e == 8 - left) {
                                    g[e] = pre[p & 1][k][0][q];
                                    u[e] = pre[p & 1][k][1][q];
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
                    store_terms<T, PL>(o.mid + i * o.ld_mid + m, o.plane_mid, left, slope);
                    short *d = o.dpre + i * o.ld_dpre + m;
                    store_terms<T, PL>(d, o.plane_dpre, left, g);
                    store_terms<T, PL>(d + o.F, o.plane_dpre, left, u);
                } else {
                    if (i >= o.rows || left <= 0) continue;
                    if (sum) store_part<float, 8>(sum + i * o.cols + m, left, x);
                    else store_part<T, 8>(static_cast<T *>(o.out) + i * o.ld_out + m, left, x);
                }
            }
        }
    });
}

template <class T, bool XT, bool YT, int OUT, bool PAIRED, int NI, int NJ>
__global__ __launch_bounds__(256, 1) void k_ffn(FfnJob job)
{
    typedef FfnLds<FfnTerms<T>::planes, XT, YT, NI, NJ> Lds;
    __shared__ __align__(16) char lds0[Lds::first];
    __shared__ __align__(16) char lds1[Lds::first];
    __shared__ __align__(16) char lds2[Lds::more];
    __shared__ __align__(16) char lds3[Lds::more];
    ffn_tile<T, XT, YT, OUT, PAIRED, NI, NJ>(job, blockIdx.x, lds0, lds1, lds2, lds3);
}

// The backward's three outputs, which do not wait for each other, in one launch:
// at small sizes each alone leaves most of the card idle, and a launch costs as
// much as a product.
struct FfnGrads {
    FfnJob x, w_in, w_out;
};
template <class T, int NI, int NJ>
__global__ __launch_bounds__(256, 1) void k_ffn_grads(FfnGrads g)
{
    constexpr int PL = FfnTerms<T>::planes;
    typedef FfnLds<PL, true, false, NI, NJ> A;
    typedef FfnLds<PL, true, true, NI, NJ> B;
    __shared__ __align__(16) char lds0[A::first > B::first ? A::first : B::first];
    __shared__ __align__(16) char lds1[A::first > B::first ? A::first : B::first];
    __shared__ __align__(16) char lds2[A::more > B::more ? A::more : B::more];
    __shared__ __align__(16) char lds3[A::more > B::more ? A::more : B::more];
    unsigned b = blockIdx.x;
    if (b < g.x.grid) {
        ffn_tile<T, true, false, FFN_OUT, false, NI, NJ>(g.x, b, lds0, lds1, lds2, lds3);
        return;
    }
    b -= g.x.grid;
    const bool in = b < g.w_in.grid;
    ffn_tile<T, true, true, FFN_OUT, false, NI, NJ>(in ? g.w_in : g.w_out, in ? b : b - g.w_in.grid, lds0, lds1, lds2,
                                                    lds3);
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

template <class T>
__global__ __launch_bounds__(256) void k_ffn_clear(T *p, int64_t ld, int64_t rows, int64_t cols)
{
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < rows * cols; c += step)
        p[c / cols * ld + c % cols] = (T)0.f;
}

// --------------------------------------------------------------- few rows

// Products of few rows, forward: the weight's bytes bound them, so it is read
// once, as it lies in memory, straight into the registers of the matrix
// instructions (16x16x32, fp32 16x16x4), and rows of any place and length serve.
// A block has 16 rows of the weight (PAIR: 16 of each projection) and 16 NB rows
// of the operand; its waves take chunks of the sum in turn, the next chunk's
// loads in flight while one is multiplied, and meet in LDS.  Lane l holds row l %
// 16 and the l / 16-th 16 bytes of each 64 of a chunk.
//
// Blocks begin at different places of the sum: rows lie a multiple of a KB apart
// as a rule, and equal columns of all of them meet in few channels of the L2 (4
// rows of 4096 x 16384 bf16: 84 us when all begin with the first, 72 so, 5.6 TB/s).
struct FewArgs {
    const void *w, *x;
    int64_t ld_w, ld_x;
    int64_t K, split_k; // summed values, of a block
    int64_t n, rows;    // operand rows; outputs (PAIR: of each projection)
    int act;
    float *pre;
    int64_t ld_pre;
    void *out;          // a (PAIR) or y
    int64_t ld_out;
    float *sum;         // [splits][n][rows]
};

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <class T>
struct FewStep {
    static constexpr int VEC = 16 / (int)sizeof(T), K = 4 * VEC; // values of a load, of a step
    typedef typename VecOf<T, VEC>::raw raw;
    static __device__ __forceinline__ f32x4 mma(raw a, raw b, f32x4 c)
    {
        if constexpr (std::is_same<T, float>::value) {
#pragma unroll
            for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
            return c;
        } else if constexpr (std::is_same<T, bf16>::value) {
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
        } else {
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
        }
    }
};

template <class T, bool PAIR, int NB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_ffn_few(FewArgs a)
{
    typedef FewStep<T> Step;
    typedef typename VecOf<T, Step::VEC>::type vec;
    constexpr int MB = PAIR ? 2 : 1, U = NB > 4 ? 2 : 4, CHUNK = U * Step::K, P = 16 * MB + 4;
    __shared__ __align__(16) float red[WAVES][16 * NB][P];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m0 = (int64_t)blockIdx.x * 16, k0 = blockIdx.y * a.split_k;
    const int64_t K = a.K - k0 < a.split_k ? a.K - k0 : a.split_k;
    const int at = (lane >> 4) * Step::VEC;
    const T *w[MB], *x[NB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int64_t r = m0 + (lane & 15);
        w[b] = static_cast<const T *>(a.w) + ((r < a.rows ? r : a.rows - 1) + b * a.rows) * a.ld_w + k0 + at;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t r = b * 16 + (lane & 15);
        x[b] = static_cast<const T *>(a.x) + (r < a.n ? r : a.n - 1) * a.ld_x + k0 + at;
    }
    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    struct Regs {
        typename Step::raw w[MB][U], x[NB][U];
    };
    auto load = [&](int64_t k, Regs &r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int b = 0; b < MB; ++b) r.w[b][u] = *reinterpret_cast<const vec *>(w[b] + k + u * Step::K);
#pragma unroll
            for (int b = 0; b < NB; ++b) r.x[b][u] = *reinterpret_cast<const vec *>(x[b] + k + u * Step::K);
        }
    };
    auto mma = [&](const Regs &r) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) acc[i][j] = Step::mma(r.w[i][u], r.x[j][u], acc[i][j]);
    };
    const int chunks = (int)(K / CHUNK), first = chunks ? (int)(blockIdx.x * 5 % (unsigned)chunks) : 0;
    auto place = [&](int c) { return (int64_t)(c + first < chunks ? c + first : c + first - chunks) * CHUNK; };
    Regs one, two;
    int c = wave;
    if (c < chunks) load(place(c), one);
    while (c < chunks) { // (a chunk past the last is the last again, and not used)
        const int c1 = c + WAVES, c2 = c + 2 * WAVES;
        load(place(c1 < chunks ? c1 : c), two);
        __builtin_amdgcn_sched_barrier(0); // (the loads would be moved behind the products, to save registers)
        mma(one);
        if (c1 >= chunks) break;
        load(place(c2 < chunks ? c2 : c1), one);
        __builtin_amdgcn_sched_barrier(0);
        mma(two);
        c = c2;
    }
    if (wave == chunks % WAVES) { // the rest of the sum, zeros past its end
        for (int64_t k = (int64_t)chunks * CHUNK; k < K; k += Step::K) {
            const int64_t left = K - k - at;
            typename Step::raw p[MB], q[NB];
            auto part = [&](const T *row) {
                typename Step::raw v;
#pragma unroll
                for (int e = 0; e < Step::VEC; ++e) v[e] = e < left ? row[k + e] : (T)0.f;
                return v;
            };
#pragma unroll
            for (int b = 0; b < MB; ++b) p[b] = part(w[b]);
#pragma unroll
            for (int b = 0; b < NB; ++b) q[b] = part(x[b]);
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) acc[i][j] = Step::mma(p[i], q[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            *reinterpret_cast<f32x4 *>(&red[wave][j * 16 + (lane & 15)][i * 16 + (lane >> 4) * 4]) = acc[i][j];
    __syncthreads();
    // eight outputs of a row per thread
    for (int e = threadIdx.x; e < 16 * NB * 2; e += 64 * WAVES) {
        const int64_t i = e >> 1, m = m0 + (e & 1) * 8;
        const int left = (int)(a.rows - m < 8 ? a.rows - m : 8);
        if (i >= a.n || left <= 0) continue;
        float v[MB][8];
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int q = 0; q < 8; ++q) v[b][q] = 0.f;
#pragma unroll 4
        for (int s = 0; s < WAVES; ++s)
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                float y[8];
                load_vec<float, 8>(&red[s][i][b * 16 + (e & 1) * 8], y);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[b][q] += y[q];
            }
        if constexpr (PAIR) {
            if (a.pre) {
                store_part<float, 8>(a.pre + i * a.ld_pre + m, left, v[0]);
                store_part<float, 8>(a.pre + i * a.ld_pre + a.rows + m, left, v[1]);
            }
            float value[8], slope[8];
            activations<sizeof(T) == 2>(a.act, v[0], value, slope);
#pragma unroll
            for (int q = 0; q < 8; ++q) value[q] *= v[1][q];
            store_part<T, 8>(static_cast<T *>(a.out) + i * a.ld_out + m, left, value);
        } else if (a.sum) {
            store_part<float, 8>(a.sum + (blockIdx.y * a.n + i) * a.rows + m, left, v[0]);
        } else {
            store_part<T, 8>(static_cast<T *>(a.out) + i * a.ld_out + m, left, v[0]);
        }
    }
}

// ------------------------------------------------------------ host: plans

unsigned blocks_for(int64_t threads)
{
    const int64_t b = (threads + 255) / 256;
    return (unsigned)(b < 16384 ? b : 16384);
}

// Side of a product's tiles: 256 where such tiles fill the compute units.
template <int PL>
int64_t ffn_side(int64_t M, int64_t N, int splits)
{
    if (PL > 1 || M <= 128 || N <= 128) return 128;
    return ((M + 255) / 256) * ((N + 255) / 256) * splits < kCUs ? 128 : 256;
}

// Parts of the summed index: where the tiles are fewer than the compute units
// take at a time, the sum is shared out.
struct FfnSplit {
    int parts;
    int64_t each;
};
FfnSplit ffn_split(int64_t M, int64_t N, int64_t K)
{
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
    int64_t s = 2 * kCUs / tiles;
    if (s > K / kSplit) s = K / kSplit;
    if (s < 1) s = 1;
    const int64_t each = up((K + s - 1) / s, kPad);
    return {(int)((K + each - 1) / each), each};
}
size_t split_bytes(int64_t M, int64_t N, int64_t K)
{
    const FfnSplit s = ffn_split(M, N, K);
    return s.parts > 1 ? round256((size_t)s.parts * M * N * sizeof(float)) : 0;
}

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

struct FfnPlan {
    short *x, *w_in, *w_out, *gy, *mid, *dpre;
    float *sum;
    int64_t Dp, Fp, Pp; // padded columns of x and gy, of a, of dp
    int64_t ldD, ldF, ldP;
    size_t bytes;
};
// Distance of rows of so many columns: an odd number of cache lines where it would
// be a multiple of 1 KB, at which a tile's rows meet in few channels of the L2
// (8192 x 4096 x 16384, rows of a 32 KB apart: y in 997 us, 902 with one line more).
inline int64_t apart(int64_t cols) { return cols % 512 ? cols : cols + 64; }

FfnPlan plan_ffn(int64_t n, int64_t D, int64_t F, int PL, bool grad, const FfnCopies &c, char *base)
{
    size_t off = TT_EMB_STATUS_BYTES;
    auto take = [&](int64_t rows, int64_t cols) {
        char *r = base ? base + off : nullptr;
        off += round256((size_t)PL * rows * cols * 2);
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
    if (c.x) p.x = take(n, p.ldD);
    if (c.w_in) p.w_in = take(grad ? 2 * F : 2 * up(F, 32), p.ldD);
    if (c.w_out) p.w_out = take(D, p.ldF);
    if (c.gy) p.gy = take(n, p.ldD);
    p.mid = take(n, p.ldF);
    size_t sums;
    if (grad) {
        p.dpre = take(n, p.ldP);
        sums = split_bytes(D, n, p.Pp) + split_bytes(D, 2 * F, up(n, kPad)) + split_bytes(F, D, up(n, kPad));
    } else {
        sums = few_rows(n, PL > 1) ? few_bytes(n, D, F) : split_bytes(D, n, p.Fp);
    }
    p.sum = reinterpret_cast<float *>(base ? base + off : nullptr);
    off += sums;
    p.bytes = off;
    return p;
}
FfnCopies copies_of(const FfnArgs &a, int dtype, bool grad)
{
    return ffn_copies(dtype == TT_EMB_DTYPE_FLOAT, grad, a.n, a.D, a.F, lies_well(a.x, a.ld_x), lies_well(a.w_in, a.ld_in),
                      lies_well(a.w_out, a.ld_out), lies_well(a.gy, a.ld_gy));
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
        return Operand{dst, ldp, to * ldp, to, width};
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

FfnJob job_of(const Operand &x, const Operand &y, int64_t M, int64_t N, int64_t K, int64_t side, const FfnOut &o)
{
    const int64_t mt = (M + side - 1) / side, nt = (N + side - 1) / side;
    FfnJob job{x, y, K, mt, nt, 0, {}, o};
    if (in_patches(mt, nt)) job.grid = tile_grid(mt, nt, 1);
    else job.xcds = xcd_parts(mt, nt, o.splits, job.grid);
    return job;
}

template <class T, bool XT, bool YT, int OUT, bool PAIRED>
void launch(const FfnJob &job, int64_t side, hipStream_t s)
{
    if constexpr (FfnTerms<T>::planes == 1) {
        if (side == 256) {
            hipLaunchKernelGGL((k_ffn<T, XT, YT, OUT, PAIRED, 4, 4>), dim3(job.grid), dim3(256), 0, s, job);
            return;
        }
    }
    hipLaunchKernelGGL((k_ffn<T, XT, YT, OUT, PAIRED, 2, 2>), dim3(job.grid), dim3(256), 0, s, job);
}

template <class T, bool XT, bool YT, int OUT, bool PAIRED>
void product(const Operand &x, const Operand &y, int64_t M, int64_t N, int64_t K, const FfnOut &o, hipStream_t s)
{
    const int64_t side = ffn_side<FfnTerms<T>::planes>(M, N, o.splits);
    launch<T, XT, YT, OUT, PAIRED>(job_of(x, y, M, N, K, side, o), side, s);
}

// Outputs [N][M] of T, whose sums are split where that fills the card: each job
// takes what it needs of the room for partial sums.
template <class T>
struct Outputs {
    float *sum;
    Joins joins{};
    int n = 0;

    FfnJob operator()(const Operand &x, const Operand &y, int64_t M, int64_t N, int64_t K, void *out, int64_t ld,
                      int64_t &side)
    {
        FfnOut o{};
        o.rows = N;
        o.cols = M;
        o.out = out;
        o.ld_out = ld;
        const FfnSplit split = ffn_split(M, N, K);
        o.splits = split.parts;
        if (split.parts > 1) {
            o.sum = sum;
            o.split_k = split.each;
            sum += split_bytes(M, N, K) / sizeof(float);
            joins.job[n] = Join{o.sum, split.parts, N, M, out, ld};
            joins.first[n + 1] = joins.first[n] + (int)blocks_for(N * ((M + 3) / 4));
            ++n;
        }
        side = ffn_side<FfnTerms<T>::planes>(M, N, o.splits);
        return job_of(x, y, M, N, K, side, o);
    }
    void join(hipStream_t s)
    {
        if (!n) return;
        for (int k = n; k < 3; ++k) joins.first[k + 1] = joins.first[k];
        hipLaunchKernelGGL(k_ffn_join<T>, dim3((unsigned)joins.first[n]), dim3(256), 0, s, joins);
    }
};

template <class T, bool PAIR>
void few(const FewArgs &a, int splits, hipStream_t s)
{
    const dim3 grid((unsigned)((a.rows + 15) / 16), (unsigned)splits);
    constexpr std::integral_constant<int, 4> four;
    constexpr std::integral_constant<int, 8> eight;
    const bool idle = (int64_t)grid.x * splits <= 2 * kCUs; // few blocks: more waves in each
    auto run = [&](auto nb, auto waves) {
        constexpr int NB = decltype(nb)::value, WAVES = decltype(waves)::value;
        hipLaunchKernelGGL((k_ffn_few<T, PAIR, NB, WAVES>), grid, dim3(64 * WAVES), 0, s, a);
    };
    if constexpr (sizeof(T) == 4) {
        if (a.n > 64) return run(std::integral_constant<int, 8>(), four);
        if (a.n > 32) return idle ? run(four, eight) : run(four, four);
        if (a.n > 16) return idle ? run(std::integral_constant<int, 2>(), eight) : run(std::integral_constant<int, 2>(), four);
    }
    constexpr std::integral_constant<int, 1> one;
    return idle ? run(one, eight) : run(one, four);
}

template <class T>
hipError_t ffn_few(const FfnArgs &a, int dtype, hipStream_t s)
{
    const FfnPlan p = plan_ffn(a.n, a.D, a.F, FfnTerms<T>::planes, false, copies_of(a, dtype, false), a.ws);
    FewArgs in{};
    in.w = a.w_in;
    in.ld_w = a.ld_in;
    in.x = a.x;
    in.ld_x = a.ld_x;
    in.K = in.split_k = a.D;
    in.n = a.n;
    in.rows = a.F;
    in.act = a.act;
    in.pre = a.pre;
    in.ld_pre = a.ld_pre;
    in.out = p.mid;
    in.ld_out = p.ldF;
    few<T, true>(in, 1, s);
    FewArgs out{};
    out.w = a.w_out;
    out.ld_w = a.ld_out;
    out.x = p.mid;
    out.ld_x = p.ldF;
    out.K = a.F;
    out.n = a.n;
    out.rows = a.D;
    out.out = a.y;
    out.ld_out = a.ld_y;
    const FfnSplit split = few_split(a.D, a.F);
    out.split_k = split.each;
    if (split.parts > 1) out.sum = p.sum;
    few<T, false>(out, split.parts, s);
    if (split.parts > 1) {
        Joins j{};
        j.job[0] = Join{p.sum, split.parts, a.n, a.D, a.y, a.ld_y};
        j.first[1] = j.first[2] = j.first[3] = (int)blocks_for(a.n * ((a.D + 3) / 4));
        hipLaunchKernelGGL(k_ffn_join<T>, dim3((unsigned)j.first[1]), dim3(256), 0, s, j);
    }
    return hipGetLastError();
}

template <class T>
hipError_t ffn_forward(const FfnArgs &a, int dtype, hipStream_t s)
{
    if (few_rows(a.n, FfnTerms<T>::planes > 1)) return ffn_few<T>(a, dtype, s);
    constexpr int PL = FfnTerms<T>::planes;
    const FfnPlan p = plan_ffn(a.n, a.D, a.F, PL, false, copies_of(a, dtype, false), a.ws);
    Packing<T> pack;
    const Operand x = pack(a.x, a.ld_x, a.n, a.D, p.x, p.Dp, 0);
    const Operand w_in = pack(a.w_in, a.ld_in, 2 * a.F, a.D, p.w_in, p.Dp, a.F);
    const Operand w_out = pack(a.w_out, a.ld_out, a.D, a.F, p.w_out, p.Fp, 0);
    pack.run(s);
    FfnOut o{};
    o.rows = a.n;
    o.splits = 1;
    o.F = a.F;
    o.act = a.act;
    o.pre = a.pre;
    o.ld_pre = a.ld_pre;
    o.mid = p.mid;
    o.ld_mid = p.ldF;
    o.plane_mid = a.n * p.ldF;
    const int64_t M = 2 * up(a.F, 32);
    bool done = false;
    if constexpr (PL == 1) {
        if (!p.w_in) {
            product<T, false, false, FFN_IN, true>(w_in, x, M, a.n, p.Dp, o, s);
            done = true;
        }
    }
    if (!done) product<T, false, false, FFN_IN, false>(w_in, x, M, a.n, p.Dp, o, s);
    const Operand mid{p.mid, p.ldF, o.plane_mid, a.n, p.Fp};
    Outputs<T> out{p.sum};
    int64_t side;
    const FfnJob y = out(w_out, mid, a.D, a.n, p.Fp, a.y, a.ld_y, side);
    launch<T, false, false, FFN_OUT, false>(y, side, s);
    out.join(s);
    return hipGetLastError();
}

template <class T>
hipError_t ffn_backward(const FfnArgs &a, int dtype, hipStream_t s)
{
    constexpr int PL = FfnTerms<T>::planes;
    const FfnPlan p = plan_ffn(a.n, a.D, a.F, PL, true, copies_of(a, dtype, true), a.ws);
    Packing<T> pack;
    const Operand gy = pack(a.gy, a.ld_gy, a.n, a.D, p.gy, p.Dp, 0);
    const Operand x = pack(a.x, a.ld_x, a.n, a.D, p.x, p.Dp, 0);
    const Operand w_in = pack(a.w_in, a.ld_in, 2 * a.F, a.D, p.w_in, p.Dp, 0);
    const Operand w_out = pack(a.w_out, a.ld_out, a.D, a.F, p.w_out, p.Fp, 0);
    // the products along dp's columns meet its padding
    if (p.Pp > 2 * a.F) pack.add(Pack{nullptr, 0, a.n, 0, p.dpre + p.Pp - kPad, kPad, p.ldP, a.n * p.ldP, 0});
    pack.run(s);
    FfnOut o{};
    o.rows = a.n;
    o.splits = 1;
    o.cols = o.F = a.F;
    o.act = a.act;
    o.pre = a.pre;
    o.ld_pre = a.ld_pre;
    o.mid = p.mid;
    o.ld_mid = p.ldF;
    o.plane_mid = a.n * p.ldF;
    o.dpre = p.dpre;
    o.ld_dpre = p.ldP;
    o.plane_dpre = a.n * p.ldP;
    product<T, true, false, FFN_MID, false>(w_out, gy, a.F, a.n, p.Dp, o, s);
    const Operand mid{p.mid, p.ldF, o.plane_mid, a.n, p.Fp}, dpre{p.dpre, p.ldP, o.plane_dpre, a.n, p.Pp};
    const int64_t rows = up(a.n, kPad);
    Outputs<T> out{p.sum};
    int64_t side_x, side_in, side_out;
    const FfnGrads g{out(w_in, dpre, a.D, a.n, p.Pp, a.gx, a.ld_gx, side_x),
                     out(x, dpre, a.D, 2 * a.F, rows, a.gw_in, a.ld_gin, side_in),
                     out(mid, gy, a.F, a.D, rows, a.gw_out, a.ld_gout, side_out)};
    if (side_x == 128 && side_in == 128 && side_out == 128) {
        hipLaunchKernelGGL((k_ffn_grads<T, 2, 2>), dim3(g.x.grid + g.w_in.grid + g.w_out.grid), dim3(256), 0, s, g);
    } else {
        launch<T, true, false, FFN_OUT, false>(g.x, side_x, s);
        launch<T, true, true, FFN_OUT, false>(g.w_in, side_in, s);
        launch<T, true, true, FFN_OUT, false>(g.w_out, side_out, s);
    }
    out.join(s);
    return hipGetLastError();
}

// No rows: the weights' gradients are zero.
template <class T>
hipError_t ffn_clear(const FfnArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(k_ffn_clear<T>, dim3(blocks_for(2 * a.F * a.D)), dim3(256), 0, s, static_cast<T *>(a.gw_in),
                       a.ld_gin, 2 * a.F, a.D);
    hipLaunchKernelGGL(k_ffn_clear<T>, dim3(blocks_for(a.D * a.F)), dim3(256), 0, s, static_cast<T *>(a.gw_out),
                       a.ld_gout, a.D, a.F);
    return hipGetLastError();
}

} // namespace

// what: TT_EMB_FFN_GRAD and TT_EMB_FFN_ALIGNED.
size_t ffn_workspace(int64_t n, int64_t D, int64_t F, int dtype, int what)
{
    const bool fp32 = dtype == TT_EMB_DTYPE_FLOAT, grad = what & TT_EMB_FFN_GRAD, well = what & TT_EMB_FFN_ALIGNED;
    return plan_ffn(n, D, F, fp32 ? 3 : 1, grad, ffn_copies(fp32, grad, n, D, F, well, well, well, well), nullptr).bytes;
}

size_t ffn_needs(const FfnArgs &a, int dtype, bool grad)
{
    return plan_ffn(a.n, a.D, a.F, dtype == TT_EMB_DTYPE_FLOAT ? 3 : 1, grad, copies_of(a, dtype, grad), nullptr).bytes;
}

hipError_t launch_ffn_forward(const FfnArgs &a, int dtype, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    if (dtype == TT_EMB_DTYPE_FLOAT) return ffn_forward<float>(a, dtype, s);
    if (dtype == TT_EMB_DTYPE_BFLOAT) return ffn_forward<bf16>(a, dtype, s);
    return ffn_forward<f16>(a, dtype, s);
}

hipError_t launch_ffn_backward(const FfnArgs &a, int dtype, hipStream_t s)
{
    if (dtype == TT_EMB_DTYPE_FLOAT) return a.n == 0 ? ffn_clear<float>(a, s) : ffn_backward<float>(a, dtype, s);
    if (dtype == TT_EMB_DTYPE_BFLOAT) return a.n == 0 ? ffn_clear<bf16>(a, s) : ffn_backward<bf16>(a, dtype, s);
    return a.n == 0 ? ffn_clear<f16>(a, s) : ffn_backward<f16>(a, dtype, s);
}

} // namespace ttemb
