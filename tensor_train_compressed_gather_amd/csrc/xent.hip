// xent.hip -- softmax cross entropy of hidden rows against a large vocabulary
// without keeping the logits, and both gradients (gfx950).
//
// Three products of the same sizes: the logits z = H W^T, and with d the
// gradient of the loss by the logits, dH = d W and dW = d^T H.  All run on the
// bf16 matrix cores with fp32 accumulators.  The logits never leave the
// registers of the tile that makes them: a first pass keeps each row's maximum
// and sum of exponentials per tile, from which lse and the loss follow; for
// the gradients a piece of the vocabulary's logits is made again, turned into
// d, and multiplied into both gradients before the next piece.  Rows of up to
// 128 values take kernels of their own, which never write d.
//
// Matrix instructions bound the large sizes, the weight's bytes those of few
// rows, launches the smallest.  8192 rows against 131072 x 4096 in bf16: 26.7 ms
// with both gradients, four products (the logits are made twice) of 8.8 TFLOP
// at 1320 TFLOP/s; 5 rows, loss only: 179 us, 6.0 TB/s.
//
// bf16 inputs: d is rounded to bf16, by at most 2^-8 of each value, because two
// terms of it would double both gradients' products.  The gradients' own rounding
// to bf16 is as large: 8192 rows against 131072 x 4096 are 1.9e-3 from 64 bits,
// 1.7e-3 with d in fp32.
//
// fp32 inputs are scaled by powers of two (to a largest magnitude in
// [2^14, 2^15): each hidden row for the logits, the hidden rows that count times
// their dL/dloss as a whole for the weight's gradient, the weight as a whole) and
// split into two fp16 terms of 11 bits each, and the three products of terms
// above 2^-22 are added up: five times the rate of the fp32 matrix instructions.
// d without dL/dloss (at most 1) is split the same way in units of 2^-15; the
// sums of dH take dL/dloss at the end, so a row's precision does not depend on
// the other rows' gradients.  A value keeps 22 bits, or an absolute 2^-39 of the
// largest where that is more.
#include "primitives.h"
#include "tiles.h"

namespace ttemb {

namespace {

constexpr size_t kPieceBytes = (size_t)256 << 20; // d of one piece of the vocabulary, at most
constexpr int kSplitK = 512;           // least summed values of a split
constexpr int kRound = 256;            // columns of d are padded to this
constexpr int kLeast = 128;            // rows and columns of the smallest tile
constexpr int kPadK = 64;              // packed rows are padded to this
constexpr int kMaxParts = 1024;        // blocks of the weight's largest magnitude
constexpr int64_t kFewRows = 128;      // fp32 rows whose statistics take no packed operands
constexpr int kUnitExp = 15;           // fp16 terms: d is kept in units of 2^-15

// PL planes of 16-bit terms: one of bf16, or two of fp16.
template <int PL>
struct Terms {
    typedef std::conditional_t<PL == 1, bf16, f16> type;
    static __device__ __forceinline__ f32x16 mma(s16x8 a, s16x8 b, f32x16 c) { return mma16<type>(a, b, c); }
};
template <int PL>
__device__ __forceinline__ void split(float x, short (&t)[PL])
{
    split_terms<typename Terms<PL>::type, PL>(x, t);
}

__device__ __forceinline__ bool row_counts(int64_t target, int64_t ignore, int64_t V)
{
    return target != ignore && target >= 0 && target < V;
}

// What a product's tiles become: maxima and sums of exponentials, d, partial
// sums in fp32, or rows of the weight's gradient.
enum { OUT_STATS, OUT_D, OUT_SUM, OUT_WEIGHT };

struct Output {
    int64_t n, V, v0;         // rows, vocabulary, first column of this piece
    const int64_t *targets;
    int64_t ignore;
    float2 *part;             // [vocabulary tiles][n] maximum and sum
    float *target_logit;      // [n]
    const float *lse, *grad;  // [n]
    const float *top_grad;    // the unit of d (bf16)
    // fp16 terms: exponents by which each row (for the logits), all rows (for
    // the weight's gradient) and the weight were scaled
    const int *h_exp, *all_exp, *w_exp;
    const float4 *rows;       // [n] scale, lse and factor of d, of rows that are streamed
    short *d;                 // [planes][rows][ldd]
    int64_t ldd, plane_d;
    float *sum;               // fp32 sums, [splits][sum_rows][D]
    int64_t sum_rows;
    int splits;               // parts of the summed index
    int64_t split_k;          // summed values of each
    int first;                // overwrite the sums, do not add to them
    void *out;                // dW
    int64_t ld_out, D;
};

// Two (maximum, sum of exponentials relative to it) as one.
__device__ __forceinline__ float2 join_sums(float2 a, float2 b)
{
    const float m = fmaxf(a.x, b.x), ref = m == -INFINITY ? 0.f : m;
    return make_float2(m, a.y * __expf(a.x - ref) + b.y * __expf(b.x - ref));
}

// Maximum and sum of exponentials of one column of a wave's NI 32 x 32 tiles of
// logits (both halves of the wave), whose values are z / unit; the target's
// logit is stored where it is among them.  `left`: rows of the tile that exist,
// first: the wave's first row.  The maximum is taken and subtracted before the
// values are scaled.
template <bool CUT, int NI, int NJ, class R>
__device__ __forceinline__ void column_sums(const f32x16 (&acc)[NI][NJ], int j, R row_of, int64_t left, float unit,
                                            float &top, float &sum)
{
    auto z = [&](int a, int r) { return CUT && row_of(a, r) >= left ? -INFINITY : acc[a][j][r]; };
    top = -INFINITY;
    sum = 0.f;
#pragma unroll
    for (int a = 0; a < NI; ++a)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, z(a, r));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float ref = top == -INFINITY ? 0.f : top, base = unit * 1.44269504f;
#pragma unroll
    for (int a = 0; a < NI; ++a)
#pragma unroll
        for (int r = 0; r < 16; ++r) sum += __builtin_amdgcn_exp2f((z(a, r) - ref) * base);
    top *= unit;
    sum += __shfl_xor(sum, 32, 64);
}
template <int NI, int NJ, class R>
__device__ __forceinline__ void column_stats(const f32x16 (&acc)[NI][NJ], int j, R row_of, int64_t left, int tile_rows,
                                             int64_t t, int first, float unit, float *target_logit, float &top,
                                             float &sum)
{
    if (__any(t >= first && t < first + 32 * NI)) {
#pragma unroll
        for (int a = 0; a < NI; ++a)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (row_of(a, r) == t) *target_logit = acc[a][j][r] * unit;
    }
    if (left < tile_rows) column_sums<true>(acc, j, row_of, left, unit, top, sum); // the vocabulary ends in this tile
    else column_sums<false>(acc, j, row_of, left, unit, top, sum);
}

// C[m][n] = sum_k X[m][k] Y[n][k] over tiles of (64 NI) x (64 NJ).
template <int PL, bool XT, bool YT, int OUT, int NI, int NJ>
__global__ __launch_bounds__(256, 1) void k_product(Operand X, Operand Y, int64_t K, int64_t mt, int64_t nt, Output o)
{
    constexpr int TM = 64 * NI, TN = 64 * NJ, BK = Stages<PL, XT>::values, NB = Stages<PL, XT>::buffers;
    constexpr int XB = PL * TileLds<XT, TM, BK>::bytes, YB = PL * TileLds<YT, TN, BK>::bytes, STAGE = XB + YB;
    // how the tile leaves through LDS: values E, in parts of 64 rows and all or
    // half of each wave's TM / 2 columns, PW of them; pitch P
    typedef std::conditional_t<OUT == OUT_WEIGHT && PL == 1, bf16, float> E32;
    typedef std::conditional_t<OUT == OUT_D, short, E32> E;
    typedef E E4 __attribute__((ext_vector_type(4)));
    constexpr int ES = (int)sizeof(E), EV = 16 / ES, PLANES = OUT == OUT_D ? PL : 1;
    constexpr int PM = ES == 4 && NB == 4 ? 2 : 1, PW = TM / 2 / PM;
    constexpr int P = 2 * PW * ES + 16, PART = 64 * P, ROWV = 2 * PW / EV, PIECES = 64 * ROWV / 256;
    constexpr int BUFFER = OUT != OUT_STATS && PLANES * PART > STAGE ? PLANES * PART : STAGE;
    __shared__ __align__(16) char lds0[BUFFER];
    __shared__ __align__(16) char lds1[BUFFER];
    __shared__ __align__(16) char lds2[NB == 4 ? STAGE : 16];
    __shared__ __align__(16) char lds3[NB == 4 ? STAGE : 16];
    int64_t mi, ni;
    int sp;
    if (!tile_of(blockIdx.x, gridDim.x, mt, nt, OUT == OUT_SUM ? o.splits : 1, mi, ni, sp)) return;
    if constexpr (OUT == OUT_SUM) { // this split's part of the sum (X is turned)
        const int64_t k0 = sp * o.split_k;
        if (k0 >= K) return;
        X.p += k0 * X.ld;
        X.rows -= k0;
        if constexpr (YT) {
            Y.p += k0 * Y.ld;
            Y.rows -= k0;
        } else {
            Y.p += k0;
            Y.cols -= k0;
        }
        K = K - k0 < o.split_k ? K - k0 : o.split_k;
        o.sum += sp * o.sum_rows * o.D;
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
    {
        const int stages = (int)(K / BK);
        TileLoader<XT, TM, BK, PL> x(X, m0, stages);
        TileLoader<YT, TN, BK, PL> y(Y, n0, stages);
        multiply<typename Terms<PL>::type, PL, XT, YT>(x, y, stages, lds0, lds1, lds2, lds3, acc);
    }
    auto row_of = [&](int i, int r) { return wm * (TM / 2) + i * 32 + 8 * (r / 4) + 4 * (lane >> 5) + (r % 4); };
    if constexpr (OUT == OUT_STATS) {
        float(*red)[2][TN] = reinterpret_cast<float(*)[2][TN]>(lds0);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            keep_columns(acc, j);
            const int nl = wn * (TN / 2) + j * 32 + (lane & 31);
            const int64_t i = n0 + nl;
            const int64_t t = i < o.n ? o.targets[i] - m0 : -1;
            const int64_t left = o.V - m0;
            // the accumulators are logits times a power of two
            const float unit = PL == 2 && i < o.n ? ldexpf(1.f, -(o.h_exp[i] + *o.w_exp)) : 1.f;
            float top, sum;
            column_stats(acc, j, row_of, left, TM, t, wm * (TM / 2), unit, o.target_logit + (i < o.n ? i : 0), top,
                         sum);
            if (lane < 32) {
                red[0][wm][nl] = top;
                red[1][wm][nl] = sum;
            }
        }
        __syncthreads();
        if (tid < TN && n0 + tid < o.n) {
            const float a = red[0][0][tid], b = red[0][1][tid], top = fmaxf(a, b);
            const float ref = top == -INFINITY ? 0.f : top;
            const float s = red[1][0][tid] * __expf(a - ref) + red[1][1][tid] * __expf(b - ref);
            o.part[mi * o.n + n0 + tid] = make_float2(top, s);
        }
    } else {
        // 64 rows at a time pass through LDS, so that they are written in whole
        // lines: a lane holds four columns of one row, a wave 32 rows
        float unit = 1.f;
        if constexpr (OUT == OUT_D && PL == 1) unit = *o.top_grad;
        if constexpr (OUT == OUT_WEIGHT) unit = PL == 2 ? ldexpf(1.f, -(kUnitExp + *o.all_exp)) : *o.top_grad;
        const int64_t left = o.V - o.v0 - m0; // of the vocabulary, in d
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            keep_columns(acc, j);
            const int64_t i = n0 + wn * (TN / 2) + j * 32 + (lane & 31);
            // rows that do not count (packed as zeros), or lie past the last: d = 0 (exp - 0)
            float lse = 0.f, g = 0.f, scale = 1.f;
            int64_t t = -1;
            if (OUT == OUT_D && i < o.n) {
                const int64_t target = o.targets[i];
                lse = o.lse[i];
                if (row_counts(target, o.ignore, o.V)) {
                    if constexpr (PL == 2) scale = ldexpf(1.f, -(o.h_exp[i] + *o.w_exp));
                    t = target - o.v0 - m0;
                    g = PL == 2 ? (float)(1 << kUnitExp) : o.grad[i] / unit;
                } else {
                    lse = INFINITY;
                }
            }
            const bool special = __any(t >= wm * (TM / 2) && t < (wm + 1) * (TM / 2)) || left < TM;
#pragma unroll
            for (int h = 0; h < PM; ++h) {
                char *part = (j * PM + h) & 1 ? lds1 : lds0; // one is written while the last is read
#pragma unroll
                for (int a = h * (NI / PM); a < (h + 1) * (NI / PM); ++a)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int m = row_of(a, 4 * q), mp = m - h * PW - wm * (TM / 2 - PW);
                        E4 w[PLANES];
                        float x[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] = acc[a][j][4 * q + r];
                        if constexpr (OUT == OUT_D) {
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                x[r] = __builtin_amdgcn_exp2f(fmaf(x[r], scale, -lse) * 1.44269504f);
                            if (special) { // a target, or the vocabulary's end
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    if (m + r == t) x[r] -= 1.f;
                                    if (m + r >= left) x[r] = 0.f;
                                }
                            }
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                short s[PL];
                                split<PL>(g * x[r], s);
#pragma unroll
                                for (int q2 = 0; q2 < PL; ++q2) w[q2][r] = s[q2];
                            }
                        } else {
#pragma unroll
                            for (int r = 0; r < 4; ++r) w[0][r] = (E)(x[r] * unit);
                        }
#pragma unroll
                        for (int q2 = 0; q2 < PLANES; ++q2)
                            *reinterpret_cast<E4 *>(part + q2 * PART + (wn * 32 + (lane & 31)) * P + mp * ES) = w[q2];
                    }
                __syncthreads();
#pragma unroll
                for (int q2 = 0; q2 < PLANES; ++q2)
#pragma unroll
                    for (int k = 0; k < PIECES; ++k) {
                        const int c = tid + k * 256, r = c / ROWV, mp = c % ROWV * EV;
                        const int64_t row = n0 + (r >> 5) * (TN / 2) + j * 32 + (r & 31);
                        const int64_t m = m0 + mp / PW * (TM / 2) + h * PW + mp % PW;
                        const char *from = part + q2 * PART + r * P + c % ROWV * 16;
                        if constexpr (OUT == OUT_D) {
                            *reinterpret_cast<u32x4 *>(o.d + q2 * o.plane_d + row * o.ldd + m) =
                                *reinterpret_cast<const u32x4 *>(from);
                        } else {
                            const int64_t to = OUT == OUT_WEIGHT ? o.v0 + row : row;
                            if (to >= (OUT == OUT_WEIGHT ? o.V : o.sum_rows) || m >= o.D) continue;
                            const int have = o.D - m < EV ? (int)(o.D - m) : EV;
                            float x[EV];
                            load_vec<E, EV>(reinterpret_cast<const E *>(from), x);
                            if constexpr (OUT == OUT_SUM) {
                                float *s = o.sum + to * o.D + m;
                                if (!o.first) {
                                    float old[EV];
                                    load_part<float, EV>(s, have, old);
#pragma unroll
                                    for (int e = 0; e < EV; ++e) x[e] += old[e];
                                }
                                store_part<float, EV>(s, have, x);
                            } else {
                                store_part<E, EV>(static_cast<E *>(o.out) + to * o.ld_out + m, have, x);
                            }
                        }
                    }
            }
        }
    }
}

// ------------------------------------------------- rows of at most 128 values
//
// With so short a sum a product's tile is over before its start and its end are
// hidden, and d, written and read twice, costs more than the products.  Here a
// wave keeps 32 NO rows of one operand in registers as fragments and streams
// the rows of the other through LDS, 32 at a step: the logits of a step stay in
// the wave's registers, where their layout (lane l: own row l % 32, streamed
// rows 8 (r / 4) + 4 (l / 32) + r % 4) is the layout of the left operand of the
// next product if that takes its summed index in the same order, which the
// transposing reads of the streamed rows can.  So d is never written.
//
//   ROW_STATS  own: hidden rows, streamed: the weight.  Maximum and sum.
//   ROW_GRAD   the same, and d times the streamed rows: dH of a part of the vocabulary.
//   VOC_GRAD   own: rows of the weight, streamed: hidden rows: dW.
//
// The logits are made three times instead of twice, and matrix instructions
// bound it: 2048 fp32 rows of 128 against 10^6, 6.9 ms with both gradients, of
// which five sums of three products are 5.2 at the card's rate (10.7 by the
// products above); bf16 2.7 ms, where the exponentials' vector instructions take
// as long as the products.  fp16 terms: the hidden rows keep their own scales in
// dW's product too, so there d_i carries dL/dloss and the ratio of the row's
// scale to that of the largest product of the two, at most 1.
enum { ROW_STATS, ROW_GRAD, VOC_GRAD };
constexpr int kNarrowStep = 32;
constexpr int64_t kNarrowSteps = 8;    // least steps of a split
// fp32: steps after which a sum is added to memory.  Six additions a step to one
// accumulator would round 10^6 rows' sum to 2^-19.6, in parts of 8192 rows to 2^-21.
constexpr int kNarrowChain = 256;
constexpr int64_t kNarrow = 128;       // longest rows

// Which of a streamed row's 16-byte pieces change places: sixteen rows' equal
// pieces, and the 64 bytes of four neighbouring rows, lie in different banks.
template <int KD>
__device__ __forceinline__ int piece_turn(int row)
{
    return KD == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : ((row & 2) << 1) | ((row >> 2) & 3);
}

template <class T, int PL, int KD, int MODE, int NO>
__global__ __launch_bounds__(256, 2) void k_narrow(Operand own, Operand str, int64_t owns, int64_t per, Output o)
{
    constexpr int KB = KD / 16, CB = KD / 32, P = KD * 2, PLANE = kNarrowStep * P, STAGE = PL * PLANE;
    constexpr int PR = KD / 8, N = kNarrowStep * PR / 256;
    constexpr bool VOC = MODE == VOC_GRAD;
    __shared__ __align__(256) char lds0[STAGE];
    __shared__ __align__(256) char lds1[STAGE];
    __shared__ __align__(16) float of_row[2][3][kNarrowStep]; // VOC_GRAD: scale, lse and gradient of the streamed rows
    __shared__ __align__(16) int hit_row[2][kNarrowStep];     // and their targets in this block's rows
    const int64_t id = (int64_t)(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
    const int64_t sp = id / owns, ob = id % owns, all = (str.rows + kNarrowStep - 1) / kNarrowStep, s0 = sp * per;
    if (s0 >= all) return;
    const int steps = (int)(all - s0 < per ? all - s0 : per);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;
    const int64_t block0 = ob * 128 * NO, own0 = block0 + wave * 32 * NO;

    s16x8 of[PL][NO][KB];
    float scale[NO], lse[NO], g[NO], top[NO], sum[NO];
    int hit[NO], hit_row_of[NO]; // step of this row's target and its row there
    const float unit = MODE != ROW_STATS && PL == 1 ? *o.top_grad : 1.f;
#pragma unroll
    for (int b = 0; b < NO; ++b) {
        const int64_t i = own0 + b * 32 + (lane & 31), ic = i < own.rows ? i : own.rows - 1;
#pragma unroll
        for (int q = 0; q < PL; ++q)
#pragma unroll
            for (int k = 0; k < KB; ++k)
                of[q][b][k] =
                    *reinterpret_cast<const s16x8 *>(own.p + q * own.plane + ic * own.ld + k * 16 + half * 8);
        scale[b] = 1.f;
        lse[b] = g[b] = sum[b] = 0.f;
        top[b] = -INFINITY;
        hit[b] = -1;
        hit_row_of[b] = 0;
        if constexpr (!VOC) {
            const int64_t target = o.targets[ic], t = target - s0 * kNarrowStep;
            bool takes = i < own.rows && t >= 0 && t < (int64_t)steps * kNarrowStep;
            if constexpr (PL == 2) scale[b] = ldexpf(1.f, -(o.h_exp[ic] + *o.w_exp));
            if constexpr (MODE == ROW_GRAD) {
                const bool counts = i < own.rows && row_counts(target, o.ignore, o.V);
                if (!counts) scale[b] = 1.f;
                lse[b] = counts ? o.lse[ic] : INFINITY;
                g[b] = !counts ? 0.f : PL == 2 ? (float)(1 << kUnitExp) : o.grad[ic] / unit;
                takes = takes && counts;
            }
            if (takes) {
                hit[b] = (int)(t / kNarrowStep);
                hit_row_of[b] = (int)(t % kNarrowStep);
            }
        }
    }
    f32x16 acc[MODE == ROW_STATS ? 1 : NO][CB];

    // streamed rows: straight to one of two LDS buffers a step ahead, a round of
    // the loop being two steps (as for tiles); rows past this split's are zeros
    const int64_t rows_end = (s0 + steps) * kNarrowStep < str.rows ? (s0 + steps) * kNarrowStep : str.rows;
    const short *sp_next = str.p + s0 * kNarrowStep * str.ld;
    const int ld = (int)str.ld;
    int rows_left = (int)(rows_end - s0 * kNarrowStep); // of the steps not asked for yet
    const int off = ((tid / PR) * ld + ((tid % PR) ^ piece_turn<KD>(tid / PR)) * 8) * 2, apart = 256 / PR * ld * 2;
    const int to_lds = __builtin_amdgcn_readfirstlane(tid >> 6) * 1024;
    float4 c_row = make_float4(0.f, INFINITY, 0.f, 0.f);
    int c_hit = -1;
    int64_t c_next = s0 * kNarrowStep;
    auto load = [&](char *to) {
        const int have = rows_left < kNarrowStep ? rows_left : kNarrowStep;
        const unsigned bytes = have > 0 ? (unsigned)((have - 1) * ld + KD) * 2 : 0;
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<short *>(sp_next + q * str.plane), 0, bytes, 0x00027000);
#pragma unroll
            for (int i = 0; i < N; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void)(to + q * PLANE + i * 4096 + to_lds), 16, off,
                                                         i * apart, 0, 0);
        }
        sp_next += kNarrowStep * str.ld;
        rows_left -= kNarrowStep;
    };
    // what the weight's gradient needs of the streamed rows: registers a step
    // ahead, then LDS
    auto load_rows = [&]() {
        if (VOC && tid < kNarrowStep) {
            const int64_t i = c_next + tid;
            c_row = make_float4(0.f, INFINITY, 0.f, 0.f);
            c_hit = -1;
            if (i < rows_end) {
                c_row = o.rows[i];
                const int64_t target = o.targets[i], t = target - block0;
                if (row_counts(target, o.ignore, o.V) && t >= 0 && t < 128 * NO) c_hit = (int)t;
            }
        }
        c_next += kNarrowStep;
    };
    auto store_rows = [&](int buf) {
        if (VOC && tid < kNarrowStep) {
            of_row[buf][0][tid] = c_row.x;
            of_row[buf][1][tid] = c_row.y;
            of_row[buf][2][tid] = c_row.z;
            hit_row[buf][tid] = c_hit;
        }
    };
    auto row_of = [&](int r) { return 8 * (r / 4) + 4 * half + r % 4; };
    const int straight = (lane & 31) * P, turn = (piece_turn<KD>(lane & 31) ^ half) * 16;
    const int four = (lane & 15) >> 2, piece = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
    const int turned = (4 * half + four) * P + (((KD == 128 ? four : four >> 1) << 2 | (piece ^ half)) << 4) +
                       (lane & 1) * 8;

    load_rows();
    store_rows(0);
    load_rows();
    load(lds0);
    loads_meet<0>();
    auto step = [&](int st, auto which) {
        constexpr int buf = decltype(which)::value;
        char *here = buf ? lds1 : lds0;
        load(buf ? lds0 : lds1); // (behind the barrier that ends its last reads)
        store_rows(buf ^ 1);
        load_rows();
        f32x16 z[NO];
#pragma unroll
        for (int b = 0; b < NO; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) z[b][r] = 0.f;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            s16x8 f[PL];
#pragma unroll
            for (int q = 0; q < PL; ++q)
                f[q] = *reinterpret_cast<const s16x8 *>(here + straight + q * PLANE + ((k * 32) ^ turn));
            if constexpr (PL == 2) {
#pragma unroll
                for (int b = 0; b < NO; ++b) z[b] = Terms<PL>::mma(f[PL - 1], of[0][b][k], z[b]);
#pragma unroll
                for (int b = 0; b < NO; ++b) z[b] = Terms<PL>::mma(f[0], of[PL - 1][b][k], z[b]);
            }
#pragma unroll
            for (int b = 0; b < NO; ++b) z[b] = Terms<PL>::mma(f[0], of[0][b][k], z[b]);
        }
        const int left = (int)(rows_end - s0 * kNarrowStep) - st * kNarrowStep; // streamed rows that exist
        if constexpr (MODE == ROW_STATS) {
#pragma unroll
            for (int b = 0; b < NO; ++b) {
                if (left < kNarrowStep) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (row_of(r) >= left) z[b][r] = -INFINITY;
                }
                if (__any(hit[b] == st)) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (hit[b] == st && row_of(r) == hit_row_of[b])
                            o.target_logit[own0 + b * 32 + (lane & 31)] = z[b][r] * scale[b];
                }
                float m = top[b];
#pragma unroll
                for (int r = 0; r < 16; ++r) m = fmaxf(m, z[b][r]);
                const float ref = m == -INFINITY ? 0.f : m, base = scale[b] * 1.44269504f;
                float s = 0.f; // of the step first: a row's sum is as many additions long as it has steps
#pragma unroll
                for (int r = 0; r < 16; ++r) s += __builtin_amdgcn_exp2f((z[b][r] - ref) * base);
                sum[b] = fmaf(sum[b], __builtin_amdgcn_exp2f((top[b] - ref) * base), s);
                top[b] = m;
            }
        } else {
            s16x8 d[PL][NO][2];
            bool here_hit[NO];
#pragma unroll
            for (int b = 0; b < NO; ++b) {
                if constexpr (VOC) {
                    const int t = hit_row[buf][lane & 31] - (wave * NO + b) * 32;
                    here_hit[b] = __any(t >= 0 && t < 32);
                } else {
                    here_hit[b] = __any(hit[b] == st);
                }
            }
            // exponentials
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float ls[4], sc[4];
                if constexpr (VOC) {
                    load_vec<float, 4>(&of_row[buf][0][8 * e + 4 * half], sc);
                    load_vec<float, 4>(&of_row[buf][1][8 * e + 4 * half], ls);
                }
#pragma unroll
                for (int b = 0; b < NO; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        z[b][4 * e + r] = __builtin_amdgcn_exp2f(
                            fmaf(z[b][4 * e + r], VOC ? sc[r] : scale[b], VOC ? -ls[r] : -lse[b]) * 1.44269504f);
            }
            // targets, and streamed rows past the vocabulary's end
#pragma unroll
            for (int b = 0; b < NO; ++b) {
                if (here_hit[b]) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const bool is = VOC ? hit_row[buf][row_of(r)] == (wave * NO + b) * 32 + (lane & 31)
                                            : hit[b] == st && row_of(r) == hit_row_of[b];
                        if (is) z[b][r] -= 1.f;
                    }
                }
                if (!VOC && left < kNarrowStep) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (row_of(r) >= left) z[b][r] = 0.f;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float gr[4];
                if constexpr (VOC) load_vec<float, 4>(&of_row[buf][2][8 * e + 4 * half], gr);
#pragma unroll
                for (int b = 0; b < NO; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        short w[PL];
                        split<PL>(z[b][4 * e + r] * (VOC ? gr[r] : g[b]), w);
#pragma unroll
                        for (int q = 0; q < PL; ++q) d[q][b][e >> 1][(e & 1) * 4 + r] = w[q];
                    }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int c = 0; c < CB; ++c) {
                    s16x8 f[PL];
#pragma unroll
                    for (int q = 0; q < PL; ++q) {
                        typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;
                        const char *from = here + q * PLANE + 16 * u * P;
                        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (lds_s16x4)(from + (turned ^ (c << 6))));
                        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (lds_s16x4)(from + 8 * P + (turned ^ (c << 6) ^ 32)));
                        f[q] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                    }
                    if constexpr (PL == 2) {
#pragma unroll
                        for (int b = 0; b < NO; ++b) acc[b][c] = Terms<PL>::mma(d[PL - 1][b][u], f[0], acc[b][c]);
#pragma unroll
                        for (int b = 0; b < NO; ++b) acc[b][c] = Terms<PL>::mma(d[0][b][u], f[PL - 1], acc[b][c]);
                    }
#pragma unroll
                    for (int b = 0; b < NO; ++b) acc[b][c] = Terms<PL>::mma(d[0][b][u], f[0], acc[b][c]);
                }
        }
        __builtin_amdgcn_sched_barrier(0);
        loads_meet<0>();
        __builtin_amdgcn_sched_barrier(0);
    };
    auto run = [&](int first, int last) { // an odd number of steps ends with one of no rows
        for (int st = first; st < last; st += 2) {
            step(st, std::integral_constant<int, 0>());
            step(st + 1, std::integral_constant<int, 1>());
        }
    };
    if constexpr (MODE == ROW_STATS) {
        run(0, steps);
#pragma unroll
        for (int b = 0; b < NO; ++b) {
            const int64_t i = own0 + b * 32 + (lane & 31);
            const float2 other = make_float2(__shfl_xor(top[b], 32, 64) * scale[b], __shfl_xor(sum[b], 32, 64));
            const float2 both = join_sums(make_float2(top[b] * scale[b], sum[b]), other);
            if (lane < 32 && i < own.rows) o.part[sp * o.n + i] = both;
        }
    } else {
        const float by = PL == 2 && VOC ? ldexpf(1.f, -(kUnitExp + *o.all_exp)) : unit;
        for (int first = 0; first < steps; first += kNarrowChain) {
            const int last = PL == 2 && steps - first > kNarrowChain ? first + kNarrowChain : steps;
#pragma unroll
            for (int b = 0; b < NO; ++b)
#pragma unroll
                for (int c = 0; c < CB; ++c)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[b][c][r] = 0.f;
            run(first, last);
#pragma unroll
            for (int b = 0; b < NO; ++b)
#pragma unroll
                for (int c = 0; c < CB; ++c)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int64_t i = own0 + b * 32 + row_of(r);
                        const int k = c * 32 + (lane & 31);
                        if (i >= own.rows || k >= o.D) continue;
                        if (VOC && o.splits == 1) {
                            T *to = static_cast<T *>(o.out) + i * o.ld_out + k;
                            const float x = acc[b][c][r] * by;
                            *to = (T)(PL == 2 && first ? (float)*to + x : x);
                        } else {
                            float *to = o.sum + (sp * own.rows + i) * o.D + k;
                            *to = PL == 2 && first ? *to + acc[b][c][r] : acc[b][c][r];
                        }
                    }
            if (PL == 1) break; // all steps
        }
    }
}

// The statistics of at most 32 NB rows of fp32: the weight is read once, as it
// is, by the fp32 matrix instructions.  Splitting it into fp16 terms first
// costs three more passes over it, more than the slower products do here
// (50000 x 1024: 1 row 60 us against 198, 64 rows 87 against 204).  A wave has 32
// MA rows of the weight; a lane reads four values of a row at a time, and each
// instruction takes the same one of the four from both halves of the wave.
template <int MA, int NB>
__global__ __launch_bounds__(256) void k_xent_few(const float *w, int64_t ld_w, const float *h, int64_t ld_h, int64_t D,
                                                  Output o)
{
    constexpr int TM = 128 * MA, STEP = 32;
    __shared__ float red[2][4][32 * NB];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = (lane >> 5) * 4;
    const int64_t m0 = (int64_t)blockIdx.x * TM;
    const float *wr[MA], *hr[NB];
#pragma unroll
    for (int a = 0; a < MA; ++a) {
        const int64_t r = m0 + wave * 32 * MA + a * 32 + (lane & 31);
        wr[a] = w + (r < o.V ? r : o.V - 1) * ld_w + half;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t r = b * 32 + (lane & 31);
        hr[b] = h + (r < o.n ? r : o.n - 1) * ld_h + half;
    }
    f32x16 acc[MA][NB];
#pragma unroll
    for (int a = 0; a < MA; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;
    auto steps = [&](int64_t k, auto whole) {
        constexpr int C = STEP / 8;
        float x[MA][C][4], y[NB][C][4];
        auto take = [&](const float *p, int c, float (&v)[4]) {
            const int64_t at = k + c * 8, left = D - half - at;
            if constexpr (decltype(whole)::value) load_vec<float, 4>(p + at, v);
            else load_part<float, 4>(p + (left > 0 ? at : 0), (int)(left < 0 ? 0 : left < 4 ? left : 4), v);
        };
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int a = 0; a < MA; ++a) take(wr[a], c, x[a][c]);
#pragma unroll
            for (int b = 0; b < NB; ++b) take(hr[b], c, y[b][c]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int a = 0; a < MA; ++a)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x2f32(x[a][c][e], y[b][c][e], acc[a][b], 0, 0, 0);
    };
    int64_t k = 0;
    for (; k + STEP <= D; k += STEP) steps(k, std::true_type());
    if (k < D) steps(k, std::false_type());
    auto row_of = [&](int a, int r) { return wave * 32 * MA + a * 32 + 8 * (r / 4) + 4 * (lane >> 5) + (r % 4); };
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t i = b * 32 + (lane & 31);
        const int64_t t = i < o.n ? o.targets[i] - m0 : -1;
        float top, sum;
        column_stats(acc, b, row_of, o.V - m0, TM, t, wave * 32 * MA, 1.f, o.target_logit + (i < o.n ? i : 0), top,
                     sum);
        if (lane < 32) {
            red[0][wave][i] = top;
            red[1][wave][i] = sum;
        }
    }
    __syncthreads();
    const int i = threadIdx.x;
    if (i < 32 * NB && i < o.n) {
        float2 all = make_float2(red[0][0][i], red[1][0][i]);
#pragma unroll
        for (int q = 1; q < 4; ++q) all = join_sums(all, make_float2(red[0][q][i], red[1][q][i]));
        o.part[blockIdx.x * o.n + i] = all;
    }
}

// What a gradient's sums are in: bf16 inputs, the unit of d; fp16 terms, the
// operand's scale, and for the hidden rows their own dL/dloss.
struct SumUnit {
    const float *top_grad; // bf16
    const int *exp;        // fp16 terms
    const float *grad;     // with targets: of rows that count
    const int64_t *targets;
    int64_t ignore, V;
};

// A gradient from its splits' sums.  `groups` (a power of two) threads share
// four values and the splits, so that many splits of few rows are not one
// thread's chain (512 of 40 x 64: 129 us by one, 10 by 32); their sums meet in
// LDS in order.
template <class T>
__global__ __launch_bounds__(256) void k_xent_sum(const float *sum, int splits, int groups, int64_t rows, int64_t D,
                                                  SumUnit u, T *out, int64_t ld)
{
    __shared__ float4 part[256];
    const int each = 256 / groups, grp = threadIdx.x / each, in = threadIdx.x % each;
    const int64_t chunks = (D + 3) / 4, all = rows * chunks, step = (int64_t)gridDim.x * each;
    const float unit = u.exp ? ldexpf(1.f, -(kUnitExp + *u.exp)) : *u.top_grad;
    for (int64_t c0 = (int64_t)blockIdx.x * each; c0 < all; c0 += step) {
        const int64_t c = c0 + in < all ? c0 + in : all - 1;
        const int64_t i = c / chunks, k = (c - i * chunks) * 4;
        const int left = (int)(D - k < 4 ? D - k : 4);
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int q = grp; q < splits; q += groups) {
            float y[4];
            load_part<float, 4>(sum + ((int64_t)q * rows + i) * D + k, left, y);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] += y[r];
        }
        if (groups > 1) {
            __syncthreads(); // the last round's parts have been read
            part[threadIdx.x] = make_float4(x[0], x[1], x[2], x[3]);
            __syncthreads();
            for (int q = 1; q < groups && grp == 0; ++q) {
                const float4 y = part[q * each + in];
                x[0] += y.x;
                x[1] += y.y;
                x[2] += y.z;
                x[3] += y.w;
            }
        }
        // the sums of a row that does not count are 0 whatever its dL/dloss
        const float g = u.targets && row_counts(u.targets[i], u.ignore, u.V) ? u.grad[i] : 1.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = x[r] * unit * g;
        if (grp == 0 && c0 + in < all) store_part<T, 4>(out + i * ld + k, left, x);
    }
}

// The exponent that brings a largest magnitude into [2^14, 2^15).
__device__ __forceinline__ int scale_exp(float top)
{
    return top > 0.f ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
}
__device__ __forceinline__ float finite_abs(float x)
{
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;
}

// One piece of a row, times `by` and scaled, split; zeros where it is cleared.
template <class T, int PL>
__device__ __forceinline__ void pack_piece(const T *src, int64_t left, float by, int e, bool clear, short *dst,
                                           int64_t plane)
{
    float x[8];
    load_part<T, 8>(src, (int)(left < 0 ? 0 : left < 8 ? left : 8), x);
    s16x8 w[PL];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        short s[PL];
        split<PL>(clear ? 0.f : PL == 2 ? ldexpf(x[i] * by, e) : x[i], s);
#pragma unroll
        for (int q = 0; q < PL; ++q) w[q][i] = s[q];
    }
#pragma unroll
    for (int q = 0; q < PL; ++q) *reinterpret_cast<s16x8 *>(dst + q * plane) = w[q];
}

// Jobs around the products, each done by blocks [0, blocks) of `threads`
// threads.  Jobs that do not wait for each other share a launch: at small sizes
// a launch costs more than they do.
template <class A, class B>
struct Both {
    static constexpr int threads = A::threads;
    static_assert(A::threads == B::threads, "one block size");
    A a;
    B b;
    int na;
    __device__ void operator()(int block, int blocks) const
    {
        if (block < na) a(block, na);
        else b(block - na, blocks - na);
    }
};
template <int THREADS>
struct NoJobOf {
    static constexpr int threads = THREADS;
    __device__ void operator()(int, int) const {}
};
template <class F>
__global__ __launch_bounds__(F::threads) void k_jobs(F f)
{
    f((int)blockIdx.x, (int)gridDim.x);
}

// Hidden rows as planes with `ld` columns, zero past D; a wave per row.  fp16
// terms: each row scaled by a power of two of its own, and with targets the
// largest magnitude of each row that counts left in `tops`.
template <class T, int PL>
struct PackRows {
    static constexpr int threads = 256;
    const T *src;
    int64_t ld_src, rows, D;
    short *dst;
    int64_t ld, plane;
    int *exps;
    float *tops;
    const int64_t *targets;
    int64_t ignore, V;

    __device__ void operator()(int block, int blocks) const
    {
        const int lane = threadIdx.x & 63;
        for (int64_t r = (int64_t)block * 4 + (threadIdx.x >> 6); r < rows; r += (int64_t)blocks * 4) {
            const T *row = src + r * ld_src;
            int e = 0;
            if constexpr (PL == 2) {
                float top = 0.f;
                for (int64_t k = lane * 8; k < D; k += 512) {
                    float x[8];
                    load_part<T, 8>(row + k, (int)(D - k < 8 ? D - k : 8), x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_abs(x[i]));
                }
#pragma unroll
                for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
                e = scale_exp(top);
                if (lane == 0) {
                    exps[r] = e;
                    if (targets) tops[r] = row_counts(targets[r], ignore, V) ? top : 0.f;
                }
            }
            for (int64_t k = lane * 8; k < ld; k += 512)
                pack_piece<T, PL>(row + (k < D ? k : 0), D - k, 1.f, e, false, dst + r * ld + k, plane);
        }
    }
};

// Packed rows that do not count become zeros once their statistics are known:
// whatever they held (NaN, or a finite value whose logits overflow), their
// logits are then 0, d is 0 and so is what they add to the weight's gradient.
// A wave per row.
template <int PL>
struct ClearRows {
    static constexpr int threads = 1024;
    short *dst;
    int64_t ld, plane, rows;
    const int64_t *targets;
    int64_t ignore, V;

    __device__ void operator()(int block, int blocks) const
    {
        const int lane = threadIdx.x & 63;
        for (int64_t r = (int64_t)block * 16 + (threadIdx.x >> 6); r < rows; r += (int64_t)blocks * 16) {
            if (row_counts(targets[r], ignore, V)) continue;
            const s16x8 none = {};
#pragma unroll
            for (int q = 0; q < PL; ++q)
                for (int64_t k = lane * 8; k < ld; k += 512)
                    *reinterpret_cast<s16x8 *>(dst + q * plane + r * ld + k) = none;
        }
    }
};

// The rows that count times their dL/dloss as fp16 planes scaled by one power of
// two, the others as zeros: the operand of the weight's gradient.
struct PackCounting {
    static constexpr int threads = 1024;
    const float *src;
    int64_t ld_src, rows, D;
    short *dst;
    int64_t ld, plane;
    const int *exp;
    const float *grad;
    const int64_t *targets;
    int64_t ignore, V;

    __device__ void operator()(int block, int blocks) const
    {
        const int64_t chunks = ld / 8, step = (int64_t)blocks * threads;
        const int e = *exp;
        for (int64_t c = (int64_t)block * threads + threadIdx.x; c < rows * chunks; c += step) {
            const int64_t r = c / chunks, k = (c - r * chunks) * 8;
            // the factor's exponent goes with the scale: their product may pass what fp32 holds
            const float g = grad[r];
            pack_piece<float, 2>(src + r * ld_src + (k < D ? k : 0), D - k, __builtin_amdgcn_frexp_mantf(g),
                                 e + __builtin_amdgcn_frexp_expf(g), !row_counts(targets[r], ignore, V),
                                 dst + r * ld + k, plane);
        }
    }
};

// Largest finite magnitude of the weight, per block.
struct WeightTop {
    static constexpr int threads = 256;
    const float *src;
    int64_t ld, rows, D;
    float *part;

    __device__ void operator()(int block, int blocks) const
    {
        __shared__ float sm[4];
        const int64_t chunks = (D + 7) / 8, step = (int64_t)blocks * 256;
        float top = 0.f;
        for (int64_t c = (int64_t)block * 256 + threadIdx.x; c < rows * chunks; c += step) {
            const int64_t r = c / chunks, k = (c - r * chunks) * 8;
            float x[8];
            load_part<float, 8>(src + r * ld + k, (int)(D - k < 8 ? D - k : 8), x);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_abs(x[i]));
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
        if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = top;
        __syncthreads();
        if (threadIdx.x == 0) part[block] = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    }
};

// The weight as planes with `ld` columns, zero past D.  fp16 terms: scaled by
// one power of two, from the largest of the `parts` magnitudes.
template <class T, int PL>
struct PackWeight {
    static constexpr int threads = 256;
    const T *src;
    int64_t ld_src, rows, D;
    short *dst;
    int64_t ld, plane;
    const float *part;
    int parts;
    int *exp;

    __device__ void operator()(int block, int blocks) const
    {
        int e = 0;
        if constexpr (PL == 2) {
            float top = 0.f;
            for (int i = threadIdx.x & 63; i < parts; i += 64) top = fmaxf(top, part[i]);
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
            e = scale_exp(top);
            if (block == 0 && threadIdx.x == 0) *exp = e;
        }
        const int64_t chunks = ld / 8, step = (int64_t)blocks * 256;
        for (int64_t c = (int64_t)block * 256 + threadIdx.x; c < rows * chunks; c += step) {
            const int64_t r = c / chunks, k = (c - r * chunks) * 8;
            pack_piece<T, PL>(src + r * ld_src + (k < D ? k : 0), D - k, 1.f, e, false, dst + r * ld + k, plane);
        }
    }
};

// bf16: the unit of d, the largest |grad_loss| of the rows that count.  With
// equal gradients (a mean over the rows) d is exp(z - lse) - [v = target] in this
// unit, and the target's -1 + p, the largest term of both gradients, rounds to
// bf16 without error for small p.  1 where there is nothing to scale.  fp16
// terms: the exponent for all rows together, from the largest exponent of a
// row's gradient and its largest value together.  One block.
struct Units {
    static constexpr int threads = 256;
    static constexpr int kNone = -(1 << 20);
    const float *grad;
    const int64_t *targets;
    int64_t ignore, n, V;
    const float *tops; // null for bf16
    float *unit;
    int *all_exp;

    __device__ void operator()(int, int) const
    {
        __shared__ float sm[4];
        __shared__ int se[4];
        float m = 0.f;
        int e = kNone;
        constexpr int U = 16; // loads in flight: their latency is what the one block waits for
        for (int64_t i0 = threadIdx.x; i0 < n; i0 += 256 * U) {
            int64_t t[U];
            float a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + u * 256 < n ? i0 + u * 256 : i0;
                t[u] = targets[i];
                a[u] = finite_abs(grad[i]);
                b[u] = tops ? tops[i] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!row_counts(t[u], ignore, V)) continue;
                m = fmaxf(m, a[u]);
                if (a[u] > 0.f && b[u] > 0.f) {
                    const int both = __builtin_amdgcn_frexp_expf(a[u]) + __builtin_amdgcn_frexp_expf(b[u]);
                    e = e > both ? e : both;
                }
            }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            m = fmaxf(m, __shfl_xor(m, o, 64));
            const int other = __shfl_xor(e, o, 64);
            e = e > other ? e : other;
        }
        if ((threadIdx.x & 63) == 0) {
            sm[threadIdx.x >> 6] = m;
            se[threadIdx.x >> 6] = e;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 4; ++w) {
                m = fmaxf(m, sm[w]);
                e = e > se[w] ? e : se[w];
            }
            *unit = m > 0.f ? m : 1.f;
            *all_exp = e == kNone ? 0 : 15 - e;
        }
    }
};

// lse and loss of sixteen rows per block from the tiles' maxima and sums, 64
// groups of tiles joined in order.
struct Join {
    static constexpr int threads = 1024;
    const float2 *part;
    int64_t tiles, n, V;
    const int64_t *targets;
    int64_t ignore;
    const float *target_logit;
    float *loss, *lse;
    int *status;
    // with `rows`: what the streamed rows of the weight's gradient need, too
    float4 *rows;
    const float *grad, *unit;
    const float *tops; // null for bf16
    const int *h_exp, *w_exp, *all_exp;

    __device__ void operator()(int block, int) const
    {
        __shared__ float2 sm[64][16];
        const int r = threadIdx.x & 15, g = threadIdx.x >> 4;
        const int64_t i = (int64_t)block * 16 + r, ic = i < n ? i : n - 1;
        float2 all = make_float2(-INFINITY, 0.f);
        for (int64_t t = g; t < tiles; t += 4 * 64) {
            float2 p[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                p[u] = part[(t + u * 64 < tiles ? t + u * 64 : t) * n + ic];
                if (t + u * 64 >= tiles) p[u] = make_float2(-INFINITY, 0.f);
            }
            all = join_sums(all, join_sums(join_sums(p[0], p[1]), join_sums(p[2], p[3])));
        }
        sm[g][r] = all;
        __syncthreads();
        if (g || i >= n) return;
        float top = -INFINITY, sum = 0.f;
#pragma unroll 8
        for (int q = 0; q < 64; ++q) top = fmaxf(top, sm[q][r].x);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 8
        for (int q = 0; q < 64; ++q) sum += sm[q][r].y * __expf(sm[q][r].x - ref);
        const float z = (top == -INFINITY ? 0.f : top) + logf(sum);
        const int64_t t = targets[i];
        const bool in = t >= 0 && t < V;
        if (!in && t != ignore) atomicOr(status + ST_ERR, (int)STB_INDEX);
        lse[i] = z;
        loss[i] = in && t != ignore ? z - target_logit[i] : 0.f;
        if (!rows) return;
        float4 c = make_float4(1.f, INFINITY, 0.f, 0.f);
        if (in && t != ignore) {
            c.y = z;
            if (tops) {
                c.x = ldexpf(1.f, -(h_exp[i] + *w_exp));
                // (a row of zeros has no scale, and no part in the sum)
                c.z = tops[i] > 0.f ? ldexpf(grad[i], kUnitExp + *all_exp - h_exp[i]) : grad[i] * 0.f;
            } else {
                c.z = grad[i] / *unit;
            }
        }
        rows[i] = c;
    }
};

template <class T>
__global__ __launch_bounds__(256) void k_xent_clear(T *p, int64_t ld, int64_t rows, int64_t D)
{
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < rows * D; c += step)
        p[c / D * ld + c % D] = (T)0.f;
}

struct XentPlan {
    float *target_logit, *top_grad, *w_part, *tops, *lse;
    int *h_exp, *all_exp, *w_exp;
    float2 *part;
    float4 *rows;
    short *h, *h_all, *w; // packed operands, of those that are packed
    float *sum, *w_sum;
    short *d;
    int64_t Kp, nr, piece;
    int splits, w_splits; // of the sums over the vocabulary (dH) and over the rows (dW)
    int parts;            // of dH's splits, those that the first piece fills: later pieces add to these only
    size_t bytes;
};

// Side of a product's tiles.  256 x 256 tiles read each operand least often
// (logits of 8192 x 16384, bf16: K = 4096 at 1315 TFLOP/s, against 1139 in tiles
// of 128).  Tiles of 128, of which a compute unit holds two, hide the start and
// the end of one behind the products of the other and win where those are long
// beside the sum (bf16 logits, K = 512: 170 us against 182, equal at 1024; fp32,
// whose sums are three products long, K = 256: 256 against 261, 460 against 432
// at 512; the other products' ends are shorter), and take outputs with a side of
// at most 128 and grids that would leave compute units idle.
constexpr int64_t kShortSum = 256, kShortLogits = 512;
inline int64_t tile_side(int64_t M, int64_t N, int64_t K, int splits, bool short_terms)
{
    if (M <= 128 || N <= 128 || K <= (short_terms ? kShortLogits : kShortSum)) return 128;
    return ((M + 255) / 256) * ((N + 255) / 256) * splits < kCUs ? 128 : 256;
}

// How often the sum of a gradient (D columns, `rows` rows, K summed values) is
// split: where its tiles are fewer than the compute units take at a time, the
// sum is shared out.
int sum_splits(int64_t rows, int64_t D, int64_t K)
{
    const bool small = rows <= 128 || D <= 128;
    const int64_t side = small ? 128 : 256, slots = small ? 2 * kCUs : kCUs;
    int64_t s = slots / (((D + side - 1) / side) * ((rows + side - 1) / side));
    if (s > K / kSplitK) s = K / kSplitK;
    return (int)(s < 1 ? 1 : s);
}

// A sum over K values in at most `most` parts of `each` values (whole steps);
// every part begins before K's end.
struct SumParts {
    int64_t each;
    int parts;
};
inline SumParts sum_parts(int64_t K, int most)
{
    const int64_t each = up((K + most - 1) / most, kPadK);
    return {each, (int)((K + each - 1) / each)};
}

// Rows of d: whole tiles, so that they are written without a test.
inline int64_t d_rows(int64_t n) { return n <= 128 ? 128 : up(n, 256); }

// Narrow kernels: 32-row blocks that a wave owns (as many as 256 registers hold;
// a streamed fragment read from LDS serves all of them; bf16 rows of 128 with
// gradients: 3.3 ms with one, 4.2 with two, which spill), and how often the
// streamed rows are split so that the blocks fill rounds of two on each compute
// unit.
constexpr int narrow_blocks(int PL, int mode, int64_t Kp)
{
    return mode == ROW_STATS || (PL == 1 && Kp == 64) ? 2 : 1;
}
inline bool narrow_rows(int64_t D) { return D <= kNarrow; }
inline int whole_splits(int64_t streamed, int64_t s) // s, less the splits that equal parts leave empty
{
    const int64_t steps = (streamed + kNarrowStep - 1) / kNarrowStep;
    if (s < 1) s = 1;
    const int64_t per = (steps + s - 1) / s;
    return (int)((steps + per - 1) / per);
}
int narrow_splits(int64_t own, int64_t streamed, int blocks)
{
    const int64_t owns = (own + 128 * blocks - 1) / (128 * blocks), slots = 2 * kCUs;
    const int64_t steps = (streamed + kNarrowStep - 1) / kNarrowStep;
    int64_t s = owns < slots ? slots / owns : 1;
    auto full = [&](int64_t k) { return 4 * owns * k >= 3 * up(owns * k, slots); };
    while (owns * s < 8 * slots && !full(s)) ++s;
    if (s > steps / kNarrowSteps) s = steps / kNarrowSteps;
    return whole_splits(streamed, s);
}

int64_t best_piece(int64_t n, int64_t V, int64_t D, int PL)
{
    if (narrow_rows(D)) return -narrow_splits(n, V, narrow_blocks(PL, ROW_GRAD, up(D, kPadK)));
    int64_t c = (int64_t)(kPieceBytes / ((size_t)PL * d_rows(n) * 2)) / kRound * kRound;
    if (c < 8 * kRound) c = 8 * kRound;
    return up(V < c ? V : c, kRound);
}

// Which operands are packed copies.  The statistics of few fp32 rows take none;
// a bf16 weight serves in place where its rows are laid out as the loads need
// them, and so do bf16 hidden rows without gradients (with them, rows that do
// not count are cleared in the copy).
struct Packed {
    bool h, w;
};
Packed packed(int64_t n, int PL, bool grad, bool h_fits, bool w_fits)
{
    const bool few = PL == 2 && n <= kFewRows;
    return {grad || (!few && !h_fits), (grad || !few) && !w_fits};
}

// `piece` columns of d (0: forward only; below 0: gradients by the narrow
// kernels, -piece splits of dH).
XentPlan plan_xent(int64_t n, int64_t V, int64_t D, int PL, Packed pack, int64_t piece, char *base)
{
    size_t off = TT_EMB_STATUS_BYTES;
    auto take = [&](size_t bytes) {
        char *r = base ? base + off : nullptr;
        off += round256(bytes > 0 ? bytes : 1);
        return r;
    };
    XentPlan p{};
    p.Kp = up(D, kPadK);
    p.nr = d_rows(n);
    p.piece = piece;
    p.target_logit = (float *)take(4 * n);
    p.top_grad = (float *)take(4);
    p.part = (float2 *)take(8 * (size_t)n * ((V + kLeast - 1) / kLeast));
    p.w_part = (float *)take(4 * kMaxParts);
    p.h_exp = (int *)take(4 * n);
    p.w_exp = (int *)take(4);
    p.all_exp = (int *)take(4);
    p.tops = (float *)take(4 * n);
    if (piece && PL == 2 && n <= kFewRows) p.lse = (float *)take(4 * n);
    if (pack.h) p.h = (short *)take((size_t)PL * n * p.Kp * 2);
    if (pack.w) p.w = (short *)take((size_t)PL * V * p.Kp * 2);
    if (piece < 0) {
        p.rows = (float4 *)take(16 * (size_t)n);
        p.splits = (int)-piece;
        p.sum = (float *)take(4 * (size_t)p.splits * n * D);
        p.w_splits = narrow_splits(V, n, narrow_blocks(PL, VOC_GRAD, p.Kp));
        if (p.w_splits > 1) p.w_sum = (float *)take(4 * (size_t)p.w_splits * V * D);
    } else if (piece) {
        if (PL == 2) p.h_all = (short *)take((size_t)PL * n * p.Kp * 2);
        p.splits = sum_splits(n, D, piece);
        p.parts = sum_parts(V < piece ? V : piece, p.splits).parts;
        p.sum = (float *)take(4 * (size_t)p.splits * n * D);
        p.w_splits = piece >= V ? sum_splits(V, D, n) : 1;
        if (p.w_splits > 1) p.w_sum = (float *)take(4 * (size_t)p.w_splits * V * D);
        p.d = (short *)take((size_t)PL * p.nr * piece * 2);
    }
    p.bytes = off;
    return p;
}

// The plan whose pieces fit the workspace.
XentPlan fit_xent(int64_t n, int64_t V, int64_t D, int PL, Packed pack, bool grad, char *base, size_t ws_bytes)
{
    int64_t piece = grad ? best_piece(n, V, D, PL) : 0;
    auto fits = [&]() { return plan_xent(n, V, D, PL, pack, piece, nullptr).bytes <= ws_bytes; };
    while (piece < -1 && !fits()) piece = -whole_splits(V, -piece / 2);
    while (piece > kRound && !fits()) piece = up(piece / 2, kRound);
    return plan_xent(n, V, D, PL, pack, piece, base);
}

// Whether rows of an operand serve in place: bf16 rows of whole steps at
// multiples of 16 bytes (rows further apart would pass the 31 bits of a tile's loads).
bool fits_in_place(int PL, int64_t D) { return PL == 1 && D % kPadK == 0; }
bool in_place(const void *src, int64_t ld, int64_t D, int PL)
{
    return fits_in_place(PL, D) && ld % 8 == 0 && ld <= (1 << 20) && (reinterpret_cast<uintptr_t>(src) & 15u) == 0;
}
Packed packed(const XentArgs &a, int PL, bool grad)
{
    return packed(a.n, PL, grad, in_place(a.hidden, a.ld_h, a.D, PL), in_place(a.weight, a.ld_w, a.D, PL));
}

unsigned blocks_for(int64_t threads)
{
    const int64_t b = (threads + 255) / 256;
    return (unsigned)(b < 65536 ? b : 65536);
}

// A product with M contiguous outputs in each of N rows; returns the tiles along M.
template <int PL, bool XT, bool YT, int OUT>
int64_t product(const Operand &x, const Operand &y, int64_t M, int64_t N, int64_t K, const Output &o, hipStream_t s)
{
    const int splits = OUT == OUT_SUM ? o.splits : 1;
    const int64_t side = tile_side(M, N, K, splits, PL == 1 && (OUT == OUT_STATS || OUT == OUT_D));
    const int64_t mt = (M + side - 1) / side, nt = (N + side - 1) / side;
    const dim3 grid(tile_grid(mt, nt, splits));
    if (side == 256)
        hipLaunchKernelGGL((k_product<PL, XT, YT, OUT, 4, 4>), grid, dim3(256), 0, s, x, y, K, mt, nt, o);
    else
        hipLaunchKernelGGL((k_product<PL, XT, YT, OUT, 2, 2>), grid, dim3(256), 0, s, x, y, K, mt, nt, o);
    return mt;
}

template <class T>
void sum_up(const float *sum, int splits, int64_t rows, int64_t D, const SumUnit &unit, void *out, int64_t ld,
            hipStream_t s)
{
    const int groups = splits >= 64 ? 32 : splits >= 8 ? 8 : 1;
    hipLaunchKernelGGL(k_xent_sum<T>, dim3(blocks_for(rows * ((D + 3) / 4) * groups)), dim3(256), 0, s, sum, splits,
                       groups, rows, D, unit, static_cast<T *>(out), ld);
}

// A pass of the narrow kernels; `splits` as planned.
template <class T, int PL, int MODE>
void narrow(const Operand &own, const Operand &streamed, int64_t Kp, int splits, const Output &o, hipStream_t s)
{
    auto run = [&](auto kd) {
        constexpr int KD = decltype(kd)::value, NO = narrow_blocks(PL, MODE, KD);
        const int64_t owns = (own.rows + 128 * NO - 1) / (128 * NO);
        const int64_t steps = (streamed.rows + kNarrowStep - 1) / kNarrowStep, per = (steps + splits - 1) / splits;
        hipLaunchKernelGGL((k_narrow<T, PL, KD, MODE, NO>), dim3((unsigned)up(owns * splits, 8)), dim3(256), 0, s, own,
                           streamed, owns, per, o);
    };
    if (Kp == 64) run(std::integral_constant<int, 64>());
    else run(std::integral_constant<int, 128>());
}

// One launch for two jobs of na and nb blocks (none for none).
template <class A, class B>
void run_jobs(const A &a, int na, const B &b, int nb, hipStream_t s)
{
    if (na + nb == 0) return;
    typedef Both<A, B> F;
    hipLaunchKernelGGL(k_jobs<F>, dim3((unsigned)(na + nb)), dim3(F::threads), 0, s, F{a, b, na});
}

// Statistics of at most 128 fp32 rows without packed operands; returns the tiles.
int64_t few_rows(const XentArgs &a, const Output &o, hipStream_t s)
{
    const float *w = static_cast<const float *>(a.weight), *h = static_cast<const float *>(a.hidden);
    const int64_t side = a.n <= 32 ? 128 : 256, tiles = (a.V + side - 1) / side;
    const dim3 grid((unsigned)tiles);
    if (a.n <= 32) hipLaunchKernelGGL((k_xent_few<1, 1>), grid, dim3(256), 0, s, w, a.ld_w, h, a.ld_h, a.D, o);
    else if (a.n <= 64) hipLaunchKernelGGL((k_xent_few<2, 2>), grid, dim3(256), 0, s, w, a.ld_w, h, a.ld_h, a.D, o);
    else hipLaunchKernelGGL((k_xent_few<2, 4>), grid, dim3(256), 0, s, w, a.ld_w, h, a.ld_h, a.D, o);
    return tiles;
}

template <class T, int PL>
hipError_t xent(const XentArgs &a, bool grad, hipStream_t s)
{
    const bool narrow_all = narrow_rows(a.D);
    const Packed pack = packed(a, PL, grad);
    const XentPlan p = fit_xent(a.n, a.V, a.D, PL, pack, grad, a.ws, a.ws_bytes);
    const int64_t piece = p.piece;
    Output o{};
    o.n = a.n;
    o.V = a.V;
    o.D = a.D;
    o.targets = a.targets;
    o.ignore = a.ignore;
    o.part = p.part;
    o.target_logit = p.target_logit;
    o.grad = a.grad_loss;
    o.top_grad = p.top_grad;
    o.h_exp = p.h_exp;
    o.w_exp = p.w_exp;
    o.all_exp = p.all_exp;
    o.d = p.d;
    o.ldd = piece;
    o.plane_d = p.nr * piece;
    const bool few = PL == 2 && a.n <= kFewRows;
    const T *hs = static_cast<const T *>(a.hidden), *ws = static_cast<const T *>(a.weight);
    Operand h{reinterpret_cast<const short *>(hs), a.ld_h, 0, a.n, a.D};
    Operand w{reinterpret_cast<const short *>(ws), a.ld_w, 0, a.V, a.D};
    if (pack.h) h = Operand{p.h, p.Kp, a.n * p.Kp, a.n, p.Kp};
    if (pack.w) w = Operand{p.w, p.Kp, a.V * p.Kp, a.V, p.Kp};
    const int row_blocks = pack.h ? (int)blocks_for(a.n * 64) : 0;
    const int unit_blocks = grad ? 1 : 0; // one block over all rows: begins first
    const int w_blocks = pack.w ? (int)blocks_for(a.V * (p.Kp / 8)) : 0;
    const PackRows<T, PL> rows_job{hs, a.ld_h, a.n, a.D, p.h, p.Kp, a.n * p.Kp, p.h_exp, p.tops,
                                   grad ? a.targets : nullptr, a.ignore, a.V};
    PackWeight<T, PL> w_job{ws, a.ld_w, a.V, a.D, p.w, p.Kp, a.V * p.Kp, p.w_part, 0, p.w_exp};
    const Units units_job{a.grad_loss, a.targets, a.ignore, a.n, a.V, PL == 2 ? p.tops : nullptr, p.top_grad,
                          p.all_exp};
    if constexpr (PL == 2) {
        // the rows and the weight's largest value, then the weight and the units
        int parts = pack.w ? (int)blocks_for(a.V * ((a.D + 7) / 8) / 4 + 1) : 0;
        if (parts > kMaxParts) parts = kMaxParts;
        w_job.parts = parts;
        run_jobs(rows_job, row_blocks, WeightTop{ws, a.ld_w, a.V, a.D, p.w_part}, parts, s);
        run_jobs(units_job, unit_blocks, w_job, w_blocks, s);
    } else {
        typedef Both<Units, PackWeight<T, PL>> First;
        run_jobs(First{units_job, w_job, unit_blocks}, unit_blocks + w_blocks, rows_job, row_blocks, s);
    }
    int64_t tiles;
    if (few && !grad) {
        tiles = few_rows(a, o, s);
    } else if (narrow_all) {
        tiles = narrow_splits(a.n, a.V, narrow_blocks(PL, ROW_STATS, p.Kp));
        narrow<T, PL, ROW_STATS>(h, w, p.Kp, (int)tiles, o, s);
    } else {
        tiles = product<PL, false, false, OUT_STATS>(w, h, a.V, a.n, p.Kp, o, s);
    }
    Join join_job{p.part, tiles, a.n, a.V, a.targets, a.ignore, p.target_logit, a.loss, few && grad ? p.lse : a.lse,
                  reinterpret_cast<int *>(a.ws)};
    if (piece < 0) {
        join_job.rows = p.rows;
        join_job.grad = a.grad_loss;
        join_job.unit = p.top_grad;
        if constexpr (PL == 2) {
            join_job.tops = p.tops;
            join_job.h_exp = p.h_exp;
            join_job.w_exp = p.w_exp;
            join_job.all_exp = p.all_exp;
        }
    }
    const int join_blocks = (int)((a.n + 15) / 16);
    if (!grad) {
        run_jobs(join_job, join_blocks, NoJobOf<1024>(), 0, s);
        return hipGetLastError();
    }
    const ClearRows<PL> clear_job{p.h, p.Kp, a.n * p.Kp, a.n, a.targets, a.ignore, a.V};
    typedef Both<Join, ClearRows<PL>> Stats;
    const Stats stats_job{join_job, clear_job, join_blocks};
    const int stats_blocks = join_blocks + (join_blocks < 1024 ? join_blocks : 1024);
    Operand h_all = h;
    if constexpr (PL == 2) {
        h_all.p = p.h_all;
        const PackCounting count_job{hs, a.ld_h, a.n, a.D, p.h_all, p.Kp, a.n * p.Kp, p.all_exp, a.grad_loss, a.targets,
                                     a.ignore, a.V};
        run_jobs(stats_job, stats_blocks, count_job,
                 piece > 0 ? (int)((blocks_for(a.n * (p.Kp / 8)) + 3) / 4) : 0, s);
    } else {
        run_jobs(stats_job, stats_blocks, NoJobOf<1024>(), 0, s);
    }
    o.lse = join_job.lse;
    if (few) {
        // d takes the lse of its own logits: the errors of the two then cancel
        // where a row is peaked (25 rows against 1437 x 870: gradients 2.3e-6
        // from 64 bits with the lse of the other sums, 3.5e-7 with this one).  What
        // the caller gets is what the call without gradients gives.
        tiles = few_rows(a, o, s);
        const Join out_job{p.part, tiles, a.n, a.V, a.targets, a.ignore, p.target_logit, a.loss, a.lse,
                           reinterpret_cast<int *>(a.ws)};
        run_jobs(out_job, join_blocks, NoJobOf<1024>(), 0, s);
    }
    SumUnit h_unit{p.top_grad}, w_unit{p.top_grad};
    if constexpr (PL == 2) {
        h_unit = SumUnit{nullptr, p.w_exp, a.grad_loss, a.targets, a.ignore, a.V};
        w_unit = SumUnit{nullptr, p.all_exp};
    }
    if (piece < 0) {
        o.rows = p.rows;
        o.sum = p.sum;
        o.splits = p.splits;
        narrow<T, PL, ROW_GRAD>(h, w, p.Kp, p.splits, o, s);
        o.sum = p.w_sum;
        o.splits = p.w_splits;
        o.out = a.dw;
        o.ld_out = a.ld_dw;
        narrow<T, PL, VOC_GRAD>(w, h, p.Kp, p.w_splits, o, s);
        if (p.w_splits > 1)
            sum_up<T>(p.w_sum, p.w_splits, a.V, a.D, w_unit, a.dw, a.ld_dw, s);
        sum_up<T>(p.sum, p.splits, a.n, a.D, h_unit, a.dh, a.ld_dh, s);
        return hipGetLastError();
    }
    for (int64_t v0 = 0; v0 < a.V; v0 += piece) {
        const int64_t here = a.V - v0 < piece ? a.V - v0 : piece, cols = up(here, kRound);
        Operand wp = w;
        wp.p += v0 * w.ld;
        wp.rows = here;
        o.v0 = v0;
        o.first = v0 == 0;
        // d in whole tiles: what lies past the rows and the vocabulary is written as zeros
        product<PL, false, false, OUT_D>(wp, h, cols, p.nr, p.Kp, o, s);
        const Operand d{p.d, piece, p.nr * piece, p.nr, cols};
        o.sum = p.sum;
        o.sum_rows = a.n;
        const SumParts over_v = sum_parts(here, p.parts);
        o.splits = over_v.parts;
        o.split_k = over_v.each;
        product<PL, true, false, OUT_SUM>(wp, d, a.D, a.n, up(here, kPadK), o, s);
        const int64_t rows = up(a.n, kPadK);
        if (p.w_splits == 1) {
            o.out = a.dw;
            o.ld_out = a.ld_dw;
            product<PL, true, true, OUT_WEIGHT>(h_all, d, a.D, here, rows, o, s);
            continue;
        }
        o.sum = p.w_sum;
        o.sum_rows = a.V;
        const SumParts over_n = sum_parts(a.n, p.w_splits);
        o.splits = over_n.parts;
        o.split_k = over_n.each;
        product<PL, true, true, OUT_SUM>(h_all, d, a.D, a.V, rows, o, s);
        sum_up<T>(p.w_sum, over_n.parts, a.V, a.D, w_unit, a.dw, a.ld_dw, s);
    }
    sum_up<T>(p.sum, p.parts, a.n, a.D, h_unit, a.dh, a.ld_dh, s);
    return hipGetLastError();
}

} // namespace

static void workspace_of(int64_t n, int64_t V, int64_t D, int PL, Packed pack, bool grad, size_t *best, size_t *least)
{
    const int64_t most = grad ? best_piece(n, V, D, PL) : 0;
    if (best) *best = plan_xent(n, V, D, PL, pack, most, nullptr).bytes;
    if (least) *least = plan_xent(n, V, D, PL, pack, most < 0 ? -1 : most > 0 ? kRound : 0, nullptr).bytes;
}

void xent_workspace(int64_t n, int64_t V, int64_t D, int dtype, int what, size_t *best, size_t *least)
{
    const int PL = dtype == TT_EMB_DTYPE_FLOAT ? 2 : 1;
    const bool grad = what & TT_EMB_XENT_GRAD, fits = (what & TT_EMB_XENT_ALIGNED) && fits_in_place(PL, D);
    if (n < 1) n = 1; // no rows: the least workspace
    workspace_of(n, V, D, PL, packed(n, PL, grad, fits, fits), grad, best, least);
}

size_t xent_least(const XentArgs &a, int dtype, bool grad)
{
    const int PL = dtype == TT_EMB_DTYPE_FLOAT ? 2 : 1;
    size_t least = 0;
    workspace_of(a.n < 1 ? 1 : a.n, a.V, a.D, PL, packed(a, PL, grad), grad, nullptr, &least);
    return least;
}

int64_t xent_parts(int64_t n, int64_t V, int64_t D, int dtype, int what, size_t ws_bytes, tt_emb_xent_part *parts,
                   int64_t cap, int32_t *slots)
{
    const int PL = dtype == TT_EMB_DTYPE_FLOAT ? 2 : 1;
    const bool fits = (what & TT_EMB_XENT_ALIGNED) && fits_in_place(PL, D);
    const XentPlan p = fit_xent(n, V, D, PL, packed(n, PL, true, fits, fits), true, nullptr, ws_bytes);
    int64_t count = 0;
    auto add = [&](int64_t begin, int64_t end, int slot, bool first) {
        if (count < cap) parts[count] = tt_emb_xent_part{begin, end, slot, first};
        ++count;
    };
    if (p.piece < 0) { // narrow rows: whole steps of the streamed vocabulary
        const int64_t steps = (V + kNarrowStep - 1) / kNarrowStep, per = (steps + p.splits - 1) / p.splits;
        for (int q = 0; q < p.splits; ++q) {
            const int64_t end = (q + 1) * per * kNarrowStep;
            add(q * per * kNarrowStep, end < V ? end : V, q, true);
        }
        *slots = p.splits;
        return count;
    }
    for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
        const int64_t here = V - v0 < p.piece ? V - v0 : p.piece;
        const SumParts over_v = sum_parts(here, p.parts);
        for (int q = 0; q < over_v.parts; ++q) {
            const int64_t end = (q + 1) * over_v.each;
            add(v0 + q * over_v.each, v0 + (end < here ? end : here), q, v0 == 0);
        }
    }
    *slots = p.parts;
    return count;
}

hipError_t launch_xent_forward(const XentArgs &a, int dtype, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    return dtype == TT_EMB_DTYPE_FLOAT ? xent<float, 2>(a, false, s) : xent<bf16, 1>(a, false, s);
}

hipError_t launch_xent_loss_grad(const XentArgs &a, int dtype, hipStream_t s)
{
    if (a.n == 0) { // no rows: the weight's gradient is zero
        const unsigned blocks = (unsigned)(a.V * a.D / 256 < 4096 ? a.V * a.D / 256 + 1 : 4096);
        if (dtype == TT_EMB_DTYPE_FLOAT)
            hipLaunchKernelGGL(k_xent_clear<float>, dim3(blocks), dim3(256), 0, s, static_cast<float *>(a.dw), a.ld_dw,
                               a.V, a.D);
        else
            hipLaunchKernelGGL(k_xent_clear<bf16>, dim3(blocks), dim3(256), 0, s, static_cast<bf16 *>(a.dw), a.ld_dw,
                               a.V, a.D);
        return hipGetLastError();
    }
    return dtype == TT_EMB_DTYPE_FLOAT ? xent<float, 2>(a, true, s) : xent<bf16, 1>(a, true, s);
}

} // namespace ttemb
