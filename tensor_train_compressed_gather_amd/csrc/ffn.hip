// ffn.hip -- the gated feed-forward block's forward (gfx950): products by tiles, and
// those of few rows by kernels of their own.
#include "ffn.h"

namespace ttemb {

namespace {

// --------------------------------------------------------------- few rows

// Products of few rows, forward: the weight's bytes bound them, so it is read
// once, as it lies in memory, straight into the registers of the matrix
// instructions (16x16x32, fp32 16x16x4), and rows of any place and length serve.
// A block has 16 rows of the weight (PAIR: 16 of each projection) and 16 NB rows
// of the operand; its waves take chunks of the sum in turn, the next chunk's
// loads in flight while one is multiplied, and meet in LDS.  Lane l holds row l %
// 16 and the l / 16-th 16 bytes of each 64 of a chunk.
//
// TERMS: where a has two terms (two_terms), they are rows i and 8 + i of one operand
// up to 8 rows, and their products meet where the waves' do; with more rows they are
// an operand each.  (4096 x 16384 bf16 with one term and with two: 1 row 72.5 and 72.7 us,
// 8 rows 77 and 83, 16 rows 86 and 101: what the blocks read of a, not the products.)
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
    int64_t second;     // elements from a (out, PAIR; else x) to its second term, 0 for none
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

enum { ONE, ROWS_OF_ONE, TWO }; // terms of the operand

template <class T, bool PAIR, int TERMS, int NB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_ffn_few(FewArgs a)
{
    typedef FewStep<T> Step;
    typedef typename VecOf<T, Step::VEC>::type vec;
    constexpr int MB = PAIR ? 2 : 1, U = NB > 4 ? 2 : 4, CHUNK = U * Step::K, P = 16 * MB + 4;
    constexpr int NX = TERMS == TWO ? 2 * NB : NB;
    constexpr bool ROWS = TERMS == ROWS_OF_ONE;
    __shared__ __align__(16) float red[WAVES][16 * NB][P];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m0 = (int64_t)blockIdx.x * 16, k0 = blockIdx.y * a.split_k;
    const int64_t K = a.K - k0 < a.split_k ? a.K - k0 : a.split_k;
    const int at = (lane >> 4) * Step::VEC;
    const T *w[MB], *x[NX];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int64_t r = m0 + (lane & 15);
        w[b] = static_cast<const T *>(a.w) + ((r < a.rows ? r : a.rows - 1) + b * a.rows) * a.ld_w + k0 + at;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t r = b * 16 + (lane & (ROWS ? 7 : 15));
        x[b] = static_cast<const T *>(a.x) + (r < a.n ? r : a.n - 1) * a.ld_x + k0 + at;
        if constexpr (ROWS) x[b] += lane & 8 ? a.second : 0;
        if constexpr (TERMS == TWO) x[NB + b] = x[b] + a.second;
    }
    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    struct Regs {
        typename Step::raw w[MB][U], x[NX][U];
    };
    auto load = [&](int64_t k, Regs &r) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int b = 0; b < MB; ++b) r.w[b][u] = *reinterpret_cast<const vec *>(w[b] + k + u * Step::K);
#pragma unroll
            for (int b = 0; b < NX; ++b) r.x[b][u] = *reinterpret_cast<const vec *>(x[b] + k + u * Step::K);
        }
    };
    auto mma = [&](const Regs &r) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NX; ++j) acc[i][j % NB] = Step::mma(r.w[i][u], r.x[j][u], acc[i][j % NB]);
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
            typename Step::raw p[MB], q[NX];
            auto part = [&](const T *row) {
                typename Step::raw v;
#pragma unroll
                for (int e = 0; e < Step::VEC; ++e) v[e] = e < left ? row[k + e] : (T)0.f;
                return v;
            };
#pragma unroll
            for (int b = 0; b < MB; ++b) p[b] = part(w[b]);
#pragma unroll
            for (int b = 0; b < NX; ++b) q[b] = part(x[b]);
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NX; ++j) acc[i][j % NB] = Step::mma(p[i], q[j], acc[i][j % NB]);
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
                if constexpr (ROWS) {
                    load_vec<float, 8>(&red[s][8 + i][b * 16 + (e & 1) * 8], y);
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[b][q] += y[q];
                }
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
            if (sizeof(T) == 2 && a.second)
                store_terms<T, 2>(static_cast<short *>(a.out) + i * a.ld_out + m, a.second, left, value);
            else store_part<T, 8>(static_cast<T *>(a.out) + i * a.ld_out + m, left, value);
        } else if (a.sum) {
            store_part<float, 8>(a.sum + (blockIdx.y * a.n + i) * a.rows + m, left, v[0]);
        } else {
            store_part<T, 8>(static_cast<T *>(a.out) + i * a.ld_out + m, left, v[0]);
        }
    }
}

template <class T, bool PAIR>
void few(const FewArgs &a, int splits, hipStream_t s)
{
    const dim3 grid((unsigned)((a.rows + 15) / 16), (unsigned)splits);
    constexpr std::integral_constant<int, 4> four;
    constexpr std::integral_constant<int, 8> eight;
    const bool idle = (int64_t)grid.x * splits <= 2 * kCUs; // few blocks: more waves in each
    auto launch = [&](auto terms, auto nb, auto waves) {
        constexpr int TERMS = decltype(terms)::value, NB = decltype(nb)::value, WAVES = decltype(waves)::value;
        hipLaunchKernelGGL((k_ffn_few<T, PAIR, TERMS, NB, WAVES>), grid, dim3(64 * WAVES), 0, s, a);
    };
    auto run = [&](auto nb, auto waves) { launch(std::integral_constant<int, ONE>(), nb, waves); };
    if constexpr (sizeof(T) == 4) {
        if (a.n > 64) return run(std::integral_constant<int, 8>(), four);
        if (a.n > 32) return idle ? run(four, eight) : run(four, four);
        constexpr std::integral_constant<int, 2> two;
        if (a.n > 16) return idle ? run(two, eight) : run(two, four);
    }
    constexpr std::integral_constant<int, 1> one;
    if constexpr (sizeof(T) == 2 && !PAIR) {
        constexpr std::integral_constant<int, ROWS_OF_ONE> rows;
        constexpr std::integral_constant<int, TWO> two;
        if (a.second && a.n <= 8) return idle ? launch(rows, one, eight) : launch(rows, one, four);
        if (a.second) return idle ? launch(two, one, eight) : launch(two, one, four);
    }
    return idle ? run(one, eight) : run(one, four);
}

template <class T>
hipError_t ffn_few(const FfnArgs &a, int dtype, hipStream_t s)
{
    const FfnPlan p = plan_ffn(a.n, a.D, a.F, FfnTerms<T>::planes, false, copies_of(a, dtype, false), a.ws);
    FewArgs in{}, out{};
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
    in.second = out.second = p.two_mid ? a.n * p.ldF : 0;
    few<T, true>(in, 1, s);
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
    o.two_mid = p.two_mid;
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
    int shape;
    const FfnSize z = y_size(a.n, a.D, a.F, PL, &shape);
    launch<T, false, false, FFN_OUT, false>(out(w_out, mid, z, shape, a.y, a.ld_y), shape, s);
    out.join(s);
    return hipGetLastError();
}

} // namespace

// what: TT_EMB_FFN_GRAD and TT_EMB_FFN_ALIGNED.
size_t ffn_workspace(int64_t n, int64_t D, int64_t F, int dtype, int what)
{
    const bool fp32 = dtype == TT_EMB_DTYPE_FLOAT, grad = what & TT_EMB_FFN_GRAD, well = what & TT_EMB_FFN_ALIGNED;
    const FfnCopies copies = ffn_copies(fp32, grad, n, D, F, well, well, well, well);
    return plan_ffn(n, D, F, fp32 ? 3 : 1, grad, copies, nullptr).bytes;
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

} // namespace ttemb
