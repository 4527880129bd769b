// norm.hip -- layer norm over the last axis, forward and backward (gfx950).
//
// One row belongs to TPR neighbouring threads, each of which holds NV vectors
// of 16 bytes of it in registers, so a row is read once: the mean, then the
// sum of the centred values and of their squares (a second pass over
// registers, not the difference of two large sums), then the output.  Blocks
// walk over rows and keep gamma, beta and the column sums of the backward in
// registers across them.
//
// Memory bounds it: 16384 rows of 4096 bf16 in 49 us forward (268 MB, 5.5 TB/s)
// and 87 backward (403 MB), 32768 rows of 128 fp32 in 10 and 15 us; 4 rows cost a
// launch, 4 us.
#include "lm.h"
#include "primitives.h"

namespace ttemb {

namespace {

constexpr int kNormBlocks = 5 * kCUs;      // forward: blocks at most, all of them resident
// Backward: rows of partial column sums, at most.  Two blocks on each compute
// unit where a block holds one row (16384 x 4096 bf16: 84 us, 95 with four),
// four where it holds several (32768 x 128 fp32: 10.6 us, 11.5 with two).
constexpr int kNormGradBlocks = 4 * kCUs;
template <int TPR>
constexpr int norm_grad_blocks() { return TPR >= 256 ? 2 * kCUs : kNormGradBlocks; }

template <int TPR>
struct NormShape {
    static constexpr int threads = TPR > 256 ? TPR : 256;
    static constexpr int rows = threads / TPR; // rows a block holds at a time
};

// Sum over the TPR threads of a row of K values each.  TPR <= 64: shuffles
// inside the wave.  Larger rows own the block: wave sums meet in LDS, in one
// of two slots in turn, so one barrier per reduction is enough.
template <int TPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*sm)[16][2], int &slot)
{
    constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], o, 64);
    if constexpr (TPR > 64) {
        constexpr int NW = TPR / 64;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) sm[slot][threadIdx.x >> 6][k] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) s += sm[slot][w][k];
            v[k] = s;
        }
        slot ^= 1;
    }
}

// The next row is on its way while this one is reduced.
template <class T, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__(NormShape<TPR>::threads) void k_norm_fwd(NormArgs a)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    __shared__ float sm[2][16][2];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int D = (int)a.D;
    const int64_t step = (int64_t)gridDim.x * NormShape<TPR>::rows, last = a.n - 1;
    int64_t r0 = (int64_t)blockIdx.x * NormShape<TPR>::rows;
    typename VecOf<T, VEC>::raw next[NV];
    auto load = [&](int64_t row) {
        const T *x = static_cast<const T *>(a.x) + (row < a.n ? row : last) * a.ld_x;
#pragma unroll
        for (int j = 0; j < NV; ++j) next[j] = load_row<T, VEC, WHOLE>(x, (t + j * TPR) * VEC, D);
    };
    load(r0 + sub);
    float gam[NV][VEC], bet[NV][VEC];
    int left[NV]; // elements of each vector that exist
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (t + j * TPR) * VEC;
        left[j] = D - c;
        load_params<VEC, WHOLE>(a.gamma, a.param_dtype, c, D, 1.f, gam[j]);
        load_params<VEC, WHOLE>(a.beta, a.param_dtype, c, D, 0.f, bet[j]);
    }
    int slot = 0;
    for (; r0 < a.n; r0 += step) {
        const int64_t r = r0 + sub;
        float v[NV][VEC];
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[j][i] = (float)next[j][i];
                s[0] += v[j][i];
            }
        load(r + step);
        row_sum<TPR, 1>(s, sm, slot);
        // a division, so that a row of equal values has their exact mean
        const float mean0 = s[0] / (float)D;
        float q[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[j][i] = i < left[j] ? v[j][i] - mean0 : 0.f;
                q[0] += v[j][i];
                q[1] = fmaf(v[j][i], v[j][i], q[1]);
            }
        row_sum<TPR, 2>(q, sm, slot);
        // what the first mean's rounding left: it matters where a row's
        // offset is large beside its spread
        const float slip = q[0] / (float)D, mean = slip == slip ? mean0 + slip : mean0; // (an infinite mean has none)
        const float var = fmaf(-slip, slip, q[1] / (float)D);
        const float rstd = 1.f / sqrtf((var < 0.f ? 0.f : var) + a.eps); // (a maximum would pass NaN over)
        if (r >= a.n) continue;
        T *y = static_cast<T *>(a.y) + r * a.ld_y;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = fmaf((v[j][i] - slip) * rstd, gam[j][i], bet[j][i]);
            store_part<T, VEC>(y + (t + j * TPR) * VEC, left[j], o);
        }
        if (t == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// Gradients of a block's rows; the block's sums over its rows of dy xhat and
// dy go to part[0][block][D] and part[1][block][D].
template <class T, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__(NormShape<TPR>::threads) void k_norm_bwd(NormArgs a, float *part)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    // sixteen waves have 128 registers each: with 16 elements per thread
    // nothing is loaded ahead and the column sums live in LDS
    constexpr bool LEAN = TPR == 1024 && NV * VEC == 16;
    __shared__ float col_sums[LEAN ? 2 * NV * VEC : 1][LEAN ? 1024 : 1];
    __shared__ float sm[2][16][2];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int D = (int)a.D;
    const float invD = 1.f / (float)D;
    const int64_t step = (int64_t)gridDim.x * NormShape<TPR>::rows, last = a.n - 1;
    int64_t r0 = (int64_t)blockIdx.x * NormShape<TPR>::rows;
    typename VecOf<T, VEC>::raw nx[NV], ng[NV];
    float nmean, nrstd;
    auto load = [&](int64_t row) {
        const int64_t r = row < a.n ? row : last;
        const T *x = static_cast<const T *>(a.x) + r * a.ld_x, *dy = static_cast<const T *>(a.dy) + r * a.ld_dy;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            nx[j] = load_row<T, VEC, WHOLE>(x, (t + j * TPR) * VEC, D);
            ng[j] = load_row<T, VEC, WHOLE>(dy, (t + j * TPR) * VEC, D);
        }
        nmean = a.mean[r];
        nrstd = a.rstd[r];
    };
    if constexpr (!LEAN) load(r0 + sub);
    float gam[NV][VEC], sg[NV][VEC], sb[NV][VEC];
    int left[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (t + j * TPR) * VEC;
        left[j] = D - c;
        load_params<VEC, WHOLE>(a.gamma, a.param_dtype, c, D, 1.f, gam[j]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if constexpr (LEAN) {
                col_sums[2 * (j * VEC + i)][threadIdx.x] = 0.f;
                col_sums[2 * (j * VEC + i) + 1][threadIdx.x] = 0.f;
            } else {
                sg[j][i] = sb[j][i] = 0.f;
            }
        }
    }
    int slot = 0;
    for (; r0 < a.n; r0 += step) {
        const int64_t r = r0 + sub;
        const bool live = r < a.n;
        if constexpr (LEAN) load(r);
        const float mean = nmean, rstd = nrstd;
        float xh[NV][VEC], g[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                xh[j][i] = (float)nx[j][i];
                g[j][i] = (float)ng[j][i];
            }
        if constexpr (!LEAN) load(r + step);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                xh[j][i] = (xh[j][i] - mean) * rstd;
                if constexpr (LEAN) {
                    if (i < left[j]) {
                        float *c = &col_sums[2 * (j * VEC + i)][threadIdx.x];
                        c[0] = fmaf(g[j][i], xh[j][i], c[0]);
                        c[1024] += g[j][i];
                    }
                } else if (live && i < left[j]) {
                    sg[j][i] = fmaf(g[j][i], xh[j][i], sg[j][i]);
                    sb[j][i] += g[j][i];
                }
                g[j][i] *= gam[j][i]; // 0 past the row's end
                s[0] += g[j][i];
                s[1] = fmaf(g[j][i], xh[j][i], s[1]);
            }
        row_sum<TPR, 2>(s, sm, slot);
        if (!live) continue;
        const float ma = s[0] * invD, mx = s[1] * invD;
        T *dx = static_cast<T *>(a.y) + r * a.ld_y;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = (g[j][i] - ma - xh[j][i] * mx) * rstd;
            store_part<T, VEC>(dx + (t + j * TPR) * VEC, left[j], o);
        }
    }
    if (!part) return;
    if constexpr (LEAN) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                sg[j][i] = col_sums[2 * (j * VEC + i)][threadIdx.x];
                sb[j][i] = col_sums[2 * (j * VEC + i) + 1][threadIdx.x];
            }
    }
    // the block's sums: sub-rows of one wave by shuffles, the waves through LDS
    if constexpr (NormShape<TPR>::rows > 1) {
        constexpr int W = TPR < 64 ? TPR : 64, COLS = TPR * NV * VEC, WAVES = NormShape<TPR>::threads / 64;
        __shared__ float col[2][WAVES][COLS];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
#pragma unroll
                for (int o = W; o < 64; o <<= 1) {
                    sg[j][i] += __shfl_xor(sg[j][i], o, 64);
                    sb[j][i] += __shfl_xor(sb[j][i], o, 64);
                }
                if ((threadIdx.x & 63) < W) {
                    col[0][threadIdx.x >> 6][(t + j * TPR) * VEC + i] = sg[j][i];
                    col[1][threadIdx.x >> 6][(t + j * TPR) * VEC + i] = sb[j][i];
                }
            }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * D; c += NormShape<TPR>::threads) {
            const int which = c >= D, cc = which ? c - D : c;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) s += col[which][w][cc];
            part[((int64_t)which * gridDim.x + blockIdx.x) * D + cc] = s;
        }
    } else {
        float *pg = part + (int64_t)blockIdx.x * D, *pb = part + ((int64_t)gridDim.x + blockIdx.x) * D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            store_part<float, VEC>(pg + (t + j * TPR) * VEC, left[j], sg[j]);
            store_part<float, VEC>(pb + (t + j * TPR) * VEC, left[j], sb[j]);
        }
    }
}

// Column sums of the blocks' partials: 64 columns per block, four per lane, 64
// groups of rows; the four groups of a wave meet in shuffles, the waves in LDS,
// always in the same order.
template <bool WHOLE>
__global__ __launch_bounds__(1024) void k_norm_cols(const float *part, int blocks, int D, void *dgamma, void *dbeta,
                                                    int param_dtype)
{
    __shared__ float sm[16][64];
    const int lane = threadIdx.x & 15, grp = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane * 4;
    const float *p = part + (int64_t)blockIdx.y * blocks * D;
    void *dst = blockIdx.y ? dbeta : dgamma;
    if (!dst) return;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int b = grp; b < blocks; b += 64) {
        const VecOf<float, 4>::raw v = load_row<float, 4, WHOLE>(p + (int64_t)b * D, c, D);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s[i] += __shfl_xor(s[i], 16, 64);
        s[i] += __shfl_xor(s[i], 32, 64);
        if ((threadIdx.x & 63) < 16) sm[wave][lane * 4 + i] = s[i];
    }
    __syncthreads();
    const int col = blockIdx.x * 64 + threadIdx.x;
    if (threadIdx.x < 64 && col < D) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 16; ++w) t += sm[w][threadIdx.x];
        store_param(dst, param_dtype, col, t);
    }
}

// Threads per row and vectors per thread: the fewest threads that hold a row
// of nv vectors with at most 16 elements each (80 registers in the backward).
template <class T, class F>
hipError_t norm_shape(int64_t D, F &&g)
{
    auto f = [&](auto tpr, auto nv) {
        if (D % (16 / (int)sizeof(T)) == 0) return g(tpr, nv, std::true_type());
        return g(tpr, nv, std::false_type());
    };
    constexpr int VEC = 16 / (int)sizeof(T), MAX = 16 / VEC;
    const int64_t nv = (D + VEC - 1) / VEC;
    auto one = [&](auto tpr) {
        constexpr int TPR = decltype(tpr)::value;
        if constexpr (MAX == 4) {
            if (nv > 2 * TPR) return f(tpr, std::integral_constant<int, 4>());
        }
        if (nv > TPR) return f(tpr, std::integral_constant<int, 2>());
        return f(tpr, std::integral_constant<int, 1>());
    };
    if (nv <= 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
    if (nv <= 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
    if (nv <= 64 * MAX) return one(std::integral_constant<int, 64>());
    if (nv <= 256 * MAX) return one(std::integral_constant<int, 256>());
    return one(std::integral_constant<int, 1024>());
}

template <class T>
hipError_t norm_forward(const NormArgs &a, hipStream_t s)
{
    return norm_shape<T>(a.D, [&](auto tpr, auto nv, auto whole) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        const int64_t need = (a.n + NormShape<TPR>::rows - 1) / NormShape<TPR>::rows;
        const int grid = (int)(need < kNormBlocks ? need : kNormBlocks);
        hipLaunchKernelGGL((k_norm_fwd<T, TPR, NV, decltype(whole)::value>), dim3(grid),
                           dim3(NormShape<TPR>::threads), 0, s, a);
        return hipGetLastError();
    });
}

template <class T>
hipError_t norm_backward(const NormArgs &a, hipStream_t s)
{
    return norm_shape<T>(a.D, [&](auto tpr, auto nv, auto whole) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        const int64_t need = (a.n + NormShape<TPR>::rows - 1) / NormShape<TPR>::rows;
        const int grid = (int)(need < norm_grad_blocks<TPR>() ? need : norm_grad_blocks<TPR>());
        float *part = (a.dgamma || a.dbeta) ? reinterpret_cast<float *>(a.ws + TT_EMB_STATUS_BYTES) : nullptr;
        hipLaunchKernelGGL((k_norm_bwd<T, TPR, NV, decltype(whole)::value>), dim3(grid),
                           dim3(NormShape<TPR>::threads), 0, s, a, part);
        if (part) {
            const dim3 cols((unsigned)((a.D + 63) / 64), 2);
            if (a.D % 4 == 0)
                hipLaunchKernelGGL(k_norm_cols<true>, cols, dim3(1024), 0, s, part, grid, (int)a.D, a.dgamma, a.dbeta,
                                   a.param_dtype);
            else
                hipLaunchKernelGGL(k_norm_cols<false>, cols, dim3(1024), 0, s, part, grid, (int)a.D, a.dgamma, a.dbeta,
                                   a.param_dtype);
        }
        return hipGetLastError();
    });
}

// No rows: the sums over them are zero.
__global__ __launch_bounds__(256) void k_norm_zero(void *dgamma, void *dbeta, int D, int param_dtype)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= D) return;
    if (dgamma) store_param(dgamma, param_dtype, c, 0.f);
    if (dbeta) store_param(dbeta, param_dtype, c, 0.f);
}

} // namespace

size_t norm_workspace(int64_t n, int64_t D)
{
    const int64_t blocks = n < kNormGradBlocks ? n : kNormGradBlocks;
    return TT_EMB_STATUS_BYTES + round256((size_t)(2 * blocks * D) * sizeof(float));
}

hipError_t launch_norm_forward(const NormArgs &a, int dtype, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    if (dtype == TT_EMB_DTYPE_FLOAT) return norm_forward<float>(a, s);
    if (dtype == TT_EMB_DTYPE_BFLOAT) return norm_forward<bf16>(a, s);
    return norm_forward<f16>(a, s);
}

hipError_t launch_norm_backward(const NormArgs &a, int dtype, hipStream_t s)
{
    if (a.n == 0) {
        if (!a.dgamma && !a.dbeta) return hipSuccess;
        hipLaunchKernelGGL(k_norm_zero, dim3((unsigned)((a.D + 255) / 256)), dim3(256), 0, s, a.dgamma, a.dbeta,
                           (int)a.D, a.param_dtype);
        return hipGetLastError();
    }
    if (dtype == TT_EMB_DTYPE_FLOAT) return norm_backward<float>(a, s);
    if (dtype == TT_EMB_DTYPE_BFLOAT) return norm_backward<bf16>(a, s);
    return norm_backward<f16>(a, s);
}

} // namespace ttemb
