// blocknorm.hip -- what stands between two blocks of a model (gfx950): the norm
// of a block's output, its gate and scale, the residual sum, and the norm before
// the next block.
//
//   u = N(x) gp + bp  (or x),  h = a r + b gate u,  y = N(h) g + beta
//
// with N the layer norm or the division by the root of the mean square.  Rows
// are held in registers as by the layer norm: x and r are read once and y and
// h written once, and the second norm works on h before it is rounded.
#include "blocknorm.h"

namespace ttemb {

namespace {

constexpr int kBlockBlocks = 5 * kCUs; // blocks at most

// v normalised in place; its elements past the row's end are zero and stay so.
template <int TPR, int NV, int VEC>
__device__ __forceinline__ void normalise(float (&v)[NV][VEC], const int (&left)[NV], bool layer, int D, float eps,
                                          float (*sm)[16][2], int &slot, float &mean, float &rstd)
{
    float q[2] = {0.f, 0.f}, slip = 0.f;
    mean = 0.f;
    if (layer) {
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] += v[j][i];
        row_sum<TPR, 1>(s, sm, slot);
        mean = s[0] / (float)D; // a division, so that a row of equal values has their exact mean
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][i] = i < left[j] ? v[j][i] - mean : 0.f;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            q[0] += v[j][i];
            q[1] = fmaf(v[j][i], v[j][i], q[1]);
        }
    row_sum<TPR, 2>(q, sm, slot);
    float var = q[1] / (float)D;
    if (layer) { // what the first mean's rounding left
        slip = q[0] / (float)D;
        if (slip == slip) mean += slip; // (an infinite mean has none)
        var = fmaf(-slip, slip, var);
    }
    rstd = 1.f / sqrtf((var < 0.f ? 0.f : var) + eps); // (a maximum would pass NaN over)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] = i < left[j] ? (v[j][i] - slip) * rstd : 0.f;
}

// Rows of more than 4096 values have 128 registers a thread: parameters are
// then read again for each row (they stay in the caches).
template <class T, class R, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__(NormShape<TPR>::threads) void k_block_fwd(BlockNormArgs a)
{
    constexpr int VEC = kBlockVec;
    constexpr bool LEAN = TPR == 1024;
    __shared__ float sm[2][16][2];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int D = (int)a.D;
    const int64_t step = (int64_t)gridDim.x * NormShape<TPR>::rows, last = a.n - 1;
    int64_t r0 = (int64_t)blockIdx.x * NormShape<TPR>::rows;
    typename VecOf<T, VEC>::raw nx[NV], ng[NV];
    typename VecOf<R, VEC>::raw nr[NV];
    auto load = [&](int64_t row) {
        const int64_t r = row < a.n ? row : last;
        const T *x = static_cast<const T *>(a.x) + r * a.ld_x, *g = static_cast<const T *>(a.gate) + r * a.ld_gate;
        const R *res = static_cast<const R *>(a.residual) + r * a.ld_r;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (t + j * TPR) * VEC;
            nx[j] = load_row<T, VEC, WHOLE>(x, c, D);
            nr[j] = load_row<R, VEC, WHOLE>(res, c, D);
            if (a.gate_rows) ng[j] = load_row<T, VEC, WHOLE>(g, c, D);
        }
    };
    if constexpr (!LEAN) load(r0 + sub);
    constexpr int PV = LEAN ? 1 : NV;
    float gam[PV][VEC], bet[PV][VEC], pgam[PV][VEC], pbet[PV][VEC], gate[PV][VEC];
    auto params = [&](int j, int p) {
        const int64_t c = (t + j * TPR) * VEC;
        load_params<VEC, WHOLE>(a.gamma, a.param_dtype, c, D, 1.f, gam[p]);
        load_params<VEC, WHOLE>(a.beta, a.param_dtype, c, D, 0.f, bet[p]);
    };
    auto post_params = [&](int j, int p) {
        const int64_t c = (t + j * TPR) * VEC;
        load_params<VEC, WHOLE>(a.post_gamma, a.param_dtype, c, D, 1.f, pgam[p]);
        load_params<VEC, WHOLE>(a.post_beta, a.param_dtype, c, D, 0.f, pbet[p]);
        load_params<VEC, WHOLE>(a.gate_rows ? nullptr : a.gate, a.param_dtype, c, D, 1.f, gate[p]);
    };
    int left[NV]; // elements of each vector that exist
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        left[j] = D - (t + j * TPR) * VEC;
        if constexpr (!LEAN) {
            params(j, j);
            post_params(j, j);
        }
    }
    int slot = 0;
    for (; r0 < a.n; r0 += step) {
        const int64_t r = r0 + sub;
        if constexpr (LEAN) load(r);
        float v[NV][VEC], res[NV][VEC], gr[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[j][i] = (float)nx[j][i];
                res[j][i] = (float)nr[j][i];
                gr[j][i] = a.gate_rows ? (float)ng[j][i] : 1.f;
            }
        if constexpr (!LEAN) load(r + step); // the next row is on its way while this one is reduced
        float pmean = 0.f, prstd = 1.f, mean, rstd;
        if (a.post) normalise<TPR>(v, left, a.layer, D, a.eps, sm, slot, pmean, prstd);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (LEAN) {
                __builtin_amdgcn_sched_barrier(0); // one vector's parameters at a time
                post_params(j, 0);
            }
            const int p = LEAN ? 0 : j;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float u = a.post ? fmaf(v[j][i], pgam[p][i], pbet[p][i]) : v[j][i];
                v[j][i] = fmaf(a.scale_block * (gate[p][i] * gr[j][i]), u, a.scale_residual * res[j][i]);
            }
        }
        if (r < a.n) {
            R *h = static_cast<R *>(a.h) + r * a.ld_h;
#pragma unroll
            for (int j = 0; j < NV; ++j) store_part<R, VEC>(h + (t + j * TPR) * VEC, left[j], v[j]);
        }
        normalise<TPR>(v, left, a.layer, D, a.eps, sm, slot, mean, rstd);
        if (r >= a.n) continue;
        T *y = static_cast<T *>(a.y) + r * a.ld_y;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (LEAN) {
                __builtin_amdgcn_sched_barrier(0);
                params(j, 0);
            }
            const int p = LEAN ? 0 : j;
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = fmaf(v[j][i], gam[p][i], bet[p][i]);
            store_part<T, VEC>(y + (t + j * TPR) * VEC, left[j], o);
        }
        if (t == 0 && a.stats) {
            float *st = a.stats + r * 4;
            st[0] = pmean;
            st[1] = prstd;
            st[2] = mean;
            st[3] = rstd;
        }
    }
}

template <class T, class R>
hipError_t block_forward(const BlockNormArgs &a, hipStream_t s)
{
    return block_shape(a.D, [&](auto tpr, auto nv, auto whole) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        const int64_t need = (a.n + NormShape<TPR>::rows - 1) / NormShape<TPR>::rows;
        const int grid = (int)(need < kBlockBlocks ? need : kBlockBlocks);
        hipLaunchKernelGGL((k_block_fwd<T, R, TPR, NV, decltype(whole)::value>), dim3(grid),
                           dim3(NormShape<TPR>::threads), 0, s, a);
        return hipGetLastError();
    });
}

} // namespace

hipError_t launch_block_forward(const BlockNormArgs &a, int dtype, int res_dtype, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    return block_types(dtype, res_dtype, [&](auto t, auto r) { return block_forward<decltype(t), decltype(r)>(a, s); });
}

} // namespace ttemb
