// blocknorm.hip -- what stands between two blocks of a model (gfx950): the norm
// of a block's output, its gate and scale, the residual sum, and the norm before
// the next block.
//
//   u = N(x) gp + bp  (or x),  h = a r + b gate u,  y = N(h) g + beta
//
// with N the layer norm or the division by the root of the mean square.  Rows of
// up to 4096 values are held in registers: x and r are read once and y and h
// written once, and the second norm works on h before it is rounded.  Longer
// rows are read again, from the caches, for each of the norms' sums.
//
// Memory bounds it: 16384 x 4096 bf16 in 115 us (4.7 TB/s), 32768 x 128 fp32 in
// 14.8 (4.5 TB/s), 3001 x 1001 fp16 beside an fp32 residual and a gate per row in
// 16.8.  Each thread has the next row's loads in flight while it reduces one; two
// rows ahead cost a wave in four and 152 us for the first of these.
#include "blocknorm.h"

namespace ttemb {

namespace {

constexpr int kBlockBlocks = 5 * kCUs; // blocks at most

// v normalised in place; its elements past the row's end are zero and stay so.
template <int TPR>
__device__ __forceinline__ void normalise(float (&v)[kBlockVec], int left, bool layer, int D, float eps,
                                          float (*sm)[16][2], int &slot, float &mean, float &rstd)
{
    float q[2] = {0.f, 0.f}, slip = 0.f;
    mean = 0.f;
    if (layer) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < kBlockVec; ++i) s[0] += v[i];
        row_sum<TPR, 1>(s, sm, slot);
        mean = s[0] / (float)D; // a division, so that a row of equal values has their exact mean
#pragma unroll
        for (int i = 0; i < kBlockVec; ++i) v[i] = i < left ? v[i] - mean : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kBlockVec; ++i) {
        q[0] += v[i];
        q[1] = fmaf(v[i], v[i], q[1]);
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
    for (int i = 0; i < kBlockVec; ++i) v[i] = i < left ? (v[i] - slip) * rstd : 0.f;
}

template <class T, class R, int TPR, bool WHOLE>
__global__ __launch_bounds__(NormShape<TPR>::threads) void k_block_fwd(BlockNormArgs a)
{
    constexpr int VEC = kBlockVec;
    __shared__ float sm[2][16][2];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, c = t * VEC;
    const int D = (int)a.D, left = D - c; // elements of the vector that exist
    const int64_t step = (int64_t)gridDim.x * NormShape<TPR>::rows, last = a.n - 1;
    int64_t r0 = (int64_t)blockIdx.x * NormShape<TPR>::rows;
    struct Row {
        typename VecOf<T, VEC>::raw x, gate;
        typename VecOf<R, VEC>::raw res;
    };
    auto load = [&](int64_t row, Row &to) {
        const int64_t r = row < a.n ? row : last;
        to.x = load_cols<T, WHOLE>(static_cast<const T *>(a.x) + r * a.ld_x, c, D);
        to.res = load_cols<R, WHOLE>(static_cast<const R *>(a.residual) + r * a.ld_r, c, D);
        if (a.gate_rows) to.gate = load_cols<T, WHOLE>(static_cast<const T *>(a.gate) + r * a.ld_gate, c, D);
    };
    Row row;
    load(r0 + sub, row);
    float gam[VEC], bet[VEC], pgam[VEC], pbet[VEC], gate[VEC];
    load_params<VEC, WHOLE>(a.gamma, a.param_dtype, c, D, 1.f, gam);
    load_params<VEC, WHOLE>(a.beta, a.param_dtype, c, D, 0.f, bet);
    load_params<VEC, WHOLE>(a.post_gamma, a.param_dtype, c, D, 1.f, pgam);
    load_params<VEC, WHOLE>(a.post_beta, a.param_dtype, c, D, 0.f, pbet);
    load_params<VEC, WHOLE>(a.gate_rows ? nullptr : a.gate, a.param_dtype, c, D, 1.f, gate);
    int slot = 0;
    for (; r0 < a.n; r0 += step) {
        const int64_t r = r0 + sub;
        float v[VEC], res[VEC], w[VEC];
        values<T, WHOLE>(row.x, left, D, v);
        values<R, WHOLE>(row.res, left, D, res);
        if (a.gate_rows) values<T, WHOLE>(row.gate, left, D, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = a.scale_block * (a.gate_rows ? w[i] : gate[i]);
        load(r + step, row); // the next row is on its way while this one is reduced
        float pmean = 0.f, prstd = 1.f, mean, rstd;
        if (a.post) normalise<TPR>(v, left, a.layer, D, a.eps, sm, slot, pmean, prstd);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float u = a.post ? fmaf(v[i], pgam[i], pbet[i]) : v[i];
            v[i] = fmaf(w[i], u, a.scale_residual * res[i]);
        }
        if (r < a.n) store_part<R, VEC>(static_cast<R *>(a.h) + r * a.ld_h + c, left, v);
        normalise<TPR>(v, left, a.layer, D, a.eps, sm, slot, mean, rstd);
        if (r >= a.n) continue;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = fmaf(v[i], gam[i], bet[i]);
        store_part<T, VEC>(static_cast<T *>(a.y) + r * a.ld_y + c, left, v);
        if (t == 0 && a.stats) store_part<float, 4>(a.stats + r * 4, 4, {pmean, prstd, mean, rstd});
    }
}

// Rows of more than 4096 values: a block's threads go over the row once for
// each sum that the next step needs.
template <class T, class R, bool WHOLE>
__global__ __launch_bounds__(kBlockLong) void k_block_fwd_long(BlockNormArgs a)
{
    constexpr int VEC = kBlockVec;
    __shared__ float sm[2][16][2];
    const int D = (int)a.D;
    int slot = 0;
    for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + r * a.ld_x, *g = static_cast<const T *>(a.gate) + r * a.ld_gate;
        const R *res = static_cast<const R *>(a.residual) + r * a.ld_r;
        auto each = [&](auto f) {
#pragma clang loop unroll(disable)
            for (int c = threadIdx.x * VEC; c < D; c += kBlockLong * VEC) f(c, D - c);
        };
        auto take_x = [&](int c, int left, float(&v)[VEC]) {
            values<T, WHOLE>(load_cols<T, WHOLE>(x, c, D), left, D, v);
        };
        // mean and rstd of what take(c, left, v) gives
        auto stats = [&](auto take, float &mean, float &rstd) {
            mean = 0.f;
            if (a.layer) {
                float s[1] = {0.f};
                each([&](int c, int left) {
                    float v[VEC];
                    take(c, left, v);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) s[0] += v[i];
                });
                row_sum<kBlockLong, 1>(s, sm, slot);
                mean = s[0] / (float)D;
            }
            float q[2] = {0.f, 0.f};
            each([&](int c, int left) {
                float v[VEC];
                take(c, left, v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = i < left ? v[i] - mean : 0.f;
                    q[0] += d;
                    q[1] = fmaf(d, d, q[1]);
                }
            });
            row_sum<kBlockLong, 2>(q, sm, slot);
            float var = q[1] / (float)D;
            if (a.layer) {
                const float slip = q[0] / (float)D;
                if (slip == slip) mean += slip;
                var = fmaf(-slip, slip, var);
            }
            rstd = 1.f / sqrtf((var < 0.f ? 0.f : var) + a.eps);
        };
        float pmean = 0.f, prstd = 1.f, mean, rstd;
        if (a.post) stats(take_x, pmean, prstd);
        auto take_h = [&](int c, int left, float(&v)[VEC]) {
            float re[VEC], w[VEC], pg[VEC], pb[VEC];
            take_x(c, left, v);
            values<R, WHOLE>(load_cols<R, WHOLE>(res, c, D), left, D, re);
            if (a.gate_rows) values<T, WHOLE>(load_cols<T, WHOLE>(g, c, D), left, D, w);
            else load_params<VEC, WHOLE>(a.gate, a.param_dtype, c, D, 1.f, w);
            load_params<VEC, WHOLE>(a.post_gamma, a.param_dtype, c, D, 1.f, pg);
            load_params<VEC, WHOLE>(a.post_beta, a.param_dtype, c, D, 0.f, pb);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float u = a.post ? fmaf((v[i] - pmean) * prstd, pg[i], pb[i]) : v[i];
                v[i] = i < left ? fmaf(a.scale_block * w[i], u, a.scale_residual * re[i]) : 0.f;
            }
        };
        stats(take_h, mean, rstd);
        // (h may be the residual and y may be x: every thread writes where it alone has read)
        each([&](int c, int left) {
            float v[VEC], gam[VEC], bet[VEC];
            take_h(c, left, v);
            load_params<VEC, WHOLE>(a.gamma, a.param_dtype, c, D, 1.f, gam);
            load_params<VEC, WHOLE>(a.beta, a.param_dtype, c, D, 0.f, bet);
            store_part<R, VEC>(static_cast<R *>(a.h) + r * a.ld_h + c, left, v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = fmaf((v[i] - mean) * rstd, gam[i], bet[i]);
            store_part<T, VEC>(static_cast<T *>(a.y) + r * a.ld_y + c, left, v);
        });
        if (threadIdx.x == 0 && a.stats) store_part<float, 4>(a.stats + r * 4, 4, {pmean, prstd, mean, rstd});
    }
}

template <class T, class R>
hipError_t block_forward(const BlockNormArgs &a, hipStream_t s)
{
    if (a.D > kBlockRegs) {
        const dim3 grid(block_grid(a.n, 4 * kCUs));
        if (a.D % kBlockVec == 0)
            hipLaunchKernelGGL((k_block_fwd_long<T, R, true>), grid, dim3(kBlockLong), 0, s, a);
        else
            hipLaunchKernelGGL((k_block_fwd_long<T, R, false>), grid, dim3(kBlockLong), 0, s, a);
        return hipGetLastError();
    }
    return block_shape(a.D, [&](auto tpr, auto whole) {
        constexpr int TPR = decltype(tpr)::value;
        const int64_t need = (a.n + NormShape<TPR>::rows - 1) / NormShape<TPR>::rows;
        hipLaunchKernelGGL((k_block_fwd<T, R, TPR, decltype(whole)::value>), dim3(block_grid(need, kBlockBlocks)),
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
