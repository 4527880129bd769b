// norm.h -- what the row norms share: the threads of a row and their sums, the
// column sums of the backward passes.
#pragma once

#include "lm.h"

namespace ttemb {

namespace {

template <int TPR>
struct NormShape {
    static constexpr int threads = TPR > 256 ? TPR : 256;
    static constexpr int rows = threads / TPR; // rows a block holds at a time
};

// Sum over the TPR threads of a row of K values each.  TPR <= 64: shuffles
// inside the wave.  Larger rows: the sums of a row's waves meet in LDS, in one of
// two slots in turn, so one barrier per reduction is enough.
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
        const int first = NormShape<TPR>::rows > 1 ? (threadIdx.x >> 6) / NW * NW : 0; // the row's first wave
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) s += sm[slot][first + w][k];
            v[k] = s;
        }
        slot ^= 1;
    }
}

// Where the column sums go; none where it is null.
struct ColumnSums {
    void *dst[5];
    int dtype[5];
};

// Column sums of the blocks' partials, rows of `ld`: 64 columns per block, four per lane, 64
// groups of rows; the four groups of a wave meet in shuffles, the waves in LDS,
// always in the same order.
template <bool WHOLE>
__global__ __launch_bounds__(1024) void k_norm_cols(const float *part, int blocks, int D, int ld, ColumnSums out)
{
    __shared__ float sm[16][64];
    const int lane = threadIdx.x & 15, grp = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane * 4;
    const float *p = part + (int64_t)blockIdx.y * blocks * ld;
    void *dst = out.dst[blockIdx.y];
    if (!dst) return;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int b = grp; b < blocks; b += 64) {
        const VecOf<float, 4>::raw v = load_row<float, 4, WHOLE>(p + (int64_t)b * ld, c, ld);
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
        store_param(dst, out.dtype[blockIdx.y], col, t);
    }
}

inline void norm_cols(const float *part, int blocks, int64_t D, int64_t ld, int sums, const ColumnSums &out,
                      hipStream_t s)
{
    const dim3 grid((unsigned)((D + 63) / 64), (unsigned)sums);
    if (ld % 4 == 0) hipLaunchKernelGGL(k_norm_cols<true>, grid, dim3(1024), 0, s, part, blocks, (int)D, (int)ld, out);
    else hipLaunchKernelGGL(k_norm_cols<false>, grid, dim3(1024), 0, s, part, blocks, (int)D, (int)ld, out);
}

} // namespace

} // namespace ttemb
