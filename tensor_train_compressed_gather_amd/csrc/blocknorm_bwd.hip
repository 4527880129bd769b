// blocknorm_bwd.hip -- the backward of the norms between two blocks (gfx950).
//
// With u, h and y as in blocknorm.hip, and gy, gh the gradients that arrive at
// y and h:
//
//   dh = gh + rstd (q - mean(q) - hhat mean(q hhat)),  q = gy g,  hhat = N(h)
//   dr = a dh,  du = b gate dh,  dgate = b u dh
//   dx = the same of du gp and N(x);  column sums of gy hhat, gy, du N(x), du, b u dh
//
// (without the means of q where N is the root mean square).  It reads x and r,
// from which it makes h again in fp32: as many bytes as reading h, which a
// caller may then overwrite, and without its rounding.  The column sums of rows
// of up to 4096 values stay in registers across a block's rows.  Longer rows
// leave too few registers for five of them: a second kernel adds them up by
// columns, from the same inputs and two sums of each row.
#include "blocknorm.h"

namespace ttemb {

namespace {

constexpr int kBlockGradBlocks = 4 * kCUs; // rows of partial column sums, at most
constexpr int kBlockCols = 64 * kBlockVec; // columns of a block that adds up long rows
constexpr int kBlockSums = 5;              // dgamma, dbeta, dpost_gamma, dpost_beta, dgate

// What a thread knows of its elements of a row, and the gradient on the way.
struct BlockGrad {
    float xhat, u, weight, hhat; // N(x), u, b gate, N(h)
};
__device__ __forceinline__ BlockGrad block_forward(const BlockNormArgs &a, const float *st, float x, float res,
                                                   float gate, float pgam, float pbet)
{
    BlockGrad v;
    v.xhat = (x - st[0]) * st[1];
    v.u = a.post ? fmaf(v.xhat, pgam, pbet) : x;
    v.weight = a.scale_block * gate;
    v.hhat = (fmaf(v.weight, v.u, a.scale_residual * res) - st[2]) * st[3];
    return v;
}

// Gradients of a block's rows; its sums over its rows go to part[sum][block][D].
// LEAN: no sums, the two sums of each row go to `dots`.
template <class T, class R, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__(NormShape<TPR>::threads) void k_block_bwd(BlockNormArgs a, float *part, float2 *dots)
{
    constexpr int VEC = kBlockVec;
    constexpr bool LEAN = TPR == 1024;
    constexpr int SUMS = LEAN ? 1 : kBlockSums, SV = LEAN ? 1 : NV;
    __shared__ float sm[2][16][2];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int D = (int)a.D;
    const float invD = 1.f / (float)D;
    const int64_t step = (int64_t)gridDim.x * NormShape<TPR>::rows, last = a.n - 1;
    int64_t r0 = (int64_t)blockIdx.x * NormShape<TPR>::rows;
    typename VecOf<T, VEC>::raw nx[NV], ny[NV], ng[NV];
    typename VecOf<R, VEC>::raw nr[NV], nh[NV];
    float nst[4];
    auto load = [&](int64_t row) {
        const int64_t r = row < a.n ? row : last;
        const T *x = static_cast<const T *>(a.x) + r * a.ld_x, *g = static_cast<const T *>(a.gate) + r * a.ld_gate;
        const T *gy = static_cast<const T *>(a.grad_y) + r * a.ld_gy;
        const R *res = static_cast<const R *>(a.residual) + r * a.ld_r;
        const R *gh = static_cast<const R *>(a.grad_h) + r * a.ld_gh;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (t + j * TPR) * VEC;
            nx[j] = load_row<T, VEC, WHOLE>(x, c, D);
            nr[j] = load_row<R, VEC, WHOLE>(res, c, D);
            ny[j] = load_row<T, VEC, WHOLE>(gy, c, D);
            if (a.grad_h) nh[j] = load_row<R, VEC, WHOLE>(gh, c, D);
            if (a.gate_rows) ng[j] = load_row<T, VEC, WHOLE>(g, c, D);
        }
        load_vec<float, 4>(a.stats + r * 4, nst);
    };
    if constexpr (!LEAN) load(r0 + sub);
    float sums[SUMS][SV][VEC];
    constexpr int PV = LEAN ? 1 : NV;
    float gam[PV][VEC], pgam[PV][VEC], pbet[PV][VEC], gate[PV][VEC];
    auto params = [&](int j, int p) {
        const int64_t c = (t + j * TPR) * VEC;
        load_params<VEC, WHOLE>(a.gamma, a.param_dtype, c, D, 1.f, gam[p]);
        load_params<VEC, WHOLE>(a.post_gamma, a.param_dtype, c, D, 1.f, pgam[p]);
        load_params<VEC, WHOLE>(a.post_beta, a.param_dtype, c, D, 0.f, pbet[p]);
        load_params<VEC, WHOLE>(a.gate_rows ? nullptr : a.gate, a.param_dtype, c, D, 1.f, gate[p]);
    };
    int left[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        left[j] = D - (t + j * TPR) * VEC;
        if constexpr (!LEAN) {
            params(j, j);
#pragma unroll
            for (int k = 0; k < SUMS; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) sums[k][j][i] = 0.f;
        }
    }
    int slot = 0;
    for (; r0 < a.n; r0 += step) {
        const int64_t r = r0 + sub;
        const bool live = r < a.n;
        if constexpr (LEAN) load(r);
        float x[NV][VEC], res[NV][VEC], gy[NV][VEC], gh[NV][VEC], gr[NV][VEC], st[4];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                x[j][i] = (float)nx[j][i];
                res[j][i] = (float)nr[j][i];
                gy[j][i] = (float)ny[j][i];
                gh[j][i] = a.grad_h ? (float)nh[j][i] : 0.f;
                gr[j][i] = a.gate_rows ? (float)ng[j][i] : 1.f;
            }
#pragma unroll
        for (int k = 0; k < 4; ++k) st[k] = nst[k];
        if constexpr (!LEAN) load(r + step);
        float s[2] = {0.f, 0.f};
        BlockGrad v[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (LEAN) {
                __builtin_amdgcn_sched_barrier(0);
                params(j, 0);
            }
            const int p = LEAN ? 0 : j;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[j][i] = block_forward(a, st, x[j][i], res[j][i], gate[p][i] * gr[j][i], pgam[p][i], pbet[p][i]);
                const float q = gy[j][i] * gam[p][i]; // 0 past the row's end
                if constexpr (!LEAN) {
                    if (live && i < left[j]) {
                        sums[0][j][i] = fmaf(gy[j][i], v[j][i].hhat, sums[0][j][i]);
                        sums[1][j][i] += gy[j][i];
                    }
                }
                gy[j][i] = q;
                s[0] += q;
                s[1] = fmaf(q, v[j][i].hhat, s[1]);
            }
        }
        row_sum<TPR, 2>(s, sm, slot);
        const float m0 = a.layer ? s[0] * invD : 0.f, m1 = s[1] * invD;
        if (LEAN && live && t == 0) dots[r] = make_float2(m0, m1);
        float w[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (LEAN) {
                __builtin_amdgcn_sched_barrier(0);
                params(j, 0);
            }
            const int p = LEAN ? 0 : j;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float dh = gh[j][i] + (gy[j][i] - m0 - v[j][i].hhat * m1) * st[3];
                const float du = i < left[j] ? v[j][i].weight * dh : 0.f;
                gh[j][i] = dh;
                if constexpr (!LEAN) {
                    if (live && i < left[j]) {
                        sums[2][j][i] = fmaf(du, v[j][i].xhat, sums[2][j][i]);
                        sums[3][j][i] += du;
                        sums[4][j][i] = fmaf(a.scale_block * dh, v[j][i].u, sums[4][j][i]);
                    }
                }
                gy[j][i] = a.post ? du * pgam[p][i] : du;
                w[0] += gy[j][i];
                w[1] = fmaf(gy[j][i], v[j][i].xhat, w[1]);
            }
        }
        if (a.post) row_sum<TPR, 2>(w, sm, slot);
        if (!live) continue;
        const float n0 = a.post && a.layer ? w[0] * invD : 0.f, n1 = a.post ? w[1] * invD : 0.f;
        T *dx = static_cast<T *>(a.grad_x) + r * a.ld_gx, *dg = static_cast<T *>(a.grad_gate) + r * a.ld_gg;
        R *dr = static_cast<R *>(a.grad_r) + r * a.ld_gr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (t + j * TPR) * VEC;
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                o[i] = a.post ? (gy[j][i] - n0 - v[j][i].xhat * n1) * st[1] : gy[j][i];
            store_part<T, VEC>(dx + c, left[j], o);
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = a.scale_residual * gh[j][i];
            store_part<R, VEC>(dr + c, left[j], o);
            if (a.gate_rows) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = a.scale_block * gh[j][i] * v[j][i].u;
                store_part<T, VEC>(dg + c, left[j], o);
            }
        }
    }
    if constexpr (!LEAN) {
        // the block's sums: sub-rows of one wave by shuffles, the waves through LDS
        constexpr int W = TPR < 64 ? TPR : 64, COLS = TPR * NV * VEC, WAVES = NormShape<TPR>::threads / 64;
        constexpr bool JOIN = NormShape<TPR>::rows > 1;
        __shared__ float col[JOIN ? WAVES : 1][JOIN ? COLS : 1];
#pragma unroll
        for (int k = 0; k < kBlockSums; ++k) {
            if (!a.sums[k]) continue;
            float *to = part + ((int64_t)k * gridDim.x + blockIdx.x) * D;
            if constexpr (JOIN) {
                __syncthreads(); // the last sum's columns have been read
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
#pragma unroll
                        for (int o = W; o < 64; o <<= 1) sums[k][j][i] += __shfl_xor(sums[k][j][i], o, 64);
                        if ((threadIdx.x & 63) < W) col[threadIdx.x >> 6][(t + j * TPR) * VEC + i] = sums[k][j][i];
                    }
                __syncthreads();
                for (int c = threadIdx.x; c < D; c += NormShape<TPR>::threads) {
                    float s = 0.f;
#pragma unroll
                    for (int w = 0; w < WAVES; ++w) s += col[w][c];
                    to[c] = s;
                }
            } else {
#pragma unroll
                for (int j = 0; j < NV; ++j) store_part<float, VEC>(to + (t + j * TPR) * VEC, left[j], sums[k][j]);
            }
        }
    }
}

// Column sums of long rows: a block has 64 vectors of columns and every fourth
// row of its share goes to one of its waves; the waves meet in LDS.
template <class T, class R, bool WHOLE>
__global__ __launch_bounds__(256) void k_block_cols(BlockNormArgs a, float *part, const float2 *dots)
{
    constexpr int VEC = kBlockVec;
    __shared__ float col[4][64 * VEC + 4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, D = (int)a.D;
    const int64_t c = ((int64_t)blockIdx.x * 64 + lane) * VEC;
    float gam[VEC], pgam[VEC], pbet[VEC], gate[VEC], sums[kBlockSums][VEC];
    load_params<VEC, WHOLE>(a.gamma, a.param_dtype, c, D, 1.f, gam);
    load_params<VEC, WHOLE>(a.post_gamma, a.param_dtype, c, D, 1.f, pgam);
    load_params<VEC, WHOLE>(a.post_beta, a.param_dtype, c, D, 0.f, pbet);
    load_params<VEC, WHOLE>(a.gate_rows ? nullptr : a.gate, a.param_dtype, c, D, 1.f, gate);
#pragma unroll
    for (int k = 0; k < kBlockSums; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sums[k][i] = 0.f;
    for (int64_t r = (int64_t)blockIdx.y * 4 + wave; r < a.n; r += (int64_t)gridDim.y * 4) {
        float st[4];
        load_vec<float, 4>(a.stats + r * 4, st);
        const float2 m = dots[r];
        const auto x = load_row<T, VEC, WHOLE>(static_cast<const T *>(a.x) + r * a.ld_x, c, D);
        const auto gy = load_row<T, VEC, WHOLE>(static_cast<const T *>(a.grad_y) + r * a.ld_gy, c, D);
        const auto res = load_row<R, VEC, WHOLE>(static_cast<const R *>(a.residual) + r * a.ld_r, c, D);
        typename VecOf<R, VEC>::raw gh = {};
        typename VecOf<T, VEC>::raw gr = {};
        if (a.grad_h) gh = load_row<R, VEC, WHOLE>(static_cast<const R *>(a.grad_h) + r * a.ld_gh, c, D);
        if (a.gate_rows) gr = load_row<T, VEC, WHOLE>(static_cast<const T *>(a.gate) + r * a.ld_gate, c, D);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float g = (float)gy[i];
            const BlockGrad v = block_forward(a, st, (float)x[i], (float)res[i],
                                              a.gate_rows ? gate[i] * (float)gr[i] : gate[i], pgam[i], pbet[i]);
            const float dh = (float)gh[i] + (g * gam[i] - m.x - v.hhat * m.y) * st[3], du = v.weight * dh;
            sums[0][i] = fmaf(g, v.hhat, sums[0][i]);
            sums[1][i] += g;
            sums[2][i] = fmaf(du, v.xhat, sums[2][i]);
            sums[3][i] += du;
            sums[4][i] = fmaf(a.scale_block * dh, v.u, sums[4][i]);
        }
    }
#pragma unroll
    for (int k = 0; k < kBlockSums; ++k) {
        if (!a.sums[k]) continue;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VEC; ++i) col[wave][lane * VEC + i] = sums[k][i];
        __syncthreads();
        float *to = part + ((int64_t)k * gridDim.y + blockIdx.y) * D + (int64_t)blockIdx.x * 64 * VEC;
        for (int i = threadIdx.x; i < 64 * VEC && (int64_t)blockIdx.x * 64 * VEC + i < D; i += 256)
            to[i] = (col[0][i] + col[1][i]) + (col[2][i] + col[3][i]);
    }
}

// No rows: the sums over them are zero.
__global__ __launch_bounds__(256) void k_block_zero(ColumnSums out, int D)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= D) return;
    for (int k = 0; k < kBlockSums; ++k)
        if (out.dst[k]) store_param(out.dst[k], out.dtype[k], c, 0.f);
}

ColumnSums block_sums(const BlockNormArgs &a)
{
    ColumnSums c{};
    for (int k = 0; k < kBlockSums; ++k) {
        c.dst[k] = a.sums[k];
        c.dtype[k] = a.param_dtype;
    }
    return c;
}

template <class T, class R>
hipError_t block_backward(const BlockNormArgs &a, hipStream_t s)
{
    const ColumnSums out = block_sums(a);
    float *part = reinterpret_cast<float *>(a.ws + TT_EMB_STATUS_BYTES);
    float2 *dots = reinterpret_cast<float2 *>(a.ws + TT_EMB_STATUS_BYTES + block_parts_bytes(a.n, a.D));
    return block_shape(a.D, [&](auto tpr, auto nv, auto whole) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        constexpr bool WHOLE = decltype(whole)::value;
        const int64_t need = (a.n + NormShape<TPR>::rows - 1) / NormShape<TPR>::rows;
        int parts = (int)(need < kBlockGradBlocks ? need : kBlockGradBlocks);
        hipLaunchKernelGGL((k_block_bwd<T, R, TPR, NV, WHOLE>), dim3(parts), dim3(NormShape<TPR>::threads), 0, s, a,
                           part, dots);
        if constexpr (TPR == 1024) {
            parts = block_col_parts(a.n, a.D);
            const dim3 grid((unsigned)((a.D + kBlockCols - 1) / kBlockCols), (unsigned)parts);
            hipLaunchKernelGGL((k_block_cols<T, R, WHOLE>), grid, dim3(256), 0, s, a, part, dots);
        }
        norm_cols(part, parts, a.D, kBlockSums, out, s);
        return hipGetLastError();
    });
}

} // namespace

// Shares of the rows in the kernel that adds up long rows' columns: some four
// blocks for each compute unit, of sixteen rows at least.
int block_col_parts(int64_t n, int64_t D)
{
    const int64_t strips = (D + kBlockCols - 1) / kBlockCols, most = (n + 15) / 16;
    int64_t parts = (4 * kCUs + strips - 1) / strips;
    if (parts > most) parts = most;
    return (int)(parts < 1 ? 1 : parts);
}

size_t block_parts_bytes(int64_t n, int64_t D)
{
    int64_t parts = n < kBlockGradBlocks ? n : kBlockGradBlocks;
    if (D > kBlockRegs) parts = block_col_parts(n, D);
    return round256((size_t)(kBlockSums * parts * D) * sizeof(float));
}

size_t block_workspace(int64_t n, int64_t D)
{
    return TT_EMB_STATUS_BYTES + block_parts_bytes(n, D) + (D > kBlockRegs ? round256((size_t)n * sizeof(float2)) : 0);
}

hipError_t launch_block_backward(const BlockNormArgs &a, int dtype, int res_dtype, hipStream_t s)
{
    if (a.n == 0) {
        hipLaunchKernelGGL(k_block_zero, dim3((unsigned)((a.D + 255) / 256)), dim3(256), 0, s, block_sums(a), (int)a.D);
        return hipGetLastError();
    }
    return block_types(dtype, res_dtype,
                       [&](auto t, auto r) { return block_backward<decltype(t), decltype(r)>(a, s); });
}

} // namespace ttemb
