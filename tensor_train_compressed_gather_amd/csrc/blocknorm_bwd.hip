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
// those that the forward was given, and makes h again in fp32: as many bytes as
// reading h, which a caller may overwrite after the forward, and without its
// rounding.  The column sums of rows of up to 4096 values stay in registers across
// a block's rows.  Longer rows are read again, from the caches, for each pair of
// sums, and a second kernel adds up their columns, from the same inputs and two
// sums of each row.
//
// Memory bounds it: 16384 x 4096 bf16 in 153 us (six tensors, 5.3 TB/s) and 5 for
// the sums of the blocks' columns; 32768 x 128 fp32 in 22 (4.6 TB/s) and 3.8.
#include "blocknorm.h"

namespace ttemb {

namespace {

// Rows of partial column sums, at most: as many blocks as the registers let the
// compute units hold (eight waves of them, in one block or in two).
constexpr int kBlockGradBlocks = 2 * kCUs;
constexpr int kBlockCols = 64 * kBlockVec; // columns of a block that adds up long rows
// Distance of the rows of partial sums: they are read four at a time.
__host__ __device__ inline int64_t part_row(int64_t D) { return (D + 3) / 4 * 4; }
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
template <class T, class R, int TPR, bool WHOLE>
__global__ __launch_bounds__(NormShape<TPR>::threads) void k_block_bwd(BlockNormArgs a, float *part)
{
    constexpr int VEC = kBlockVec;
    constexpr bool TWO = sizeof(T) == 2 && sizeof(R) == 2; // rows on their way (fp32 rows are as many bytes each)
    __shared__ float sm[2][16][2];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, c = t * VEC;
    const int D = (int)a.D, left = D - c;
    const float invD = 1.f / (float)D;
    const int64_t step = (int64_t)gridDim.x * NormShape<TPR>::rows, last = a.n - 1;
    int64_t r0 = (int64_t)blockIdx.x * NormShape<TPR>::rows;
    struct Row {
        typename VecOf<T, VEC>::raw x, gy, gate;
        typename VecOf<R, VEC>::raw res, gh;
        float st[4];
    };
    auto load = [&](int64_t row, Row &to) {
        const int64_t r = row < a.n ? row : last;
        to.x = load_cols<T, WHOLE>(static_cast<const T *>(a.x) + r * a.ld_x, c, D);
        to.res = load_cols<R, WHOLE>(static_cast<const R *>(a.residual) + r * a.ld_r, c, D);
        to.gy = load_cols<T, WHOLE>(static_cast<const T *>(a.grad_y) + r * a.ld_gy, c, D);
        if (a.grad_h) to.gh = load_cols<R, WHOLE>(static_cast<const R *>(a.grad_h) + r * a.ld_gh, c, D);
        if (a.gate_rows) to.gate = load_cols<T, WHOLE>(static_cast<const T *>(a.gate) + r * a.ld_gate, c, D);
        load_vec<float, 4>(a.stats + r * 4, to.st);
    };
    Row one, two;
    load(r0 + sub, one);
    if constexpr (TWO) load(r0 + step + sub, two);
    float sums[kBlockSums][VEC], gam[VEC], pgam[VEC], pbet[VEC], gate[VEC];
    load_params<VEC, WHOLE>(a.gamma, a.param_dtype, c, D, 1.f, gam);
    load_params<VEC, WHOLE>(a.post_gamma, a.param_dtype, c, D, 1.f, pgam);
    load_params<VEC, WHOLE>(a.post_beta, a.param_dtype, c, D, 0.f, pbet);
    load_params<VEC, WHOLE>(a.gate_rows ? nullptr : a.gate, a.param_dtype, c, D, 1.f, gate);
#pragma unroll
    for (int k = 0; k < kBlockSums; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sums[k][i] = 0.f;
    int slot = 0;
    auto pass = [&](int64_t r, Row &row) {
        const bool live = r < a.n;
        float x[VEC], res[VEC], gy[VEC], gh[VEC], gr[VEC], st[4];
        values<T, WHOLE>(row.x, left, D, x);
        values<R, WHOLE>(row.res, left, D, res);
        values<T, WHOLE>(row.gy, left, D, gy);
        if (a.grad_h) values<R, WHOLE>(row.gh, left, D, gh);
        if (a.gate_rows) values<T, WHOLE>(row.gate, left, D, gr);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            gh[i] = a.grad_h ? gh[i] : 0.f;
            gr[i] = a.gate_rows ? gr[i] : gate[i];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) st[k] = row.st[k];
        load(r + (TWO ? 2 : 1) * step, row);
        float s[2] = {0.f, 0.f};
        BlockGrad v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            v[i] = block_forward(a, st, x[i], res[i], gr[i], pgam[i], pbet[i]);
            const float q = gy[i] * gam[i]; // 0 past the row's end
            if (live && i < left) {
                sums[0][i] = fmaf(gy[i], v[i].hhat, sums[0][i]);
                sums[1][i] += gy[i];
            }
            gy[i] = q;
            s[0] += q;
            s[1] = fmaf(q, v[i].hhat, s[1]);
        }
        row_sum<TPR, 2>(s, sm, slot);
        const float m0 = a.layer ? s[0] * invD : 0.f, m1 = s[1] * invD;
        float w[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float dh = gh[i] + (gy[i] - m0 - v[i].hhat * m1) * st[3];
            const float du = i < left ? v[i].weight * dh : 0.f;
            gh[i] = dh;
            if (live && i < left) {
                sums[2][i] = fmaf(du, v[i].xhat, sums[2][i]);
                sums[3][i] += du;
                sums[4][i] = fmaf(a.scale_block * dh, v[i].u, sums[4][i]);
            }
            gy[i] = a.post ? du * pgam[i] : du;
            w[0] += gy[i];
            w[1] = fmaf(gy[i], v[i].xhat, w[1]);
        }
        if (a.post) row_sum<TPR, 2>(w, sm, slot);
        if (!live) return;
        const float n0 = a.layer ? w[0] * invD : 0.f, n1 = w[1] * invD;
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = a.post ? (gy[i] - n0 - v[i].xhat * n1) * st[1] : gy[i];
        store_part<T, VEC>(static_cast<T *>(a.grad_x) + r * a.ld_gx + c, left, x);
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = a.scale_residual * gh[i];
        store_part<R, VEC>(static_cast<R *>(a.grad_r) + r * a.ld_gr + c, left, x);
        if (a.gate_rows) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[i] = a.scale_block * gh[i] * v[i].u;
            store_part<T, VEC>(static_cast<T *>(a.grad_gate) + r * a.ld_gg + c, left, x);
        }
    };
    while (r0 < a.n) {
        pass(r0 + sub, one);
        r0 += step;
        if constexpr (TWO) {
            if (r0 >= a.n) break;
            pass(r0 + sub, two);
            r0 += step;
        }
    }
    // the block's sums: sub-rows of one wave by shuffles, the others through LDS
    constexpr int W = TPR < 64 ? TPR : 64, COLS = TPR * VEC;
    constexpr bool JOIN = NormShape<TPR>::rows > 1;
    constexpr int PARTS = TPR <= 64 ? NormShape<TPR>::threads / 64 : NormShape<TPR>::rows;
    const int mine = TPR <= 64 ? threadIdx.x >> 6 : sub;
    __shared__ float col[JOIN ? PARTS : 1][JOIN ? COLS : 1];
#pragma unroll
    for (int k = 0; k < kBlockSums; ++k) {
        if (!a.sums[k]) continue;
        float *to = part + ((int64_t)k * gridDim.x + blockIdx.x) * part_row(D);
        if constexpr (JOIN) {
            __syncthreads(); // the last sum's columns have been read
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
#pragma unroll
                for (int o = W; o < 64; o <<= 1) sums[k][i] += __shfl_xor(sums[k][i], o, 64);
                if ((threadIdx.x & 63) < W) col[mine][c + i] = sums[k][i];
            }
            __syncthreads();
            for (int q = threadIdx.x; q < D; q += NormShape<TPR>::threads) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < PARTS; ++w) s += col[w][q];
                to[q] = s;
            }
        } else {
            store_part<float, VEC>(to + c, left, sums[k]);
        }
    }
}

// Rows of more than 4096 values: a block's threads go over the row once for each
// of the two pairs of sums, and once more for the gradients; the column sums are
// another kernel's, which takes m0 and m1 of each row from `dots`.
template <class T, class R, bool WHOLE>
__global__ __launch_bounds__(kBlockLong) void k_block_bwd_long(BlockNormArgs a, float2 *dots)
{
    constexpr int VEC = kBlockVec;
    __shared__ float sm[2][16][2];
    const int D = (int)a.D;
    const float invD = 1.f / (float)D;
    int slot = 0;
    for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
        float st[4];
        load_vec<float, 4>(a.stats + r * 4, st);
        // f(column, elements that exist, N(x) .. N(h), grad_y gamma, grad_h, post_gamma)
        auto each = [&](auto f) {
#pragma clang loop unroll(disable)
            for (int c = threadIdx.x * VEC; c < D; c += kBlockLong * VEC) {
                const int left = D - c;
                float x[VEC], res[VEC], q[VEC], gh[VEC], gate[VEC], gam[VEC], pgam[VEC], pbet[VEC];
                values<T, WHOLE>(load_cols<T, WHOLE>(static_cast<const T *>(a.x) + r * a.ld_x, c, D), left, D, x);
                values<R, WHOLE>(load_cols<R, WHOLE>(static_cast<const R *>(a.residual) + r * a.ld_r, c, D), left, D,
                                 res);
                values<T, WHOLE>(load_cols<T, WHOLE>(static_cast<const T *>(a.grad_y) + r * a.ld_gy, c, D), left, D, q);
                if (a.grad_h)
                    values<R, WHOLE>(load_cols<R, WHOLE>(static_cast<const R *>(a.grad_h) + r * a.ld_gh, c, D), left, D,
                                     gh);
                if (a.gate_rows)
                    values<T, WHOLE>(load_cols<T, WHOLE>(static_cast<const T *>(a.gate) + r * a.ld_gate, c, D), left, D,
                                     gate);
                else load_params<VEC, WHOLE>(a.gate, a.param_dtype, c, D, 1.f, gate);
                load_params<VEC, WHOLE>(a.gamma, a.param_dtype, c, D, 1.f, gam);
                load_params<VEC, WHOLE>(a.post_gamma, a.param_dtype, c, D, 1.f, pgam);
                load_params<VEC, WHOLE>(a.post_beta, a.param_dtype, c, D, 0.f, pbet);
                BlockGrad v[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    v[i] = block_forward(a, st, x[i], res[i], gate[i], pgam[i], pbet[i]);
                    q[i] *= gam[i];
                    gh[i] = a.grad_h ? gh[i] : 0.f;
                }
                f(c, left, v, q, gh, pgam);
            }
        };
        typedef BlockGrad(&Grads)[VEC];
        typedef float(&Values)[VEC];
        float s[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
        each([&](int, int, Grads v, Values q, Values, Values) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) { // (q is 0 past the row's end)
                s[0] += q[i];
                s[1] = fmaf(q[i], v[i].hhat, s[1]);
            }
        });
        row_sum<kBlockLong, 2>(s, sm, slot);
        const float m0 = a.layer ? s[0] * invD : 0.f, m1 = s[1] * invD;
        if (threadIdx.x == 0) dots[r] = make_float2(m0, m1);
        auto dh_of = [&](const BlockGrad &v, float q, float gh) { return gh + (q - m0 - v.hhat * m1) * st[3]; };
        if (a.post) {
            each([&](int, int left, Grads v, Values q, Values gh, Values pgam) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float p = i < left ? v[i].weight * dh_of(v[i], q[i], gh[i]) * pgam[i] : 0.f;
                    w[0] += p;
                    w[1] = fmaf(p, v[i].xhat, w[1]);
                }
            });
            row_sum<kBlockLong, 2>(w, sm, slot);
        }
        const float n0 = a.layer ? w[0] * invD : 0.f, n1 = w[1] * invD;
        each([&](int c, int left, Grads v, Values q, Values gh, Values pgam) {
            float dx[VEC], dg[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float dh = dh_of(v[i], q[i], gh[i]), du = v[i].weight * dh;
                dx[i] = a.post ? (du * pgam[i] - n0 - v[i].xhat * n1) * st[1] : du;
                dg[i] = a.scale_block * dh * v[i].u;
                q[i] = a.scale_residual * dh;
            }
            store_part<T, VEC>(static_cast<T *>(a.grad_x) + r * a.ld_gx + c, left, dx);
            store_part<R, VEC>(static_cast<R *>(a.grad_r) + r * a.ld_gr + c, left, q);
            if (a.gate_rows) store_part<T, VEC>(static_cast<T *>(a.grad_gate) + r * a.ld_gg + c, left, dg);
        });
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
        float *to = part + ((int64_t)k * gridDim.y + blockIdx.y) * part_row(D) + (int64_t)blockIdx.x * 64 * VEC;
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
    return round256((size_t)(kBlockSums * parts * part_row(D)) * sizeof(float));
}

template <class T, class R>
hipError_t block_backward(const BlockNormArgs &a, hipStream_t s)
{
    const ColumnSums out = block_sums(a);
    float *part = reinterpret_cast<float *>(a.ws + TT_EMB_STATUS_BYTES);
    float2 *dots = reinterpret_cast<float2 *>(a.ws + TT_EMB_STATUS_BYTES + block_parts_bytes(a.n, a.D));
    if (a.D > kBlockRegs) {
        const int parts = block_col_parts(a.n, a.D);
        const dim3 rows(block_grid(a.n, 4 * kCUs)), cols((unsigned)((a.D + kBlockCols - 1) / kBlockCols), parts);
        auto run = [&](auto whole) {
            constexpr bool WHOLE = decltype(whole)::value;
            hipLaunchKernelGGL((k_block_bwd_long<T, R, WHOLE>), rows, dim3(kBlockLong), 0, s, a, dots);
            hipLaunchKernelGGL((k_block_cols<T, R, WHOLE>), cols, dim3(256), 0, s, a, part, dots);
        };
        if (a.D % kBlockVec == 0) run(std::true_type());
        else run(std::false_type());
        norm_cols(part, parts, a.D, part_row(a.D), kBlockSums, out, s);
        return hipGetLastError();
    }
    return block_shape(a.D, [&](auto tpr, auto whole) {
        constexpr int TPR = decltype(tpr)::value;
        const int64_t need = (a.n + NormShape<TPR>::rows - 1) / NormShape<TPR>::rows;
        const int parts = block_grid(need, TPR == 512 ? kCUs : kBlockGradBlocks);
        hipLaunchKernelGGL((k_block_bwd<T, R, TPR, decltype(whole)::value>), dim3(parts),
                           dim3(NormShape<TPR>::threads), 0, s, a, part);
        norm_cols(part, parts, a.D, part_row(a.D), kBlockSums, out, s);
        return hipGetLastError();
    });
}

} // namespace

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
