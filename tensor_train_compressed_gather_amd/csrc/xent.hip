// xent.hip -- softmax cross entropy of hidden rows against a large vocabulary
// without keeping the logits, and both gradients (gfx950).
//
// Three products of the same sizes: the logits z = H W^T, and with d the
// gradient of the loss by the logits, dH = d W and dW = d^T H.  All run on the
// bf16 matrix cores with fp32 accumulators.  The logits never leave the
// registers of the tile that makes them: a first pass keeps each row's maximum
// and sum of exponentials per tile, from which lse and the loss follow; for
// the gradients a piece of the vocabulary's logits is made again, turned into
// d, and multiplied into both gradients before the next piece.
//
// fp32 inputs are split into three bf16 terms (24 bits of mantissa) and the
// six products of terms that matter at 2^-24 are added up, which is more than
// twice the rate of the fp32 matrix instructions; d is split the same way.
#include "lm.h"
#include "primitives.h"

namespace ttemb {

namespace {

typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTile = 128;    // rows and columns of a product's tile
constexpr int kTileK = 64;
constexpr int kPad = 8;       // elements between rows of a tile in LDS
constexpr int64_t kPiece = 16384; // columns of d at a time, at most

inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// An operand of a product: `planes` bf16 matrices.  Straight: row r holds the
// summed index.  Turned: row k of the summed index holds the outputs.
struct Operand {
    const bf16 *p;
    int64_t ld, plane; // elements between rows, between planes
    int64_t rows, cols; // of the stored matrix; reads past them are clamped
};

enum { OUT_STATS, OUT_D, OUT_HIDDEN, OUT_WEIGHT };

struct Output {
    int64_t n, V, v0;         // rows, vocabulary, first column of this piece
    const int64_t *targets;
    int64_t ignore;
    float2 *part;             // [vocabulary tiles][n] maximum and sum
    float *target_logit;      // [n]
    const float *lse, *grad;  // [n]
    const float *top_grad;    // the largest |grad| of a row that counts
    bf16 *d;                  // [planes][rows][ldd]
    int64_t ldd, plane_d;
    float *sum;               // dH in fp32, [n][D]
    void *out;                // dH or dW
    int64_t ld_out, D;
    int out_f32, first, last;
};

// x as a sum of PL bf16 values
template <int PL>
__device__ __forceinline__ void split(float x, bf16 (&t)[PL])
{
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        t[i] = (bf16)x;
        x -= (float)t[i];
    }
}

// C[m][n] = sum_k X[m][k] Y[n][k] over tiles of 128 x 128; 32x32x16 matrix
// instructions, two by two tiles per wave.  Lane l of a wave holds column
// n = l % 32 and the rows m = 8 (r / 4) + 4 (l / 32) + r % 4, so the contiguous
// output index is m and the row of the output is n.
template <int PL, bool XT, bool YT, int OUT>
__global__ __launch_bounds__(256) void k_product(Operand X, Operand Y, int64_t K, Output o)
{
    __shared__ bf16 xs[kTile][kTileK + kPad], ys[kTile][kTileK + kPad];
    __shared__ float red[2][2][kTile];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave & 1, wn = wave >> 1;
    const int64_t m0 = (int64_t)blockIdx.x * kTile, n0 = (int64_t)blockIdx.y * kTile;
    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    auto stage = [&](const Operand &a, bool turned, int plane, int64_t r0, int64_t k0, bf16 (*dst)[kTileK + kPad]) {
        const bf16 *p = a.p + plane * a.plane;
        if (!turned) {
#pragma unroll
            for (int i = 0; i < kTile * kTileK / 8 / 256; ++i) {
                const int c = tid + i * 256, r = c / (kTileK / 8), k = (c % (kTileK / 8)) * 8;
                const int64_t row = r0 + r < a.rows ? r0 + r : a.rows - 1;
                *reinterpret_cast<bf16x8 *>(&dst[r][k]) = *reinterpret_cast<const bf16x8 *>(p + row * a.ld + k0 + k);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kTile * kTileK / 8 / 256; ++i) {
                const int c = tid + i * 256, k = c / (kTile / 8), r = (c % (kTile / 8)) * 8;
                const int64_t row = k0 + k < a.rows ? k0 + k : a.rows - 1;
                const int64_t col = r0 + r < a.cols - 8 ? r0 + r : a.cols - 8;
                const bf16x8 v = *reinterpret_cast<const bf16x8 *>(p + row * a.ld + col);
#pragma unroll
                for (int j = 0; j < 8; ++j) dst[r + j][k] = v[j];
            }
        }
    };
    // products of terms, the small ones first
    constexpr int SEG = PL == 1 ? 1 : 6;
    constexpr int sx[6] = {2, 0, 1, 1, 0, 0}, sy[6] = {0, 2, 1, 0, 1, 0};
    for (int g = 0; g < SEG; ++g) {
        const int px = PL == 1 ? 0 : sx[g], py = PL == 1 ? 0 : sy[g];
        for (int64_t k0 = 0; k0 < K; k0 += kTileK) {
            __syncthreads();
            stage(X, XT, px, m0, k0, xs);
            stage(Y, YT, py, n0, k0, ys);
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kTileK; k += 16) {
                bf16x8 a[2], b[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    a[i] = *reinterpret_cast<const bf16x8 *>(&xs[wm * 64 + i * 32 + (lane & 31)][k + (lane >> 5) * 8]);
                    b[i] = *reinterpret_cast<const bf16x8 *>(&ys[wn * 64 + i * 32 + (lane & 31)][k + (lane >> 5) * 8]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
            }
        }
    }
    auto row_of = [&](int i, int r) { return wm * 64 + i * 32 + 8 * (r / 4) + 4 * (lane >> 5) + (r % 4); };
    if constexpr (OUT == OUT_STATS) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int nl = wn * 64 + j * 32 + (lane & 31);
            const int64_t i = n0 + nl;
            const int64_t t = i < o.n ? o.targets[i] : -1;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t v = m0 + row_of(a, r);
                    if (v < o.V) {
                        top = fmaxf(top, acc[a][j][r]);
                        if (v == t) o.target_logit[i] = acc[a][j][r];
                    }
                }
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (m0 + row_of(a, r) < o.V) sum += __expf(acc[a][j][r] - ref);
            sum += __shfl_xor(sum, 32, 64);
            if (lane < 32) {
                red[0][wm][nl] = top;
                red[1][wm][nl] = sum;
            }
        }
        __syncthreads();
        if (tid < kTile && n0 + tid < o.n) {
            const float a = red[0][0][tid], b = red[0][1][tid], top = fmaxf(a, b);
            const float ref = top == -INFINITY ? 0.f : top;
            const float s = red[1][0][tid] * __expf(a - ref) + red[1][1][tid] * __expf(b - ref);
            o.part[(int64_t)blockIdx.x * o.n + n0 + tid] = make_float2(top, s);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t i = n0 + wn * 64 + j * 32 + (lane & 31);
            float lse = 0.f, g = 0.f;
            int64_t t = -1;
            if constexpr (OUT == OUT_D) {
                if (i < o.n) {
                    t = o.targets[i] - o.v0;
                    const bool counts = o.targets[i] != o.ignore && o.targets[i] >= 0 && o.targets[i] < o.V;
                    g = counts ? o.grad[i] / *o.top_grad : 0.f;
                    lse = o.lse[i];
                }
            }
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t m = m0 + row_of(a, 4 * q);
                    float x[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[r] = acc[a][j][4 * q + r];
                    if constexpr (OUT == OUT_D) {
                        bf16x4 w[PL];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const bool in = g != 0.f && o.v0 + m + r < o.V;
                            const float d = in ? g * (__expf(x[r] - lse) - (m + r == t ? 1.f : 0.f)) : 0.f;
                            bf16 s[PL];
                            split<PL>(d, s);
#pragma unroll
                            for (int q2 = 0; q2 < PL; ++q2) w[q2][r] = s[q2];
                        }
#pragma unroll
                        for (int q2 = 0; q2 < PL; ++q2)
                            *reinterpret_cast<bf16x4 *>(o.d + q2 * o.plane_d + i * o.ldd + m) = w[q2];
                    } else if constexpr (OUT == OUT_HIDDEN) {
                        if (i >= o.n) continue;
                        const float scale = *o.top_grad;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (m + r >= o.D) continue;
                            float *s = o.sum + i * o.D + m + r;
                            float v = o.first ? x[r] : *s + x[r];
                            if (o.last) v *= scale;
                            if (!o.last) *s = v;
                            else if (o.out_f32) static_cast<float *>(o.out)[i * o.ld_out + m + r] = v;
                            else static_cast<bf16 *>(o.out)[i * o.ld_out + m + r] = (bf16)v;
                        }
                    } else {
                        if (o.v0 + i >= o.V) continue;
                        const float scale = *o.top_grad;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (m + r >= o.D) continue;
                            const int64_t at = (o.v0 + i) * o.ld_out + m + r;
                            if (o.out_f32) static_cast<float *>(o.out)[at] = x[r] * scale;
                            else static_cast<bf16 *>(o.out)[at] = (bf16)(x[r] * scale);
                        }
                    }
                }
        }
    }
}

// Rows of a matrix as PL bf16 planes with `ld` columns, zero past D.
template <class T, int PL>
__global__ __launch_bounds__(256) void k_pack(const T *src, int64_t ld_src, int64_t rows, int64_t D, bf16 *dst,
                                              int64_t ld, int64_t plane)
{
    const int64_t chunks = ld / 8;
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < rows * chunks; c += step) {
        const int64_t r = c / chunks, k = (c - r * chunks) * 8;
        float x[8];
        const int left = D - k < 8 ? (int)(D - k < 0 ? 0 : D - k) : 8;
        load_part<T, 8>(src + r * ld_src + (left ? k : 0), left, x);
        bf16x8 w[PL];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            bf16 s[PL];
            split<PL>(x[i], s);
#pragma unroll
            for (int q = 0; q < PL; ++q) w[q][i] = s[q];
        }
#pragma unroll
        for (int q = 0; q < PL; ++q) *reinterpret_cast<bf16x8 *>(dst + q * plane + r * ld + k) = w[q];
    }
}

// lse and loss of sixteen rows per block from the tiles' maxima and sums.
__global__ __launch_bounds__(256) void k_xent_join(const float2 *part, int64_t tiles, int64_t n, int64_t V,
                                                   const int64_t *targets, int64_t ignore, const float *target_logit,
                                                   float *loss, float *lse, int *status)
{
    __shared__ float2 sm[16][16];
    const int r = threadIdx.x & 15, g = threadIdx.x >> 4;
    const int64_t i = (int64_t)blockIdx.x * 16 + r, ic = i < n ? i : n - 1;
    float top = -INFINITY, sum = 0.f;
    for (int64_t t = g; t < tiles; t += 16) {
        const float2 p = part[t * n + ic];
        const float m = fmaxf(top, p.x);
        const float ref = m == -INFINITY ? 0.f : m;
        sum = sum * __expf(top - ref) + p.y * __expf(p.x - ref);
        top = m;
    }
    sm[r][g] = make_float2(top, sum);
    __syncthreads();
    if (g || i >= n) return;
    for (int q = 1; q < 16; ++q) {
        const float2 p = sm[r][q];
        const float m = fmaxf(top, p.x);
        const float ref = m == -INFINITY ? 0.f : m;
        sum = sum * __expf(top - ref) + p.y * __expf(p.x - ref);
        top = m;
    }
    const float z = (top == -INFINITY ? 0.f : top) + logf(sum);
    const int64_t t = targets[i];
    const bool in = t >= 0 && t < V;
    if (!in && t != ignore) atomicOr(status + ST_ERR, (int)STB_INDEX);
    lse[i] = z;
    loss[i] = in && t != ignore ? z - target_logit[i] : 0.f;
}

// The largest |grad_loss| of the rows that count.  d is kept in units of it:
// with equal gradients (a mean over the rows) d is exp(z - lse) - [v = target],
// and the target's -1 + p, the largest term of both gradients, rounds to bf16
// without error for small p.  1 where there is nothing to scale.
__global__ __launch_bounds__(1024) void k_xent_top_grad(const float *grad, const int64_t *targets, int64_t ignore,
                                                        int64_t n, int64_t V, float *top)
{
    __shared__ float sm[16];
    float m = 0.f;
    for (int64_t i = threadIdx.x; i < n; i += 1024) {
        const int64_t t = targets[i];
        if (t != ignore && t >= 0 && t < V) m = fmaxf(m, fabsf(grad[i]));
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) m = fmaxf(m, sm[w]);
        *top = m > 0.f && m < INFINITY ? m : 1.f;
    }
}

template <class T>
__global__ __launch_bounds__(256) void k_xent_clear(T *p, int64_t ld, int64_t rows, int64_t D)
{
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < rows * D; c += step)
        p[c / D * ld + c % D] = (T)0.f;
}

struct XentPlan {
    float *target_logit, *top_grad;
    float2 *part;
    bf16 *h, *w;     // packed operands (nullptr: used in place)
    float *sum;
    bf16 *d;
    int64_t Kp, nr, piece;
    size_t bytes;
};

// `piece` columns of d (0: forward only).  Packed copies of the operands are
// planned whether or not an aligned bf16 operand needs them, so that the size
// does not depend on the pointers.
XentPlan plan_xent(int64_t n, int64_t V, int64_t D, int PL, int64_t piece, char *base)
{
    size_t off = TT_EMB_STATUS_BYTES;
    auto take = [&](size_t bytes) {
        char *r = base ? base + off : nullptr;
        off += round256(bytes > 0 ? bytes : 1);
        return r;
    };
    XentPlan p{};
    p.Kp = up(D, kTileK);
    p.nr = up(n, kTile);
    p.piece = piece;
    p.target_logit = (float *)take(4 * n);
    p.top_grad = (float *)take(4);
    p.part = (float2 *)take(8 * (size_t)n * ((V + kTile - 1) / kTile));
    p.h = (bf16 *)take((size_t)PL * n * p.Kp * 2);
    p.w = (bf16 *)take((size_t)PL * V * p.Kp * 2);
    if (piece) {
        p.sum = (float *)take(4 * (size_t)n * D);
        p.d = (bf16 *)take((size_t)PL * p.nr * piece * 2);
    }
    p.bytes = off;
    return p;
}

int64_t best_piece(int64_t V) { return up(V < kPiece ? V : kPiece, kTile); }

template <class T, int PL>
Operand operand(const T *src, int64_t ld, int64_t rows, int64_t D, bf16 *room, int64_t Kp, hipStream_t s)
{
    if constexpr (PL == 1) {
        if (D == Kp && ld % 8 == 0 && (reinterpret_cast<uintptr_t>(src) & 15u) == 0)
            return Operand{src, ld, 0, rows, D};
    }
    int64_t blocks = (rows * (Kp / 8) + 255) / 256;
    if (blocks > 65536) blocks = 65536;
    hipLaunchKernelGGL((k_pack<T, PL>), dim3((unsigned)blocks), dim3(256), 0, s, src, ld, rows, D, room, Kp,
                       rows * Kp);
    return Operand{room, Kp, rows * Kp, rows, Kp};
}

template <class T, int PL>
hipError_t xent(const XentArgs &a, bool grad, hipStream_t s)
{
    int64_t piece = grad ? best_piece(a.V) : 0;
    while (piece > kTile && plan_xent(a.n, a.V, a.D, PL, piece, nullptr).bytes > a.ws_bytes)
        piece = up(piece / 2, kTile);
    const XentPlan p = plan_xent(a.n, a.V, a.D, PL, piece, a.ws);
    const Operand h = operand<T, PL>(static_cast<const T *>(a.hidden), a.ld_h, a.n, a.D, p.h, p.Kp, s);
    const Operand w = operand<T, PL>(static_cast<const T *>(a.weight), a.ld_w, a.V, a.D, p.w, p.Kp, s);
    const unsigned nt = (unsigned)(p.nr / kTile);
    Output o{};
    o.n = a.n;
    o.V = a.V;
    o.D = a.D;
    o.targets = a.targets;
    o.ignore = a.ignore;
    o.part = p.part;
    o.target_logit = p.target_logit;
    o.lse = a.lse;
    o.grad = a.grad_loss;
    o.top_grad = p.top_grad;
    o.d = p.d;
    o.ldd = piece;
    o.plane_d = p.nr * piece;
    o.sum = p.sum;
    o.out_f32 = sizeof(T) == 4;
    const int64_t tiles = (a.V + kTile - 1) / kTile;
    hipLaunchKernelGGL((k_product<PL, false, false, OUT_STATS>), dim3((unsigned)tiles, nt), dim3(256), 0, s, w, h,
                       p.Kp, o);
    hipLaunchKernelGGL(k_xent_join, dim3((unsigned)((a.n + 15) / 16)), dim3(256), 0, s, p.part, tiles, a.n, a.V,
                       a.targets, a.ignore, p.target_logit, a.loss, a.lse, reinterpret_cast<int *>(a.ws));
    if (!grad) return hipGetLastError();
    hipLaunchKernelGGL(k_xent_top_grad, dim3(1), dim3(1024), 0, s, a.grad_loss, a.targets, a.ignore, a.n, a.V,
                       p.top_grad);
    const unsigned dt = (unsigned)((a.D + kTile - 1) / kTile);
    for (int64_t v0 = 0; v0 < a.V; v0 += piece) {
        const int64_t here = a.V - v0 < piece ? a.V - v0 : piece, cols = up(here, kTile);
        Operand wp = w;
        wp.p += v0 * w.ld;
        wp.rows = here;
        o.v0 = v0;
        o.first = v0 == 0;
        o.last = v0 + piece >= a.V;
        hipLaunchKernelGGL((k_product<PL, false, false, OUT_D>), dim3((unsigned)(cols / kTile), nt), dim3(256), 0, s,
                           wp, h, p.Kp, o);
        const Operand d{p.d, piece, p.nr * piece, p.nr, cols};
        o.out = a.dh;
        o.ld_out = a.ld_dh;
        hipLaunchKernelGGL((k_product<PL, true, false, OUT_HIDDEN>), dim3(dt, nt), dim3(256), 0, s, wp, d, cols, o);
        o.out = a.dw;
        o.ld_out = a.ld_dw;
        hipLaunchKernelGGL((k_product<PL, true, true, OUT_WEIGHT>), dim3(dt, (unsigned)(cols / kTile)), dim3(256), 0,
                           s, h, d, p.nr, o);
    }
    return hipGetLastError();
}

} // namespace

void xent_workspace(int64_t n, int64_t V, int64_t D, int dtype, bool grad, size_t *best, size_t *least)
{
    const int PL = dtype == TT_EMB_DTYPE_FLOAT ? 3 : 1;
    if (best) *best = plan_xent(n, V, D, PL, grad ? best_piece(V) : 0, nullptr).bytes;
    if (least) *least = plan_xent(n, V, D, PL, grad ? kTile : 0, nullptr).bytes;
}

hipError_t launch_xent_forward(const XentArgs &a, int dtype, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    return dtype == TT_EMB_DTYPE_FLOAT ? xent<float, 3>(a, false, s) : xent<bf16, 1>(a, false, s);
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
    return dtype == TT_EMB_DTYPE_FLOAT ? xent<float, 3>(a, true, s) : xent<bf16, 1>(a, true, s);
}

} // namespace ttemb
