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
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileK = 64;             // summed index per stage
constexpr int kRowPitch = kTileK * 2 + 16; // bytes of a straight tile's row in LDS
constexpr int kTurnPad = 64;           // bytes past a turned tile's row in LDS
constexpr int kPatchM = 8, kPatchN = 4; // tiles that one XCD works on at a time
constexpr size_t kPieceBytes = (size_t)256 << 20; // d of one piece of the vocabulary, at most
constexpr int kSplitK = 1024;          // least summed values of a split of dH
constexpr int kRound = 256;            // rows and columns of d are padded to this

constexpr int kLeast = 128;             // rows and columns of the smallest tile

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
    float *sum;               // dH in fp32, [splits][n][D]
    int64_t split_k;          // summed values per split of dH
    void *out;                // dW
    int64_t ld_out, D;
    int first;                // dH's first piece
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

// How an operand's tile of R outputs and 64 summed values lies in LDS.
// Straight: R rows of 64 values, 144 bytes apart, so that the 16-byte reads of
// sixteen lanes (sixteen rows) meet different banks.  Turned: 64 rows of R
// values and 64 bytes, so that the four rows of 64 bytes that half a wave's
// transposing read touches do.
template <bool TURNED, int R>
struct TileLds {
    static constexpr int pitch = TURNED ? R * 2 + kTurnPad : kRowPitch;
    static constexpr int bytes = TURNED ? kTileK * pitch : R * pitch;
    static constexpr int vecs = R * kTileK / 8 / 256; // 16-byte pieces per thread
};

// One operand's way from memory to registers to LDS.  Loads go through a
// buffer descriptor that ends with the matrix, so rows past it (of the outputs
// or of the summed index) read as zeros and no address needs a clamp.
template <bool TURNED, int R>
struct TileLoader {
    static constexpr int N = TileLds<TURNED, R>::vecs;
    static constexpr int ROWV = TURNED ? R / 8 : kTileK / 8; // pieces in a tile's row
    const bf16 *p;  // plane 0, moved to the tile's first row (straight) or column (turned)
    int64_t ld, plane, end; // end: elements from p to the end of plane 0
    int off;        // byte offset of this thread's first piece; the others are 256 / ROWV rows apart
    int step;
    u32x4 v[N];

    __device__ __forceinline__ TileLoader(const Operand &a, int64_t r0)
    {
        ld = a.ld;
        plane = a.plane;
        p = a.p + (TURNED ? r0 : r0 * a.ld);
        end = (a.rows - 1) * a.ld + a.cols - (TURNED ? r0 : r0 * a.ld);
        const int t = threadIdx.x;
        off = ((t / ROWV) * (int)ld + (t % ROWV) * 8) * 2;
        step = 256 / ROWV * (int)ld * 2;
    }
    __device__ __forceinline__ void load(int pl, int64_t k0)
    {
        const int64_t skip = TURNED ? k0 * ld : k0;
        const int64_t left = (end - skip) * 2;
        const unsigned bytes = left > 0x7fffffff ? 0x7fffffffu : left < 0 ? 0u : (unsigned)left;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<bf16 *>(p + pl * plane + skip), 0, bytes, 0x00027000);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b128(r, off, i * step, 0);
    }
    __device__ __forceinline__ void store(char *lds) const
    {
        const int t = threadIdx.x;
        constexpr int P = TileLds<TURNED, R>::pitch;
        char *q = lds + (t / ROWV) * P + (t % ROWV) * 16;
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4 *>(q + i * (256 / ROWV) * P) = v[i];
    }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Fragments of N 32-row blocks from row `r0` of a tile, summed values
// [ks * 16, ks * 16 + 16): lane l gets row l % 32, values 8 (l / 32) .. + 7.
// A transposing read gives each of sixteen lanes one column of the four rows
// that the sixteen lanes' 8-byte addresses name.
template <bool TURNED, int R, int N>
__device__ __forceinline__ void fragments(const char *lds, int r0, int ks, bf16x8 (&f)[N])
{
    const int l = threadIdx.x & 63;
    if constexpr (!TURNED) {
        const char *q = lds + (r0 + (l & 31)) * kRowPitch + ks * 32 + (l >> 5) * 16;
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = *reinterpret_cast<const bf16x8 *>(q + i * 32 * kRowPitch);
    } else {
        constexpr int P = TileLds<TURNED, R>::pitch;
        const char *q = lds + (ks * 16 + (l >> 5) * 8 + ((l & 15) >> 2)) * P +
                        (r0 + ((l >> 4) & 1) * 16 + (l & 3) * 4) * 2;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(q + i * 64));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(q + i * 64 + 4 * P));
            f[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
}

// Tile of a thread block: consecutive blocks go to the eight XCDs in turn, so
// each XCD takes patches of kPatchM x kPatchN tiles (its 32 compute units) whose
// operands meet in its L2, and the patches that run at the same time lie along
// n, where they share the X operand in the memory-side cache.
__device__ __forceinline__ bool tile_of(int64_t mt, int64_t nt, int64_t &m, int64_t &n)
{
    constexpr int P = kPatchM * kPatchN;
    const int64_t b = blockIdx.x, local = b >> 3;
    const int64_t patch = local / P * 8 + (b & 7), in = local % P;
    const int64_t pn = (nt + kPatchN - 1) / kPatchN;
    m = patch / pn * kPatchM + in % kPatchM;
    n = patch % pn * kPatchN + in / kPatchM;
    return m < mt && n < nt;
}
inline unsigned tile_grid(int64_t mt, int64_t nt)
{
    const int64_t patches = ((mt + kPatchM - 1) / kPatchM) * ((nt + kPatchN - 1) / kPatchN);
    return (unsigned)(up(patches, 8) * kPatchM * kPatchN);
}

// Order of a step's instructions: the reads of the next step's fragments two
// to a matrix instruction, so that they are there when that step begins; then
// the stores of a stage's pieces to LDS, each followed by the load of the same
// piece of a later stage (a whole stage ahead of its use).
template <int M, int READS, int PIECES>
__device__ __forceinline__ void interleave()
{
    constexpr int mfma = 0x008, vmem_read = 0x020, ds_read = 0x100, ds_write = 0x200;
    constexpr int by = (READS + 1) / 2 < M ? 2 : (READS + M - 1) / M, first = READS / by;
    constexpr int rest = M - first > 0 ? M - first : 1, each = (PIECES + rest - 1) / rest;
#pragma unroll
    for (int i = 0; i < M; ++i) {
        __builtin_amdgcn_sched_group_barrier(mfma, 1, 0);
        if (i < first) __builtin_amdgcn_sched_group_barrier(ds_read, by, 0);
        else if (PIECES) {
            __builtin_amdgcn_sched_group_barrier(ds_write, each, 0);
            __builtin_amdgcn_sched_group_barrier(vmem_read, each, 0);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
}

// C[m][n] = sum_k X[m][k] Y[n][k] over tiles of (64 NI) x (64 NJ); four waves,
// 32x32x16 matrix instructions, NI x NJ of them per wave.  Lane l of a wave
// holds column n = l % 32 and the rows m = 8 (r / 4) + 4 (l / 32) + r % 4 of
// each, so the contiguous output index is m and the row of the output is n.
//
// Tiles go from memory to registers a stage ahead and from there to one of two
// LDS buffers, and fragments are read one step of 16 ahead of the matrix
// instructions that use them; the one barrier per stage stands before its last
// step, whose fragments are in registers by then.
template <int PL, bool XT, bool YT, int OUT, int NI, int NJ>
__global__ __launch_bounds__(256, 1) void k_product(Operand X, Operand Y, int64_t K, int64_t mt, int64_t nt, Output o)
{
    constexpr int TM = 64 * NI, TN = 64 * NJ;
    constexpr int XB = TileLds<XT, TM>::bytes, YB = TileLds<YT, TN>::bytes, STAGE = XB + YB;
    __shared__ __align__(16) char lds[2 * STAGE];
    int64_t mi, ni;
    if (!tile_of(mt, nt, mi, ni)) return;
    if constexpr (OUT == OUT_HIDDEN) { // this split's part of the sum
        const int64_t k0 = blockIdx.y * o.split_k;
        if (k0 >= K) return;
        X.p += k0 * X.ld;
        X.rows -= k0;
        Y.p += k0;
        K = K - k0 < o.split_k ? K - k0 : o.split_k;
        o.sum += blockIdx.y * o.n * o.D;
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
        TileLoader<XT, TM> x(X, m0);
        TileLoader<YT, TN> y(Y, n0);
        // products of terms, the small ones first
        constexpr int SEG = PL == 1 ? 1 : 6;
        const int per = (int)(K / kTileK), stages = SEG * per;
        int seg = 0, in = 0; // of the next stage to load; the last one is loaded again past the end
        // planes (2,0) (0,2) (1,1) (1,0) (0,1) (0,0), two bits each
        auto load_x = [&]() { x.load(PL == 1 ? 0 : (0x052 >> (2 * seg)) & 3, (int64_t)in * kTileK); };
        auto load_y = [&]() {
            y.load(PL == 1 ? 0 : (0x118 >> (2 * seg)) & 3, (int64_t)in * kTileK);
            const bool over = in + 1 == per, more = !over || seg + 1 < SEG;
            seg += over && more;
            in = over ? (more ? 0 : in) : in + 1;
        };
        auto mma = [&](const bf16x8 (&a)[NI], const bf16x8 (&b)[NJ]) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
        };
        load_x();
        load_y();
        x.store(lds);
        y.store(lds + XB);
        load_x();
        load_y();
        __syncthreads();
        bf16x8 a0[NI], b0[NJ], a1[NI], b1[NJ];
        const int rx = wm * (TM / 2), ry = wn * (TN / 2);
        fragments<XT, TM>(lds, rx, 0, a0);
        fragments<YT, TN>(lds + XB, ry, 0, b0);
        // reads of a step's fragments, pieces of an operand moved, matrix instructions of a step
        constexpr int RD = NI * (XT ? 2 : 1) + NJ * (YT ? 2 : 1), XV = TM / 32, YV = TN / 32, MM = NI * NJ;
        int cur = 0;
        for (int t = 0; t < stages; ++t) {
            const char *here = lds + cur;
            char *next = lds + (STAGE - cur);
            fragments<XT, TM>(here, rx, 1, a1);
            fragments<YT, TN>(here + XB, ry, 1, b1);
            x.store(next);
            load_x();
            mma(a0, b0);
            interleave<MM, RD, XV>();
            fragments<XT, TM>(here, rx, 2, a0);
            fragments<YT, TN>(here + XB, ry, 2, b0);
            y.store(next + XB);
            load_y();
            mma(a1, b1);
            interleave<MM, RD, YV>();
            fragments<XT, TM>(here, rx, 3, a1);
            fragments<YT, TN>(here + XB, ry, 3, b1);
            mma(a0, b0);
            interleave<MM, RD, 0>();
            __syncthreads();
            __builtin_amdgcn_sched_barrier(0); // the last step's products stay behind the barrier
            fragments<XT, TM>(next, rx, 0, a0);
            fragments<YT, TN>(next + XB, ry, 0, b0);
            mma(a1, b1);
            interleave<MM, RD, 0>();
            cur = STAGE - cur;
        }
    }
    auto row_of = [&](int i, int r) { return wm * (TM / 2) + i * 32 + 8 * (r / 4) + 4 * (lane >> 5) + (r % 4); };
    if constexpr (OUT == OUT_STATS) {
        float(*red)[2][TN] = reinterpret_cast<float(*)[2][TN]>(lds);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int nl = wn * (TN / 2) + j * 32 + (lane & 31);
            const int64_t i = n0 + nl;
            const int64_t t = i < o.n ? o.targets[i] - m0 : -1;
            const int64_t left = o.V - m0;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int a = 0; a < NI; ++a)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int v = row_of(a, r);
                    if (v >= left) acc[a][j][r] = -INFINITY;
                    top = fmaxf(top, acc[a][j][r]);
                    if (v == t) o.target_logit[i] = acc[a][j][r];
                }
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int a = 0; a < NI; ++a)
#pragma unroll
                for (int r = 0; r < 16; ++r) sum += __expf(acc[a][j][r] - ref);
            sum += __shfl_xor(sum, 32, 64);
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
        const float scale = *o.top_grad;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int64_t i = n0 + wn * (TN / 2) + j * 32 + (lane & 31);
            float lse = 0.f, g = 0.f;
            int64_t t = -1;
            if constexpr (OUT == OUT_D) {
                if (i < o.n) {
                    t = o.targets[i] - o.v0;
                    const bool counts = o.targets[i] != o.ignore && o.targets[i] >= 0 && o.targets[i] < o.V;
                    g = counts ? o.grad[i] / scale : 0.f;
                    lse = o.lse[i];
                }
            }
#pragma unroll
            for (int a = 0; a < NI; ++a)
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
                    } else {
                        const int left = (int)(o.D - m < 4 ? o.D - m : 4);
                        if (left <= 0) continue;
                        const int64_t row = o.v0 + i;
                        if constexpr (OUT == OUT_HIDDEN) {
                            if (i >= o.n) continue;
                            float *s = o.sum + i * o.D + m;
                            if (!o.first) {
                                float old[4];
                                load_part<float, 4>(s, left, old);
#pragma unroll
                                for (int r = 0; r < 4; ++r) x[r] += old[r];
                            }
                            store_part<float, 4>(s, left, x);
                            continue;
                        }
                        if (row >= o.V) continue;
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] *= scale;
                        if (PL > 1) store_part<float, 4>(static_cast<float *>(o.out) + row * o.ld_out + m, left, x);
                        else store_part<bf16, 4>(static_cast<bf16 *>(o.out) + row * o.ld_out + m, left, x);
                    }
                }
        }
    }
}

// dH from the splits' sums, in order, in units of the loss.
template <class T>
__global__ __launch_bounds__(256) void k_xent_hidden(const float *sum, int splits, int64_t n, int64_t D,
                                                     const float *top_grad, T *out, int64_t ld)
{
    const int64_t chunks = (D + 3) / 4, step = (int64_t)gridDim.x * 256;
    const float scale = *top_grad;
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < n * chunks; c += step) {
        const int64_t i = c / chunks, k = (c - i * chunks) * 4;
        const int left = (int)(D - k < 4 ? D - k : 4);
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        for (int q = 0; q < splits; ++q) {
            float y[4];
            load_part<float, 4>(sum + ((int64_t)q * n + i) * D + k, left, y);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] += y[r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] *= scale;
        store_part<T, 4>(out + i * ld + k, left, x);
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
    int splits;
    size_t bytes;
};

// Rows and columns of a product's tile, and how often dH's sum over a piece of
// the vocabulary is split: its output is small (n x D) beside what it adds up,
// so where its tiles are fewer than the compute units the sum is shared out.
inline int64_t tile_side(int64_t size) { return size <= 128 ? 128 : 256; }
int hidden_splits(int64_t n, int64_t D, int64_t piece)
{
    const int64_t tm = tile_side(D), tn = tile_side(n);
    const int64_t tiles = ((D + tm - 1) / tm) * ((n + tn - 1) / tn);
    int64_t s = kCUs / tiles;
    if (s > piece / kSplitK) s = piece / kSplitK;
    return (int)(s < 1 ? 1 : s);
}

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
    p.nr = up(n, kRound);
    p.piece = piece;
    p.target_logit = (float *)take(4 * n);
    p.top_grad = (float *)take(4);
    p.part = (float2 *)take(8 * (size_t)n * ((V + kLeast - 1) / kLeast));
    p.h = (bf16 *)take((size_t)PL * n * p.Kp * 2);
    p.w = (bf16 *)take((size_t)PL * V * p.Kp * 2);
    if (piece) {
        p.splits = hidden_splits(n, D, piece);
        p.sum = (float *)take(4 * (size_t)p.splits * n * D);
        p.d = (bf16 *)take((size_t)PL * p.nr * piece * 2);
    }
    p.bytes = off;
    return p;
}

int64_t best_piece(int64_t n, int64_t V, int PL)
{
    int64_t c = (int64_t)(kPieceBytes / ((size_t)PL * up(n, kRound) * 2)) / kRound * kRound;
    if (c < 8 * kRound) c = 8 * kRound;
    return up(V < c ? V : c, kRound);
}

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

// A product with M contiguous outputs in each of N rows; returns the tiles
// along M.  256 x 256 tiles read each operand least often; a side of at most
// 128 takes half of that, and where the tiles would leave compute units idle
// 128 x 128 ones spread the work further.
template <int PL, bool XT, bool YT, int OUT>
int64_t product(const Operand &x, const Operand &y, int64_t M, int64_t N, int64_t K, const Output &o, hipStream_t s,
                int splits = 1)
{
    const int64_t tm = tile_side(M), tn = tile_side(N);
    int64_t mt = (M + tm - 1) / tm, nt = (N + tn - 1) / tn;
    const bool small = mt * nt * splits < kCUs;
    if (small) {
        mt = (M + 127) / 128;
        nt = (N + 127) / 128;
    }
    const dim3 grid(tile_grid(mt, nt), (unsigned)splits);
    auto go = [&](auto i, auto j) {
        constexpr int NI = decltype(i)::value, NJ = decltype(j)::value;
        hipLaunchKernelGGL((k_product<PL, XT, YT, OUT, NI, NJ>), grid, dim3(256), 0, s, x, y, K, mt, nt, o);
    };
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 4> four;
    if (!small && tm == 256 && tn == 256) go(four, four);
    else if (!small && tm == 256) go(four, two);
    else if (!small && tn == 256) go(two, four);
    else go(two, two);
    return mt;
}

template <class T, int PL>
hipError_t xent(const XentArgs &a, bool grad, hipStream_t s)
{
    int64_t piece = grad ? best_piece(a.n, a.V, PL) : 0;
    while (piece > kRound && plan_xent(a.n, a.V, a.D, PL, piece, nullptr).bytes > a.ws_bytes)
        piece = up(piece / 2, kRound);
    const XentPlan p = plan_xent(a.n, a.V, a.D, PL, piece, a.ws);
    const Operand h = operand<T, PL>(static_cast<const T *>(a.hidden), a.ld_h, a.n, a.D, p.h, p.Kp, s);
    const Operand w = operand<T, PL>(static_cast<const T *>(a.weight), a.ld_w, a.V, a.D, p.w, p.Kp, s);
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
    const int64_t tiles = product<PL, false, false, OUT_STATS>(w, h, a.V, a.n, p.Kp, o, s);
    hipLaunchKernelGGL(k_xent_join, dim3((unsigned)((a.n + 15) / 16)), dim3(256), 0, s, p.part, tiles, a.n, a.V,
                       a.targets, a.ignore, p.target_logit, a.loss, a.lse, reinterpret_cast<int *>(a.ws));
    if (!grad) return hipGetLastError();
    hipLaunchKernelGGL(k_xent_top_grad, dim3(1), dim3(1024), 0, s, a.grad_loss, a.targets, a.ignore, a.n, a.V,
                       p.top_grad);
    for (int64_t v0 = 0; v0 < a.V; v0 += piece) {
        const int64_t here = a.V - v0 < piece ? a.V - v0 : piece, cols = up(here, kRound);
        Operand wp = w;
        wp.p += v0 * w.ld;
        wp.rows = here;
        o.v0 = v0;
        o.first = v0 == 0;
        // d of whole 256 x 256 blocks: what lies past the rows and the vocabulary is written as zeros
        product<PL, false, false, OUT_D>(wp, h, cols, p.nr, p.Kp, o, s);
        const Operand d{p.d, piece, p.nr * piece, p.nr, cols};
        o.split_k = up((cols + p.splits - 1) / p.splits, kTileK);
        product<PL, true, false, OUT_HIDDEN>(wp, d, a.D, a.n, cols, o, s, p.splits);
        o.out = a.dw;
        o.ld_out = a.ld_dw;
        product<PL, true, true, OUT_WEIGHT>(h, d, a.D, here, p.nr, o, s);
    }
    // splits past the first piece's end have written nothing
    const int64_t first = up(a.V < piece ? a.V : piece, kRound);
    const int64_t per = up((first + p.splits - 1) / p.splits, kTileK);
    int64_t blocks = (a.n * ((a.D + 3) / 4) + 255) / 256;
    if (blocks > 65536) blocks = 65536;
    hipLaunchKernelGGL(k_xent_hidden<T>, dim3((unsigned)blocks), dim3(256), 0, s, p.sum, (int)((first + per - 1) / per),
                       a.n, a.D, p.top_grad, static_cast<T *>(a.dh), a.ld_dh);
    return hipGetLastError();
}

} // namespace

void xent_workspace(int64_t n, int64_t V, int64_t D, int dtype, bool grad, size_t *best, size_t *least)
{
    const int PL = dtype == TT_EMB_DTYPE_FLOAT ? 3 : 1;
    if (n < 1) n = 1; // no rows: the least workspace
    if (best) *best = plan_xent(n, V, D, PL, grad ? best_piece(n, V, PL) : 0, nullptr).bytes;
    if (least) *least = plan_xent(n, V, D, PL, grad ? kRound : 0, nullptr).bytes;
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
