// tiles.h -- products of matrices of 16-bit values by the matrix instructions:
// operands' tiles from memory to LDS, fragments, the order of a tile's steps and
// which compute unit takes which tile.
#pragma once

#include "lm.h"

namespace ttemb {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8))); // a fragment: eight bf16 or fp16 values
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// 32x32x16 matrix instructions of 16-bit values.
template <class E>
__device__ __forceinline__ f32x16 mma16(s16x8 a, s16x8 b, f32x16 c)
{
    if constexpr (std::is_same<E, bf16>::value)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// x as a sum of PL terms of 16 bits.  What makes x is kept out of the
// conversions: fused with a product, one of the two uses of a term rounded the
// exact product and the other the rounded one, and where they differ (one value
// in some thousand) the terms were off by a unit of the first.
template <class E, int PL>
__device__ __forceinline__ void split_terms(float x, short (&t)[PL])
{
    if constexpr (PL > 1) asm("" : "+v"(x));
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const E y = (E)x;
        t[i] = __builtin_bit_cast(short, y);
        x -= (float)y;
    }
}

// Summed values per stage and stages in LDS.  Straight rows of 64 bf16 are
// whole cache lines, and half the barriers; turned ones are lines anyway, and
// more and shorter stages leave their loads more time (8192 rows, K = 4096 and
// 8192: logits 7.24 ms with stages of 32, 6.86 of 64; the weight's gradient 770
// and 826 us a piece).  DEEP: three stages ahead, for grids that leave a compute
// unit one block of small tiles, where a stage's loads take longer than its products.
template <int PL, bool XT, bool DEEP = false>
struct Stages {
    static constexpr int values = PL == 1 && (DEEP || !XT) ? 64 : 32, buffers = DEEP || (PL == 1 && XT) ? 4 : 2;
};

// An operand of a product: PL matrices of 16-bit values.  Straight: row r holds
// the summed index.  Turned: row k of the summed index holds the outputs.
struct Operand {
    const short *p;
    int64_t ld, plane;  // elements between rows, between planes
    int64_t rows, cols; // of the stored matrix; what lies past them reads as zero
};

// How one plane of an operand's tile, R outputs and BK summed values, lies in
// LDS: rows of 16-byte pieces without gaps, as loads that go there directly
// write them.  Straight: R rows of BK values; turned: BK rows of R values.
// Which of a row's pieces change places (`turn`) is chosen so that the sixteen
// rows that sixteen lanes read lie in different banks (straight), and so do
// the four rows of 64 bytes that half a wave's transposing read touches.
template <bool TURNED, int R, int BK>
struct TileLds {
    static constexpr int pitch = (TURNED ? R : BK) * 2;
    static constexpr int bytes = R * BK * 2;
    static constexpr int vecs = R * BK / 8 / 256; // 16-byte pieces per thread
    static __device__ __forceinline__ int turn(int row)
    {
        if constexpr (TURNED) return R == 64 ? (row & 2) << 1 : (row & 3) << 2; // (rows of 64 have eight pieces)
        else return BK == 64 ? (row >> 1) & 7 : (row >> 2) & 3;
    }
};

typedef __attribute__((address_space(3))) void *lds_void;

// One operand's way from memory to LDS, without registers between: a wave's
// load fills 1 KB of LDS in the order of its lanes, so the pieces change places
// by the address that each lane reads.  Loads go through a buffer descriptor
// that ends with the matrix, so rows past it (of the outputs or of the summed
// index) are written as zeros and no address needs a clamp; so are stages past
// the last.  What a stage's descriptor takes is kept up by additions.
// ROT: the stages begin with `first` and go round.
template <bool TURNED, int R, int BK, int PL, bool ROT = false>
struct TileLoader {
    typedef TileLds<TURNED, R, BK> L;
    static constexpr int N = L::vecs, ROWV = L::pitch / 16; // pieces in a tile's row
    const short *p;     // plane 0, the next stage
    int64_t plane, next; // elements to the next plane, to the next stage
    int whole;          // stages to come that lie inside the matrix
    unsigned bytes, rest; // of those, of the one at the matrix's end (turned)
    int off;            // byte offset of this thread's first piece; the others are 256 / ROWV rows apart
    int step, to;       // to: the wave's place in LDS
    int at, all, todo;  // ROT: the next stage's number, of how many, stages to come (whole: those before the rest)

    __device__ __forceinline__ TileLoader(const Operand &a, int64_t r0, int stages, int first = 0)
    {
        const int ld = (int)a.ld;
        plane = a.plane;
        p = a.p + (TURNED ? r0 : r0 * a.ld);
        next = TURNED ? BK * a.ld : BK;
        if constexpr (TURNED) {
            const int64_t have = a.rows > 0 ? a.rows : 0; // (a part that begins past the rows has none)
            const int64_t full = have / BK;
            const int cols = (int)(a.cols - r0 < R ? a.cols - r0 : R), left = (int)(have - full * BK);
            whole = cols > 0 ? (int)(full < stages ? full : stages) : 0;
            bytes = (unsigned)((BK - 1) * ld + cols) * 2;
            rest = full < stages && left && cols > 0 ? (unsigned)((left - 1) * ld + cols) * 2 : 0;
        } else {
            const int rows = (int)(a.rows - r0 < R ? a.rows - r0 : R);
            whole = rows > 0 ? stages : 0; // (a tile of d's padding has none)
            bytes = (unsigned)((rows - 1) * ld + (int)a.cols) * 2;
            rest = 0;
        }
        const int t = threadIdx.x, row = t / ROWV;
        off = (row * ld + ((t % ROWV) ^ L::turn(row)) * 8) * 2;
        step = 256 / ROWV * ld * 2;
        to = __builtin_amdgcn_readfirstlane(t >> 6) * 1024;
        if constexpr (ROT) {
            at = first;
            all = todo = stages;
            p += first * next;
            if constexpr (!TURNED) bytes -= first * BK * 2;
        }
    }
    __device__ __forceinline__ void load(char *lds)
    {
        unsigned now;
        if constexpr (ROT) now = todo <= 0 ? 0 : at < whole ? bytes : at == whole ? rest : 0;
        else now = whole > 0 ? bytes : whole == 0 ? rest : 0;
#pragma unroll
        for (int q = 0; q < PL; ++q) {
            const __amdgpu_buffer_rsrc_t r =
                __builtin_amdgcn_make_buffer_rsrc(const_cast<short *>(p + q * plane), 0, now, 0x00027000);
#pragma unroll
            for (int i = 0; i < N; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void)(lds + q * L::bytes + i * 4096 + to), 16, off,
                                                         i * step, 0, 0);
        }
        p += next;
        if constexpr (!TURNED) bytes -= BK * 2;
        if constexpr (ROT) {
            --todo;
            if (++at == all) {
                at = 0;
                p -= all * next;
                if constexpr (!TURNED) bytes += all * BK * 2;
            }
        } else {
            --whole;
        }
    }
};

// Every wave's reads of LDS are done, and so are all but its last N loads.  A
// barrier of the language would wait for every load in flight; the fences here
// order the compiler's accesses and cost nothing.
template <int N>
__device__ __forceinline__ void loads_meet()
{
    static_assert(N < 64, "a counter of six bits");
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14); // lgkmcnt(0) vmcnt(N)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Fragments of N 32-row blocks from row `r0` of a tile, summed values
// [ks * 16, ks * 16 + 16): lane l gets row l % 32, values 8 (l / 32) .. + 7.
// A transposing read gives each of sixteen lanes one column of the four rows
// that the sixteen lanes' 8-byte addresses name.
template <bool TURNED, int R, int BK, int PL, int N>
__device__ __forceinline__ void fragments(const char *lds, int r0, int ks, s16x8 (&f)[PL][N])
{
    typedef TileLds<TURNED, R, BK> L;
    constexpr int P = L::pitch;
    const int l = threadIdx.x & 63, half = l >> 5;
    if constexpr (!TURNED) {
        const int at = (r0 + (l & 31)) * P + ((half ^ L::turn(l & 31)) * 16 ^ ks * 32);
#pragma unroll
        for (int q = 0; q < PL; ++q)
#pragma unroll
            for (int i = 0; i < N; ++i)
                f[q][i] = *reinterpret_cast<const s16x8 *>(lds + at + q * L::bytes + i * 32 * P);
    } else {
        const int row = half * 8 + ((l & 15) >> 2);
        const int at = row * P + ((r0 * 2 + ((l >> 4) & 1) * 32 + (l & 3) * 8) ^ L::turn(row) * 16);
#pragma unroll
        for (int q = 0; q < PL; ++q)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;
                const char *from = lds + q * L::bytes + ks * 16 * P + (at ^ i * 64);
                const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)from);
                const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(from + 4 * P));
                f[q][i] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
            }
    }
}

constexpr int kPatchM = 8, kPatchN = 4; // tiles that one XCD works on at a time

// Tile (and split of the sum) of block b of a grid.  Consecutive blocks go to the
// eight XCDs in turn.  Grids of many rounds: each XCD takes patches of kPatchM x
// kPatchN tiles (its 32 compute units) whose operands meet in its L2, and the
// patches that run at the same time lie along n, where they share the X operand
// in the memory-side cache.  Smaller grids: each XCD takes an eighth of the
// tiles in a row, split by split.
__host__ __device__ inline bool in_patches(int64_t mt, int64_t nt)
{
    return mt >= kPatchM && nt >= kPatchN && mt * nt >= 4 * kCUs;
}
__device__ __forceinline__ bool tile_of(int64_t b, int64_t grid, int64_t mt, int64_t nt, int splits, int64_t &m,
                                        int64_t &n, int &split)
{
    const int64_t local = b >> 3;
    split = 0;
    if (in_patches(mt, nt)) {
        constexpr int P = kPatchM * kPatchN;
        const int64_t patch = local / P * 8 + (b & 7), in = local % P;
        const int64_t pn = (nt + kPatchN - 1) / kPatchN;
        m = patch / pn * kPatchM + in % kPatchM;
        n = patch % pn * kPatchN + in / kPatchM;
        return m < mt && n < nt;
    }
    const int64_t id = (b & 7) * (grid >> 3) + local, t = id % (mt * nt);
    split = (int)(id / (mt * nt));
    m = t % mt;
    n = t / mt;
    return split < splits;
}
inline unsigned tile_grid(int64_t mt, int64_t nt, int splits)
{
    if (!in_patches(mt, nt)) return (unsigned)up(mt * nt * splits, 8);
    const int64_t patches = ((mt + kPatchM - 1) / kPatchM) * ((nt + kPatchN - 1) / kPatchN);
    return (unsigned)(up(patches, 8) * kPatchM * kPatchN);
}

// Order of a step's instructions: the reads of the next step's fragments two
// to a matrix instruction, so that they are there when that step begins; then
// loads, evenly: where they follow each other faster than the cache delivers,
// the wave waits at each.
template <int M, int READS, int LOADS>
__device__ __forceinline__ void interleave()
{
    constexpr int mfma = 0x008, vmem = 0x010, ds_read = 0x100;
    constexpr int by = (READS + 1) / 2 < M ? 2 : (READS + M - 1) / M, first = READS / by;
    constexpr int rest = M - first > 0 ? M - first : 1;
#pragma unroll
    for (int i = 0; i < M; ++i) {
        __builtin_amdgcn_sched_group_barrier(mfma, 1, 0);
        if (i < first) {
            __builtin_amdgcn_sched_group_barrier(ds_read, by, 0);
        } else {
            const int now = (i - first + 1) * LOADS / rest - (i - first) * LOADS / rest;
#pragma unroll
            for (int k = 0; k < now; ++k) __builtin_amdgcn_sched_group_barrier(vmem, 1, 0);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Columns from `j` on stay in the accumulator registers: read there all at
// once, behind the products, they would not fit the others and go to memory.
template <int NI, int NJ>
__device__ __forceinline__ void keep_columns(f32x16 (&acc)[NI][NJ], int j)
{
#pragma unroll
    for (int a = 0; a < NI; ++a)
#pragma unroll
        for (int i = 0; i < NJ; ++i)
            if (i >= j) asm volatile("" : "+a"(acc[a][i]));
}

// Products of terms, the small ones first: of two terms those above 2^-22 of
// the values' product, of three those above 2^-25.
template <int PL>
struct TermPairs {
    static constexpr int count = PL == 1 ? 1 : PL == 2 ? 3 : 6;
    static constexpr int a(int i) { return PL == 1 ? 0 : PL == 2 ? i == 0 : (0x001102 >> (4 * (i)) & 15); }
    static constexpr int b(int i) { return PL == 1 ? 0 : PL == 2 ? i == 1 : (0x010120 >> (4 * (i)) & 15); }
};

// acc[m][n] += sum_k X[m][k] Y[n][k] for a tile of (64 NI) x (64 NJ) whose
// operands the loaders bring: four waves, 32x32x16 matrix instructions, NI x NJ
// of them per wave.  Lane l of a wave holds column n = l % 32 and the rows m = 8
// (r / 4) + 4 (l / 32) + r % 4 of each, so the contiguous output index is m and
// the row of the output is n.
//
// Stages of both tiles go from memory to LDS buffers ahead of their use, and
// fragments are read one step of 16 ahead of the matrix instructions that use
// them; the one barrier per stage stands before products whose fragments are in
// registers by then, and the loads into the buffer that it frees begin behind
// it.  The buffers are the caller's variables and a round of the loop passes all
// of them, so that the compiler knows which one a load or a read means and does
// not wait for the others.
template <class E, int PL, bool XT, bool YT, bool DEEP = false, int NI, int NJ, class LoadX, class LoadY>
__device__ __forceinline__ void multiply(LoadX &x, LoadY &y, int stages, char *lds0, char *lds1, char *lds2, char *lds3,
                                         f32x16 (&acc)[NI][NJ])
{
    typedef TermPairs<PL> Pairs;
    constexpr int TM = 64 * NI, TN = 64 * NJ;
    constexpr int BK = Stages<PL, XT, DEEP>::values, NB = Stages<PL, XT, DEEP>::buffers;
    constexpr int XB = PL * TileLds<XT, TM, BK>::bytes;
    const int wave = threadIdx.x >> 6, wm = wave & 1, wn = wave >> 1;
    auto load_x = [&](char *to) { x.load(to); };
    auto load_y = [&](char *to) { y.load(to + XB); };
    // Three terms: the small products have sums of their own, so that the large ones'
    // are rounded once a step and not six times (sums of 4000 values: 6e-7 off, 1.7e-6
    // in one sum, in the same time).  256 x 128 tiles have no registers for them.
    constexpr bool APART = PL == 3 && NI * NJ <= 2;
    f32x16 low[APART ? NI : 1][APART ? NJ : 1];
    if constexpr (APART) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) low[i][j][r] = 0.f;
    }
    auto mma = [&](const s16x8 (&a)[NI], const s16x8 (&b)[NJ], bool small = false) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                f32x16 &to = APART && small ? low[APART ? i : 0][APART ? j : 0] : acc[i][j];
                to = mma16<E>(a[i], b[j], to);
            }
    };
    s16x8 a0[PL][NI], b0[PL][NJ], a1[PL][NI], b1[PL][NJ];
    const int rx = wm * (TM / 2), ry = wn * (TN / 2);
    // reads of a step's fragments, loads of a stage, matrix instructions of a product
    constexpr int RD = PL * (NI * (XT ? 2 : 1) + NJ * (YT ? 2 : 1)), MM = NI * NJ;
    constexpr int LX = PL * TileLds<XT, TM, BK>::vecs, LY = PL * TileLds<YT, TN, BK>::vecs;
    auto read = [&](const char *from, int ks, s16x8 (&a)[PL][NI], s16x8 (&b)[PL][NJ]) {
        fragments<XT, TM, BK, PL>(from, rx, ks, a);
        fragments<YT, TN, BK, PL>(from + XB, ry, ks, b);
    };
    // A buffer's loads begin behind the barrier that follows its last reads;
    // one term: X's there, Y's in the next stage's first step.
    auto stage = [&](char *last, char *here, char *next) {
        read(here, 1, a1, b1);
        if constexpr (PL == 1) {
            load_y(last);
            mma(a0[0], b0[0]);
            interleave<MM, RD, LY>();
            if constexpr (BK == 64) {
                read(here, 2, a0, b0);
                mma(a1[0], b1[0]);
                interleave<MM, RD, 0>();
                read(here, 3, a1, b1);
                mma(a0[0], b0[0]);
                interleave<MM, RD, 0>();
            }
        } else {
#pragma unroll
            for (int i = 0; i < Pairs::count; ++i) mma(a0[Pairs::a(i)], b0[Pairs::b(i)], i + 1 < Pairs::count);
            interleave<Pairs::count * MM, RD, 0>();
#pragma unroll
            for (int i = 0; i < PL - 1; ++i) mma(a1[Pairs::a(i)], b1[Pairs::b(i)], true);
        }
        __builtin_amdgcn_sched_barrier(0);
        loads_meet<(NB - 2) * (LX + LY)>(); // the next stage is there
        __builtin_amdgcn_sched_barrier(0);  // the last products stay behind the barrier
        read(next, 0, a0, b0);
        load_x(here);
        if constexpr (PL == 1) {
            mma(a1[0], b1[0]);
            interleave<MM, RD, LX>();
        } else {
            load_y(here);
#pragma unroll
            for (int i = PL - 1; i < Pairs::count; ++i)
                mma(a1[Pairs::a(i)], b1[Pairs::b(i)], i + 1 < Pairs::count);
            interleave<(Pairs::count - PL + 1) * MM, RD, LX + LY>();
        }
    };
    // all but the last buffer's Y, which the first stage asks for (one term)
    load_x(lds0);
    load_y(lds0);
    load_x(lds1);
    if constexpr (NB == 4 || PL > 1) load_y(lds1);
    if constexpr (NB == 4) {
        load_x(lds2);
        load_y(lds2);
        load_x(lds3);
        if constexpr (PL > 1) load_y(lds3);
    }
    loads_meet<(NB - 1) * (LX + LY) - (PL == 1 ? LY : 0)>();
    read(lds0, 0, a0, b0);
    for (int t = 0; t < stages; t += NB) { // (what the last round has too many are stages of zeros)
        if constexpr (NB == 4) {
            stage(lds3, lds0, lds1);
            stage(lds0, lds1, lds2);
            stage(lds1, lds2, lds3);
            stage(lds2, lds3, lds0);
        } else {
            stage(lds1, lds0, lds1);
            stage(lds0, lds1, lds0);
        }
    }
    loads_meet<0>(); // none is on its way into the buffers that the caller uses again
    if constexpr (APART) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] += low[i][j];
    }
}

} // namespace

} // namespace ttemb
