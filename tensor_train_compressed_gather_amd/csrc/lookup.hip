// lookup.hip -- rows of a dense table for token ids, and the gradient of the
// table summed by sorted tokens (gfx950).
//
// Both are copies of rows: a row (or a piece of a long one) belongs to LPR
// neighbouring lanes of NV 16-byte vectors each.  The gradient is not
// scattered with atomics, whose order would change the result: positions are
// sorted stably by token, fixed tiles of the sorted positions are summed by
// one worker each, and only runs of one token that cover a whole tile are cut
// and joined by a second kernel in a fixed order.
//
// Memory bounds the large sizes: 65536 tokens of 131072 x 1024 bf16 in 47 us
// (268 MB), their gradient in 135 us, of which 92 are the sums and the rows of
// zeros (402 MB), 28 the sort, 14 the joins.  32768 tokens of 64 fp32 columns
// are bound by the chain of six dependent launches: 5 us and 43.
#include "lm.h"
#include "primitives.h"

namespace ttemb {

namespace {

constexpr int kSumBatch = 8;       // gradient rows a worker has in flight
constexpr int kSumTile = 8;        // sorted positions per worker, at least
constexpr int64_t kSumTiles = 8192; // workers per row piece, at most
constexpr int kJoinGroups = 16;    // waves of a joining block
constexpr int64_t kMaxGrid = 1 << 20; // blocks of the forward, which walks over rows past them
constexpr int kTokThreads = 512, kTokItems = 4, kTokTile = kTokThreads * kTokItems; // token sort
constexpr int kTokBits = 10, kTokDigits = 1 << kTokBits;
constexpr int64_t kTokSortMax = 131072; // tokens that the token sort takes

// Lanes per row (piece) and vectors per lane for rows of D elements: the
// whole row where 64 lanes of two vectors hold it, pieces of that size else.
template <class T, class F>
hipError_t row_shape(int64_t D, F &&f)
{
    const int64_t nv = (D * (int64_t)sizeof(T) + 15) / 16;
    if (nv <= 8) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
    if (nv <= 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
    if (nv <= 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
    if (nv <= 64) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
    return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
}

template <class T, int LPR, int NV>
__global__ __launch_bounds__(256) void k_lookup(LookupArgs a, int pieces)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    const int lane = threadIdx.x % LPR;
    const int64_t step = (int64_t)gridDim.x * 256 / LPR;
    for (int64_t w = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPR; w < a.n * pieces; w += step) {
        const int64_t i = w / pieces;
        const int64_t c0 = (w - i * pieces) * (LPR * NV * VEC) + lane * VEC;
        const int64_t tok = a.tokens[i];
        const bool ok = tok >= 0 && tok < a.V;
        if (!ok && lane == 0) atomicOr(reinterpret_cast<int *>(a.ws) + ST_ERR, (int)STB_INDEX);
        const T *src = static_cast<const T *>(a.src) + (ok ? tok : 0) * a.ld_src;
        T *dst = static_cast<T *>(a.dst) + i * a.ld_dst;
        float x[NV][VEC];
        int left[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = c0 + (int64_t)j * LPR * VEC, l = a.D - c;
            left[j] = l < VEC ? (int)(l < 0 ? 0 : l) : VEC;
            load_part<T, VEC>(src + (left[j] ? c : 0), left[j], x[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = c0 + (int64_t)j * LPR * VEC;
#pragma unroll
            for (int k = 0; k < VEC; ++k) x[j][k] = ok ? x[j][k] * a.scale : 0.f;
            if (left[j]) store_part<T, VEC>(dst + c, left[j], x[j]);
        }
    }
}

// Sort key of every position: its token, or V (sorted last, never summed) for
// padding and for tokens out of range.
__device__ __forceinline__ uint32_t token_key(const LookupArgs &a, int64_t i)
{
    const int64_t t = a.tokens[i];
    const bool pad = a.pad >= 0 && t == a.pad, ok = t >= 0 && t < a.V;
    if (!ok && !pad) atomicOr(reinterpret_cast<int *>(a.ws) + ST_ERR, (int)STB_INDEX);
    return ok && !pad ? (uint32_t)t : (uint32_t)a.V;
}

__global__ __launch_bounds__(256) void k_lookup_keys(LookupArgs a, uint32_t *key, int32_t *val)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.n) return;
    key[i] = token_key(a, i);
    val[i] = (int32_t)i;
}

// ------------------------------------------------------------- token sort
//
// Stable LSD radix sort of up to kTokSortMax tokens in few launches, which is
// what bounds so small a sort: digits of up to ten bits (two passes for
// vocabularies below 2^20), every tile's block adding up the other tiles'
// digit counts itself instead of a scan between two kernels (32768 tokens: 25 us
// in four launches; tiles of 1024 take the same, of 512 longer).  One tile is
// sorted in LDS by one launch.
struct RankLds {
    uint16_t wave[kTokThreads / 64][kTokDigits];
    uint32_t start[kTokDigits];
    uint32_t part[kTokThreads / 64];
};

// Exclusive scan of two values per thread (digits 2 tid and 2 tid + 1).
__device__ __forceinline__ void scan_digits(uint32_t *part, uint32_t a, uint32_t b, uint32_t &ea, uint32_t &eb)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const uint32_t x = wave_inclusive_scan(a + b);
    if (lane == 63) part[w] = x;
    __syncthreads();
    uint32_t pre = 0;
#pragma unroll
    for (int i = 0; i < kTokThreads / 64; ++i) pre += i < w ? part[i] : 0;
    ea = pre + x - a - b;
    eb = ea + a;
    __syncthreads();
}

// Place of every key of the tile among the tile's keys in stable order of the
// digit; lds.start then holds the digits' first places.
__device__ __forceinline__ void tile_rank(RankLds &lds, const uint32_t (&digit)[kTokItems],
                                          const bool (&valid)[kTokItems], int bits, uint32_t (&place)[kTokItems])
{
    constexpr int W = kTokThreads / 64;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    for (int i = tid; i < W * kTokDigits / 2; i += kTokThreads) reinterpret_cast<uint32_t *>(&lds.wave[0][0])[i] = 0;
    __syncthreads();
    const uint64_t lt = (1ull << lane) - 1ull;
#pragma unroll
    for (int r = 0; r < kTokItems; ++r) {
        uint64_t m = __ballot(valid[r]);
        for (int b = 0; b < bits; ++b) {
            const bool bit = (digit[r] >> b) & 1u;
            const uint64_t bb = __ballot(bit);
            m &= bit ? bb : ~bb;
        }
        const uint32_t below = (uint32_t)__popcll(m & lt);
        const uint32_t prior = lds.wave[w][digit[r]];
        __builtin_amdgcn_wave_barrier();
        if (valid[r] && below == 0) lds.wave[w][digit[r]] = (uint16_t)(prior + (uint32_t)__popcll(m));
        __builtin_amdgcn_wave_barrier();
        place[r] = prior + below;
    }
    __syncthreads();
    uint32_t tot[2] = {0, 0}; // of digits 2 tid and 2 tid + 1
#pragma unroll
    for (int i = 0; i < W; ++i) {
        uint32_t *c = reinterpret_cast<uint32_t *>(&lds.wave[i][0]) + tid;
        const uint32_t v = *c;
        *c = tot[0] | (tot[1] << 16);
        tot[0] += v & 0xFFFFu;
        tot[1] += v >> 16;
    }
    uint32_t e0, e1;
    scan_digits(lds.part, tot[0], tot[1], e0, e1);
    lds.start[2 * tid] = e0;
    lds.start[2 * tid + 1] = e1;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kTokItems; ++r) place[r] += lds.start[digit[r]] + lds.wave[w][digit[r]];
}

// Position of item r of this thread in the tile: each wave has 256 positions in a row.
__device__ __forceinline__ int tile_item(int r)
{
    return (threadIdx.x >> 6) * (64 * kTokItems) + r * 64 + (threadIdx.x & 63);
}

// All of at most kTokTile tokens by one block.
__global__ __launch_bounds__(kTokThreads) void k_token_sort(LookupArgs a, int bits, uint32_t *key_out,
                                                            int32_t *val_out)
{
    __shared__ RankLds lds;
    __shared__ uint32_t skey[kTokTile];
    __shared__ uint16_t sval[kTokTile];
    const int n = (int)a.n;
    uint32_t key[kTokItems], val[kTokItems];
#pragma unroll
    for (int r = 0; r < kTokItems; ++r) {
        const int i = tile_item(r);
        key[r] = i < n ? token_key(a, i) : 0;
        val[r] = (uint32_t)i;
    }
    const int passes = (bits + kTokBits - 1) / kTokBits, wd = (bits + passes - 1) / passes;
    for (int pass = 0; pass < passes; ++pass) {
        uint32_t digit[kTokItems], place[kTokItems];
        bool valid[kTokItems];
        if (pass) {
#pragma unroll
            for (int r = 0; r < kTokItems; ++r) {
                const int i = tile_item(r);
                key[r] = i < n ? skey[i] : 0;
                val[r] = i < n ? sval[i] : 0;
            }
        }
#pragma unroll
        for (int r = 0; r < kTokItems; ++r) {
            valid[r] = tile_item(r) < n;
            digit[r] = (key[r] >> (pass * wd)) & ((1u << wd) - 1u);
        }
        tile_rank(lds, digit, valid, wd, place); // its barriers stand between the reads above and the writes below
#pragma unroll
        for (int r = 0; r < kTokItems; ++r)
            if (valid[r]) {
                skey[place[r]] = key[r];
                sval[place[r]] = (uint16_t)val[r];
            }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < n; i += kTokThreads) {
        key_out[i] = skey[i];
        val_out[i] = sval[i];
    }
}

// Digit counts of each tile.  FIRST: keys are made from the tokens.
template <bool FIRST>
__global__ __launch_bounds__(kTokThreads) void k_token_count(LookupArgs a, const uint32_t *key, int shift, int wd,
                                                             uint32_t *count)
{
    __shared__ uint32_t cnt[kTokDigits];
    uint32_t digit[kTokItems];
    bool valid[kTokItems];
#pragma unroll
    for (int r = 0; r < kTokItems; ++r) {
        const int64_t i = (int64_t)blockIdx.x * kTokTile + tile_item(r);
        valid[r] = i < a.n;
        const int64_t ic = valid[r] ? i : a.n - 1;
        digit[r] = ((FIRST ? token_key(a, ic) : key[ic]) >> shift) & ((1u << wd) - 1u);
    }
    for (int d = threadIdx.x; d < kTokDigits; d += kTokThreads) cnt[d] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kTokItems; ++r)
        if (valid[r]) atomicAdd(&cnt[digit[r]], 1u);
    __syncthreads();
    for (int d = threadIdx.x; d < kTokDigits; d += kTokThreads)
        count[(int64_t)blockIdx.x * kTokDigits + d] = cnt[d];
}

// One pass: the tile's keys to their places.
template <bool FIRST>
__global__ __launch_bounds__(kTokThreads) void k_token_place(LookupArgs a, const uint32_t *key_in,
                                                             const int32_t *val_in, uint32_t *key_out,
                                                             int32_t *val_out, int shift, int wd,
                                                             const uint32_t *count)
{
    __shared__ RankLds lds;
    __shared__ uint32_t base[kTokDigits];
    const int tiles = gridDim.x, tile = blockIdx.x, tid = threadIdx.x;
    const uint32_t mask = (1u << wd) - 1u;
    uint32_t key[kTokItems], digit[kTokItems], place[kTokItems];
    int32_t val[kTokItems];
    bool valid[kTokItems];
#pragma unroll
    for (int r = 0; r < kTokItems; ++r) {
        const int64_t i = (int64_t)tile * kTokTile + tile_item(r);
        valid[r] = i < a.n;
        const int64_t ic = valid[r] ? i : a.n - 1;
        key[r] = FIRST ? token_key(a, ic) : key_in[ic];
        val[r] = FIRST ? (int32_t)i : val_in[ic];
        digit[r] = (key[r] >> shift) & mask;
    }
    uint32_t tot[2] = {0, 0}, before[2] = {0, 0}; // digits 2 tid, 2 tid + 1: of all tiles, of those before
#pragma unroll 8
    for (int q = 0; q < tiles; ++q) {
        const uint2 c = *reinterpret_cast<const uint2 *>(count + (int64_t)q * kTokDigits + 2 * tid);
        tot[0] += c.x;
        tot[1] += c.y;
        before[0] += q < tile ? c.x : 0;
        before[1] += q < tile ? c.y : 0;
    }
    uint32_t e0, e1;
    scan_digits(lds.part, tot[0], tot[1], e0, e1);
    base[2 * tid] = e0 + before[0];
    base[2 * tid + 1] = e1 + before[1];
    tile_rank(lds, digit, valid, wd, place);
#pragma unroll
    for (int r = 0; r < kTokItems; ++r) {
        if (!valid[r]) continue;
        const uint32_t to = base[digit[r]] + place[r] - lds.start[digit[r]];
        key_out[to] = key[r];
        val_out[to] = val[r];
    }
}

// The run of equal keys across a tile's edge is cut there when it covers a
// whole tile next to the edge.  Shorter runs belong to the worker of the tile
// they begin in, which reads past its end (by less than a tile).

template <class T, int VEC, int NV>
__device__ __forceinline__ void add_row_out(const LookupArgs &a, int64_t v, const int64_t (&c)[NV],
                                            const int (&left)[NV], const float (&acc)[NV][VEC])
{
    T *dst = static_cast<T *>(a.dst) + v * a.ld_dst;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!left[j]) continue;
        float o[VEC];
        if (a.accumulate) load_part<T, VEC>(dst + c[j], left[j], o);
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = a.accumulate ? fmaf(acc[j][i], a.scale, o[i]) : acc[j][i] * a.scale;
        store_part<T, VEC>(dst + c[j], left[j], o);
    }
}

// First position whose key is at least v, by a whole wave: each step looks at
// 64 places together, so 65536 positions take three dependent loads.
__device__ __forceinline__ int64_t first_at_least(const uint32_t *key, int64_t n, int64_t v)
{
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, len = n; // the answer is in [lo, lo + len]
    while (len > 0) {
        const int64_t step = (len + 63) / 64, at = lo + (lane + 1) * step - 1; // the last place of this lane's part
        const bool less = at < lo + len && (int64_t)key[at] < v;
        const int parts = (int)__popcll(__ballot(less)); // whole parts below v
        lo += parts * step;
        len = len - parts * step < step - 1 ? len - parts * step : step - 1;
        if (len < 0) len = 0;
    }
    return lo;
}

// Rows of the table that no position names, written as zeros.  A wave has 64
// rows: their keys lie side by side among the sorted ones, where every lane
// looks for one row's; then the wave writes the rows that are not there, several
// rows at a time where a row is shorter than 64 vectors (350000 rows of 44 fp32:
// 22 us with a row at a time and a search from the start by every lane, 14 now).
template <class T>
__device__ void zero_rows(const LookupArgs &a, const uint32_t *key, int64_t wave)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    const int lane = threadIdx.x & 63;
    const int64_t v0 = wave * 64;
    if (v0 >= a.V) return;
    const int64_t v = v0 + lane;
    int64_t lo = first_at_least(key, a.n, v0), hi = first_at_least(key, a.n, v0 + 64);
    const int64_t end = hi;
    while (lo < hi) { // first position whose key is >= v
        const int64_t mid = (lo + hi) >> 1;
        if ((int64_t)key[mid] < v) lo = mid + 1;
        else hi = mid;
    }
    const bool absent = v < a.V && (lo >= end || (int64_t)key[lo] != v);
    uint64_t m = __ballot(absent);
    const float z[VEC] = {};
    const int64_t nv = (a.D + VEC - 1) / VEC;
    if (nv < 64) {
        const int n = (int)nv, down = 64 / n, across = 64 % n;
        for (int row = lane / n, c = lane % n; row < 64;) {
            const int left = (int)a.D - c * VEC;
            if (m >> row & 1)
                store_part<T, VEC>(static_cast<T *>(a.dst) + (v0 + row) * a.ld_dst + c * VEC, left < VEC ? left : VEC,
                                   z);
            row += down;
            c += across;
            if (c >= n) {
                c -= n;
                ++row;
            }
        }
        return;
    }
    while (m) {
        const int k = __builtin_ctzll(m);
        m &= m - 1;
        T *dst = static_cast<T *>(a.dst) + (v0 + k) * a.ld_dst;
        for (int64_t c = lane * VEC; c < a.D; c += 64 * VEC)
            store_part<T, VEC>(dst + c, (int)(a.D - c < VEC ? a.D - c : VEC), z);
    }
}

// Blocks of both kinds alternate, so that the writes of zeros and the reads of
// the sums overlap.
template <class T, int LPR, int NV, bool WHOLE>
__global__ __launch_bounds__(256) void k_lookup_sum(LookupArgs a, const uint32_t *key, const int32_t *perm, int tile,
                                                    int tiles, int pieces, float *slots, int sum_blocks)
{
    constexpr int VEC = 16 / (int)sizeof(T), U = kSumBatch;
    static_assert(LPR >= U, "a lane of the worker for each row in flight");
    const int zero_blocks = (int)gridDim.x - sum_blocks, both = sum_blocks < zero_blocks ? sum_blocks : zero_blocks;
    int b = blockIdx.x;
    bool zero;
    if (b < 2 * both) {
        zero = b & 1;
        b >>= 1;
    } else {
        zero = zero_blocks > sum_blocks;
        b -= both;
    }
    if (zero) {
        zero_rows<T>(a, key, (int64_t)b * 4 + (threadIdx.x >> 6));
        return;
    }
    const int lane = threadIdx.x % LPR;
    const int64_t w = ((int64_t)b * 256 + threadIdx.x) / LPR;
    const int64_t j = w / pieces;
    if (j >= tiles) return;
    const int64_t n = a.n, tb = j * tile, te = tb + tile < n ? tb + tile : n;
    auto at = [&](int64_t p) { return p < 0 ? 0 : p < n ? p : n - 1; };
    // the six keys that say how the tile's first and last runs continue, one per lane
    const int64_t probe = lane == 0 ? tb - tile : lane == 1 ? tb - 1 : lane == 2 ? tb : lane == 3 ? te - 1
                          : lane == 4 ? te : te + tile - 1;
    const uint32_t pk = key[at(probe)];
    const uint32_t k_before = __shfl(pk, 0, LPR), k_left = __shfl(pk, 1, LPR), k_first = __shfl(pk, 2, LPR);
    const uint32_t k_last = __shfl(pk, 3, LPR), k_right = __shfl(pk, 4, LPR), k_beyond = __shfl(pk, 5, LPR);
    const uint32_t none = (uint32_t)a.V;
    uint32_t cur = k_first;
    if (cur == none) return;
    int64_t c[NV];
    int left[NV];
    float acc[NV][VEC];
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        c[q] = (w - j * pieces) * (LPR * NV * VEC) + (q * LPR + lane) * VEC;
        const int64_t l = a.D - c[q];
        left[q] = l < VEC ? (int)(l < 0 ? 0 : l) : VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[q][i] = 0.f;
    }
    // where the open run goes: the table's row, nowhere (an earlier worker's
    // run), or this tile's left or right slot
    enum { ROW, SKIP, LEFT, RIGHT };
    int dest = ROW;
    if (tb > 0 && k_left == cur)
        dest = k_before == cur || (tb + tile - 1 < n && k_last == cur) ? LEFT : SKIP;
    int64_t end = te;
    bool cut = false;
    if (te < n && k_right == k_last && k_right != none) {
        cut = k_first == k_right || (te + tile - 1 < n && k_beyond == k_right);
        if (!cut) { // the run ends less than a tile further on
            const int base = (threadIdx.x & 63) / LPR * LPR;
            const uint64_t full = LPR == 64 ? ~0ull : (1ull << (LPR & 63)) - 1ull;
            for (;;) {
                const bool same = end + lane < n && key[at(end + lane)] == k_right;
                const uint64_t m = (__ballot(same) >> base) & full;
                if (m == full) {
                    end += LPR;
                    continue;
                }
                end += __builtin_ctzll(~m);
                break;
            }
        }
    }
    auto flush = [&]() {
        if (dest == SKIP) return;
        if (dest == ROW) {
            add_row_out<T, VEC, NV>(a, cur, c, left, acc);
            return;
        }
        float *slot = slots + (2 * j + (dest == RIGHT)) * a.D;
#pragma unroll
        for (int q = 0; q < NV; ++q)
            if (left[q]) store_part<float, VEC>(slot + c[q], left[q], acc[q]);
    };
    for (int64_t p = tb; p < end; p += U) {
        const int64_t mine = p + lane < end ? p + lane : end - 1;
        const uint32_t keys = key[mine];
        const int32_t rows = perm[mine];
        typename VecOf<T, VEC>::raw x[U][NV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const T *src = static_cast<const T *>(a.src) + (int64_t)__shfl(rows, u, LPR) * a.ld_src;
#pragma unroll
            for (int v = 0; v < NV; ++v) x[u][v] = load_row<T, VEC, WHOLE>(src, c[v], a.D);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t k = __shfl(keys, u, LPR);
            if (p + u >= end || k == none) continue;
            if (k != cur) {
                flush();
                cur = k;
                dest = ROW;
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) acc[v][i] = 0.f;
            }
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[v][i] += (float)x[u][v][i];
        }
    }
    if (cut && dest == ROW) dest = RIGHT;
    flush();
}

// Runs that were cut: the block of 64 tiles and 256 columns adds up the runs
// that begin in its tiles.  A wave takes a short run by itself; the sums of a
// long one are shared out over the waves and joined in order.  What bounds it
// is the chain of dependent loads of one run, so the keys that say which runs
// begin are read together, a row that is added to before its sum is known,
// and where a row has fewer than 256 columns a wave's lanes take several slots
// at a time.
template <class T>
__global__ __launch_bounds__(64 * kJoinGroups) void k_lookup_join(LookupArgs a, const uint32_t *key, int tile,
                                                                  int tiles, const float *slots)
{
    constexpr int kShort = 2 * kJoinGroups;
    __shared__ float sm[kJoinGroups][256];
    __shared__ int3 longs[64]; // tile, last tile, key
    __shared__ int count;
    if (threadIdx.x == 0) count = 0;
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int64_t n = a.n, j0 = (int64_t)blockIdx.x * 64;
    auto at = [&](int64_t p) { return key[p < 0 ? 0 : p < n ? p : n - 1]; };
    bool begins; // a cut run begins in this lane's tile
    uint32_t edge;
    {
        const int64_t j = j0 + lane, tb = j * tile, b = tb + tile;
        const uint32_t before = at(tb - 1), first = at(tb), last = at(b - 1), beyond = at(b + tile - 1);
        edge = at(b);
        const bool cut = b < n && last == edge && (first == edge || (b + tile - 1 < n && beyond == edge));
        begins = cut && edge != (uint32_t)a.V && !(tb > 0 && first == edge && before == edge);
    }
    __syncthreads();
    // the last tile that the run of tile j reaches: the next 64 tiles are
    // looked at together, then every 64th of those that follow
    auto last_of = [&](int64_t j, uint32_t k) {
        auto reach = [&](int64_t q, int64_t by) { // how many of tiles q, q + by, .. begin in the run
            const int64_t p = q + lane * by;
            const uint64_t m = __ballot(p < tiles && key[(p < tiles ? p : tiles - 1) * tile] == k);
            return m == ~0ull ? 64 : __builtin_ctzll(~m);
        };
        int64_t q = j + 1;
        for (;;) {
            const int c = reach(q, 1);
            if (c < 64) return q + c - 1;
            const int steps = reach(q, 64); // tile q is in the run: at least one
            q += (int64_t)(steps > 1 ? steps - 1 : 1) * 64;
        }
    };
    // lanes side by side in a row of columns, and rows of lanes
    const int64_t wide = a.D - (int64_t)blockIdx.y * 256;
    const int across = wide > 128 ? 64 : wide > 64 ? 32 : 16, rows = 64 / across, sub = lane / across;
    const int64_t c = (int64_t)blockIdx.y * 256 + lane % across * 4;
    const int left = (int)(a.D - c < 4 ? (a.D - c < 0 ? 0 : a.D - c) : 4);
    auto add = [&](int64_t j, int64_t from, int64_t to, int by, float (&s)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = 0.f;
#pragma unroll 8
        for (int64_t q = from + sub * by; q <= to; q += rows * by) {
            float x[4];
            load_part<float, 4>(slots + (2 * q + (q == j)) * a.D + (left ? c : 0), left, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += x[i];
        }
        for (int o = across; o < 64; o <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += __shfl_xor(s[i], o, 64);
    };
    auto row = [&](uint32_t k) { return static_cast<T *>(a.dst) + (int64_t)k * a.ld_dst + c; };
    auto fetch = [&](uint32_t k, float (&o)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = 0.f;
        if (a.accumulate) load_part<T, 4>(row(k), left, o);
    };
    auto out = [&](uint32_t k, const float (&s)[4], const float (&old)[4]) {
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = fmaf(s[i], a.scale, old[i]);
        if (sub == 0 && left) store_part<T, 4>(row(k), left, o);
    };
    float s[4], old[4];
    int turn = 0;
    for (uint64_t m = __ballot(begins); m; m &= m - 1, ++turn) {
        if (turn % kJoinGroups != grp) continue;
        const int t = __builtin_ctzll(m);
        const uint32_t k = __shfl(edge, t, 64);
        fetch(k, old);
        const int64_t last = last_of(j0 + t, k);
        if (last - (j0 + t) >= kShort) { // left to all waves
            if (lane == 0) longs[atomicAdd(&count, 1)] = make_int3(t, (int)last, (int)k);
            continue;
        }
        add(j0 + t, j0 + t, last, 1, s);
        out(k, s, old);
    }
    __syncthreads();
    for (int i = 0; i < count; ++i) { // each is summed by itself: their order does not matter
        const int64_t j = j0 + longs[i].x;
        const uint32_t k = (uint32_t)longs[i].z;
        fetch(k, old);
        add(j, j + grp, longs[i].y, kJoinGroups, s);
#pragma unroll
        for (int q = 0; q < 4; ++q) sm[grp][lane * 4 + q] = s[q];
        __syncthreads();
        if (grp == 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                s[q] = 0.f;
#pragma unroll
                for (int g = 0; g < kJoinGroups; ++g) s[q] += sm[g][lane * 4 + q];
            }
            out(k, s, old);
        }
        __syncthreads();
    }
}

// Positions per worker: few enough that the workers of `lanes` lanes fill the
// compute units (eight waves on each), since what each one does is a chain of
// loads; no fewer, because every tile edge may cut a run.  lanes = 0: the
// fewest there can be, which the workspace allows for.
int sum_tile(int64_t n, int64_t lanes)
{
    int t = kSumTile;
    while (t < 4 * kSumTile && n / (2 * t) * lanes >= (int64_t)kCUs * 8 * 64) t *= 2;
    while ((n + t - 1) / t > kSumTiles) t *= 2;
    return t;
}

struct LookupPlan {
    uint32_t *key0, *key1;
    int32_t *val0, *val1;
    Plan sort;                  // of the general sort
    uint32_t *count;            // of the token sort
    float *slots;
};

size_t plan_lookup(int64_t n, int64_t D, char *base, LookupPlan *p)
{
    size_t off = TT_EMB_STATUS_BYTES;
    auto take = [&](size_t bytes) {
        char *r = base ? base + off : nullptr;
        off += round256(bytes > 0 ? bytes : 1);
        return r;
    };
    LookupPlan q{};
    q.key0 = (uint32_t *)take(4 * n);
    q.key1 = (uint32_t *)take(4 * n);
    q.val0 = (int32_t *)take(4 * n);
    q.val1 = (int32_t *)take(4 * n);
    if (n > kTokTile) { // a vocabulary past 2^20 takes the general sort too
        q.sort.ws.hist = (uint32_t *)take(4 * 256 * (size_t)sort_blocks(n));
        q.sort.ws.part = (uint64_t *)take(8 * (kScanBlocks + 1));
        const size_t tiles = (size_t)((n + kTokTile - 1) / kTokTile);
        if (n <= kTokSortMax) q.count = (uint32_t *)take(4 * kTokDigits * tiles);
    }
    const int64_t tile = sum_tile(n, 0);
    q.slots = (float *)take((size_t)(2 * ((n + tile - 1) / tile) * D) * 4);
    if (p) *p = q;
    return off;
}

template <class T>
hipError_t lookup_forward(const LookupArgs &a, hipStream_t s)
{
    return row_shape<T>(a.D, [&](auto lpr, auto nv) {
        constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value, COLS = LPR * NV * 16 / (int)sizeof(T);
        const int64_t pieces = (a.D + COLS - 1) / COLS;
        int64_t blocks = (a.n * pieces * LPR + 255) / 256;
        if (blocks > kMaxGrid) blocks = kMaxGrid;
        hipLaunchKernelGGL((k_lookup<T, LPR, NV>), dim3((unsigned)blocks), dim3(256), 0, s, a, (int)pieces);
        return hipGetLastError();
    });
}

template <class T>
hipError_t lookup_backward(const LookupArgs &a, hipStream_t s)
{
    LookupPlan p;
    plan_lookup(a.n, a.D, a.ws, &p);
    int bits = 0;
    while ((a.V >> bits) != 0) ++bits;
    hipError_t e = hipSuccess;
    bool in_1 = false;
    const int passes = (bits + kTokBits - 1) / kTokBits, wd = (bits + passes - 1) / passes;
    if (a.n <= kTokTile) {
        hipLaunchKernelGGL(k_token_sort, dim3(1), dim3(kTokThreads), 0, s, a, bits, p.key0, p.val0);
    } else if (a.n <= kTokSortMax && passes <= 2) {
        const unsigned tiles = (unsigned)((a.n + kTokTile - 1) / kTokTile);
        hipLaunchKernelGGL(k_token_count<true>, dim3(tiles), dim3(kTokThreads), 0, s, a, nullptr, 0, wd, p.count);
        hipLaunchKernelGGL(k_token_place<true>, dim3(tiles), dim3(kTokThreads), 0, s, a, nullptr, nullptr, p.key1,
                           p.val1, 0, wd, p.count);
        in_1 = passes == 1;
        if (passes == 2) {
            hipLaunchKernelGGL(k_token_count<false>, dim3(tiles), dim3(kTokThreads), 0, s, a, p.key1, wd, wd, p.count);
            hipLaunchKernelGGL(k_token_place<false>, dim3(tiles), dim3(kTokThreads), 0, s, a, p.key1, p.val1, p.key0,
                               p.val0, wd, wd, p.count);
        }
    } else {
        hipLaunchKernelGGL(k_lookup_keys, dim3((unsigned)((a.n + 255) / 256)), dim3(256), 0, s, a, p.key0, p.val0);
        e = radix_sort_pairs(p.sort, p.key0, p.val0, p.key1, p.val1, a.n, nullptr, bits, &in_1, s);
    }
    if (e != hipSuccess) return e;
    const uint32_t *key = in_1 ? p.key1 : p.key0;
    const int32_t *perm = in_1 ? p.val1 : p.val0;
    int tile = 0, tiles = 0;
    e = row_shape<T>(a.D, [&](auto lpr, auto nv) {
        constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value, COLS = LPR * NV * 16 / (int)sizeof(T);
        const int64_t pieces = (a.D + COLS - 1) / COLS;
        tile = sum_tile(a.n, pieces * LPR);
        tiles = (int)((a.n + tile - 1) / tile);
        const int64_t sum = ((int64_t)tiles * pieces * LPR + 255) / 256;
        const int64_t zero = a.accumulate ? 0 : (a.V + 255) / 256;
        auto go = [&](auto whole) {
            hipLaunchKernelGGL((k_lookup_sum<T, LPR, NV, decltype(whole)::value>), dim3((unsigned)(sum + zero)),
                               dim3(256), 0, s, a, key, perm, tile, tiles, (int)pieces, p.slots, (int)sum);
            return hipGetLastError();
        };
        return a.D % (16 / (int)sizeof(T)) == 0 ? go(std::true_type()) : go(std::false_type());
    });
    if (e != hipSuccess) return e;
    if (tiles > 1)
        hipLaunchKernelGGL(k_lookup_join<T>, dim3((unsigned)((tiles + 63) / 64), (unsigned)((a.D + 255) / 256)),
                           dim3(64 * kJoinGroups), 0, s, a, key, tile, tiles, p.slots);
    return hipGetLastError();
}

// No tokens: an overwritten gradient is zero.
template <class T>
__global__ __launch_bounds__(256) void k_lookup_clear(LookupArgs a)
{
    zero_rows<T>(a, nullptr, (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6));
}

template <class T>
hipError_t lookup_grad(const LookupArgs &a, hipStream_t s)
{
    if (a.n > 0) return lookup_backward<T>(a, s);
    if (a.accumulate) return hipSuccess;
    hipLaunchKernelGGL(k_lookup_clear<T>, dim3((unsigned)((a.V + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace

size_t lookup_workspace(int64_t n, int64_t V, int64_t D)
{
    (void)V;
    return plan_lookup(n, D, nullptr, nullptr);
}

hipError_t launch_lookup_forward(const LookupArgs &a, int dtype, hipStream_t s)
{
    if (a.n == 0) return hipSuccess;
    if (dtype == TT_EMB_DTYPE_FLOAT) return lookup_forward<float>(a, s);
    if (dtype == TT_EMB_DTYPE_BFLOAT) return lookup_forward<bf16>(a, s);
    return lookup_forward<f16>(a, s);
}

hipError_t launch_lookup_backward(const LookupArgs &a, int dtype, hipStream_t s)
{
    if (dtype == TT_EMB_DTYPE_FLOAT) return lookup_grad<float>(a, s);
    if (dtype == TT_EMB_DTYPE_BFLOAT) return lookup_grad<bf16>(a, s);
    return lookup_grad<f16>(a, s);
}

} // namespace ttemb
