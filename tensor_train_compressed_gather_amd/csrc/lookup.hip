// lookup.hip -- rows of a dense table for token ids, and the gradient of the
// table summed by sorted tokens (gfx950).
//
// Both are copies of rows: a row (or a piece of a long one) belongs to LPR
// neighbouring lanes of NV 16-byte vectors each.  The gradient is not
// scattered with atomics, whose order would change the result: positions are
// sorted stably by token, fixed tiles of the sorted positions are summed by
// one worker each, and only runs of one token that cover a whole tile are cut
// and joined by a second kernel in tile order.
#include "lm.h"
#include "primitives.h"

namespace ttemb {

namespace {

constexpr int kSumBatch = 8;       // gradient rows a worker has in flight
constexpr int kSumTile = 32;       // sorted positions per worker, at least
constexpr int64_t kMaxGrid = 1 << 20; // blocks of the forward, which walks over rows past them
constexpr int64_t kSumTiles = 4096; // workers per row piece, at most

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
__global__ __launch_bounds__(256) void k_lookup_keys(LookupArgs a, uint32_t *key, int32_t *val)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.n) return;
    const int64_t t = a.tokens[i];
    const bool pad = a.pad >= 0 && t == a.pad, ok = t >= 0 && t < a.V;
    if (!ok && !pad) atomicOr(reinterpret_cast<int *>(a.ws) + ST_ERR, (int)STB_INDEX);
    key[i] = ok && !pad ? (uint32_t)t : (uint32_t)a.V;
    val[i] = (int32_t)i;
}

// Whether the run of equal keys across the boundary b (a multiple of the
// tile) is cut there: it is when it covers a whole tile next to b.  Shorter
// runs belong to the worker of the tile they begin in, which reads past its
// end (by less than a tile).
__device__ __forceinline__ bool run_cut(const uint32_t *key, int64_t n, int64_t b, int tile)
{
    if (b <= 0 || b >= n) return false;
    const uint32_t k = key[b];
    if (key[b - 1] != k) return false;
    return key[b - tile] == k || (b + tile - 1 < n && key[b + tile - 1] == k);
}

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

// Rows of the table that no position names, written as zeros: every lane
// looks for one row's token among the sorted keys, then the wave writes the
// rows that are not there.
template <class T>
__device__ void zero_rows(const LookupArgs &a, const uint32_t *key, int64_t wave)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    const int lane = threadIdx.x & 63;
    const int64_t v0 = wave * 64;
    if (v0 >= a.V) return;
    const int64_t v = v0 + lane;
    int64_t lo = 0, hi = a.n; // first position whose key is >= v
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if ((int64_t)key[mid] < v) lo = mid + 1;
        else hi = mid;
    }
    const bool absent = v < a.V && (lo >= a.n || (int64_t)key[lo] != v);
    uint64_t m = __ballot(absent);
    const float z[VEC] = {};
    while (m) {
        const int k = __builtin_ctzll(m);
        m &= m - 1;
        T *dst = static_cast<T *>(a.dst) + (v0 + k) * a.ld_dst;
        for (int64_t c = lane * VEC; c < a.D; c += 64 * VEC)
            store_part<T, VEC>(dst + c, (int)(a.D - c < VEC ? a.D - c : VEC), z);
    }
}

template <class T, int LPR, int NV>
__global__ __launch_bounds__(256) void k_lookup_sum(LookupArgs a, const uint32_t *key, const int32_t *perm, int tile,
                                                    int tiles, int pieces, float *slots, int sum_blocks)
{
    constexpr int VEC = 16 / (int)sizeof(T), U = kSumBatch;
    if ((int)blockIdx.x >= sum_blocks) {
        zero_rows<T>(a, key, (int64_t)((int)blockIdx.x - sum_blocks) * 4 + (threadIdx.x >> 6));
        return;
    }
    const int lane = threadIdx.x % LPR;
    const int64_t w = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPR;
    const int64_t j = w / pieces;
    if (j >= tiles) return;
    const int64_t n = a.n, tb = j * tile, te = tb + tile < n ? tb + tile : n;
    uint32_t cur = key[tb];
    const uint32_t none = (uint32_t)a.V;
    if (cur == none) return;
    int64_t c[NV];
    int left[NV];
    float acc[NV][VEC];
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        c[q] = (w - j * pieces) * (LPR * NV * VEC) + (q * LPR + lane) * VEC;
        const int64_t l = a.D - c[q];
        left[q] = l < VEC ? (int)(l < 0 ? 0 : l) : VEC;
        if (!left[q]) c[q] = 0;
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[q][i] = 0.f;
    }
    // where the open run goes: the table's row, nowhere (an earlier worker's
    // run), or this tile's left or right slot
    enum { ROW, SKIP, LEFT, RIGHT };
    int dest = ROW;
    if (tb > 0 && key[tb - 1] == cur) dest = run_cut(key, n, tb, tile) ? LEFT : SKIP;
    int64_t end = te;
    bool cut = false;
    if (te < n && key[te] == key[te - 1] && key[te] != none) {
        cut = run_cut(key, n, te, tile);
        const uint32_t k = key[te];
        if (!cut)
            while (end < n && key[end] == k) ++end;
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
        uint32_t k[U];
        float x[U][NV][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t q = p + u < end ? p + u : end - 1;
            k[u] = key[q];
            const T *src = static_cast<const T *>(a.src) + (int64_t)perm[q] * a.ld_src;
#pragma unroll
            for (int v = 0; v < NV; ++v) load_part<T, VEC>(src + c[v], left[v], x[u][v]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p + u >= end || k[u] == none) continue;
            if (k[u] != cur) {
                flush();
                cur = k[u];
                dest = ROW;
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) acc[v][i] = 0.f;
            }
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[v][i] += x[u][v][i];
        }
    }
    if (cut && dest == ROW) dest = RIGHT;
    flush();
}

// Runs that were cut: block (tile, 64 columns) adds up the run that begins in
// the tile, sixteen groups of slots joined in order.
template <class T>
__global__ __launch_bounds__(1024) void k_lookup_join(LookupArgs a, const uint32_t *key, int tile, int tiles,
                                                      const float *slots)
{
    __shared__ float sm[16][64];
    const int64_t j = blockIdx.x, n = a.n, b = (j + 1) * (int64_t)tile;
    if (!run_cut(key, n, b, tile)) return;
    const uint32_t k = key[b];
    if (k == (uint32_t)a.V) return;
    const int64_t tb = j * (int64_t)tile;
    if (tb > 0 && key[tb] == k && key[tb - 1] == k) return; // it begins further left
    // last tile the run reaches: the first tile boundary past its end
    int64_t lo = j + 1, hi = tiles - 1; // largest tile whose first key is k
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (key[mid * tile] <= k) lo = mid;
        else hi = mid - 1;
    }
    const int64_t last = lo;
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.y * 64 + lane;
    float s = 0.f;
    if (c < a.D)
        for (int64_t q = j + grp; q <= last; q += 16) s += slots[(2 * q + (q == j)) * a.D + c];
    sm[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && c < a.D) {
        float t = 0.f;
#pragma unroll
        for (int g = 0; g < 16; ++g) t += sm[g][lane];
        T *dst = static_cast<T *>(a.dst) + (int64_t)k * a.ld_dst + c;
        *dst = (T)(a.accumulate ? fmaf(t, a.scale, (float)*dst) : t * a.scale);
    }
}

int sum_tile(int64_t n)
{
    int t = kSumTile;
    while ((n + t - 1) / t > kSumTiles) t *= 2;
    return t;
}

struct LookupPlan {
    uint32_t *key0, *key1;
    int32_t *val0, *val1;
    Plan sort;
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
    q.sort.ws.hist = (uint32_t *)take(4 * 256 * (size_t)sort_blocks(n));
    q.sort.ws.part = (uint64_t *)take(8 * (kScanBlocks + 1));
    const int64_t tile = sum_tile(n);
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
    hipLaunchKernelGGL(k_lookup_keys, dim3((unsigned)((a.n + 255) / 256)), dim3(256), 0, s, a, p.key0, p.val0);
    bool in_1 = false;
    hipError_t e = radix_sort_pairs(p.sort, p.key0, p.val0, p.key1, p.val1, a.n, nullptr, bits, &in_1, s);
    if (e != hipSuccess) return e;
    const uint32_t *key = in_1 ? p.key1 : p.key0;
    const int32_t *perm = in_1 ? p.val1 : p.val0;
    const int tile = sum_tile(a.n), tiles = (int)((a.n + tile - 1) / tile);
    e = row_shape<T>(a.D, [&](auto lpr, auto nv) {
        constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value, COLS = LPR * NV * 16 / (int)sizeof(T);
        const int64_t pieces = (a.D + COLS - 1) / COLS;
        const int64_t sum = ((int64_t)tiles * pieces * LPR + 255) / 256;
        const int64_t zero = a.accumulate ? 0 : (a.V + 255) / 256;
        hipLaunchKernelGGL((k_lookup_sum<T, LPR, NV>), dim3((unsigned)(sum + zero)), dim3(256), 0, s, a, key, perm,
                           tile, tiles, (int)pieces, p.slots, (int)sum);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    if (tiles > 1)
        hipLaunchKernelGGL(k_lookup_join<T>, dim3((unsigned)tiles, (unsigned)((a.D + 63) / 64)), dim3(1024), 0, s, a,
                           key, tile, tiles, p.slots);
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
