// clip.hip -- global norm of the gradients of many tensors and their scaling
// to a bound (gfx950).
//
// N = sqrt(sum g^2) over all tensors, factor = min(1, max_norm / (N + eps)).
// The squares are taken and added in fp64: those of fp32 values are exact
// there, none over- or underflows, and a sum of 10^9 of them is off by 2^-53
// its few hundred additions per thread.  Memory bounds the kernels: 25.2 M fp32
// values are read in 17.3 us (5.8 TB/s) and scaled in 33.5 (6.0 TB/s).  Of 16-bit
// values fp64 takes the same instructions for half the bytes (159 M of bf16: 82
// us, 3.9 TB/s), the price of sums that no value can overflow.
//
// Each block adds up the chunks it owns and leaves one partial sum; the next
// launch begins by adding up the partial sums, every block for itself in the
// same order, so that no block waits for another and the bits repeat.  Few
// values are one block's work from the first load to the last store.
#include "lm.h"

namespace ttemb {

namespace {

constexpr int kClipChunk = 8192; // elements that a block takes at a time
// Chunks of all tensors up to which one block does everything.  One launch less is 3 us
// less of a call (the 3 cores of a 1000-row table, 1760 fp32 values, call after call: 12.1
// us, 15.3 with two launches).  In a graph the kernels take 5.4 and 5.0 us there; 4 chunks
// 4.4 and 4.4 where they are whole, 13.8 and 6.9 as ragged tensors of bf16, whose loads
// are waited for one by one; 8 chunks 7.2 and 4.7, ragged 26 and 7.3.
constexpr int kClipOne = 4;

// A chunk's values by this thread: 16 bytes at a time, zeros past the end.
template <class T>
struct Chunk {
    static constexpr int VEC = 16 / (int)sizeof(T), N = kClipChunk / 256 / VEC;
    float x[N][VEC];

    __device__ __forceinline__ void load(const T *g, int64_t left)
    {
        const int c = threadIdx.x * VEC;
        if (left >= kClipChunk) { // (a load under a condition is waited for before the next one)
#pragma unroll
            for (int j = 0; j < N; ++j) load_vec<T, VEC>(g + c + j * 256 * VEC, x[j]);
            return;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int have = (int)left - (c + j * 256 * VEC);
            load_part<T, VEC>(have > 0 ? g + c + j * 256 * VEC : g, have > 0 ? have : 0, x[j]);
        }
    }
    __device__ __forceinline__ void store(T *g, int64_t left) const
    {
        const int c = threadIdx.x * VEC, whole = left >= kClipChunk ? kClipChunk : (int)left;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int have = whole - (c + j * 256 * VEC);
            if (have > 0) store_part<T, VEC>(g + c + j * 256 * VEC, have, x[j]);
        }
    }
};

template <class T>
__device__ __forceinline__ double chunk_squares(const T *g, int64_t left)
{
    Chunk<T> c;
    c.load(g, left);
    double s[2] = {0.0, 0.0};
#pragma unroll
    for (int j = 0; j < Chunk<T>::N; ++j)
#pragma unroll
        for (int i = 0; i < Chunk<T>::VEC; ++i) s[i & 1] = fma((double)c.x[j][i], (double)c.x[j][i], s[i & 1]);
    return s[0] + s[1];
}

template <class T>
__device__ __forceinline__ void chunk_scale(T *g, int64_t left, float factor)
{
    Chunk<T> c;
    c.load(g, left);
#pragma unroll
    for (int j = 0; j < Chunk<T>::N; ++j)
#pragma unroll
        for (int i = 0; i < Chunk<T>::VEC; ++i) c.x[j][i] *= factor;
    c.store(g, left);
}

// f(tensor's address at a chunk as its own type, elements from there on) for
// the chunks of a block.
template <class F>
__device__ __forceinline__ void for_chunks(const ClipTable &t, F f)
{
    int at = 0;
    for (int c = (int)blockIdx.x; c < t.first[t.n]; c += (int)gridDim.x) {
        int lo = at, hi = t.n - 1; // a block's chunks are in order
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (t.first[mid] <= c) lo = mid;
            else hi = mid - 1;
        }
        at = lo;
        const int64_t e = (int64_t)(c - t.first[lo]) * kClipChunk, left = t.cnt[lo] - e;
        if (t.dtype[lo] == TT_EMB_DTYPE_FLOAT) f(static_cast<float *>(t.g[lo]) + e, left);
        else if (t.dtype[lo] == TT_EMB_DTYPE_BFLOAT) f(static_cast<bf16 *>(t.g[lo]) + e, left);
        else f(static_cast<f16 *>(t.g[lo]) + e, left);
    }
}

__device__ __forceinline__ double block_sum(double s)
{
    __shared__ double sm[4];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = s;
    __syncthreads();
    return (sm[0] + sm[1]) + (sm[2] + sm[3]);
}

// Factor of a sum of squares.  (A NaN is not under the bound.)
__device__ __forceinline__ float factor_of(const ClipBound &b, double sum, bool store)
{
    const double norm = sqrt(sum);
    const float factor = norm + b.eps <= b.max_norm ? 1.f : (float)(b.max_norm / (norm + b.eps));
    if (store && threadIdx.x == 0) {
        if (b.norm) *b.norm = (float)norm;
        if (b.factor) *b.factor = factor;
    }
    return factor;
}

__device__ __forceinline__ double join_parts(const double *part, int parts)
{
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 256) s += part[i];
    return block_sum(s);
}

// Partial sums of a launch's blocks.
__global__ __launch_bounds__(256) void k_clip_sum(ClipTable t, double *part)
{
    double s = 0.0;
    for_chunks(t, [&](auto *g, int64_t left) { s += chunk_squares(g, left); });
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void k_clip_finish(ClipBound b, const double *part, int parts)
{
    factor_of(b, join_parts(part, parts), true);
}

// The partial sums to the factor, then the tensors times it; nothing is read
// or written where it is 1.
__global__ __launch_bounds__(256) void k_clip_scale(ClipTable t, ClipBound b, const double *part, int parts)
{
    const float factor = factor_of(b, join_parts(part, parts), blockIdx.x == 0);
    if (factor == 1.f) return;
    for_chunks(t, [&](auto *g, int64_t left) { chunk_scale(g, left, factor); });
}

// One block: the sum, the factor, and the tensors times it.  (A thread scales
// the elements that it has read.)
__global__ __launch_bounds__(256) void k_clip_one(ClipTable t, ClipBound b, int scale)
{
    double s = 0.0;
    for_chunks(t, [&](auto *g, int64_t left) { s += chunk_squares(g, left); });
    const float factor = factor_of(b, block_sum(s), true);
    if (!scale || factor == 1.f) return;
    for_chunks(t, [&](auto *g, int64_t left) { chunk_scale(g, left, factor); });
}

int64_t chunks_of(int64_t numel) { return (numel + kClipChunk - 1) / kClipChunk; }
int grid_for(int64_t chunks) { return (int)(chunks < kClipBlocks ? chunks : kClipBlocks); }

// g(table) for every launch's tensors: as many as a kernel's argument holds.
template <class G>
hipError_t for_tables(int32_t count, void *const *grads, const int32_t *dtypes, const int64_t *numel, G g)
{
    ClipTable t;
    t.n = 0;
    t.first[0] = 0;
    for (int32_t k = 0; k < count; ++k) {
        if (numel[k] == 0) continue;
        t.g[t.n] = grads[k];
        t.dtype[t.n] = (uint8_t)dtypes[k];
        t.cnt[t.n] = numel[k];
        t.first[t.n + 1] = t.first[t.n] + (int32_t)chunks_of(numel[k]);
        if (++t.n == kClipTensors) {
            g(t);
            t.n = 0;
        }
    }
    if (t.n) g(t);
    return hipGetLastError();
}

} // namespace

// Chunks of all tensors, launches and partial sums.
ClipPlan plan_clip(int32_t count, const int64_t *numel)
{
    ClipPlan p{0, 0, 0};
    int64_t here = 0;
    int n = 0;
    auto flush = [&]() {
        if (!n) return;
        ++p.launches;
        p.parts += grid_for(here);
        p.chunks += here;
        here = n = 0;
    };
    for (int32_t k = 0; k < count; ++k) {
        if (numel[k] == 0) continue;
        here += chunks_of(numel[k]);
        if (++n == kClipTensors) flush();
    }
    flush();
    return p;
}

hipError_t launch_clip(int32_t count, void *const *grads, const int32_t *dtypes, const int64_t *numel,
                       const ClipBound &b, bool scale, char *ws, hipStream_t s)
{
    const ClipPlan p = plan_clip(count, numel);
    if (p.launches <= 1 && p.chunks <= kClipOne) {
        if (p.launches == 0) { // no values: the norm is 0
            hipLaunchKernelGGL(k_clip_finish, dim3(1), dim3(256), 0, s, b, (const double *)nullptr, 0);
            return hipGetLastError();
        }
        return for_tables(count, grads, dtypes, numel, [&](const ClipTable &t) {
            hipLaunchKernelGGL(k_clip_one, dim3(1), dim3(256), 0, s, t, b, scale ? 1 : 0);
        });
    }
    double *part = reinterpret_cast<double *>(ws + TT_EMB_STATUS_BYTES);
    int at = 0;
    hipError_t e = for_tables(count, grads, dtypes, numel, [&](const ClipTable &t) {
        const int grid = grid_for(t.first[t.n]);
        hipLaunchKernelGGL(k_clip_sum, dim3(grid), dim3(256), 0, s, t, part + at);
        at += grid;
    });
    if (e != hipSuccess) return e;
    if (!scale) {
        hipLaunchKernelGGL(k_clip_finish, dim3(1), dim3(256), 0, s, b, part, at);
        return hipGetLastError();
    }
    return for_tables(count, grads, dtypes, numel, [&](const ClipTable &t) {
        hipLaunchKernelGGL(k_clip_scale, dim3(grid_for(t.first[t.n])), dim3(256), 0, s, t, b, part, at);
    });
}

} // namespace ttemb
