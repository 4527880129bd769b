// lm.h -- shared definitions of the operators around the table (lookup, norm,
// blocknorm, ffn, xent, adamw, clip): element types, vector access, block reductions, launchers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "../../include/tt_emb.h"

namespace ttemb {

typedef __bf16 bf16;
typedef _Float16 f16;

constexpr int kCUs = 256; // compute units of an MI355X
constexpr int kStatusWords = (int)(TT_EMB_STATUS_BYTES / 4);
enum StatusWord { ST_ERR = 0 };
enum { STB_INDEX = 1 };

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// N consecutive elements as one access.  The type carries the alignment of a
// single element, so rows may begin anywhere; gfx950 serves such accesses with
// the same wide instructions as aligned ones.
template <class T, int N>
struct VecOf {
    typedef T raw __attribute__((ext_vector_type(N)));
    typedef raw type __attribute__((aligned(sizeof(T))));
};

template <class T, int N>
__device__ __forceinline__ void load_vec(const T *p, float (&x)[N])
{
    const typename VecOf<T, N>::type v = *reinterpret_cast<const typename VecOf<T, N>::type *>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (float)v[i];
}

// The first `left` of N elements (the rest read as zero): the ragged end of a row.
template <class T, int N>
__device__ __forceinline__ void load_part(const T *p, int left, float (&x)[N])
{
    if (left >= N) {
        load_vec<T, N>(p, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < left ? (float)p[i] : 0.f;
}

template <class T, int N>
__device__ __forceinline__ void store_part(T *p, int left, const float (&x)[N])
{
    if (left >= N) {
        typename VecOf<T, N>::type v;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = (T)x[i];
        *reinterpret_cast<typename VecOf<T, N>::type *>(p) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < left) p[i] = (T)x[i];
}

// Vector at column c of a row of D elements, zero past its end, still in its
// own type.  WHOLE: D is a multiple of N, so a vector is inside or outside; it
// is then read without a condition (from the row's start where it is outside),
// because a load under a condition is waited for before the next one is issued.
template <class T, int N, bool WHOLE>
__device__ __forceinline__ typename VecOf<T, N>::raw load_row(const T *row, int64_t c, int64_t D)
{
    typedef typename VecOf<T, N>::type vec;
    typename VecOf<T, N>::raw v;
    if constexpr (WHOLE) {
        v = *reinterpret_cast<const vec *>(row + (c < D ? c : 0));
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = c < D ? v[i] : (T)0.f;
    } else if (c + N <= D) {
        v = *reinterpret_cast<const vec *>(row + c);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = c + i < D ? row[c + i] : (T)0.f;
    }
    return v;
}

// Columns c .. c + N - 1 of a parameter row whose type is known at run time:
// `none` where there is no array, 0 past the row's end.
template <int N, bool WHOLE>
__device__ __forceinline__ void load_params(const void *p, int dtype, int64_t c, int64_t D, float none, float (&x)[N])
{
    auto take = [&](auto *q) {
        typedef std::remove_const_t<std::remove_pointer_t<decltype(q)>> T;
        const typename VecOf<T, N>::raw v = load_row<T, N, WHOLE>(q, c, D);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = (float)v[i];
    };
    if (!p) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = c + i < D ? none : 0.f;
    } else if (dtype == TT_EMB_DTYPE_FLOAT) {
        take(static_cast<const float *>(p));
    } else if (dtype == TT_EMB_DTYPE_BFLOAT) {
        take(static_cast<const bf16 *>(p));
    } else {
        take(static_cast<const f16 *>(p));
    }
}
__device__ __forceinline__ void store_param(void *p, int dtype, int64_t j, float x)
{
    if (dtype == TT_EMB_DTYPE_FLOAT) static_cast<float *>(p)[j] = x;
    else if (dtype == TT_EMB_DTYPE_BFLOAT) static_cast<bf16 *>(p)[j] = (bf16)x;
    else static_cast<f16 *>(p)[j] = (f16)x;
}

// ----------------------------------------------------------------- launchers
struct LookupArgs {
    const void *src;      // weight (forward) or grad_out (backward)
    int64_t ld_src;
    const int64_t *tokens;
    int64_t n, V, D;
    float scale;
    void *dst;            // out (forward) or grad_weight (backward)
    int64_t ld_dst;
    int64_t pad;          // padding_idx, negative for none
    int accumulate;
    char *ws;
};
hipError_t launch_lookup_forward(const LookupArgs &a, int dtype, hipStream_t s);
hipError_t launch_lookup_backward(const LookupArgs &a, int dtype, hipStream_t s);
size_t lookup_workspace(int64_t n, int64_t V, int64_t D);

struct NormArgs {
    const void *x, *dy;
    int64_t ld_x, ld_dy, n, D;
    const void *gamma, *beta;
    int param_dtype;
    float eps;
    void *y; // y (forward) or grad_x (backward)
    int64_t ld_y;
    float *mean, *rstd;
    void *dgamma, *dbeta;
    char *ws;
};
hipError_t launch_norm_forward(const NormArgs &a, int dtype, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs &a, int dtype, hipStream_t s);
size_t norm_workspace(int64_t n, int64_t D);

struct BlockNormArgs {
    const void *x, *residual, *gate; // gate: [D] of param_dtype, or rows of x's type
    int64_t ld_x, ld_r, ld_gate, n, D;
    int gate_rows, layer, post;
    const void *gamma, *beta, *post_gamma, *post_beta;
    int param_dtype;
    float eps, scale_residual, scale_block;
    float *stats;                    // [n][4] mean and rstd of x, of h
    void *y, *h;                     // forward
    int64_t ld_y, ld_h;
    const void *grad_y, *grad_h;     // backward
    int64_t ld_gy, ld_gh;
    void *grad_x, *grad_r, *grad_gate;
    int64_t ld_gx, ld_gr, ld_gg;
    void *sums[5];                   // dgamma, dbeta, dpost_gamma, dpost_beta, dgate [D]; null for none
    char *ws;
};
hipError_t launch_block_forward(const BlockNormArgs &a, int dtype, int res_dtype, hipStream_t s);
hipError_t launch_block_backward(const BlockNormArgs &a, int dtype, int res_dtype, hipStream_t s);
size_t block_workspace(int64_t n, int64_t D);

struct FfnArgs {
    const void *x, *w_in, *w_out;
    int64_t ld_x, ld_in, ld_out, n, D, F;
    int act;
    float *pre; // written (forward, or null) or read (backward)
    int64_t ld_pre;
    void *y; // forward
    int64_t ld_y;
    const void *gy; // backward
    int64_t ld_gy;
    void *gx, *gw_in, *gw_out;
    int64_t ld_gx, ld_gin, ld_gout;
    char *ws;
};
hipError_t launch_ffn_forward(const FfnArgs &a, int dtype, hipStream_t s);
hipError_t launch_ffn_backward(const FfnArgs &a, int dtype, hipStream_t s);
size_t ffn_workspace(int64_t n, int64_t D, int64_t F, int dtype, int what);
size_t ffn_needs(const FfnArgs &a, int dtype, bool grad); // for these operands as they lie in memory

struct XentArgs {
    const void *hidden, *weight;
    int64_t ld_h, ld_w;
    const int64_t *targets;
    const float *grad_loss;
    int64_t n, V, D;
    int64_t ignore;
    float *loss, *lse;
    void *dh, *dw;
    int64_t ld_dh, ld_dw;
    char *ws;
    size_t ws_bytes;
};
hipError_t launch_xent_forward(const XentArgs &a, int dtype, hipStream_t s);
hipError_t launch_xent_loss_grad(const XentArgs &a, int dtype, hipStream_t s);
void xent_workspace(int64_t n, int64_t V, int64_t D, int dtype, int what, size_t *best, size_t *least);
size_t xent_least(const XentArgs &a, int dtype, bool grad); // for these operands as they lie in memory
int64_t xent_parts(int64_t n, int64_t V, int64_t D, int dtype, int what, size_t ws_bytes, tt_emb_xent_part *parts,
                   int64_t cap, int32_t *slots); // returns how many there are

constexpr int kAdamBlock = 256;   // elements that share one scale of an 8-bit state
constexpr int kAdamTensors = 88;  // tensors per launch (their table is a kernel argument)
struct AdamTable {
    int n;
    uint32_t key;                     // of (seed, step)
    float beta1, one_minus_beta1, beta2, one_minus_beta2;
    float decay, size, root, eps;     // 1 - lr wd, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
    void *m, *v;
    float *m_scale, *v_scale;
    const float *g_scale;             // what multiplies the gradients, null for 1
    int32_t first[kAdamTensors + 1];  // first thread block of each tensor
    int32_t qb[kAdamTensors];         // first block of kAdamBlock elements in the states
    float *p[kAdamTensors];
    const void *g[kAdamTensors];
    bf16 *copy[kAdamTensors];
    int64_t cnt[kAdamTensors];
};
static_assert(sizeof(AdamTable) <= 4096, "the table is passed as a kernel argument");
hipError_t launch_adamw(AdamTable &t, int32_t count, float *const *p, const void *const *g, int grad_dtype,
                        void *const *copies, const int64_t *numel, int bits, hipStream_t s);

constexpr int kClipTensors = 160; // tensors per launch (their table is a kernel argument)
constexpr int kClipBlocks = 8 * kCUs; // blocks of a launch, at most
struct ClipTable {
    int n;
    int32_t first[kClipTensors + 1]; // first chunk of each tensor
    void *g[kClipTensors];
    int64_t cnt[kClipTensors];
    uint8_t dtype[kClipTensors];
};
struct ClipBound {
    double max_norm, eps;
    float *norm, *factor;
};
static_assert(sizeof(ClipTable) + sizeof(ClipBound) + 16 <= 4096, "the table is passed as a kernel argument");
struct ClipPlan {
    int64_t chunks;
    int launches;
    int64_t parts; // partial sums
};
ClipPlan plan_clip(int32_t count, const int64_t *numel);
hipError_t launch_clip(int32_t count, void *const *grads, const int32_t *dtypes, const int64_t *numel,
                       const ClipBound &b, bool scale, char *ws, hipStream_t s);

} // namespace ttemb
