// adamw.hip -- one AdamW step over many tensors in few launches (gfx950).
//
// Memory-bound: per element the parameter and both moments are read and
// written and the gradient read (28 bytes with fp32 states and gradients, 16
// with 8-bit states).  A wave takes 256 consecutive elements, four per lane,
// which is also the block that shares one scale of an 8-bit state, so the
// block's largest magnitude is a reduction inside the wave.  All tensors of a
// call share launches (a table of 88 is the kernel's argument): 78 cores of 25
// million values in 133 us (5.3 TB/s), a model of 160 million with 8-bit states,
// bf16 gradients and a bf16 copy in 490 us (5.2 TB/s), three small cores in 3.6.
#include "lm.h"
#include "primitives.h"

namespace ttemb {

namespace {

constexpr int kAdamSpan = 16;            // blocks of kAdamBlock elements per thread block
constexpr float kAdamTiny = 0x1p-100f;   // least block maximum that a scale is made from

// 32 random bits of element `i` at this step: the finaliser of MurmurHash3
// (A. Appleby, public domain) of the element's number and the step's key.
__device__ __forceinline__ uint32_t adam_noise(uint32_t i, uint32_t key)
{
    uint32_t h = i ^ key;
    h ^= h >> 16;
    h *= 0x85EBCA6Bu;
    h ^= h >> 13;
    h *= 0xC2B2AE35u;
    h ^= h >> 16;
    return h;
}

__device__ __forceinline__ float wave_max(float x)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor(x, o, 64));
    return x;
}

// |x| in units of the block's scale to an 8-bit code.  16 random bits are
// added below the kept mantissa (EXP: exponent of the least normal value,
// DROP: mantissa bits of fp32 that are not kept), so a value goes to its upper
// neighbour with a probability in proportion to its distance from the lower.
template <int EXP, int DROP, int LAST, bool FLOOR_ONE>
__device__ __forceinline__ uint32_t adam_code(float a, uint32_t noise)
{
#pragma clang fp contract(off)
    constexpr int MANT = 23 - DROP;
    constexpr uint32_t BIAS = (uint32_t)(126 + EXP) << MANT;
    const float unit = __builtin_bit_cast(float, (uint32_t)(127 - EXP + MANT) << 23); // 1 / least value
    uint32_t c = ((__builtin_bit_cast(uint32_t, a) + (noise << (DROP - 16))) >> DROP) - BIAS;
    const float small = floorf(a * unit + (float)noise * 0x1p-16f);
    if (a < __builtin_bit_cast(float, (uint32_t)(127 + EXP) << 23)) c = (uint32_t)small;
    c = c > LAST ? LAST : c;
    if (FLOOR_ONE && c == 0 && a > 0.f) c = 1;
    return a != a ? 0x7Fu : c;
}

template <class G, bool BYTES>
__global__ __launch_bounds__(256) void k_adamw(AdamTable t)
{
#pragma clang fp contract(off) // the rounding of m and v is part of the 8-bit result
    int lo = 0, hi = t.n - 1; // the tensor of this thread block
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= (int)blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const int64_t cnt = t.cnt[lo];
    float *const p = t.p[lo];
    const G *const g = static_cast<const G *>(t.g[lo]);
    bf16 *const copy = t.copy[lo];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t q0 = (int64_t)((int)blockIdx.x - t.first[lo]) * kAdamSpan + wave;
#pragma unroll
    for (int k = 0; k < kAdamSpan / 4; ++k) {
        const int64_t q = q0 + 4 * k;       // block of this tensor
        const int64_t e = q * kAdamBlock + 4 * lane;
        if (q * kAdamBlock >= cnt) return;  // the whole wave
        const int64_t sq = t.qb[lo] + q, se = sq * kAdamBlock + 4 * lane; // its place in the states
        const int left = e < cnt ? (cnt - e < 4 ? (int)(cnt - e) : 4) : 0;
        float P[4], Gd[4], M[4], V[4];
        load_part<float, 4>(p + e, left, P);
        load_part<G, 4>(g + e, left, Gd);
        if constexpr (BYTES) {
            const int mq = left ? static_cast<const int *>(t.m)[se >> 2] : 0;
            const int vq = left ? static_cast<const int *>(t.v)[se >> 2] : 0;
            const float ms = t.m_scale[sq], vs = t.v_scale[sq];
            M[0] = __builtin_amdgcn_cvt_f32_fp8(mq, 0) * ms;
            M[1] = __builtin_amdgcn_cvt_f32_fp8(mq, 1) * ms;
            M[2] = __builtin_amdgcn_cvt_f32_fp8(mq, 2) * ms;
            M[3] = __builtin_amdgcn_cvt_f32_fp8(mq, 3) * ms;
            V[0] = __builtin_amdgcn_cvt_f32_bf8(vq, 0) * vs;
            V[1] = __builtin_amdgcn_cvt_f32_bf8(vq, 1) * vs;
            V[2] = __builtin_amdgcn_cvt_f32_bf8(vq, 2) * vs;
            V[3] = __builtin_amdgcn_cvt_f32_bf8(vq, 3) * vs;
        } else {
            load_part<float, 4>(static_cast<const float *>(t.m) + se, left, M);
            load_part<float, 4>(static_cast<const float *>(t.v) + se, left, V);
        }
        float mmax = 0.f, vmax = 0.f;
        bool mbad = false, vbad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            M[i] = M[i] * t.beta1 + Gd[i] * t.one_minus_beta1;
            V[i] = V[i] * t.beta2 + (Gd[i] * t.one_minus_beta2) * Gd[i];
            // hardware square root and reciprocal (1 ulp each): p's own
            // rounding is larger than what they add to it.  The root takes
            // values below 2^-126 for 0, so small ones are scaled up first.
            const bool tiny = V[i] < 0x1p-96f;
            const float root = __builtin_amdgcn_sqrtf(tiny ? V[i] * 0x1p64f : V[i]);
            const float den = (tiny ? root * 0x1p-32f : root) * t.root + t.eps;
            P[i] = P[i] * t.decay - (M[i] * t.size) * __builtin_amdgcn_rcpf(den);
            if constexpr (BYTES) {
                mmax = fmaxf(mmax, fabsf(M[i]));
                vmax = fmaxf(vmax, V[i]);
                mbad = mbad || M[i] != M[i];
                vbad = vbad || V[i] != V[i];
            }
        }
        store_part<float, 4>(p + e, left, P);
        if (copy) store_part<bf16, 4>(copy + e, left, P);
        if constexpr (BYTES) {
            mmax = wave_max(mmax);
            vmax = wave_max(vmax);
            if (__any(mbad)) mmax = __builtin_nanf(""); // a maximum passes NaN over
            if (__any(vbad)) vmax = __builtin_nanf("");
            const float ms = (mmax > kAdamTiny || mmax != mmax ? mmax : kAdamTiny) * (1.f / 448.f);
            const float vs = (vmax > kAdamTiny || vmax != vmax ? vmax : kAdamTiny) * (1.f / 57344.f);
            const float mi = 1.f / ms, vi = 1.f / vs;
            uint32_t mq = 0, vq = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t r = adam_noise((uint32_t)se + i, t.key);
                const uint32_t mc = adam_code<-6, 20, 0x7E, false>(fabsf(M[i]) * mi, r & 0xFFFFu) |
                                    (M[i] < 0.f ? 0x80u : 0u);
                const uint32_t vc = adam_code<-14, 21, 0x7B, true>(V[i] * vi, r >> 16);
                mq |= (i < left ? mc : 0u) << (8 * i);
                vq |= (i < left ? vc : 0u) << (8 * i);
            }
            static_cast<uint32_t *>(t.m)[se >> 2] = mq;
            static_cast<uint32_t *>(t.v)[se >> 2] = vq;
            if (lane == 0) {
                t.m_scale[sq] = ms;
                t.v_scale[sq] = vs;
            }
        } else {
            store_part<float, 4>(static_cast<float *>(t.m) + se, left, M);
            store_part<float, 4>(static_cast<float *>(t.v) + se, left, V);
        }
    }
}

template <class G>
hipError_t adamw_batch(const AdamTable &t, int bits, hipStream_t s)
{
    if (bits == 8) hipLaunchKernelGGL((k_adamw<G, true>), dim3(t.first[t.n]), dim3(256), 0, s, t);
    else hipLaunchKernelGGL((k_adamw<G, false>), dim3(t.first[t.n]), dim3(256), 0, s, t);
    return hipGetLastError();
}

} // namespace

// The tensors' table is the kernel's argument (no copy to the device, nothing
// to keep alive), so more than kAdamTensors of them take further launches.
hipError_t launch_adamw(AdamTable &t, int32_t count, float *const *p, const void *const *g, int grad_dtype,
                        void *const *copies, const int64_t *numel, int bits, hipStream_t s)
{
    int64_t qb = 0;
    t.n = 0;
    t.first[0] = 0;
    auto flush = [&]() -> hipError_t {
        if (t.n == 0) return hipSuccess;
        const hipError_t e = grad_dtype == TT_EMB_DTYPE_FLOAT    ? adamw_batch<float>(t, bits, s)
                             : grad_dtype == TT_EMB_DTYPE_BFLOAT ? adamw_batch<bf16>(t, bits, s)
                                                                 : adamw_batch<f16>(t, bits, s);
        t.n = 0;
        return e;
    };
    for (int32_t k = 0; k < count; ++k) {
        const int64_t blocks = (numel[k] + kAdamBlock - 1) / kAdamBlock;
        if (numel[k] > 0) {
            t.qb[t.n] = (int32_t)qb;
            t.p[t.n] = p[k];
            t.g[t.n] = g[k];
            t.copy[t.n] = copies ? static_cast<bf16 *>(copies[k]) : nullptr;
            t.cnt[t.n] = numel[k];
            t.first[t.n + 1] = t.first[t.n] + (int32_t)((blocks + kAdamSpan - 1) / kAdamSpan);
            ++t.n;
            if (t.n == kAdamTensors) {
                const hipError_t e = flush();
                if (e != hipSuccess) return e;
            }
        }
        qb += blocks;
    }
    return flush();
}

} // namespace ttemb
