// ffn_bwd.hip -- the gated feed-forward block's backward (gfx950).
#include "ffn.h"

namespace ttemb {

namespace {

// The backward's three outputs, which do not wait for each other, in one launch:
// at small sizes each alone leaves most of the card idle, and a launch costs as
// much as a product (777 x 1001 x 2731 bf16: 34 us, 51 in three launches; 8192 x
// 128 x 512 fp32: 44 us, 71).
struct FfnGrads {
    FfnJob x, w_in, w_out;
};
template <class T, int SHAPE>
__global__ __launch_bounds__(256, 1) void k_ffn_grads(FfnGrads g)
{
    constexpr int PL = FfnTerms<T>::planes;
    typedef FfnLds<PL, true, false, SHAPE> A;
    typedef FfnLds<PL, true, true, SHAPE> B;
    __shared__ __align__(16) char lds0[A::first > B::first ? A::first : B::first];
    __shared__ __align__(16) char lds1[A::first > B::first ? A::first : B::first];
    __shared__ __align__(16) char lds2[A::more > B::more ? A::more : B::more];
    __shared__ __align__(16) char lds3[A::more > B::more ? A::more : B::more];
    unsigned b = blockIdx.x;
    if (b < g.x.grid) {
        ffn_tile<T, true, false, FFN_OUT, false, SHAPE>(g.x, b, lds0, lds1, lds2, lds3);
        return;
    }
    b -= g.x.grid;
    const bool in = b < g.w_in.grid;
    ffn_tile<T, true, true, FFN_OUT, false, SHAPE>(in ? g.w_in : g.w_out, in ? b : b - g.w_in.grid, lds0, lds1, lds2,
                                                   lds3);
}

template <class T>
__global__ __launch_bounds__(256) void k_ffn_clear(T *p, int64_t ld, int64_t rows, int64_t cols)
{
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < rows * cols; c += step)
        p[c / cols * ld + c % cols] = (T)0.f;
}

template <class T>
hipError_t ffn_backward(const FfnArgs &a, int dtype, hipStream_t s)
{
    constexpr int PL = FfnTerms<T>::planes;
    const FfnPlan p = plan_ffn(a.n, a.D, a.F, PL, true, copies_of(a, dtype, true), a.ws);
    Packing<T> pack;
    const Operand gy = pack(a.gy, a.ld_gy, a.n, a.D, p.gy, p.Dp, 0);
    const Operand x = pack(a.x, a.ld_x, a.n, a.D, p.x, p.Dp, 0);
    const Operand w_in = pack(a.w_in, a.ld_in, 2 * a.F, a.D, p.w_in, p.Dp, 0);
    const Operand w_out = pack(a.w_out, a.ld_out, a.D, a.F, p.w_out, p.Fp, 0);
    // the products along dp's columns meet its padding
    for (int term = 0; term < (p.two_dpre ? 2 : 1) && p.Pp > 2 * a.F; ++term)
        pack.add(Pack{nullptr, 0, a.n, 0, p.dpre + term * a.n * p.ldP + p.Pp - kPad, kPad, p.ldP, a.n * p.ldP, 0});
    pack.run(s);
    FfnOut o{};
    o.rows = a.n;
    o.splits = 1;
    o.cols = o.F = a.F;
    o.act = a.act;
    o.pre = a.pre;
    o.ld_pre = a.ld_pre;
    o.mid = p.mid;
    o.ld_mid = p.ldF;
    o.plane_mid = a.n * p.ldF;
    o.dpre = p.dpre;
    o.ld_dpre = p.ldP;
    o.plane_dpre = a.n * p.ldP;
    o.two_mid = p.two_mid;
    o.two_dpre = p.two_dpre;
    product<T, true, false, FFN_MID, false>(w_out, gy, a.F, a.n, p.Dp, o, s);
    const Operand mid{p.mid, p.ldF, o.plane_mid, a.n, p.Fp}, dpre{p.dpre, p.ldP, o.plane_dpre, a.n, p.Pp};
    Outputs<T> out{p.sum};
    FfnSize z[3];
    const int shape = grad_sizes(z, a.n, a.D, a.F, PL);
    const FfnGrads g{out(w_in, dpre, z[0], shape, a.gx, a.ld_gx), out(x, dpre, z[1], shape, a.gw_in, a.ld_gin),
                     out(mid, gy, z[2], shape, a.gw_out, a.ld_gout)};
    const dim3 grid(g.x.grid + g.w_in.grid + g.w_out.grid);
    if (shape == BIG) hipLaunchKernelGGL((k_ffn_grads<T, BIG>), grid, dim3(256), 0, s, g);
    if (shape == SMALL) hipLaunchKernelGGL((k_ffn_grads<T, SMALL>), grid, dim3(256), 0, s, g);
    if constexpr (PL == 1) {
        if (shape == DEEP) hipLaunchKernelGGL((k_ffn_grads<T, DEEP>), grid, dim3(256), 0, s, g);
        if (shape == SLIM) hipLaunchKernelGGL((k_ffn_grads<T, SLIM>), grid, dim3(256), 0, s, g);
    }
    out.join(s);
    return hipGetLastError();
}

// No rows: the weights' gradients are zero.
template <class T>
hipError_t ffn_clear(const FfnArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL(k_ffn_clear<T>, dim3(blocks_for(2 * a.F * a.D)), dim3(256), 0, s, static_cast<T *>(a.gw_in),
                       a.ld_gin, 2 * a.F, a.D);
    hipLaunchKernelGGL(k_ffn_clear<T>, dim3(blocks_for(a.D * a.F)), dim3(256), 0, s, static_cast<T *>(a.gw_out),
                       a.ld_gout, a.D, a.F);
    return hipGetLastError();
}

} // namespace

hipError_t launch_ffn_backward(const FfnArgs &a, int dtype, hipStream_t s)
{
    if (dtype == TT_EMB_DTYPE_FLOAT) return a.n == 0 ? ffn_clear<float>(a, s) : ffn_backward<float>(a, dtype, s);
    if (dtype == TT_EMB_DTYPE_BFLOAT) return a.n == 0 ? ffn_clear<bf16>(a, s) : ffn_backward<bf16>(a, dtype, s);
    return a.n == 0 ? ffn_clear<f16>(a, s) : ffn_backward<f16>(a, dtype, s);
}

} // namespace ttemb
