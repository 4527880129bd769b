// blocknorm.h -- what the forward and the backward of the norms between blocks
// share: how many threads a row has, and the types they are built for.
#pragma once

#include "norm.h"

namespace ttemb {

namespace {

constexpr int kBlockVec = 8;         // neighbouring elements of a thread, of every type
constexpr int64_t kBlockRegs = 4096; // longest rows whose column sums stay in registers

// Threads of a row of D elements, eight each (sixteen past 8192).
template <class F>
hipError_t block_shape(int64_t D, F &&f)
{
    auto g = [&](auto tpr, auto nv) {
        if (D % kBlockVec == 0) return f(tpr, nv, std::true_type());
        return f(tpr, nv, std::false_type());
    };
    constexpr std::integral_constant<int, 1> one;
    if (D <= 128) return g(std::integral_constant<int, 16>(), one);
    if (D <= 512) return g(std::integral_constant<int, 64>(), one);
    if (D <= 2048) return g(std::integral_constant<int, 256>(), one);
    if (D <= kBlockRegs) return g(std::integral_constant<int, 512>(), one);
    if (D <= 8192) return g(std::integral_constant<int, 1024>(), one);
    return g(std::integral_constant<int, 1024>(), std::integral_constant<int, 2>());
}

// Types of x and of the residual.
template <class F>
hipError_t block_types(int dtype, int res_dtype, F f)
{
    if (dtype == TT_EMB_DTYPE_FLOAT) return f(float(), float());
    if (dtype == TT_EMB_DTYPE_BFLOAT)
        return res_dtype == TT_EMB_DTYPE_FLOAT ? f(bf16(), float()) : f(bf16(), bf16());
    return res_dtype == TT_EMB_DTYPE_FLOAT ? f(f16(), float()) : f(f16(), f16());
}

} // namespace

} // namespace ttemb
