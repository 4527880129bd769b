// blocknorm.h -- what the forward and the backward of the norms between blocks
// share: how many threads a row has, and the types they are built for.
#pragma once

#include "norm.h"

namespace ttemb {

namespace {

constexpr int kBlockVec = 8;         // neighbouring elements of a thread, of every type
constexpr int64_t kBlockRegs = 4096; // longest rows that are held in registers

// Columns c .. c + VEC - 1 of a row, still in their own type.  Not WHOLE (D is no
// multiple of VEC): the vector that the row's end cuts, and those past it, are
// the row's last VEC elements, so that every load is issued without a condition;
// `values` moves them into place.
template <class T, bool WHOLE>
__device__ __forceinline__ typename VecOf<T, kBlockVec>::raw load_cols(const T *row, int c, int D)
{
    constexpr int VEC = kBlockVec;
    typedef typename VecOf<T, VEC>::type vec;
    if constexpr (WHOLE) return *reinterpret_cast<const vec *>(row + (c < D ? c : 0));
    if (D >= VEC) return *reinterpret_cast<const vec *>(row + (c + VEC <= D ? c : D - VEC));
    typename VecOf<T, VEC>::raw v;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = c + i < D ? row[c + i] : (T)0.f;
    return v;
}
// Those of a thread whose vector has `left` elements of the row, zeros past them.
template <class T, bool WHOLE>
__device__ __forceinline__ void values(const typename VecOf<T, kBlockVec>::raw &v, int left, int D,
                                       float (&x)[kBlockVec])
{
    constexpr int VEC = kBlockVec;
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = (float)v[i];
    if constexpr (WHOLE) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = left > 0 ? x[i] : 0.f;
    } else if (left < VEC && D >= VEC) {
        for (int shift = left > 0 ? left : 0; shift < VEC; ++shift) {
#pragma unroll
            for (int i = 0; i + 1 < VEC; ++i) x[i] = x[i + 1];
            x[VEC - 1] = 0.f;
        }
    }
}

// Blocks for so many groups of rows, at most `most`, with equal shares.
inline int block_grid(int64_t need, int64_t most)
{
    const int64_t rounds = (need + most - 1) / most;
    return (int)((need + rounds - 1) / rounds);
}

// Threads of a row of D <= kBlockRegs elements, eight each: the fewest of these that
// hold it, as idle ones cost as much as others (131072 x 256 bf16: forward 52 us, backward
// 64 with 32 threads, 82 and 112 with 64; 131072 x 144 fp32: 64 and 85, 87 and 143).
template <class F>
hipError_t block_shape(int64_t D, F &&f)
{
    auto g = [&](auto tpr) {
        if (D % kBlockVec == 0) return f(tpr, std::true_type());
        return f(tpr, std::false_type());
    };
    if (D <= 128) return g(std::integral_constant<int, 16>());
    if (D <= 256) return g(std::integral_constant<int, 32>());
    if (D <= 512) return g(std::integral_constant<int, 64>());
    if (D <= 1024) return g(std::integral_constant<int, 128>());
    if (D <= 2048) return g(std::integral_constant<int, 256>());
    return g(std::integral_constant<int, 512>());
}
constexpr int kBlockLong = 512; // threads of a longer row, which take its parts of 4096 in turn

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
