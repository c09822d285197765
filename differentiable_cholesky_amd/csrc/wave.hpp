// Exchanges between the lanes of a wave that stay in its registers: within a row of 16
// lanes by data-parallel primitives, across rows by swaps.
#pragma once

#include <hip/hip_runtime.h>

namespace chol {

template <int CTRL, typename T> __device__ __forceinline__ T dpp(T x)
{
    static_assert(sizeof(T) == 4, "");
    return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
// lane K of the lane's row
template <int K, typename T> __device__ __forceinline__ T of_row(T x) { return dpp<0x150 + K>(x); }

template <typename T> struct Two {
    T a, b;
};
// a: x's lower half and y's lower half; b: x's upper half and y's upper half
template <typename T> __device__ __forceinline__ Two<T> swap_halves(T x, T y)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y), false, false);
    const unsigned p = r[0], q = r[1]; // (elements of a vector have no address to cast from)
    return {__builtin_bit_cast(T, p), __builtin_bit_cast(T, q)};
}
// a: x's even rows, with y's even rows in the odd places; b: x's odd rows in the even
// places, with y's odd rows
template <typename T> __device__ __forceinline__ Two<T> swap_rows(T x, T y)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y), false, false);
    const unsigned p = r[0], q = r[1];
    return {__builtin_bit_cast(T, p), __builtin_bit_cast(T, q)};
}

// f over the 64 lanes, in every lane and in one order.
template <typename T, typename F> __device__ __forceinline__ T over_wave(T x, F f)
{
    x = f(x, dpp<0xb1>(x));  // lanes 1 0 3 2 of four
    x = f(x, dpp<0x4e>(x));  // lanes 2 3 0 1
    x = f(x, dpp<0x141>(x)); // the other four of eight
    x = f(x, dpp<0x140>(x)); // the other eight of the row
    const Two<T> r = swap_rows(x, x);
    x = f(r.a, r.b);
    const Two<T> h = swap_halves(x, x);
    return f(h.a, h.b);
}

// LDS written by lanes of a wave and read by others of the same wave, whose operations
// on it are in order.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

} // namespace chol
