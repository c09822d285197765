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

// Lane j of a row gets the sum over the row's lanes of x[j].  Halves of the row, then of
// those, exchange what they do not keep: x[k] + its exchange goes to all lanes, and that of
// x[k + 8] (k + 4) over the upper half (the bank mask names groups of four lanes whose
// result is written).  Written with selections the compiler takes 47 instructions, this 35.
// An operand of an exchange has to be two instructions old: s_nop 1 sees to it for what
// comes in, and the order below has it for the rest.  Results are written before the last
// operand is read: none may share its register, not even where both hold one value ("&").
__device__ __forceinline__ float over_lanes(const float (&in)[16], int lane)
{
    float x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k)
        x[k] = in[k];
#define EXCHANGE(k, from, ctrl, mask) "v_add_f32_dpp %" #k ", %" #from ", %" #from " " ctrl " row_mask:0xf bank_mask:" mask "\n\t"
#define BOTH(k, far, ctrl, mask) EXCHANGE(k, k, ctrl, "0xf") EXCHANGE(k, far, ctrl, mask)
#define FAR(k, far) BOTH(k, far, "row_ror:8", "0xc")         // lanes l and l + 8
#define MID(k, far) BOTH(k, far, "row_half_mirror", "0xa")   // l and l ^ 7
    asm("s_nop 1\n\t"
        FAR(0, 8) FAR(1, 9) FAR(2, 10) FAR(3, 11) FAR(4, 12) FAR(5, 13) FAR(6, 14) FAR(7, 15)
        MID(0, 4) MID(1, 5) MID(2, 6) MID(3, 7)
        EXCHANGE(0, 0, "quad_perm:[2,3,0,1]", "0xf") EXCHANGE(1, 1, "quad_perm:[2,3,0,1]", "0xf")
        EXCHANGE(2, 2, "quad_perm:[2,3,0,1]", "0xf") EXCHANGE(3, 3, "quad_perm:[2,3,0,1]", "0xf")
        EXCHANGE(0, 0, "quad_perm:[1,0,3,2]", "0xf") EXCHANGE(1, 1, "quad_perm:[1,0,3,2]", "0xf")
        EXCHANGE(2, 2, "quad_perm:[1,0,3,2]", "0xf") EXCHANGE(3, 3, "quad_perm:[1,0,3,2]", "0xf")
        : "+&v"(x[0]), "+&v"(x[1]), "+&v"(x[2]), "+&v"(x[3]), "+&v"(x[4]), "+&v"(x[5]), "+&v"(x[6]), "+&v"(x[7])
        : "v"(x[8]), "v"(x[9]), "v"(x[10]), "v"(x[11]), "v"(x[12]), "v"(x[13]), "v"(x[14]), "v"(x[15]));
#undef MID
#undef FAR
#undef BOTH
#undef EXCHANGE
    const float lo = lane & 1 ? x[1] : x[0], hi = lane & 1 ? x[3] : x[2];
    return lane & 2 ? hi : lo;
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
