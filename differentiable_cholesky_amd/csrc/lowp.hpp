// Element types of the sequence, norm and optimiser kernels (fp32, bf16, fp16,
// and e4m3 for 8-bit outputs and states) and their loads and stores.  All
// arithmetic is fp32: a load widens, a store rounds once, to nearest even.
#pragma once

#include "common.hpp"

namespace chol {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

inline bool lowp_dtype(chol_dtype dt) { return dt == CHOL_F32 || dt == CHOL_BF16 || dt == CHOL_F16; }
inline size_t lowp_size(chol_dtype dt) { return dt == CHOL_F32 ? 4 : 2; }

template <typename T, int V> struct VecOf {
    typedef T type __attribute__((ext_vector_type(V)));
};
template <typename T> struct VecOf<T, 1> {
    typedef T type;
};
template <typename T, int V> using vec = typename VecOf<T, V>::type;

// V elements at an address aligned to one element: global loads and stores of
// up to 16 bytes take any address, so ragged rows need no variant of their own.
template <typename T, int V> __device__ __forceinline__ vec<T, V> load_vec(const T *p)
{
    vec<T, V> v;
    __builtin_memcpy(&v, p, sizeof(T) * V);
    return v;
}
template <typename T, int V> __device__ __forceinline__ void store_vec(T *p, vec<T, V> v)
{
    __builtin_memcpy(p, &v, sizeof(T) * V);
}

template <typename T, int V> __device__ __forceinline__ float lane_of(const vec<T, V> &v, int i)
{
    if constexpr (V == 1)
        return (float)v;
    else
        return (float)v[i];
}
template <typename T, int V> __device__ __forceinline__ void set_lane(vec<T, V> &v, int i, float x)
{
    if constexpr (V == 1)
        v = (T)x;
    else
        v[i] = (T)x;
}

// Runs f(T *) for the element type of a dtype code (one of lowp_dtype's).
template <typename F> inline chol_status with_lowp(chol_dtype dt, F f)
{
    switch (dt) {
    case CHOL_F32: return f((float *)nullptr);
    case CHOL_BF16: return f((bf16_t *)nullptr);
    case CHOL_F16: return f((f16_t *)nullptr);
    default: return CHOL_ERR_INVALID_VALUE;
    }
}

} // namespace chol
