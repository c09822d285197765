// Rows of a sequence held as vectors of channels, and the exponentials that the
// convolution and the scan share.
#pragma once

#include "lowp.hpp"

namespace chol {

// A [batch, len, dim] array with unit channel stride.
struct SeqRows {
    void *p;
    int64_t ld, stride;
};

// V elements from p of which the first n exist (n may be below zero), `none` past them.
template <typename T, int V> __device__ __forceinline__ vec<T, V> load_some(const T *p, int64_t n, T none = (T)0.f)
{
    if (n >= V)
        return load_vec<T, V>(p);
    vec<T, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (V == 1)
            v = i < n ? p[i] : none;
        else
            v[i] = i < n ? p[i] : none;
    }
    return v;
}
template <typename T, int V> __device__ __forceinline__ void store_some(T *p, int64_t n, vec<T, V> v)
{
    if (n >= V) {
        store_vec<T, V>(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < n)
            p[i] = (T)lane_of<T, V>(v, i);
}

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

// exp(x) from the hardware's 2^y.  Rounding y = x log2(e) changes the result by up to
// |x| 2^-24 of itself; where the result is kept in fp32 (FULL) the product's low part
// is applied as well.
template <bool FULL> __device__ __forceinline__ float expf_of(float x)
{
    const float y = x * LOG2E, e = __builtin_amdgcn_exp2f(y);
    if constexpr (!FULL)
        return e;
    const float low = fmaf(x, (float)(1.4426950408889634074 - LOG2E), fmaf(x, LOG2E, -y));
    return fabsf(y) < 128.f ? fmaf(e * LN2, low, e) : e; // (beyond, it is 0 or inf)
}

// 1 / (1 + exp(-x)); `full`: to a few units of fp32 at any x, else to |x| of them
template <bool FULL> __device__ __forceinline__ float sigmoid_of(float x)
{
    return __builtin_amdgcn_rcpf(1.f + expf_of<FULL>(-x));
}

} // namespace chol
