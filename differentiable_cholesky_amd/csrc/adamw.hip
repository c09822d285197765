// AdamW over many tensors in one launch, states in fp32 or in e4m3.
//
//   g' = grad_scale g,  m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
//   p -= lr wd p,  p -= lr / (1 - beta1^t) m / (sqrt(v) (1 - beta2^t)^(-1/2) + eps)
//
// In 8 bits m and sqrt(v) are kept as e4m3 codes of x / scale, the scale a power
// of two per 256 elements of a tensor that brings the largest of them into
// [2^7, 2^8).  The codes are rounded up or down by random bits, so that small
// changes of a state survive on average.  Products and sums of the states round
// one by one (no contraction into fused operations): a value that lies at a
// power of two then gives the same scale on any implementation of the formulas.
//
// Every element is independent and everything is read and written once, so the
// step is bound by memory.
#include <type_traits>

#include "adamw.hpp"
#include "lowp.hpp"

namespace chol {

namespace {

constexpr int THREADS = 256, V = 4; // a wave's 64 x 4 elements are one tile of 256

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x ^= x >> 16;
    x *= 0x9E3779B1u;
    x ^= x >> 15;
    x *= 0x85EBCA77u;
    return x ^ (x >> 16);
}

// V elements of which n are there (all of them, or the last of a tensor)
template <typename T> __device__ __forceinline__ void read(const void *base, uint32_t at, int n, float (&x)[V])
{
    const T *p = (const T *)base + at;
    if (n == V) {
        const vec<T, V> v = load_vec<T, V>(p);
#pragma unroll
        for (int k = 0; k < V; ++k)
            x[k] = (float)v[k];
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            x[k] = k < n ? (float)p[k] : 0.f;
    }
}
template <typename T> __device__ __forceinline__ void write(void *base, uint32_t at, int n, const float (&x)[V])
{
    T *p = (T *)base + at;
    if (n == V) {
        vec<T, V> v;
#pragma unroll
        for (int k = 0; k < V; ++k)
            v[k] = (T)x[k];
        store_vec<T, V>(p, v);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < n)
                p[k] = (T)x[k];
    }
}

// the values four codes stand for, before their scale
__device__ __forceinline__ void read_codes(const void *base, uint32_t at, int n, float (&x)[V])
{
    const unsigned char *p = (const unsigned char *)base + at;
    unsigned u = 0;
    if (n == V) {
        __builtin_memcpy(&u, p, V);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < n)
                u |= (unsigned)p[k] << (8 * k);
    }
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, true);
    x[0] = lo[0], x[1] = lo[1], x[2] = hi[0], x[3] = hi[1];
}

// e4m3 code of y (|y| < 256 unless inf or NaN), rounded away from zero where
// the 16 random bits and what is dropped carry
__device__ __forceinline__ unsigned code_of(float y, unsigned noise, bool keep)
{
    const unsigned bits = __float_as_uint(y), mag = bits & 0x7fffffffu;
    // normal codes (from 2^-6): the noise is added below the three mantissa
    // bits that stay, and the exponent's bias goes from 127 to 7
    unsigned c = ((mag + (noise << 4)) >> 20) - (120u << 3);
    // below: multiples of 2^-9
    if (mag < 0x3c800000u)
        c = (unsigned)floorf(fabsf(y) * 512.f + (float)noise * 0x1p-16f);
    if (keep && mag != 0 && c == 0)
        c = 1;
    if (mag >= 0x7f800000u)
        c = 0x7f;
    return c | ((bits >> 24) & 0x80u);
}

// Codes and scale of a tile held by the wave
__device__ __forceinline__ void write_codes(void *base, float *scale, uint32_t at, int n, const float (&x)[V],
                                            const unsigned (&noise)[V], bool keep)
{
    unsigned most = 0;
#pragma unroll
    for (int k = 0; k < V; ++k)
        most = max(most, __float_as_uint(x[k]) & 0x7fffffffu);
#pragma unroll
    for (int o = 32; o > 0; o /= 2)
        most = max(most, (unsigned)__shfl_xor((int)most, o));
    const int e = max((int)(most >> 23) - 7, 1);
    const float inv = __uint_as_float((unsigned)(254 - e) << 23);
    unsigned u = 0;
#pragma unroll
    for (int k = 0; k < V; ++k)
        u |= code_of(x[k] * inv, noise[k], keep) << (8 * k);
    unsigned char *p = (unsigned char *)base + at;
    if (n == V) {
        __builtin_memcpy(p, &u, V);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < n)
                p[k] = (unsigned char)(u >> (8 * k));
    }
    if (threadIdx.x % 64 == 0)
        scale[at / ADAMW_TILE] = __uint_as_float((unsigned)e << 23);
}

template <typename T, bool MASTER, bool BITS8>
__global__ void __launch_bounds__(THREADS) k_adamw(const AdamwChunk *table, AdamwHyper k)
{
#pragma clang fp contract(off)
    const AdamwChunk c = table[blockIdx.x];
    const float clip = k.grad_scale ? *k.grad_scale : 1.f;
    for (uint32_t at = threadIdx.x * V; at / ADAMW_TILE * ADAMW_TILE < c.n; at += THREADS * V) {
        const int n = at < c.n ? min((int)(c.n - at), V) : 0; // whole waves stay for their tile's scale
        float p[V], g[V], m[V], v[V], root[V];
        if constexpr (MASTER)
            read<float>(c.master, at, n, p);
        else
            read<T>(c.p, at, n, p);
        read<T>(c.g, at, n, g);
        if constexpr (BITS8) {
            const float ms = c.m_scale[at / ADAMW_TILE], vs = c.v_scale[at / ADAMW_TILE];
            read_codes(c.m, at, n, m);
            read_codes(c.v, at, n, v);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float r = v[i] * vs;
                m[i] = m[i] * ms;
                v[i] = r * r;
            }
        } else {
            read<float>(c.m, at, n, m);
            read<float>(c.v, at, n, v);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float x = g[i] * clip;
            m[i] = m[i] * k.beta1 + x * k.one_beta1;
            v[i] = v[i] * k.beta2 + x * x * k.one_beta2;
            root[i] = __fsqrt_rn(v[i]);
            p[i] = p[i] - p[i] * k.decay;
            p[i] = p[i] - k.rate * m[i] * __frcp_rn(root[i] * k.inv_root + k.eps);
        }
        if constexpr (MASTER)
            write<float>(c.master, at, n, p);
        write<T>(c.p, at, n, p);
        if constexpr (BITS8) {
            unsigned lo[V], hi[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t r = mix(c.first + at + i + k.key);
                lo[i] = r & 0xffffu;
                hi[i] = r >> 16;
            }
            write_codes(c.m, c.m_scale, at, n, m, lo, false);
            write_codes(c.v, c.v_scale, at, n, root, hi, true);
        } else {
            write<float>(c.m, at, n, m);
            write<float>(c.v, at, n, v);
        }
    }
}

} // namespace

uint32_t adamw_mix(uint32_t x) { return mix(x); }

chol_status adamw(chol_dtype dt, int bits, bool master, int64_t chunks, const AdamwChunk *table, const AdamwHyper &k,
                  hipStream_t st)
{
    return with_lowp(dt, [&](auto *e) {
        typedef std::remove_pointer_t<decltype(e)> T;
        const dim3 grid((unsigned)chunks), block(THREADS);
        if (master && bits == 8)
            hipLaunchKernelGGL((k_adamw<T, true, true>), grid, block, 0, st, table, k);
        else if (master)
            hipLaunchKernelGGL((k_adamw<T, true, false>), grid, block, 0, st, table, k);
        else if (bits == 8)
            hipLaunchKernelGGL((k_adamw<T, false, true>), grid, block, 0, st, table, k);
        else
            hipLaunchKernelGGL((k_adamw<T, false, false>), grid, block, 0, st, table, k);
        CHOL_LAUNCH_CHECK();
        return CHOL_OK;
    });
}

} // namespace chol
