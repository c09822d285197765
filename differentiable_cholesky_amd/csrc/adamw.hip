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
// step is bound by memory: a workgroup is one wave, with one vector of four
// elements a lane, and loads and stores leave the caches alone.  302 M elements,
// bf16 with fp32 master, us with 32-bit and with 8-bit states:
//   a workgroup of 256 that walks 4096 elements           1670   987
//   the same without the caches                           1590   949
//   a workgroup of 256 for 1024 elements                  1423   929
//   of 64 for 256                                         1351   907
//   and the tile's largest over the lanes without LDS     1352   871
// (6.3 and 5.6 TB/s; a copy reaches 5.2).  With 8-bit states the arithmetic of the
// codes and the random bits takes nearly as long as the memory.
#include <algorithm>
#include <type_traits>

#include "adamw.hpp"
#include "lowp.hpp"

namespace chol {

namespace {

constexpr int THREADS = 64, V = 4; // a wave's 64 x 4 elements are one tile of 256
constexpr int PARTS = ADAMW_CHUNK / (THREADS * V); // workgroups of a chunk

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x)
{
    x ^= x >> 16;
    x *= 0x9E3779B1u;
    x ^= x >> 15;
    x *= 0x85EBCA77u;
    return x ^ (x >> 16);
}

// V elements at an address aligned to one of them
template <typename T> __device__ __forceinline__ vec<T, V> load_once(const T *p)
{
    if constexpr (sizeof(T) == 4) {
        typedef float any __attribute__((ext_vector_type(4), aligned(4)));
        return __builtin_nontemporal_load((const any *)p);
    } else {
        typedef uint64_t any __attribute__((aligned(2)));
        return __builtin_bit_cast(vec<T, V>, __builtin_nontemporal_load((const any *)p));
    }
}
template <typename T> __device__ __forceinline__ void store_once(T *p, vec<T, V> v)
{
    if constexpr (sizeof(T) == 4) {
        typedef float any __attribute__((ext_vector_type(4), aligned(4)));
        __builtin_nontemporal_store((any)v, (any *)p);
    } else {
        typedef uint64_t any __attribute__((aligned(2)));
        __builtin_nontemporal_store(__builtin_bit_cast(uint64_t, v), (any *)p);
    }
}

// V elements of which n are there (all of them, or the last of a tensor)
template <typename T> __device__ __forceinline__ void read(const void *base, uint32_t at, int n, float (&x)[V])
{
    const T *p = (const T *)base + at;
    if (n == V) {
        const vec<T, V> v = load_once(p);
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
        store_once(p, v);
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

// e4m3 code of a finite y (|y| < 256), rounded away from zero where the 16 random
// bits and what is dropped carry
__device__ __forceinline__ unsigned code_of(float y, unsigned noise, bool keep)
{
    const unsigned bits = __float_as_uint(y), mag = bits & 0x7fffffffu;
    // normal codes (from 2^-6): the noise is added below the three mantissa
    // bits that stay, and the exponent's bias goes from 127 to 7
    const unsigned normal = ((mag + (noise << 4)) >> 20) - (120u << 3);
    // below: multiples of 2^-9, counted in 2^-16 of them
    const unsigned small = (unsigned)fmaf(fabsf(y), 0x1p25f, (float)noise) >> 16;
    unsigned c = mag < 0x3c800000u ? small : normal;
    if (keep)
        c = max(c, min(mag, 1u));
    return c | ((bits >> 24) & 0x80u);
}

// The correctly rounded root of a value in 2^-100 .. 2^100: with the hardware's
// estimate y of x^(-1/2) and s = x y, the residual r = x - s^2 is exact, and
// s + r y / 2 rounds correctly for every mantissa (all 2^24 of two binades, at
// eleven exponents, compared with 64 bits; the hardware's own root fails 15%).
__device__ __forceinline__ float root_of(float x)
{
    const float y = __builtin_amdgcn_rsqf(x), s = x * y;
    return fmaf(fmaf(-s, s, x), 0.5f * y, s);
}

__device__ __forceinline__ void roots(const float (&x)[V], float (&root)[V])
{
    unsigned far = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        far = max(far, __float_as_uint(x[i]) - (27u << 23));
    if (__all(far < (200u << 23))) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            root[i] = root_of(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool low = x[i] < 0x1p-60f, high = x[i] > 0x1p+60f;
            const float r = root_of(x[i] * (low ? 0x1p+100f : high ? 0x1p-100f : 1.f));
            const float other = x[i] < 0.f ? NAN : x[i]; // zero, inf and NaN are their own roots
            root[i] = x[i] > 0.f && x[i] < INFINITY ? r * (low ? 0x1p-50f : high ? 0x1p+50f : 1.f) : other;
        }
    }
}

// largest of the wave's values, in every lane: over the 16 lanes of a row, then
// rows 0 and 2 into 1 and 3, and 1 into 3
__device__ __forceinline__ unsigned wave_max(unsigned x)
{
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0xb1, 0xf, 0xf, false));  // lanes xor 1
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x4e, 0xf, 0xf, false));  // lanes xor 2
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xf, 0xf, false)); // mirror of 8
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xf, 0xf, false)); // mirror of 16
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xa, 0xf, false));
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xc, 0xf, false));
    return (unsigned)__builtin_amdgcn_readlane((int)x, 63);
}

// Codes and scale of a tile held by the wave
__device__ __forceinline__ void write_codes(void *base, float *scale, uint32_t at, int n, const float (&x)[V],
                                            const unsigned (&noise)[V], bool keep)
{
    unsigned most = 0;
#pragma unroll
    for (int k = 0; k < V; ++k)
        most = max(most, __float_as_uint(x[k]) & 0x7fffffffu);
    most = wave_max(most);
    const bool finite = most < 0x7f800000u; // the same for the whole wave
    if (!finite) { // the scale is that of the finite values: the others have no part in their neighbours' codes
        most = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const unsigned mag = __float_as_uint(x[k]) & 0x7fffffffu;
            most = max(most, mag < 0x7f800000u ? mag : 0u);
        }
        most = wave_max(most);
    }
    const int e = max((int)(most >> 23) - 7, 1);
    const float inv = __uint_as_float((unsigned)(254 - e) << 23);
    unsigned u = 0;
    if (finite) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            u |= code_of(x[k] * inv, noise[k], keep) << (8 * k);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const unsigned bits = __float_as_uint(x[k]), nan = 0x7fu | ((bits >> 24) & 0x80u);
            u |= ((bits & 0x7fffffffu) < 0x7f800000u ? code_of(x[k] * inv, noise[k], keep) : nan) << (8 * k);
        }
    }
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
    const AdamwChunk c = table[blockIdx.x / PARTS];
    const float clip = k.grad_scale ? *k.grad_scale : 1.f;
    const uint32_t at = (blockIdx.x % PARTS * THREADS + threadIdx.x) * V;
    if (at / ADAMW_TILE * ADAMW_TILE >= c.n) // whole waves stay for their tile's scale
        return;
    const int n = at < c.n ? min((int)(c.n - at), V) : 0;
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
    }
    roots(v, root);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        p[i] = p[i] - p[i] * k.decay;
        // (the hardware's reciprocal, within a step of fp32: the update is small beside p)
        p[i] = p[i] - k.rate * m[i] * __builtin_amdgcn_rcpf(root[i] * k.inv_root + k.eps);
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

} // namespace

uint32_t adamw_mix(uint32_t x) { return mix(x); }

chol_status adamw(chol_dtype dt, int bits, bool master, int64_t chunks, const AdamwChunk *table, const AdamwHyper &k,
                  hipStream_t st)
{
    return with_lowp(dt, [&](auto *e) {
        typedef std::remove_pointer_t<decltype(e)> T;
        constexpr int64_t MOST = (int64_t)1 << 21; // chunks of a launch: a grid holds < 2^32 threads
        for (int64_t first = 0; first < chunks; first += MOST) {
            const dim3 grid((unsigned)(std::min(MOST, chunks - first) * PARTS)), block(THREADS);
            const AdamwChunk *t = table + first;
            if (master && bits == 8)
                hipLaunchKernelGGL((k_adamw<T, true, true>), grid, block, 0, st, t, k);
            else if (master)
                hipLaunchKernelGGL((k_adamw<T, true, false>), grid, block, 0, st, t, k);
            else if (bits == 8)
                hipLaunchKernelGGL((k_adamw<T, false, true>), grid, block, 0, st, t, k);
            else
                hipLaunchKernelGGL((k_adamw<T, false, false>), grid, block, 0, st, t, k);
            CHOL_LAUNCH_CHECK();
        }
        return CHOL_OK;
    });
}

} // namespace chol
