// RMS norm with the residual's addition, an output in the input's type or in
// e4m3 with scales, and the adjoint.
//
//   h = rnd(x + r),  s = (mean h^2 + eps)^(-1/2),  y = h s w
//   adj_x = s (g - h s^2 mean(g h)) + adj_h with g = adj w,  adj_w = sum_rows adj h s
//
// A row stays in the registers of TPR threads, NV vectors of 16 bytes each, so
// the data is read once and written once, which is what bounds these kernels.
// Sums and maxima cross the lanes of a wave by shuffles and waves through LDS.
#include <algorithm>
#include <type_traits>

#include "lowp.hpp"
#include "rmsnorm.hpp"

namespace chol {

namespace {

constexpr int WAVE = 64;
constexpr float E4M3_MAX = 448.f;

template <typename T> constexpr int vec_of = 16 / (int)sizeof(T);
// threads of a workgroup: a row of more than a wave has its own, whose LDS it uses
template <int TPR> constexpr int block_of = TPR > WAVE ? TPR : 256;

// A call that moves well over the 256 MB which the last cache holds reads past it
// (STREAM), and leaves it to what is written.  Norm of n x 4096 bf16 between a
// kernel that writes its input and one that reads its output, us for the three:
// 16384 rows 177 -> 167, 12288 (403 MB) 130 -> 127, but 8192 (268 MB) 86 -> 90.
constexpr double CACHE = 320e6;

// NV vectors of one row, thread `t` of TPR holding vectors t, t + TPR, ...; zero
// past the end of the row.
template <typename T, int TPR, int NV> struct Row {
    static constexpr int V = vec_of<T>;
    vec<T, V> v[NV];
    template <bool STREAM> __device__ __forceinline__ void load(const T *p, int t, int cols)
    {
        typedef unsigned any __attribute__((ext_vector_type(4), aligned(2)));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            if (c + V <= cols) {
                if constexpr (STREAM)
                    v[i] = __builtin_bit_cast(vec<T, V>, __builtin_nontemporal_load((const any *)(p + c)));
                else
                    v[i] = load_vec<T, V>(p + c);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    v[i][k] = c + k < cols ? p[c + k] : (T)0.f;
            }
        }
    }
    __device__ __forceinline__ void store(T *p, int t, int cols) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            if (c + V <= cols) {
                store_vec<T, V>(p + c, v[i]);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (c + k < cols)
                        p[c + k] = v[i][k];
            }
        }
    }
    __device__ __forceinline__ float at(int i, int k) const { return (float)v[i][k]; }
    __device__ __forceinline__ void set(int i, int k, float x) { v[i][k] = (T)x; }
};

struct Sum {
    static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct Max {
    static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};
// largest magnitude by its bits: as integers, finite < inf < NaN
struct MaxBits {
    static __device__ __forceinline__ unsigned of(unsigned a, unsigned b) { return a > b ? a : b; }
};

// Over the TPR threads of a row (all of them get the result).  `slot`: LDS of
// TPR / WAVE values of this row's own, not used by the call before.
template <int TPR, typename Op, typename S> __device__ __forceinline__ S over_row(S x, int t, S *slot)
{
#pragma unroll
    for (int o = (TPR < WAVE ? TPR : WAVE) / 2; o > 0; o /= 2)
        x = Op::of(x, __shfl_xor(x, o));
    if constexpr (TPR > WAVE) {
        if (t % WAVE == 0)
            slot[t / WAVE] = x;
        __syncthreads();
        x = slot[0];
#pragma unroll
        for (int i = 1; i < TPR / WAVE; ++i)
            x = Op::of(x, slot[i]);
    }
    return x;
}

// e4m3 codes of V values, to nearest even, at a byte address
template <int V> __device__ __forceinline__ void store_e4m3(unsigned char *p, const float (&q)[V], int n)
{
    unsigned word[V / 4];
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
        int u = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * k], q[4 * k + 1], 0, false);
        word[k] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * k + 2], q[4 * k + 3], u, true);
    }
    if (n >= V) {
        __builtin_memcpy(p, word, V);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < n)
                p[k] = (unsigned char)(word[k / 4] >> (8 * (k % 4)));
    }
}

template <typename T, int TPR, int NV, bool QUANT, bool STREAM>
__global__ void __launch_bounds__(block_of<TPR>) k_rmsnorm(NormArgs a, int64_t first)
{
    // the low parts below are what a rounded product lost
#pragma clang fp contract(off)
    constexpr int V = vec_of<T>, BLOCK = block_of<TPR>;
    __shared__ float s_sum[TPR > WAVE ? TPR / WAVE : 1];
    __shared__ unsigned s_max[TPR > WAVE ? TPR / WAVE : 1];
    __shared__ float s_low[TPR > WAVE ? TPR / WAVE : 1];
    const int t = threadIdx.x % TPR, cols = (int)a.cols;
    const int64_t row = first + (int64_t)blockIdx.x * (BLOCK / TPR) + threadIdx.x / TPR;
    if (row >= a.rows) // whole rows: no lane of one that stays is missing
        return;
    Row<T, TPR, NV> h, w;
    h.template load<STREAM>((const T *)a.x + row * a.ldx, t, cols);
    if (a.residual) {
        Row<T, TPR, NV> r;
        r.template load<STREAM>((const T *)a.residual + row * a.ldr, t, cols);
        w.template load<false>((const T *)a.w, t, cols);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k)
                h.set(i, k, h.at(i, k) + r.at(i, k));
        h.store((T *)a.h + row * a.ldh, t, cols);
    } else {
        w.template load<false>((const T *)a.w, t, cols);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k)
            sum = fmaf(h.at(i, k), h.at(i, k), sum);
    const float s = rsqrtf(over_row<TPR, Sum>(sum, t, s_sum) / (float)cols + a.eps);
    if constexpr (!QUANT) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k)
                h.set(i, k, h.at(i, k) * s * w.at(i, k));
        h.store((T *)a.y + row * a.ldy, t, cols);
    } else {
        // s is common to the row: a code is h w / max |h w| * 448.  That is formed in
        // two parts, so that the value a code is rounded from is right to half a step
        // of fp32: the product's low part (exactly zero for 16-bit types), that of
        // the largest, and that of 448 over it.
        constexpr bool LOW = sizeof(T) == 4;
        float y[NV][V], low[NV];
        unsigned most[NV];
        const auto low_part = [&](int i, int k) { return LOW ? fmaf(h.at(i, k), w.at(i, k), -y[i][k]) : 0.f; };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            most[i] = 0;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                y[i][k] = h.at(i, k) * w.at(i, k);
                most[i] = MaxBits::of(most[i], __float_as_uint(y[i][k]) & 0x7fffffffu);
            }
        }
        // a group is `lanes` neighbouring vectors of one wave, or the row
        const int lanes = a.group / V < TPR ? a.group / V : TPR;
        if (a.group) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                for (int o = 1; o < lanes; o *= 2)
                    most[i] = MaxBits::of(most[i], __shfl_xor(most[i], o));
        } else {
#pragma unroll
            for (int i = 1; i < NV; ++i)
                most[0] = MaxBits::of(most[0], most[i]);
            most[0] = over_row<TPR, MaxBits>(most[0], t, s_max);
        }
        if constexpr (LOW) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                low[i] = -INFINITY;
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if ((__float_as_uint(y[i][k]) & 0x7fffffffu) == most[a.group ? i : 0])
                        low[i] = fmaxf(low[i], y[i][k] < 0.f ? -low_part(i, k) : low_part(i, k));
            }
            if (a.group) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    for (int o = 1; o < lanes; o *= 2)
                        low[i] = fmaxf(low[i], __shfl_xor(low[i], o));
            } else {
#pragma unroll
                for (int i = 1; i < NV; ++i)
                    low[0] = fmaxf(low[0], low[i]);
                low[0] = over_row<TPR, Max>(low[0], t, s_low);
            }
        }
        unsigned char *q = (unsigned char *)a.y + row * a.ldy;
        float *scale = a.scale + row * a.lds;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * V;
            const float m = __uint_as_float(a.group ? most[i] : most[0]), top = m * s;
            // one for a group of zeros (or with a NaN); not below the smallest
            // normal number, whose reciprocal still is one
            const bool some = top > 0.f;
            const float sc = some ? fmaxf(__fdiv_rn(top, E4M3_MAX), 0x1p-126f) : 1.f;
            const bool plain = some && sc > 0x1p-126f && m > 0x1p-110f; // 448 / m is finite
            const float inv = __fdiv_rn(plain ? E4M3_MAX : 1.f, plain ? m : sc);
            float inv_low = 0.f;
            if (plain && m < INFINITY) {
                inv_low = fmaf(-inv, m, E4M3_MAX);
                if constexpr (LOW)
                    inv_low = fmaf(-inv, low[a.group ? i : 0], inv_low);
                inv_low *= inv * (1.f / E4M3_MAX);
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float x = plain ? y[i][k] : y[i][k] * s, hi = x * inv;
                y[i][k] = hi + fmaf(x, inv_low, fmaf(x, inv, -hi) + (plain ? low_part(i, k) * inv : 0.f));
            }
            if (c < cols) {
                store_e4m3<V>(q + c, y[i], cols - c);
                if (a.group ? c % a.group == 0 : c == 0)
                    scale[a.group ? c / a.group : 0] = sc;
            }
        }
    }
}

// Rows blockIdx.x * RPB + slot, then a grid further on; every thread sums its
// columns' adj h s over its rows.  part[blockIdx.x * cols + c], or adj_w itself
// where the grid is one block.
template <typename T, int TPR, int NV, bool STREAM>
__global__ void __launch_bounds__(block_of<TPR>) k_rmsnorm_adjoint(NormAdjArgs a, float *part)
{
    constexpr int V = vec_of<T>, BLOCK = block_of<TPR>, RPB = BLOCK / TPR;
    __shared__ float s_sum[2][TPR > WAVE ? 2 * TPR / WAVE : 1];
    __shared__ float s_w[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? TPR * NV * V : 1];
    const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR, cols = (int)a.cols;
    Row<T, TPR, NV> w;
    w.template load<false>((const T *)a.w, t, cols);
    float acc[NV][V] = {};
    // the next row is on its way while this one is summed (16384 x 2048 bf16 52 -> 47
    // us, 8192 x 8192 107 -> 104), where its registers leave room: not for four
    // vectors, nor in a workgroup of 1024, which has 128 a thread
    constexpr bool AHEAD = TPR < 1024 && NV <= 2;
    Row<T, TPR, NV> h, g, p, next_h, next_g, next_p;
    const auto fetch = [&](int64_t row, Row<T, TPR, NV> &h, Row<T, TPR, NV> &g, Row<T, TPR, NV> &p) {
        h.template load<STREAM>((const T *)a.h + row * a.ldh, t, cols);
        g.template load<STREAM>((const T *)a.adj + row * a.lda, t, cols);
        if (a.adj_h)
            p.template load<STREAM>((const T *)a.adj_h + row * a.ldah, t, cols);
    };
    const int64_t start = (int64_t)blockIdx.x * RPB + slot, ahead = (int64_t)gridDim.x * RPB;
    if (AHEAD && start < a.rows)
        fetch(start, h, g, p);
    int phase = 0;
    for (int64_t row = start; row < a.rows; row += ahead, phase ^= 1) {
        if constexpr (!AHEAD)
            fetch(row, h, g, p);
        else if (row + ahead < a.rows)
            fetch(row + ahead, next_h, next_g, next_p);
        float hh = 0.f, gh = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                hh = fmaf(h.at(i, k), h.at(i, k), hh);
                gh = fmaf(g.at(i, k) * w.at(i, k), h.at(i, k), gh);
            }
#pragma unroll
        for (int o = (TPR < WAVE ? TPR : WAVE) / 2; o > 0; o /= 2) {
            hh += __shfl_xor(hh, o);
            gh += __shfl_xor(gh, o);
        }
        if constexpr (TPR > WAVE) {
            constexpr int W = TPR / WAVE;
            // two sets in turn: a wave that is a row ahead writes the other one
            if (t % WAVE == 0) {
                s_sum[phase][t / WAVE] = hh;
                s_sum[phase][W + t / WAVE] = gh;
            }
            __syncthreads();
            hh = gh = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                hh += s_sum[phase][i];
                gh += s_sum[phase][W + i];
            }
        }
        const float n = (float)cols, s = rsqrtf(hh / n + a.eps), along = s * s * (gh / n);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float hv = h.at(i, k), gv = g.at(i, k);
                acc[i][k] = fmaf(gv, hv * s, acc[i][k]);
                float d = s * (gv * w.at(i, k) - hv * along);
                if (a.adj_h)
                    d += p.at(i, k);
                h.set(i, k, d);
            }
        h.store((T *)a.adj_x + row * a.ldax, t, cols);
        if constexpr (AHEAD)
            h = next_h, g = next_g, p = next_p;
    }
    if constexpr (RPB > 1) {
        if (slot > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    s_w[slot - 1][(i * TPR + t) * V + k] = acc[i][k];
        }
        __syncthreads();
        if (slot > 0)
            return;
#pragma unroll 3
        for (int j = 0; j < RPB - 1; ++j)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    acc[i][k] += s_w[j][(i * TPR + t) * V + k];
    }
    const bool one = gridDim.x == 1;
    float *out = one ? a.adj_w : part + (int64_t)blockIdx.x * cols;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (i * TPR + t) * V + k;
            if (c < cols)
                out[c] = one && a.accumulate ? out[c] + acc[i][k] : acc[i][k];
        }
}

// adj_w[c] (+)= the sum of `count` rows of partial sums, in a fixed order: 16
// waves take every 16th row, and their sums are added in LDS.
__global__ void __launch_bounds__(1024) k_sum_rows(const float *part, int count, int cols, float *out, int accumulate)
{
    __shared__ float s[16][WAVE];
    const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE, c = (int)blockIdx.x * WAVE + lane;
    float x = 0.f;
    if (c < cols)
#pragma unroll 8
        for (int r = wave; r < count; r += 16)
            x += part[(int64_t)r * cols + c];
    s[wave][lane] = x;
    __syncthreads();
    if (wave == 0 && c < cols) {
        for (int i = 1; i < 16; ++i)
            x += s[i][lane];
        out[c] = accumulate ? out[c] + x : x;
    }
}

// no rows: adj_w has no terms
__global__ void __launch_bounds__(256) k_zero(float *out, int n)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n)
        out[i] = 0.f;
}

// Runs f(threads of a row, vectors of a thread) for rows of `n` vectors.  A row
// takes the fewest threads that hold it, so that short rows fill their waves
// (131072 x 128 bf16: 16 threads 21 us and 26 for the adjoint, 64 threads 52 and
// 126), and several vectors a thread before more threads: 2048 x 4096 bf16 10.8 us
// with 256 threads of two, 12.4 with 512 of one.  Up to 256 vectors a wave alone
// holds the row: the adjoint of 16384 x 1500 53 us, of 16384 x 2048 55, with 256
// threads 123 and 53 (most of the difference is the ragged end, which waits).
template <typename T, typename F> chol_status with_shape(int64_t n, F f)
{
    using std::integral_constant;
    if (n <= 8) return f(integral_constant<int, 8>(), integral_constant<int, 1>());
    if (n <= 16) return f(integral_constant<int, 16>(), integral_constant<int, 1>());
    if (n <= 32) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
    if (n <= 64) return f(integral_constant<int, 64>(), integral_constant<int, 1>());
    if (n <= 128) return f(integral_constant<int, 64>(), integral_constant<int, 2>());
    if (n <= 256) return f(integral_constant<int, 64>(), integral_constant<int, 4>());
    if (n <= 512) return f(integral_constant<int, 256>(), integral_constant<int, 2>());
    if (n <= 1024) return f(integral_constant<int, 512>(), integral_constant<int, 2>());
    if (n <= 2048) return f(integral_constant<int, 1024>(), integral_constant<int, 2>());
    // 16-bit rows of the longest kind end above.  (The adjoint spills 32 of its registers
    // here: 1024 threads leave 128 each, and h, adj, adj_h, w and the sums take 80.)
    if constexpr (sizeof(T) == 4)
        if (n <= 4096) return f(integral_constant<int, 1024>(), integral_constant<int, 4>());
    return CHOL_ERR_NOT_SUPPORTED;
}

template <typename T> int64_t vectors(int64_t cols) { return (cols + vec_of<T> - 1) / vec_of<T>; }

// Each workgroup of the adjoint leaves a row of partial sums of adj_w: few enough
// that these stay small beside the rows (8192 x 8192 bf16: 104 us with 256
// workgroups of 512 threads, 109 with 512), enough that the CUs stay full
// (workgroups of 256: 16384 x 4096 103 us with 512, 116 with 1024).
template <int TPR> int64_t adjoint_blocks(int64_t rows)
{
    constexpr int64_t rpb = block_of<TPR> / TPR;
    return std::min<int64_t>(block_of<TPR> > 256 ? 256 : 512, (rows + rpb - 1) / rpb);
}

} // namespace

chol_status rmsnorm(chol_dtype dt, bool quantise, const NormArgs &a, hipStream_t st)
{
    return with_lowp(dt, [&](auto *e) {
        typedef std::remove_pointer_t<decltype(e)> T;
        return with_shape<T>(vectors<T>(a.cols), [&](auto tpr, auto nv) {
            constexpr int TPR = tpr, NV = nv, BLOCK = block_of<TPR>;
            constexpr int64_t RPB = BLOCK / TPR, MOST = (int64_t)1 << 21; // workgroups of a launch: a grid holds < 2^32 threads
            const double size = (a.residual ? 3.0 : 1.0) * sizeof(T) + (quantise ? 1 : sizeof(T));
            const bool stream = size * a.rows * a.cols > CACHE;
            for (int64_t first = 0; first < a.rows; first += MOST * RPB) {
                const unsigned grid = (unsigned)std::min(MOST, (a.rows - first + RPB - 1) / RPB);
                const auto launch = [&](auto kernel) {
                    hipLaunchKernelGGL(kernel, dim3(grid), dim3(BLOCK), 0, st, a, first);
                };
                if (quantise)
                    stream ? launch(k_rmsnorm<T, TPR, NV, true, true>) : launch(k_rmsnorm<T, TPR, NV, true, false>);
                else
                    stream ? launch(k_rmsnorm<T, TPR, NV, false, true>) : launch(k_rmsnorm<T, TPR, NV, false, false>);
                CHOL_LAUNCH_CHECK();
            }
            return CHOL_OK;
        });
    });
}

size_t rmsnorm_adjoint_workspace(chol_dtype dt, int64_t rows, int64_t cols)
{
    size_t bytes = 0;
    (void)with_lowp(dt, [&](auto *e) {
        typedef std::remove_pointer_t<decltype(e)> T;
        return with_shape<T>(vectors<T>(cols), [&](auto tpr, auto) {
            constexpr int TPR = tpr;
            const int64_t blocks = adjoint_blocks<TPR>(rows);
            bytes = blocks > 1 ? (size_t)(blocks * cols) * sizeof(float) : 0;
            return CHOL_OK;
        });
    });
    return bytes;
}

chol_status rmsnorm_adjoint(chol_dtype dt, const NormAdjArgs &a, void *ws, hipStream_t st)
{
    if (a.rows == 0) {
        if (!a.accumulate)
            hipLaunchKernelGGL(k_zero, dim3((unsigned)((a.cols + 255) / 256)), dim3(256), 0, st, a.adj_w, (int)a.cols);
        CHOL_LAUNCH_CHECK();
        return CHOL_OK;
    }
    return with_lowp(dt, [&](auto *e) {
        typedef std::remove_pointer_t<decltype(e)> T;
        return with_shape<T>(vectors<T>(a.cols), [&](auto tpr, auto nv) {
            constexpr int TPR = tpr, NV = nv, BLOCK = block_of<TPR>;
            const int64_t blocks = adjoint_blocks<TPR>(a.rows);
            const auto launch = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(BLOCK), 0, st, a, (float *)ws);
            };
            const bool stream = (a.adj_h ? 4.0 : 3.0) * sizeof(T) * a.rows * a.cols > CACHE;
            stream ? launch(k_rmsnorm_adjoint<T, TPR, NV, true>) : launch(k_rmsnorm_adjoint<T, TPR, NV, false>);
            CHOL_LAUNCH_CHECK();
            if (blocks > 1) {
                hipLaunchKernelGGL(k_sum_rows, dim3((unsigned)((a.cols + WAVE - 1) / WAVE)), dim3(1024), 0, st,
                                   (const float *)ws, (int)blocks, (int)a.cols, a.adj_w, a.accumulate);
                CHOL_LAUNCH_CHECK();
            }
            return CHOL_OK;
        });
    });
}

} // namespace chol
