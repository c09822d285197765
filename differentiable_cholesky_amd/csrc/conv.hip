// The short causal convolution along a sequence, one filter of K taps a channel, and
// its adjoint.
//
//   p_t = bias + sum_k w_k x_{t-K+1+k},  y_t = silu(p_t) (or p_t);  rows before the
//   first are the kept ones (`state`) or zero
//   q_t = adj_t silu'(p_t),  adj_x_t = sum_k w_k q_{t+K-1-k} (+ adj_last),
//   adj_w_k = sum q_t x_{t-K+1+k},  adj_bias = sum q_t
//
// A few operations an element, so memory bounds it (8 x 4096 x 4096 bf16 105 us, 5.1 TB/s,
// adjoint 172, 4.7; 64 x 1 x 4096 4.4 on the GPU).  A thread walks `run` steps of V
// channels and keeps the last K - 1 rows in registers, so a row is read once, and
// K - 1 more a run (the adjoint: two rows K - 1 times).  Lanes lie along the channels
// as far as these reach and along runs from there on, so that neighbouring runs, which
// share those rows, mostly run on one CU.
//
// The adjoint walks the same way: q_t is formed once, adj_x trails it by K - 1 rows.  A
// workgroup's sums of adj_w and adj_bias are rows of the workspace, added up in one
// order by a second launch.
#include <algorithm>
#include <type_traits>

#include "conv.hpp"

namespace chol {

namespace {

constexpr int WAVE = 64, THREADS = 256;

struct Plan {
    int lanes;     // along the channels; THREADS / lanes runs a workgroup
    int run;       // steps of a thread
    int64_t across, along; // workgroups
};

template <typename T, int V> __device__ __forceinline__ vec<T, V> row_at(const SeqRows &r, int64_t z, int64_t t, int64_t c, int64_t n)
{
    return load_some<T, V>((const T *)r.p + z * r.stride + t * r.ld + c, n);
}

// Row t of the sequence with what lies before it.
template <typename T, int V, int K>
__device__ __forceinline__ vec<T, V> input_row(const ConvArgs &a, int64_t z, int64_t t, int64_t c, int64_t n)
{
    if (t >= 0)
        return row_at<T, V>(a.x, z, t, c, n);
    if (a.state)
        return load_some<T, V>((const T *)a.state + (z * (K - 1) + t + K - 1) * a.dim + c, n);
    return (vec<T, V>)(T)0.f;
}

template <typename T, int V, int K> struct Taps {
    float w[V][K], bias[V];
    __device__ __forceinline__ void load(const ConvArgs &a, int64_t c, int64_t n)
    {
        const vec<T, V> b = a.bias ? load_some<T, V>((const T *)a.bias + c, n) : (vec<T, V>)(T)0.f;
        T raw[V * K];
        const T *p = (const T *)a.w + c * K;
        if (n >= V) {
            __builtin_memcpy(raw, p, sizeof(raw));
        } else {
#pragma unroll
            for (int i = 0; i < V * K; ++i)
                raw[i] = i < n * K ? p[i] : (T)0.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            bias[v] = lane_of<T, V>(b, v);
#pragma unroll
            for (int k = 0; k < K; ++k)
                w[v][k] = (float)raw[v * K + k];
        }
    }
};

// A thread's place: batch element, first channel, how many channels from there exist, first
// step.  The last vector of a ragged row moves back to end with it, over channels of its
// neighbour (`twice` of them), which then writes the same values: whole vectors only (adjoint
// of 8 x 4096 x 1001 bf16 132 -> 58 us, forward 40 -> 30).
struct Place {
    int64_t z, c, n, t0;
    int twice;
    __device__ __forceinline__ bool set(const ConvArgs &a, const Plan &p, int V)
    {
        const unsigned block = blockIdx.x, cb = block % (unsigned)p.across, rest = block / (unsigned)p.across;
        z = rest / (unsigned)p.along;
        c = ((int64_t)cb * p.lanes + threadIdx.x % p.lanes) * V;
        t0 = (int64_t)((rest % (unsigned)p.along) * (THREADS / p.lanes) + threadIdx.x / p.lanes) * p.run;
        n = a.dim - c, twice = 0;
        // (not over kept rows that are replaced in place: the neighbour may have written them)
        if (n > 0 && n < V && a.dim >= V && !(a.state && a.state == a.last))
            twice = (int)(V - n), c -= twice, n = V;
        return n > 0;
    }
};

// GROUP rows are on their way at a time.
template <typename T, int V, int K, int GROUP, bool SILU>
__global__ void __launch_bounds__(THREADS) k_conv(ConvArgs a, Plan p)
{
    constexpr bool FULL = sizeof(T) == 4;
    Place at;
    if (!at.set(a, p, V))
        return;
    const int64_t z = at.z, c = at.c, n = at.n, t0 = at.t0;
    // the first run, which reads the kept rows, also writes them: they may be replaced
    // in place
    vec<T, V> kept[K - 1];
    if (t0 == 0 && a.last) {
#pragma unroll
        for (int i = 0; i < K - 1; ++i)
            kept[i] = input_row<T, V, K>(a, z, a.len - (K - 1) + i, c, n);
    }
    if (t0 < a.len) {
        Taps<T, V, K> taps;
        taps.load(a, c, n);
        vec<T, V> past[K - 1];
#pragma unroll
        for (int i = 0; i < K - 1; ++i)
            past[i] = input_row<T, V, K>(a, z, t0 - (K - 1) + i, c, n);
        const int64_t end = t0 + p.run < a.len ? t0 + p.run : a.len;
        T *y = (T *)a.y.p + z * a.y.stride + c;
        for (int64_t t = t0; t < end; t += GROUP) {
            vec<T, V> rows[GROUP + K - 1];
#pragma unroll
            for (int i = 0; i < K - 1; ++i)
                rows[i] = past[i];
#pragma unroll
            for (int g = 0; g < GROUP; ++g) // (a row past the end is read again, not used)
                rows[K - 1 + g] = row_at<T, V>(a.x, z, t + g < end ? t + g : end - 1, c, n);
#pragma unroll
            for (int g = 0; g < GROUP; ++g) {
                vec<T, V> out;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float s = taps.bias[v];
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        s = fmaf(taps.w[v][k], lane_of<T, V>(rows[g + k], v), s);
                    set_lane<T, V>(out, v, SILU ? s * sigmoid_of<FULL>(s) : s);
                }
                if (t + g < end)
                    store_some<T, V>(y + (t + g) * a.y.ld, n, out);
            }
#pragma unroll
            for (int i = 0; i < K - 1; ++i)
                past[i] = rows[GROUP + i];
        }
    }
    if (t0 == 0 && a.last)
#pragma unroll
        for (int i = 0; i < K - 1; ++i)
            store_some<T, V>((T *)a.last + (z * (K - 1) + i) * a.dim + c, n, kept[i]);
}

// part: a row of dim * (K + 1) sums a workgroup along the sequence
template <typename T, int V, int K, int GROUP, bool SILU>
__global__ void __launch_bounds__(THREADS) k_conv_adjoint(ConvArgs a, Plan p, float *part)
{
    constexpr bool FULL = sizeof(T) == 4;
    __shared__ float s_sum[THREADS][V + 1]; // (a sum of one tap or of the bias at a time)
    Place at;
    const bool here = at.set(a, p, V);
    const int64_t z = at.z, c = at.c, n = at.n, t0 = at.t0;
    float dw[V][K] = {}, db[V] = {};
    // adj_last's row of input row t, which it reaches directly
    const auto direct = [&](int64_t t) {
        const int64_t i = t - (a.len - (K - 1));
        return a.adj_last && i >= 0 ? load_some<T, V>((const T *)a.adj_last + (z * (K - 1) + i) * a.dim + c, n)
                                    : (vec<T, V>)(T)0.f;
    };
    if (here && (t0 < a.len || (t0 == 0 && a.last))) {
        Taps<T, V, K> taps;
        taps.load(a, c, n);
        vec<T, V> past[K - 1];
        float q[K - 1][V] = {}; // of the rows before t
#pragma unroll
        for (int i = 0; i < K - 1; ++i)
            past[i] = input_row<T, V, K>(a, z, t0 - (K - 1) + i, c, n);
        // q of a run's own rows and of the K - 1 after them; adj_x of its own, and the
        // first run's of the kept rows
        const int64_t own = t0 + p.run < a.len ? t0 + p.run : a.len, end = own + K - 1;
        const int64_t from = t0 == 0 && a.last ? -(K - 1) : t0;
        // G rows from t; `whole`: they and all of their channels exist, and are the run's own
        const auto walk = [&](int64_t t, auto rows_at_once, auto whole) {
            constexpr int G = rows_at_once;
            constexpr bool WHOLE = whole;
            vec<T, V> rows[G + K - 1], adj[G];
#pragma unroll
            for (int i = 0; i < K - 1; ++i)
                rows[i] = past[i];
            if constexpr (WHOLE) {
                const T *px = (const T *)a.x.p + z * a.x.stride + t * a.x.ld + c;
                const T *pa = (const T *)a.adj.p + z * a.adj.stride + t * a.adj.ld + c;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    rows[K - 1 + g] = load_vec<T, V>(px + g * a.x.ld);
                    adj[g] = load_vec<T, V>(pa + g * a.adj.ld);
                }
            } else {
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    rows[K - 1 + g] = (vec<T, V>)(T)0.f;
                    adj[g] = (vec<T, V>)(T)0.f;
                }
                if (a.len > 0)
#pragma unroll
                    for (int g = 0; g < G; ++g) { // (a row past the end is read again, not used)
                        const int64_t i = t + g < a.len ? t + g : a.len - 1;
                        rows[K - 1 + g] = row_at<T, V>(a.x, z, i, c, n);
                        adj[g] = row_at<T, V>(a.adj, z, i, c, n);
                    }
            }
            T *const px = WHOLE ? (T *)a.y.p + z * a.y.stride + (t - (K - 1)) * a.y.ld + c : nullptr;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int64_t now = t + g, back = now - (K - 1);
                vec<T, V> out = (vec<T, V>)(T)0.f, more = (vec<T, V>)(T)0.f;
                const bool write = (WHOLE || now < end) && back >= from;
                if constexpr (!WHOLE)
                    if (write && back >= a.len - (K - 1))
                        more = direct(back);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float s = taps.bias[v], d = lane_of<T, V>(adj[g], v);
                    if constexpr (SILU) {
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            s = fmaf(taps.w[v][k], lane_of<T, V>(rows[g + k], v), s);
                        const float sg = sigmoid_of<FULL>(s);
                        d *= sg * fmaf(s, 1.f - sg, 1.f);
                    }
                    if constexpr (!WHOLE)
                        d = now < a.len ? d : 0.f;
                    if (WHOLE || now < own) {
                        db[v] += d;
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            dw[v][k] = fmaf(d, lane_of<T, V>(rows[g + k], v), dw[v][k]);
                    }
                    // adj_x of row back: taps 0 .. K - 1 meet q of rows now .. back
                    float o = WHOLE ? taps.w[v][0] * d : fmaf(taps.w[v][0], d, lane_of<T, V>(more, v));
#pragma unroll
                    for (int k = 1; k < K; ++k)
                        o = fmaf(taps.w[v][k], q[K - 1 - k][v], o);
                    set_lane<T, V>(out, v, o);
#pragma unroll
                    for (int k = 0; k + 1 < K - 1; ++k)
                        q[k][v] = q[k + 1][v];
                    q[K - 2][v] = d;
                }
                if (write) {
                    if (WHOLE && back >= 0)
                        store_vec<T, V>(px + g * a.y.ld, out);
                    else if (back >= 0)
                        store_some<T, V>((T *)a.y.p + z * a.y.stride + back * a.y.ld + c, n, out);
                    else
                        store_some<T, V>((T *)a.last + (z * (K - 1) + back + K - 1) * a.dim + c, n, out);
                }
            }
#pragma unroll
            for (int i = 0; i < K - 1; ++i)
                past[i] = rows[G + i];
        };
        int64_t t = t0;
        if (n >= V)
            for (; t + GROUP <= own; t += GROUP)
                walk(t, std::integral_constant<int, GROUP>(), std::true_type());
        for (; t < end; t += K - 1)
            walk(t, std::integral_constant<int, K - 1>(), std::false_type());
    }
    // over the workgroup's runs, one tap at a time
    const int64_t row = blockIdx.x / (unsigned)p.across; // batch * along of them
    float *out = part + row * a.dim * (K + 1);
#pragma unroll
    for (int k = 0; k <= K; ++k) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v >= at.twice) // (the neighbour has the others)
                s_sum[threadIdx.x][v - at.twice] = k < K ? dw[v][k < K ? k : 0] : db[v];
        __syncthreads();
        // channel lane * V + v of the workgroup by thread v * lanes + lane
        for (int i = threadIdx.x; i < p.lanes * V; i += THREADS) {
            const int lane = i / V, v = i % V;
            float s = 0.f;
            for (int r = lane; r < THREADS; r += p.lanes)
                s += s_sum[r][v];
            const int64_t ch = (int64_t)(blockIdx.x % (unsigned)p.across) * p.lanes * V + i;
            if (ch < a.dim)
                out[k < K ? ch * K + k : a.dim * K + ch] = s;
        }
        __syncthreads();
    }
}

// adj_w and adj_bias from the workgroups' rows, a column a lane, sixteen lanes' sums of
// every sixteenth row joined
__global__ void __launch_bounds__(1024) k_conv_sums(const float *part, int64_t rows, int64_t taps, int64_t cols,
                                                    float *adj_w, float *adj_bias, bool accumulate)
{
    __shared__ float s_sum[16][WAVE];
    const int lane = threadIdx.x % WAVE, slot = threadIdx.x / WAVE;
    const int64_t c = (int64_t)blockIdx.x * WAVE + lane;
    float s = 0.f;
    if (c < cols)
        for (int64_t r = slot; r < rows; r += 16)
            s += part[r * cols + c];
    s_sum[slot][lane] = s;
    __syncthreads();
    if (slot > 0 || c >= cols)
        return;
#pragma unroll
    for (int i = 1; i < 16; ++i)
        s += s_sum[i][lane];
    float *out = c < taps ? adj_w + c : adj_bias ? adj_bias + (c - taps) : nullptr;
    if (out)
        *out = accumulate ? *out + s : s;
}

constexpr int GROUP = 8;
template <typename T> constexpr int forward_vec = 16 / (int)sizeof(T);
template <typename T> constexpr int adjoint_vec = 4;

Plan plan_of(const ConvArgs &a, int v, int longest)
{
    Plan p;
    const int64_t words = (a.dim + v - 1) / v;
    p.lanes = 1;
    while (p.lanes < words && p.lanes < WAVE)
        p.lanes *= 2;
    p.across = (words + p.lanes - 1) / p.lanes;
    const int runs = THREADS / p.lanes;
    // Long runs read few rows twice (adjoint of 8 x 4096 x 4096 bf16 with runs of 64 189 us,
    // of 128 172); runs are halved while workgroups are fewer than two a CU.
    p.run = longest;
    const auto along = [&] { return std::max<int64_t>(1, (a.len + (int64_t)runs * p.run - 1) / ((int64_t)runs * p.run)); };
    while (p.run > GROUP && a.batch * p.across * along() < 512)
        p.run /= 2;
    p.along = along();
    return p;
}

template <typename T> Plan forward_plan(const ConvArgs &a) { return plan_of(a, forward_vec<T>, 64); }
template <typename T> Plan adjoint_plan(const ConvArgs &a) { return plan_of(a, adjoint_vec<T>, 128); }

bool grid_ok(const ConvArgs &a, const Plan &p)
{
    return (double)a.batch * p.across * p.along * THREADS <= 4294967295.0;
}

template <typename F> chol_status with_width(int width, F f)
{
    switch (width) {
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    default: return CHOL_ERR_NOT_SUPPORTED;
    }
}

} // namespace

bool conv_fits(chol_dtype dt, const ConvArgs &a)
{
    return dt == CHOL_F32 ? grid_ok(a, forward_plan<float>(a)) : grid_ok(a, forward_plan<bf16_t>(a));
}

int64_t conv_adjoint_workspace(chol_dtype dt, const ConvArgs &a)
{
    const Plan p = dt == CHOL_F32 ? adjoint_plan<float>(a) : adjoint_plan<bf16_t>(a);
    // (and the threads of the sums)
    return grid_ok(a, p) && (double)(a.dim * (a.width + 1) + WAVE) * 16 <= 4294967295.0 ? a.batch * p.along * a.dim * (a.width + 1) * (int64_t)sizeof(float) : -1;
}

chol_status conv(chol_dtype dt, const ConvArgs &a, hipStream_t st)
{
    return with_lowp(dt, [&](auto *e) {
        typedef std::remove_pointer_t<decltype(e)> T;
        return with_width(a.width, [&](auto width) {
            constexpr int K = width, V = forward_vec<T>;
            const Plan p = forward_plan<T>(a);
            const dim3 grid((unsigned)(a.batch * p.across * p.along));
            const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(THREADS), 0, st, a, p); };
            if (a.len <= 1)
                a.silu ? launch(k_conv<T, V, K, 1, true>) : launch(k_conv<T, V, K, 1, false>);
            else
                a.silu ? launch(k_conv<T, V, K, GROUP, true>) : launch(k_conv<T, V, K, GROUP, false>);
            CHOL_LAUNCH_CHECK();
            return CHOL_OK;
        });
    });
}

chol_status conv_adjoint(chol_dtype dt, const ConvArgs &a, void *ws, hipStream_t st)
{
    return with_lowp(dt, [&](auto *e) {
        typedef std::remove_pointer_t<decltype(e)> T;
        return with_width(a.width, [&](auto width) {
            constexpr int K = width, V = adjoint_vec<T>;
            const Plan p = adjoint_plan<T>(a);
            const dim3 grid((unsigned)(a.batch * p.across * p.along));
            const auto launch = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, grid, dim3(THREADS), 0, st, a, p, (float *)ws);
            };
            if (a.batch > 0) {
                a.silu ? launch(k_conv_adjoint<T, V, K, GROUP, true>) : launch(k_conv_adjoint<T, V, K, GROUP, false>);
                CHOL_LAUNCH_CHECK();
            }
            const int64_t cols = a.dim * (K + 1);
            hipLaunchKernelGGL(k_conv_sums, dim3((unsigned)((cols + WAVE - 1) / WAVE)), dim3(1024), 0, st,
                               (const float *)ws, a.batch * p.along, a.dim * K, cols, a.adj_w, a.adj_bias, a.accumulate);
            CHOL_LAUNCH_CHECK();
            return CHOL_OK;
        });
    });
}

} // namespace chol
