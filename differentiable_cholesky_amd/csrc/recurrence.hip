// The gated linear recurrence h_t = a_t h_{t-1} + b_t and its adjoint.
//
// Both are compositions of affine maps of one fp32 number a channel.  Forward,
// step t maps x -> a_t x + b_t.  The adjoint runs from the last step to the
// first on mu_t = a_t lam_t with lam_t = adj_t + mu_{t+1}: step t maps
// x -> a_t x + a_t adj_t, so a step needs its own gate only and the walk ends
// with adj_h0 = mu_0.  A run of steps composes to x -> P x + Q.
//
// A sequence is cut into segments.  One kernel forms each segment's (P, Q); a
// second joins those before a segment, which gives the state it starts from,
// and walks the segment again, now writing.
#include <algorithm>
#include <type_traits>

#include "lowp.hpp"
#include "recurrence.hpp"

namespace chol {

namespace {

constexpr int THREADS = 256;

template <typename T> struct Rows {
    T *p;
    int64_t ld;
    explicit __device__ Rows(const RecRows &r, int64_t b, int64_t c) : p((T *)r.p + b * r.stride + c), ld(r.ld) {}
    __device__ __forceinline__ float at(int64_t t) const { return (float)p[t * ld]; }
    __device__ __forceinline__ void put(int64_t t, float x) const { p[t * ld] = (T)x; }
};

template <bool LOG> __device__ __forceinline__ float gate(float x) { return LOG ? expf(x) : x; }

// step s of the walk is row s (forward) or len - 1 - s (adjoint)
template <bool ADJ> __device__ __forceinline__ int64_t row_of(int64_t s, int64_t len) { return ADJ ? len - 1 - s : s; }

// (P, Q) of segment blockIdx.y of batch element blockIdx.z; ws[(z * segments + y) * dim + channel]
template <typename T, bool LOG, bool ADJ>
__global__ void __launch_bounds__(THREADS) k_rec_segment(RecArgs r, int64_t seg, float2 *ws)
{
    const int64_t c = (int64_t)blockIdx.x * THREADS + threadIdx.x, z = blockIdx.z;
    if (c >= r.dim)
        return;
    const Rows<T> a(r.a, z, c), b(r.b, z, c);
    const int64_t s0 = (int64_t)blockIdx.y * seg, s1 = min(s0 + seg, r.len);
    float P = 1.f, Q = 0.f;
    for (int64_t s = s0; s < s1; ++s) {
        const int64_t t = row_of<ADJ>(s, r.len);
        const float g = gate<LOG>(a.at(t)), x = b.at(t);
        Q = ADJ ? g * (Q + x) : g * Q + x;
        P *= g;
    }
    // the first segment's slot holds the state before and after it: the walk
    // may then write the end over the start
    if (blockIdx.y == 0) {
        const float x = r.start ? r.start[z * r.dim + c] : 0.f;
        Q = P * x + Q;
        P = x;
    }
    ws[(z * gridDim.y + blockIdx.y) * r.dim + c] = make_float2(P, Q);
}

template <typename T, bool LOG, bool ADJ>
__global__ void __launch_bounds__(THREADS) k_rec_walk(RecArgs r, int64_t seg, const float2 *ws)
{
    const int64_t c = (int64_t)blockIdx.x * THREADS + threadIdx.x, z = blockIdx.z;
    if (c >= r.dim)
        return;
    float x;
    if (gridDim.y == 1) {
        x = r.start ? r.start[z * r.dim + c] : 0.f;
    } else {
        const float2 first = ws[z * gridDim.y * r.dim + c];
        x = blockIdx.y ? first.y : first.x;
        for (int64_t y = 1; y < blockIdx.y; ++y) {
            const float2 pq = ws[(z * gridDim.y + y) * r.dim + c];
            x = pq.x * x + pq.y;
        }
    }
    const Rows<T> a(r.a, z, c), b(r.b, z, c), out(r.out, z, c);
    const int64_t s0 = (int64_t)blockIdx.y * seg, s1 = min(s0 + seg, r.len);
    for (int64_t s = s0; s < s1; ++s) {
        const int64_t t = row_of<ADJ>(s, r.len);
        const float g = gate<LOG>(a.at(t));
        if constexpr (ADJ) {
            const float lam = b.at(t) + x;
            const float before = t > 0 ? Rows<T>(r.h, z, c).at(t - 1) : r.h0 ? r.h0[z * r.dim + c] : 0.f;
            x = g * lam;
            Rows<T>(r.adj_a, z, c).put(t, before * (LOG ? x : lam));
            out.put(t, lam);
        } else {
            x = g * x + b.at(t);
            out.put(t, x);
        }
    }
    if (r.end && blockIdx.y == gridDim.y - 1)
        r.end[z * r.dim + c] = x;
}

// Steps of a segment: whole sequences where channels alone give 2^17 threads
// (two waves a SIMD on 256 CUs), else as many segments as bring them there.
int64_t segment_of(int64_t batch, int64_t len, int64_t dim)
{
    const int64_t threads = batch * ((dim + THREADS - 1) / THREADS) * THREADS;
    const int64_t want = std::max<int64_t>(1, ((int64_t)1 << 17) / threads);
    return std::max<int64_t>(16, (len + want - 1) / want);
}

template <typename T, bool LOG, bool ADJ> chol_status run(const RecArgs &r, void *ws, hipStream_t st)
{
    const int64_t seg = segment_of(r.batch, r.len, r.dim);
    if (r.batch > 65535)
        return CHOL_ERR_NOT_SUPPORTED;
    const int64_t parts = std::max<int64_t>(1, (r.len + seg - 1) / seg);
    const dim3 grid((unsigned)((r.dim + THREADS - 1) / THREADS), (unsigned)parts, (unsigned)r.batch);
    if (parts > 1) {
        hipLaunchKernelGGL((k_rec_segment<T, LOG, ADJ>), grid, dim3(THREADS), 0, st, r, seg, (float2 *)ws);
        CHOL_LAUNCH_CHECK();
    }
    hipLaunchKernelGGL((k_rec_walk<T, LOG, ADJ>), grid, dim3(THREADS), 0, st, r, seg, (const float2 *)ws);
    CHOL_LAUNCH_CHECK();
    return CHOL_OK;
}

} // namespace

size_t recurrence_workspace(int64_t batch, int64_t len, int64_t dim)
{
    const int64_t seg = segment_of(batch, len, dim), parts = (len + seg - 1) / seg;
    return parts > 1 ? (size_t)(batch * parts * dim) * sizeof(float2) : 0;
}

chol_status recurrence(chol_dtype dt, bool log_gate, bool adjoint, const RecArgs &r, void *ws, hipStream_t st)
{
    return with_lowp(dt, [&](auto *t) {
        typedef std::remove_pointer_t<decltype(t)> T;
        if (adjoint)
            return log_gate ? run<T, true, true>(r, ws, st) : run<T, false, true>(r, ws, st);
        return log_gate ? run<T, true, false>(r, ws, st) : run<T, false, false>(r, ws, st);
    });
}

} // namespace chol
