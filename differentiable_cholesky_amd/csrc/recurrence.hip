// The gated linear recurrence h_t = a_t h_{t-1} + b_t and its adjoint.
//
// Both are compositions of affine maps of one fp32 number a channel.  Forward,
// step t maps x -> a_t x + b_t.  The adjoint walks from the last step to the
// first on mu_t = a_t lam_t with lam_t = adj_t + mu_{t+1}: step t maps
// x -> a_t x + a_t adj_t, so a step needs its own gate only and the walk ends
// with adj_h0 = mu_0.  A run of steps composes to x -> P x + Q.
//
// One pass over memory: a lane holds R consecutive steps of one 32-bit word of
// channels (two 16-bit ones, or an fp32 one) in registers, composes them, and
// walks them again from registers once it knows the state before them.  Teams of
// lanes (waves, or parts of them for few channels) lie along the steps (`teams`,
// fewer for short sequences) and across channels, and exchange their (P, Q) through LDS.  Workgroups of one
// channel group form a chain along the sequence, cut into groups of LINKS: a
// workgroup composes what those before it in its group published, and applies
// that to the state its group starts from, which the last workgroup of the group
// before published (links.hpp).  So the chain waits once a group, every sum is formed in
// one order whatever the workgroups' timing, and equal calls give equal bits.
//
// Every element is read once and written once and costs a few operations, so
// memory bounds long sequences: 1 x 65536 x 2048 bf16 forward 151 us (5.3 TB/s),
// adjoint 260 us (5.2 TB/s), where a large copy reaches 5.2 TB/s; 8 x 4096 x 2048
// 91 us (4.4 TB/s), four rounds of workgroups, whose first loads and last stores
// overlap nothing.
#include <algorithm>
#include <type_traits>

#include "links.hpp"
#include "lowp.hpp"
#include "recurrence.hpp"

namespace chol {

namespace {

constexpr int WAVE = 64, THREADS = 512;
constexpr int NARROW = 16; // lanes of a part of a wave

template <typename T> constexpr int word_channels = 4 / (int)sizeof(T);

template <typename T> __device__ __forceinline__ float part(uint32_t w, int i)
{
    if constexpr (sizeof(T) == 4)
        return __uint_as_float(w);
    else
        return (float)__builtin_bit_cast(T, (uint16_t)(w >> (16 * i)));
}
template <typename T> __device__ __forceinline__ uint32_t pack(const float (&x)[word_channels<T>])
{
    if constexpr (sizeof(T) == 4) {
        return __float_as_uint(x[0]);
    } else {
        vec<T, 2> v;
        v[0] = (T)x[0];
        v[1] = (T)x[1];
        return __builtin_bit_cast(uint32_t, v);
    }
}
// Stores leave the caches to the loads: 8 x 4096 x 2048 bf16 forward 92 -> 88 us
// with inputs from memory, 93 -> 72 with inputs that the last cache still holds
// (only where rows share cache lines the adjoint loses: 2 x 4095 x 1999 fp32 93 ->
// 103).  Loads that do so too cost odd rows more (4 x 4095 x 1999 bf16 68 -> 91) and
// gain 5% at most elsewhere.
typedef uint32_t any_word __attribute__((aligned(2)));
template <typename T> __device__ __forceinline__ uint32_t load_word(const T *p)
{
    return *(const any_word *)p;
}
template <typename T> __device__ __forceinline__ void store_word(T *p, uint32_t w)
{
    __builtin_nontemporal_store(w, (any_word *)p);
}

// Where a word may lie past the row's or the sequence's end: its elements at the
// offsets at[], which lie inside, with `none`'s in place of those that do not
// count.  No branch, so that the loads of a run stay in flight together:
// 4 x 4095 x 1999 bf16 forward 88 -> 70 us, 16 x 500 x 333 31 -> 17 us.
template <typename T>
__device__ __forceinline__ uint32_t load_part(const T *p, const int64_t (&at)[word_channels<T>],
                                              const bool (&counts)[word_channels<T>], bool row, uint32_t none)
{
    if constexpr (sizeof(T) == 4) {
        const uint32_t w = __float_as_uint(p[at[0]]);
        return row && counts[0] ? w : none;
    } else {
        const uint32_t lo = __builtin_bit_cast(uint16_t, p[at[0]]), hi = __builtin_bit_cast(uint16_t, p[at[1]]);
        return (row && counts[0] ? lo : none & 0xffffu) | (row && counts[1] ? hi << 16 : none & 0xffff0000u);
    }
}
template <typename T> __device__ __forceinline__ void store_part(T *p, int64_t c, int64_t dim, uint32_t w)
{
#pragma unroll
    for (int i = 0; i < word_channels<T>; ++i)
        if (c + i < dim) {
            if constexpr (sizeof(T) == 4)
                p[i] = __uint_as_float(w);
            else
                p[i] = __builtin_bit_cast(T, (uint16_t)(w >> (16 * i)));
        }
}
template <typename T> __device__ __forceinline__ uint32_t one_word()
{
    float x[word_channels<T>];
    for (float &v : x)
        v = 1.f;
    return pack<T>(x);
}

// exp(x) from the hardware's 2^y.  Rounding y = x log2(e) would change the result by
// up to |x| 2^-24 of itself, so the product is carried in two parts.  A 16-bit x
// times the leading bits H of log2(e) is exact, and the rest is small: exp(x) =
// 2^(x H) exp(x (1 - H ln 2)), the last by its series (left out is 1e-7 at |x| = 88
// in bf16, with H of 15 bits, and 1e-8 in fp16, with 13).  All values of both types:
// within 1.7e-7, where one part gives 3.8e-6.  It costs the adjoint of 1 x 65536 x 2048
// bf16 256 -> 260 us.
template <typename T, bool LOG> __device__ __forceinline__ float gate(float x)
{
    constexpr double LOG2E = 1.4426950408889634074, LN2 = 0.69314718055994530942;
    if constexpr (!LOG)
        return x;
    if constexpr (sizeof(T) == 2) {
        constexpr bool BF16 = std::is_same_v<T, bf16_t>;
        constexpr float H = BF16 ? 0x1.7154p+0f : 0x1.715p+0f, REST = (float)((LOG2E - H) * LN2);
        // (the bound keeps x = -inf, whose first factor is zero, from 0 times inf)
        const float e = __builtin_amdgcn_exp2f(x * H), d = fmaxf(x * REST, -1.f);
        return fmaf(e, BF16 ? d : d * fmaf(d, 0.5f, 1.f), e);
    } else {
        constexpr float L = (float)LOG2E, L_LOW = (float)(LOG2E - L);
        const float y = x * L, e = __builtin_amdgcn_exp2f(y), low = fmaf(x, L_LOW, fmaf(x, L, -y));
        // beyond +-128 the result is 0 or inf (and low may be NaN)
        return fabsf(y) < 128.f ? fmaf(e * (float)LN2, low, e) : e;
    }
}

struct Plan {
    int lanes;          // of a team: a wave, or a part of one for few channels
    int teams;          // of a workgroup along the steps; the others lie across channels
    int steps;          // R
    int chunks, groups; // workgroups along the steps, and across a batch element's channels
};

// What a workgroup publishes (links.hpp), one 64-bit word a channel, written once and
// read whole, so that no flag or fence is needed: P and Q.  The workspace is filled with
// EMPTY first (P's NaN of all ones, which a published P never is).
constexpr uint64_t EMPTY = ~(uint64_t)0;

__device__ __forceinline__ void publish(uint64_t *p, float P, float Q)
{
    const uint32_t bits = P != P ? 0x7fc00000u : __float_as_uint(P);
    __hip_atomic_store(p, (uint64_t)bits | (uint64_t)__float_as_uint(Q) << 32, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 arrived(const uint64_t *p, uint64_t w)
{
    while ((uint32_t)w == (uint32_t)EMPTY) {
        __builtin_amdgcn_s_sleep(1);
        w = peek(p);
    }
    return make_float2(__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32)));
}

// A lane's view of its chain (links.hpp): its word of workgroup k lies k * stride on.
template <typename State> struct Words {
    uint64_t *links;
    int64_t stride;
    const float *from;
    const State &state;
    __device__ __forceinline__ float start(int v) const { return state(from, v); }
    __device__ __forceinline__ uint64_t *at(unsigned k, int v) const { return links + (int64_t)k * stride + v; }
    __device__ __forceinline__ void publish(unsigned k, int v, float P, float Q) const { chol::publish(at(k, v), P, Q); }
    __device__ __forceinline__ uint64_t peek(unsigned k, int v) const { return chol::peek(at(k, v)); }
    __device__ __forceinline__ float2 arrived(unsigned k, int v, uint64_t w) const { return chol::arrived(at(k, v), w); }
};

// Fills the workspace, two words a store; the first two are the tickets'.
constexpr int CLEAR = 4; // stores of a thread
typedef uint64_t word_pair __attribute__((ext_vector_type(2), aligned(8)));

__global__ void __launch_bounds__(256) k_rec_clear(word_pair *ws, int64_t pairs)
{
    int64_t i = (int64_t)blockIdx.x * 256 * CLEAR + threadIdx.x;
#pragma unroll
    for (int k = 0; k < CLEAR; ++k, i += 256)
        if (i < pairs)
            ws[i] = i ? (word_pair)EMPTY : (word_pair)0;
}

// (four waves a SIMD, so two workgroups a CU: without it the partial words' loads
// take the registers of one, adjoint of 1 x 65536 x 2048 bf16 256 -> 311 us)
template <typename T, bool LOG, bool ADJ, int R, int LANES>
__global__ void __launch_bounds__(THREADS, 4) k_recurrence(RecArgs r, Plan p, uint64_t *ws)
{
    constexpr int V = word_channels<T>, SPAN = LANES * V, TEAMS = THREADS / LANES;
    __shared__ float2 s_link[TEAMS][SPAN];
    __shared__ float s_in[TEAMS][SPAN];
    __shared__ unsigned s_ticket;
    const int lane = threadIdx.x % LANES;
    const int team = LANES < WAVE ? threadIdx.x / LANES : __builtin_amdgcn_readfirstlane(threadIdx.x / LANES);
    const int jw = team % p.teams, cw = team / p.teams, across = TEAMS / p.teams;
    unsigned block = blockIdx.x;
    if (p.chunks > 1) {
        // chains advance in the order in which workgroups start: whatever a
        // workgroup waits for has been started before it
        if (threadIdx.x == 0)
            s_ticket = atomicAdd((unsigned *)ws, 1u);
        __syncthreads();
        block = __builtin_amdgcn_readfirstlane(s_ticket);
    }
    const unsigned chains = (unsigned)(r.batch * p.groups);
    const unsigned chunk = block / chains, chain = block % chains;
    const int64_t z = chain / p.groups;
    const int64_t c0 = ((int64_t)(chain % p.groups) * across + cw) * SPAN, c = c0 + lane * V;
    const int64_t s0 = ((int64_t)chunk * p.teams + jw) * R;
    // walk step s is row s, or counted from the end
    const auto row = [&](int64_t s) { return ADJ ? r.len - 1 - s : s; };
    const T *pa = (const T *)r.a.p + z * r.a.stride + c0, *pb = (const T *)r.b.p + z * r.b.stride + c0;
    const T *ph = ADJ ? (const T *)r.h.p + z * r.h.stride + c0 : nullptr;
    const bool whole = c0 + SPAN <= r.dim && s0 + R + (ADJ ? 1 : 0) <= r.len;

    uint32_t a[R], b[R], h[ADJ ? R : 1]; // h: the state before the step
    if (whole) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            a[i] = load_word(pa + row(s0 + i) * r.a.ld + lane * V);
            b[i] = load_word(pb + row(s0 + i) * r.b.ld + lane * V);
        }
        if constexpr (ADJ)
#pragma unroll
            for (int i = 0; i < R; ++i)
                h[i] = load_word(ph + row(s0 + i + 1) * r.h.ld + lane * V);
    } else {
        // steps past the end and channels past dim leave the state as it is
        const uint32_t open = LOG ? 0u : one_word<T>();
        int64_t at[V];
        bool counts[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            counts[v] = c + v < r.dim;
            at[v] = (counts[v] ? c + v : r.dim - 1) - c0;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            a[i] = open, b[i] = 0u;
            if constexpr (ADJ)
                h[i] = 0u;
        }
        if (r.len > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int64_t s = s0 + i, here = row(s < r.len ? s : r.len - 1);
                a[i] = load_part(pa + here * r.a.ld, at, counts, s < r.len, open);
                b[i] = load_part(pb + here * r.b.ld, at, counts, s < r.len, 0u);
                if constexpr (ADJ)
                    h[i] = load_part(ph + row(s + 1 < r.len ? s + 1 : r.len - 1) * r.h.ld, at, counts, s + 1 < r.len, 0u);
            }
        }
    }
    const auto state = [&](const float *x, int v) { return x && c + v < r.dim ? x[z * r.dim + c + v] : 0.f; };

    float x[V];
    if (p.teams * p.chunks == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            x[v] = state(r.start, v);
    } else {
        float P[V], Q[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.f, Q[v] = 0.f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float g = gate<T, LOG>(part<T>(a[i], v)), y = part<T>(b[i], v);
                Q[v] = ADJ ? g * (Q[v] + y) : fmaf(g, Q[v], y);
                P[v] *= g;
            }
            s_link[team][lane * V + v] = make_float2(P[v], Q[v]);
        }
        __syncthreads();
        if (jw == 0) {
            for (int k = 1; k < p.teams; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float2 n = s_link[team + k][lane * V + v];
                    Q[v] = fmaf(n.x, Q[v], n.y);
                    P[v] *= n.x;
                }
            if (p.chunks > 1) {
                const int64_t stride = (int64_t)across * SPAN;
                uint64_t *const links = ws + 2 + (int64_t)chain * p.chunks * stride + cw * SPAN + lane * V;
                Words<decltype(state)> words{links, stride, r.start, state};
                state_before(words, chunk, (unsigned)p.chunks, P, Q, x);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    x[v] = state(r.start, v);
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                s_in[cw][lane * V + v] = x[v];
        }
        __syncthreads();
        if (jw > 0) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                x[v] = s_in[cw][lane * V + v];
            for (int k = 0; k < jw; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float2 n = s_link[team - jw + k][lane * V + v];
                    x[v] = fmaf(n.x, x[v], n.y);
                }
        }
    }

    // the words are unpacked again: values kept from the first walk would take
    // twice the registers, and half the waves
#pragma unroll
    for (int i = 0; i < R; ++i)
        asm volatile("" : "+v"(a[i]), "+v"(b[i]));

    T *po = (T *)r.out.p + z * r.out.stride + c0;
    T *pd = ADJ ? (T *)r.adj_a.p + z * r.adj_a.stride + c0 : nullptr;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float out[V], da[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float g = gate<T, LOG>(part<T>(a[i], v)), y = part<T>(b[i], v);
            if constexpr (ADJ) {
                const float lam = y + x[v];
                float before = part<T>(h[i], v);
                if (!whole && s0 + i + 1 == r.len)
                    before = state(r.h0, v);
                x[v] = g * lam;
                da[v] = before * (LOG ? x[v] : lam);
                out[v] = lam;
            } else {
                x[v] = fmaf(g, x[v], y);
                out[v] = x[v];
            }
        }
        T *o = po + row(s0 + i) * r.out.ld + lane * V, *d = ADJ ? pd + row(s0 + i) * r.adj_a.ld + lane * V : nullptr;
        if (whole) {
            store_word(o, pack<T>(out));
            if constexpr (ADJ)
                store_word(d, pack<T>(da));
        } else if (s0 + i < r.len) {
            store_part(o, c, r.dim, pack<T>(out));
            if constexpr (ADJ)
                store_part(d, c, r.dim, pack<T>(da));
        }
    }
    if (chunk == (unsigned)p.chunks - 1 && jw == p.teams - 1)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c + v < r.dim)
                r.end[z * r.dim + c + v] = x[v];
}

int ceil_pow2(int64_t x, int most)
{
    int p = 1;
    while (p < x && p < most)
        p *= 2;
    return p;
}

constexpr int SHORT = 8, LONG = 32, LONG_ADJOINT = 20; // R

Plan plan_of(chol_dtype dt, bool adjoint, int64_t batch, int64_t len, int64_t dim)
{
    // Few channels leave most of a wave without work: quarters of waves walk runs of
    // their own then (us forward and adjoint, bf16: 16 x 65536 x 16 142 and 247 with
    // waves, 77 and 122 with quarters; 16 x 30000 x 64 101 and 162, 61 and 98; x 96
    // 125 and 196, 85 and 135).  Not where a row would end inside a second quarter,
    // which then shares the row's cache lines: 8 x 20000 x 30 fp32 30 and 42, 40 and 45.
    const int64_t words = (dim * (int64_t)lowp_size(dt) + 3) / 4;
    const bool quarters = words <= NARROW || (words < WAVE && words % NARROW == 0);
    const int lanes = quarters ? NARROW : WAVE, all = THREADS / lanes;
    const int64_t span = lanes * (4 / (int64_t)lowp_size(dt));
    const auto with = [&](int steps) {
        Plan p;
        p.lanes = lanes;
        p.steps = steps;
        p.teams = ceil_pow2((len + steps - 1) / steps, all);
        p.chunks = (int)std::max<int64_t>(1, (len + p.teams * steps - 1) / (p.teams * steps));
        const int64_t width = span * (all / p.teams);
        p.groups = (int)((dim + width - 1) / width);
        return p;
    };
    // More steps a lane mean fewer links for the same bytes (1 x 65536 x 128 bf16
    // forward 30 us with 32 steps, 92 with 8), up to what leaves two workgroups a
    // CU (40 and more: 8 x 4096 x 2048 97 us, with 32 86).  Where one workgroup
    // holds the sequence with 8 there are no links, and the lanes' runs count:
    // 64 x 16 x 2048 bf16 forward 8.8 us with 8, 11.3 with 32; adjoint 13.3, 17.7.
    return with(len <= 1 ? 1 : len <= all * SHORT ? SHORT : adjoint ? LONG_ADJOINT : LONG);
}

int64_t links_of(chol_dtype dt, const Plan &p, int64_t batch)
{
    return p.chunks > 1 ? batch * p.groups * p.chunks * (4 / (int64_t)lowp_size(dt)) * (THREADS / p.teams) : 0;
}

template <typename T, bool LOG, bool ADJ> chol_status run(chol_dtype dt, const RecArgs &r, void *ws, hipStream_t st)
{
    const Plan p = plan_of(dt, ADJ, r.batch, r.len, r.dim);
    if (p.chunks > 1) {
        const int64_t pairs = links_of(dt, p, r.batch) / 2 + 1; // (a row of links is a multiple of 16)
        hipLaunchKernelGGL(k_rec_clear, dim3((unsigned)((pairs + 256 * CLEAR - 1) / (256 * CLEAR))), dim3(256), 0, st,
                           (word_pair *)ws, pairs);
        CHOL_LAUNCH_CHECK();
    }
    const dim3 grid((unsigned)(r.batch * p.groups * p.chunks));
    constexpr int L = ADJ ? LONG_ADJOINT : LONG;
    const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(THREADS), 0, st, r, p, (uint64_t *)ws); };
    if (p.lanes == WAVE)
        p.steps == 1       ? launch(k_recurrence<T, LOG, ADJ, 1, WAVE>)
        : p.steps == SHORT ? launch(k_recurrence<T, LOG, ADJ, SHORT, WAVE>)
                           : launch(k_recurrence<T, LOG, ADJ, L, WAVE>);
    else
        p.steps == 1       ? launch(k_recurrence<T, LOG, ADJ, 1, NARROW>)
        : p.steps == SHORT ? launch(k_recurrence<T, LOG, ADJ, SHORT, NARROW>)
                           : launch(k_recurrence<T, LOG, ADJ, L, NARROW>);
    CHOL_LAUNCH_CHECK();
    return CHOL_OK;
}

} // namespace

// bytes, or -1 where the threads are more than a grid holds
int64_t recurrence_workspace(chol_dtype dt, int64_t batch, int64_t len, int64_t dim)
{
    int64_t bytes = 0;
    for (const bool adjoint : {false, true}) {
        const Plan p = plan_of(dt, adjoint, batch, len, dim);
        if ((double)batch * p.groups * p.chunks * THREADS > 4294967295.0)
            return -1;
        const int64_t links = links_of(dt, p, batch);
        if (links)
            bytes = std::max(bytes, (links + 2) * (int64_t)sizeof(uint64_t));
    }
    return bytes;
}

chol_status recurrence(chol_dtype dt, bool log_gate, bool adjoint, const RecArgs &r, void *ws, hipStream_t st)
{
    return with_lowp(dt, [&](auto *t) {
        typedef std::remove_pointer_t<decltype(t)> T;
        if (adjoint)
            return log_gate ? run<T, true, true>(dt, r, ws, st) : run<T, false, true>(dt, r, ws, st);
        return log_gate ? run<T, true, false>(dt, r, ws, st) : run<T, false, false>(dt, r, ws, st);
    });
}

} // namespace chol
