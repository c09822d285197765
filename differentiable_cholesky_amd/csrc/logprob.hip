// Log probabilities of given tokens, entropy and the most likely alternatives of rows of
// logits, and the gradient that reaches the logits.
//
//   y = scale x,  m = max y,  s = sum e^(y - m),  lse = m + log s,  logp = (y_token - m) - log s
//   entropy = log s - sum (y - m) e^(y - m) / s
//   adj_x_j = scale (gl (1[j = token] - p_j) - ge p_j (log p_j + entropy)),  p = e^(y - lse)
//
// Memory bounds both: forward reads a row once, the adjoint reads and writes it once
// (4096 x 128000 bf16 175 us, 6.0 TB/s, and 399 us, 5.3 TB/s).  A
// row is cut into chunks that stay in the registers of a wave (short rows, four to a
// workgroup) or of a workgroup, so that the maximum, the sums relative to it and the
// search for alternatives take one reading.  Several chunks a row (long rows, or few of
// them) are joined by a second launch, one wave a row.
//
// Alternatives: the k-th largest maximum of a lane is a bound that k elements reach, so only
// lanes that reach it, hardly more than k of the workgroup, can hold one.  Their elements go
// through LDS, a lane an element; those that reach the bound are ranked against each other
// (4096 x 128000 bf16 with 1, 8 and 20 alternatives 190, 243 and 296 us, where the search's own
// vector instructions and barriers add to a kernel that fills three quarters of the units; a
// bound and a list for each wave, found by comparing all lanes, took 221, 291 and 415, and
// comparing every element in its own lane 896 for 8).  Where lanes or elements are too many
// (equal values, sorted rows, or fewer lanes with a column above -inf than alternatives, so that
// the bound is -inf) a wave finds each alternative in turn among its elements, k times the
// comparisons (with 50 columns of 128000 above -inf 8 alternatives take 5090 us, 20 12500; 16
// rows 38 for 18).  Order: by value, then by the lower index; NaN before all.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "../../include/libchol.h"
#include "logprob.hpp"
#include "rows.hpp"
#include "wave.hpp"

namespace chol {

namespace {

constexpr int WAVE = 64, THREADS = 256, WAVES = THREADS / WAVE;
constexpr int MOST_CHUNKS = WAVE; // a lane each when they are joined
constexpr int NONE = INT_MIN;     // below the key of any value
constexpr int SLOTS = 32;         // lanes whose elements are looked at

template <typename T> constexpr int vec_of = 16 / (int)sizeof(T);

// Integers in the order of the values.
__device__ __forceinline__ int key_of(float x)
{
    const int b = x != x ? 0x7fc00000 : __float_as_int(x + 0.f); // (-0 is 0)
    return b ^ (b >> 31 & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int key) { return __int_as_float(key ^ (key >> 31 & 0x7fffffff)); }

__device__ __forceinline__ float wave_max(float x)
{
    return over_wave(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float x)
{
    return over_wave(x, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ int wave_max(int x)
{
    return over_wave(x, [](int a, int b) { return max(a, b); });
}
__device__ __forceinline__ int wave_min(int x)
{
    return over_wave(x, [](int a, int b) { return min(a, b); });
}

// How many of `lanes` are before this one.
__device__ __forceinline__ int before_lane(uint64_t lanes)
{
    return __builtin_amdgcn_mbcnt_hi((unsigned)(lanes >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)lanes, 0));
}

// A key that `top` or more of the wave's keys reach (all are above NONE and `most` is the
// greatest) and, unless several are equal, exactly so many: first by steps down from the
// greatest, each eight times the last, then by halving.  A comparison a turn, the rest is scalar.
template <int N> __device__ __forceinline__ int reached_by(const int (&keys)[N], int most, int top)
{
    const auto reach = [&](int key) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            n += __popcll(__ballot(keys[i] >= key));
        return n;
    };
    int high = most, low = most, n = top > 1 ? reach(most) : 1;
    if (n >= top)
        return most;
    for (unsigned step = 1u << 20; n < top; step *= 8) {
        high = low;
        low = step != 0 && (unsigned)most - (unsigned)NONE > step ? most - (int)step : NONE;
        n = reach(low);
    }
    while (n != top && (unsigned)high - (unsigned)low > 1) {
        const int half = (int)((unsigned)low + ((unsigned)high - (unsigned)low) / 2), r = reach(half);
        if (r < top)
            high = half;
        else
            low = half, n = r;
    }
    return low;
}

struct Entry {
    int key, index;
    __device__ __forceinline__ bool after(const Entry &o) const { return o.key > key || (o.key == key && o.index < index); }
};

// The first of the lanes' entries, in every lane; NONE if there is none.
__device__ __forceinline__ Entry wave_first(Entry e)
{
    const int key = wave_max(e.key);
    return {key, wave_min(e.key == key ? e.index : INT_MAX)};
}

// A row's statistics, or a chunk's: its maximum, sum e and sum g e, with e = 2^g and g =
// (x - m) scale log2(e).  Without a value above -inf: -inf, 0, 0.
struct Stats {
    float m, s, t;
};

// Half the distance to the maximum: the whole one, like a sum of distances instead of
// exponents, may pass the largest number where a small scale makes little of it.
__device__ __forceinline__ float half_below(float x, float m) { return fmaf(x, 0.5f, -0.5f * m); }

// t, relative to a maximum above, from which g leads to its own (where e = 2^g is 0, g may be anything).
__device__ __forceinline__ float shifted(const Stats &st, float g, float e) { return e == 0.f ? 0.f : fmaf(g, st.s, st.t) * e; }

// Natural logarithm of the sum, and of a logit's probability.  The latter from the distance to the
// maximum: from lse, whose rounding grows with the logits, a likely token's could come out above 0.
__device__ __forceinline__ float log_sum(const Stats &st) { return __builtin_amdgcn_logf(st.s) * LN2; }
__device__ __forceinline__ float log_prob(float scale, const Stats &st, float x)
{
    return x == -INFINITY && st.s == st.s ? x : fmaf(2.f * scale, half_below(x, st.m), -log_sum(st));
}

__device__ __forceinline__ void finish(const LogprobArgs &a, int64_t row, Stats st, float given)
{
    const float log_s = log_sum(st);
    const float lse = st.m == -INFINITY ? -INFINITY : fmaf(a.scale, st.m, log_s);
    a.lse[row] = st.s != st.s ? st.s : lse; // NaN
    const int64_t token = a.tokens[row];
    a.logp[row] = token < 0 || token >= a.vocab ? 0.f : log_prob(a.scale, st, given);
    if (a.entropy)
        a.entropy[row] = st.m == -INFINITY && st.s == st.s ? 0.f : log_s - LN2 * (st.t / st.s);
}

template <typename T> __device__ __forceinline__ float given_logit(const LogprobArgs &a, int64_t row)
{
    const int64_t token = a.tokens[row];
    return token < 0 || token >= a.vocab ? 0.f : (float)((const T *)a.x)[row * a.ld + token];
}

// Chunk of TEAM waves with NV vectors a lane; part: a row of `chunks` statistics and
// lists a row of logits, or nothing where the chunk is the row.
template <typename T, int NV, int TEAM, bool TOP>
__global__ void __launch_bounds__(THREADS) k_logprob(LogprobArgs a, int chunks, int chunk, Stats *stats, Entry *lists)
{
    constexpr int V = vec_of<T>, LANES = TEAM * WAVE, N = NV * V, MOST = CHOL_LOGPROB_MAX_TOP;
    __shared__ Stats s_stats[WAVES];
    __shared__ Entry s_some[TOP ? WAVES : 1][WAVE], s_list[TOP ? WAVES : 1][MOST];
    __shared__ vec<T, V> s_lane[TOP ? WAVES : 1][SLOTS][NV];
    __shared__ int s_column[TOP ? WAVES : 1][SLOTS];
    __shared__ float s_max[TOP ? WAVES : 1][WAVE], s_bound;
    __shared__ int s_count;
    const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE, t = threadIdx.x % LANES;
    const int64_t unit = (int64_t)blockIdx.x * (WAVES / TEAM) + (TEAM == 1 ? wave : 0);
    if (unit >= a.rows * chunks) // (waves of their own where TEAM is 1)
        return;
    const int64_t row = unit / chunks;
    const int c0 = (int)(unit % chunks) * chunk, end = (int)(c0 + chunk < a.vocab ? c0 + chunk : a.vocab);
    const T *p = (const T *)a.x + row * a.ld;
    vec<T, V> x[NV];
    if (c0 + LANES * N <= end) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            x[i] = load_vec<T, V>(p + c0 + (i * LANES + t) * V);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + (i * LANES + t) * V;
            x[i] = load_some<T, V>(p + c, end - c, (T)-INFINITY);
        }
    }
    const float k = 2.f * a.scale * LOG2E; // (of half a distance)
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v)
            m = fmaxf(m, (float)x[i][v]);
    const float lane_max = m;
    m = wave_max(m);
    const float ref = m == -INFINITY ? 0.f : m;
    float s = 0.f, w = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float g = half_below((float)x[i][v], ref) * k, e = __builtin_amdgcn_exp2f(g);
            s += e;
            w = fmaf(fmaxf(g, -__FLT_MAX__), e, w); // (e is 0 at -inf)
        }
    const float lane_sum = s;
    s = wave_sum(s), w = wave_sum(w);
    const Stats mine{m, s, w};
    if constexpr (TEAM > 1)
        if (lane == 0)
            s_stats[wave] = mine;

    int count = 0; // elements that may be alternatives, of the workgroup (TEAM 1: of the wave)
    const int list = TEAM > 1 ? 0 : wave;
    if constexpr (TOP) {
        const int top = a.top;
        // k of the lanes' maxima, so k elements, reach the bound
        float bound;
        if constexpr (TEAM == 1) {
            const int keys[1] = {key_of(lane_max)};
            bound = value_of(reached_by(keys, __builtin_amdgcn_readfirstlane(key_of(m)), top));
        } else {
            s_max[wave][lane] = lane_max;
            if (threadIdx.x == 0)
                s_count = 0;
            __syncthreads();
            if (wave == 0) {
                int keys[TEAM];
                float most = m;
#pragma unroll
                for (int i = 0; i < TEAM; ++i) {
                    keys[i] = key_of(s_max[i][lane]);
                    most = fmaxf(most, s_stats[i].m);
                }
                s_bound = value_of(reached_by(keys, __builtin_amdgcn_readfirstlane(key_of(most)), top));
            }
            __syncthreads();
            bound = s_bound;
        }
        // (a NaN makes its lane's sum one)
        const bool holds = lane_max >= bound || lane_sum != lane_sum;
        const uint64_t holders = __ballot(holds);
        const int slots = __popcll(holders), slot = before_lane(holders);
        if (slots <= SLOTS) {
            if (holds) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    s_lane[wave][slot][i] = x[i];
                s_column[wave][slot] = c0 + t * V;
            }
            wave_sync();
            for (int at = lane; at - lane < slots * N; at += WAVE) {
                const int from = at / N, k = at % N, c = from < slots ? s_column[wave][from] + k / V * (LANES * V) + k % V : end;
                const float y = from < slots ? (float)s_lane[wave][from][k / V][k % V] : -INFINITY;
                const uint64_t who = __ballot(!(y < bound) && c < end);
                int first = count;
                if constexpr (TEAM > 1) { // (in any order: places in the list are by value and index)
                    if (who && lane == 0)
                        first = atomicAdd(&s_count, __popcll(who));
                    first = __builtin_amdgcn_readfirstlane(first);
                }
                const int place = first + before_lane(who);
                if ((who >> lane & 1) && place < WAVE)
                    s_some[list][place] = {key_of(y), c};
                if constexpr (TEAM == 1)
                    count += __popcll(who);
            }
        } else if (TEAM == 1) {
            count = WAVE + 1;
        } else if (lane == 0) {
            atomicAdd(&s_count, WAVE + 1);
        }
        if constexpr (TEAM > 1) {
            __syncthreads();
            count = s_count;
            if (count <= WAVE && wave > 0)
                return;
        } else {
            wave_sync();
        }
        if (count <= WAVE) {
            // a lane's place is the number of those before it
            Entry e{NONE, INT_MAX};
            if (lane < count)
                e = s_some[list][lane];
            int before = 0;
            for (int l = 0; l < count; ++l)
                before += e.after(s_some[list][l]) ? 1 : 0;
            if (lane < top)
                s_list[list][lane] = {NONE, INT_MAX};
            if (lane < count && before < top)
                s_list[list][before] = e;
        } else {
            // (from memory again: from registers it would be as many instructions as elements)
            Entry last{INT_MAX, -1};
            for (int r = 0; r < top; ++r) {
                Entry e{NONE, INT_MAX};
#pragma unroll 1
                for (int k = 0; k < N; ++k) {
                    const int c = c0 + (k / V * LANES + t) * V + k % V;
                    const Entry o{c < end ? key_of((float)p[c]) : NONE, c};
                    if (o.after(last) && e.after(o))
                        e = o;
                }
                last = wave_first(e);
                if (lane == 0)
                    s_list[wave][r] = last;
            }
        }
    }

    Stats all = mine;
    if constexpr (TEAM > 1) {
        if (!TOP || count > WAVE) { // (else the waves have met, and only the first is here)
            __syncthreads();
            if (wave > 0)
                return;
        }
#pragma unroll
        for (int i = 0; i < TEAM; ++i)
            all.m = fmaxf(all.m, s_stats[i].m);
        all.s = all.t = 0.f;
#pragma unroll
        for (int i = 0; i < TEAM; ++i) {
            const Stats o = s_stats[i];
            if (o.m > -INFINITY || o.s != o.s) {
                const float g = half_below(o.m, all.m) * k, e = __builtin_amdgcn_exp2f(g);
                all.s = fmaf(o.s, e, all.s);
                all.t += shifted(o, g, e);
            }
        }
    }
    if constexpr (TOP)
        wave_sync();
    if (lane == 0) {
        if (chunks > 1)
            stats[unit] = all;
        else
            finish(a, row, all, given_logit<T>(a, row));
    }
    if constexpr (TOP) {
        // The waves' lists (where there are any) together: an entry's place is its own and, in each other list, the
        // number of those before it (found by halving; entries that are none come last)
        Entry mine{NONE, INT_MAX};
        if (TEAM == 1 || count <= WAVE) {
            if (lane < a.top)
                mine = s_list[list][lane];
        } else {
            if (lane < a.top)
                s_some[0][lane] = mine;
            wave_sync();
            for (int at = lane; at < TEAM * a.top; at += WAVE) {
                const int own = at / a.top;
                const Entry e = s_list[own][at % a.top];
                int place = at % a.top;
#pragma unroll
                for (int w = 1; w < TEAM; ++w) {
                    const Entry *const list = s_list[(own + w) % TEAM];
                    int first = 0;
                    for (int size = a.top; size > 0; size /= 2) {
                        // the first of `size + 1` places from `first` on whose entry is not before e
                        const int half = first + size / 2;
                        const bool before = e.after(list[half]);
                        first = before ? half + 1 : first;
                        size -= before && size % 2 == 0 ? 1 : 0;
                    }
                    place += first;
                }
                if (place < a.top && e.key != NONE)
                    s_some[0][place] = e;
            }
            wave_sync();
            if (lane < a.top)
                mine = s_some[0][lane];
        }
        if (lane < a.top) {
            if (chunks > 1) {
                lists[unit * a.top + lane] = mine;
            } else {
                a.top_ids[row * a.top + lane] = mine.index;
                a.top_logp[row * a.top + lane] = log_prob(a.scale, all, value_of(mine.key));
            }
        }
    }
}

// Joins a row's chunks, a lane each; one wave.  The lists come to LDS together.
template <typename T>
__global__ void __launch_bounds__(WAVE) k_logprob_join(LogprobArgs a, int chunks, const Stats *stats, const Entry *lists)
{
    extern __shared__ Entry s_lists[];
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    for (int i = lane; i < chunks * a.top; i += WAVE)
        s_lists[i] = lists[row * chunks * a.top + i];
    const float k = 2.f * a.scale * LOG2E, given = given_logit<T>(a, row);
    Stats st{-INFINITY, 0.f, 0.f};
    if (lane < chunks)
        st = stats[row * chunks + lane];
    Stats all;
    all.m = wave_max(st.m);
    float s = 0.f, t = 0.f;
    if (st.m > -INFINITY || st.s != st.s) {
        const float g = half_below(st.m, all.m) * k, e = __builtin_amdgcn_exp2f(g);
        s = st.s * e;
        t = shifted(st, g, e);
    }
    all.s = wave_sum(s), all.t = wave_sum(t);
    if (lane == 0)
        finish(a, row, all, given);
    if (a.top == 0)
        return;
    wave_sync();
    const Entry *list = s_lists + lane * a.top;
    int at = 0;
    Entry mine{NONE, INT_MAX}, e = lane < chunks ? list[0] : mine;
    for (int r = 0; r < a.top; ++r) {
        const Entry f = wave_first(e);
        if (e.key == f.key && e.index == f.index) {
            ++at;
            e = at < a.top ? list[at] : Entry{NONE, INT_MAX};
        }
        if (lane == r)
            mine = f;
    }
    if (lane < a.top) {
        a.top_ids[row * a.top + lane] = mine.index;
        a.top_logp[row * a.top + lane] = log_prob(a.scale, all, value_of(mine.key));
    }
}

// LANES threads a row, NV vectors each; rows longer than that take several workgroups.
template <typename T, int NV>
__global__ void __launch_bounds__(THREADS) k_logprob_adjoint(LogprobAdjArgs a, unsigned across, int lanes)
{
    constexpr int V = vec_of<T>;
    const int t = threadIdx.x % lanes;
    const int64_t row = (int64_t)(blockIdx.x / across) * (THREADS / lanes) + threadIdx.x / lanes;
    const int c0 = (int)(blockIdx.x % across) * (THREADS * NV * V);
    if (row >= a.rows)
        return;
    const int64_t token = a.tokens[row];
    const float lse = a.lse[row], H = a.adj_entropy ? a.entropy[row] : 0.f, ge = a.adj_entropy ? a.adj_entropy[row] : 0.f;
    const float gl = a.adj_logp && token >= 0 && token < a.vocab ? a.adj_logp[row] : 0.f;
    const T *x = (const T *)a.x + row * a.ld;
    T *d = (T *)a.adj + row * a.lda;
    vec<T, V> in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + (i * lanes + t) * V;
        in[i] = load_some<T, V>(x + c, a.vocab - c);
    }
    // no token is possible, or no gradient reaches the row, whose logits may be anything: zeros
    const bool empty = lse == -INFINITY || (gl == 0.f && ge == 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + (i * lanes + t) * V;
        vec<T, V> out;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float lp = fmaf(a.scale, (float)in[i][v], -lse), p = __builtin_amdgcn_exp2f(lp * LOG2E);
            float g = -p * fmaf(ge, fmaxf(lp, -200.f) + H, gl); // (p is 0 from there on down)
            if (c + v == token)
                g += gl;
            out[v] = (T)(empty ? 0.f : a.scale * g);
        }
        store_some<T, V>(d + c, a.vocab - c, out);
    }
}

struct Plan {
    int team;     // waves
    int vectors;  // of a lane
    int chunks, chunk;
};

Plan plan_of(chol_dtype dt, int64_t rows, int64_t vocab)
{
    const int v = 16 / (int)lowp_size(dt);
    Plan p;
    p.team = vocab <= WAVE * 8 * v ? 1 : WAVES;
    const int64_t lanes = p.team * WAVE;
    // Eight vectors a lane, or two where the rows are short or would leave CUs without
    // work (fewer than two workgroups for each).
    const int64_t wide = lanes * 8 * v, narrow = lanes * 2 * v;
    const bool small = vocab <= narrow ||
                       (p.team > 1 && rows * ((vocab + wide - 1) / wide) < 512 && vocab <= narrow * MOST_CHUNKS);
    p.vectors = small ? 2 : 8;
    const int64_t most = small ? narrow : wide;
    p.chunks = (int)std::max<int64_t>(1, (vocab + most - 1) / most);
    // chunks of one size, a multiple of a vector
    p.chunk = (int)(((vocab + p.chunks - 1) / p.chunks + v - 1) / v * v);
    return p;
}

int64_t ceil_of(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int ADJ_VECTORS = 4;

} // namespace

size_t logprob_workspace(chol_dtype dt, int64_t rows, int64_t vocab, int top)
{
    const Plan p = plan_of(dt, rows, vocab);
    return p.chunks > 1 ? (size_t)(rows * p.chunks) * (sizeof(Stats) + top * sizeof(Entry)) : 0;
}

bool logprob_fits(chol_dtype dt, int64_t rows, int64_t vocab)
{
    const Plan p = plan_of(dt, rows, vocab);
    const int64_t v = 16 / (int64_t)lowp_size(dt);
    return (double)rows * std::max<int64_t>(p.chunks, ceil_of(vocab, THREADS * ADJ_VECTORS * v)) * THREADS <= 4294967295.0;
}

chol_status logprob(chol_dtype dt, const LogprobArgs &a, void *ws, hipStream_t st)
{
    const Plan p = plan_of(dt, a.rows, a.vocab);
    Stats *stats = (Stats *)ws;
    Entry *lists = (Entry *)(stats + a.rows * p.chunks);
    return with_lowp(dt, [&](auto *e) {
        typedef std::remove_pointer_t<decltype(e)> T;
        const dim3 grid((unsigned)ceil_of(a.rows * p.chunks, WAVES / p.team));
        const auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid, dim3(THREADS), 0, st, a, p.chunks, p.chunk, stats, lists);
        };
        const auto with_top = [&](auto nv, auto team) {
            a.top > 0 ? launch(k_logprob<T, nv, team, true>) : launch(k_logprob<T, nv, team, false>);
        };
        typedef std::integral_constant<int, 1> One;
        typedef std::integral_constant<int, 2> Two;
        typedef std::integral_constant<int, WAVES> All;
        typedef std::integral_constant<int, 8> Eight;
        if (p.team == 1)
            p.vectors == 2 ? with_top(Two(), One()) : with_top(Eight(), One());
        else
            p.vectors == 2 ? with_top(Two(), All()) : with_top(Eight(), All());
        CHOL_LAUNCH_CHECK();
        if (p.chunks > 1) {
            hipLaunchKernelGGL(k_logprob_join<T>, dim3((unsigned)a.rows), dim3(WAVE), p.chunks * a.top * sizeof(Entry), st, a,
                               p.chunks, (const Stats *)stats, (const Entry *)lists);
            CHOL_LAUNCH_CHECK();
        }
        return CHOL_OK;
    });
}

chol_status logprob_adjoint(chol_dtype dt, const LogprobAdjArgs &a, hipStream_t st)
{
    return with_lowp(dt, [&](auto *e) {
        typedef std::remove_pointer_t<decltype(e)> T;
        // (a workgroup takes as many rows as its threads hold: 23630 x 416 bf16 84 -> 12 us)
        const int64_t vectors = ceil_of(a.vocab, vec_of<T>), across = ceil_of(vectors, THREADS * ADJ_VECTORS);
        int lanes = 1;
        while (lanes < THREADS && lanes * ADJ_VECTORS < vectors)
            lanes *= 2;
        hipLaunchKernelGGL((k_logprob_adjoint<T, ADJ_VECTORS>), dim3((unsigned)(ceil_of(a.rows, THREADS / lanes) * across)),
                           dim3(THREADS), 0, st, a, (unsigned)across, lanes);
        CHOL_LAUNCH_CHECK();
        return CHOL_OK;
    });
}

} // namespace chol
