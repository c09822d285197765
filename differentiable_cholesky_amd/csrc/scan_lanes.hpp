// What the selective scan and its adjoint share: how lanes hold channels, states and
// steps, their loads, and the plan of a launch.
//
// A wave holds 16 channels: lane l has channel l % 16 and R consecutive states, those of
// row l / 16 of the wave (16 lanes).  Then B and C are the same along a row: one register
// holds them for 16 / R steps and an operand of the multiplication broadcasts a lane of it
// (DPP).  Sums over the states are within the lane and over four rows; four steps' sums at
// once take three swaps of rows and leave each lane the sum of one step and channel, which
// is also how u, delta and z are loaded and results are stored: nothing of a step and
// channel is computed twice.  Only dt and dt u go from the lane that has them to the
// others, in LDS of the wave's own.
//
// Where batch and channels give too few waves, sequences are cut into segments.  A first
// launch walks each from a state of zero to its end, whose state, with the sum of its
// steps, is a map x -> exp(A sum dt) x + Q; the segments' own walks compose the maps
// before them.  No workgroup waits for another, and every sum has one order.
#pragma once

#include <algorithm>
#include <type_traits>
#include <utility>

#include "scan.hpp"
#include "wave.hpp"

namespace chol {

namespace {

constexpr int WAVE = 64, ROW = 16; // lanes; channels of a wave

template <int I> using index = std::integral_constant<int, I>;
template <typename F, int... I> __device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>)
{
    (f(index<I>()), ...);
}
template <int N, typename F> __device__ __forceinline__ void each(F f)
{
    each_of(f, std::make_integer_sequence<int, N>());
}

// Row r gets the sum over the four rows of x[r].
__device__ __forceinline__ float over_rows(const float (&x)[4])
{
    const Two<float> p = swap_halves(x[0], x[2]), q = swap_halves(x[1], x[3]);
    const Two<float> s = swap_rows(p.a + p.b, q.a + q.b);
    return s.a + s.b;
}
// The sum over the rows, in every lane.
__device__ __forceinline__ float over_rows(float x)
{
    const float same[4] = {x, x, x, x};
    return over_rows(same);
}
// log(1 + exp(x)): the larger of x and 0, and log(1 + w) with w = exp(-|x|).  Where
// u = 1 + w is rounded, what it lost is added (the logarithm's slope there is 1 / u; w
// is small where it matters).  NaN stays one by the choice (a maximum would drop it).  The hardware's logarithm is within 1.2e-7 on all of (1, 2).
__device__ __forceinline__ float softplus_of(float x)
{
    // exp(-|x|) with its product's low part (expf_of); at -110, where it is 0, and below
    const float v = fmaxf(-fabsf(x), -110.f), y = v * LOG2E, e = __builtin_amdgcn_exp2f(y);
    const float low = fmaf(v, (float)(1.4426950408889634074 - LOG2E), fmaf(v, LOG2E, -y));
    const float w = fmaf(e * LN2, low, e), u = 1.f + w;
    return (x < 0.f ? 0.f : x) + fmaf(__builtin_amdgcn_logf(u), LN2, w - (u - 1.f));
}

struct Plan {
    int waves;             // of a workgroup of the adjoint
    int per_group;         // workgroups along a group's channels
    int64_t across;        // workgroups across groups and channels
    int segments;          // of a sequence
    int segment;           // steps of one
};

// An array from some row on, as buffer instructions take it: the address is the wave's, the
// offset (32 bits, unsigned) the lane's, so that a load costs no vector arithmetic.
template <typename T> struct Buffer {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ Buffer(const char *p)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), 0, -1, 0x00027000))
    {
    }
    __device__ __forceinline__ T load(unsigned lane, unsigned wave) const
    {
        if constexpr (sizeof(T) == 4)
            return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, lane, wave, 0));
        else
            return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, lane, wave, 0));
    }
    __device__ __forceinline__ void store(unsigned lane, unsigned wave, T x) const
    {
        if constexpr (sizeof(T) == 4)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, x), r, lane, wave, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, x), r, lane, wave, 0);
    }
};

// N values of a lane from a block of rows, EVERY rows apart.  KEEP: an offset for each
// value; else one, and a scalar register for each.
template <typename T, int N, int EVERY, bool KEEP> struct Feed {
    const char *p;     // the sequence's first row
    unsigned ld;       // bytes
    unsigned first, off[KEEP ? N : 1];
    // row first + k * EVERY of a block, column col
    __device__ __forceinline__ Feed(const SeqRows &r, int64_t z, int64_t c0, int row, int col)
        : p((const char *)((const T *)r.p + z * r.stride + c0)), ld((unsigned)r.ld * (unsigned)sizeof(T)), first(row)
    {
#pragma unroll
        for (int k = 0; k < (KEEP ? N : 1); ++k)
            off[k] = (first + k * EVERY) * ld + col * (unsigned)sizeof(T);
    }
    __device__ __forceinline__ Buffer<T> block(int t) const { return Buffer<T>(p + (uint64_t)(unsigned)t * ld); }
    __device__ __forceinline__ unsigned lane(int k) const { return off[KEEP ? k : 0]; }
    __device__ __forceinline__ unsigned wave(int k) const { return KEEP ? 0u : k * EVERY * ld; }
    // the block from step t; rows past `left` of them are read again at the last one
    // (WHOLE: there are none)
    template <bool WHOLE = false> __device__ __forceinline__ void load(T (&v)[N], int t, int left) const
    {
        const Buffer<T> b = block(t);
        if (WHOLE || left >= N * EVERY) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                v[k] = b.load(lane(k), wave(k));
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const unsigned last = (unsigned)left - 1u, row = min(first + k * EVERY, last);
                v[k] = b.load(off[0] + (row - first) * ld, 0);
            }
        }
    }
    __device__ __forceinline__ void store(int t, int k, T x) const { block(t).store(lane(k), wave(k), x); }
    __device__ __forceinline__ bool inside(int k, int left) const { return (int)first + k * EVERY < left; }
};

// A lane's place: its channel and its first state.
template <int R> struct Place {
    int row, j;            // of the wave; lane of the row
    int g, c, n0;          // group, channel, first state
    int64_t z;             // batch element
    int from, to, seg;     // steps; segment
    int first;             // the wave's first channel
    bool real;             // the channel exists (c is a real one in any case)
    // values of one step and channel a lane: steps 4 k + row of a block, channel c
    template <typename T, int STEPS, bool KEEP = true>
    __device__ __forceinline__ Feed<T, STEPS / 4, 4, KEEP> column(const SeqRows &r) const
    {
        return {r, z, first, row, c - first};
    }
    // B or C: value k holds steps k * 16 / R on of a block, lane j of a row the step j / R
    // and the row's state j % R of them
    template <typename T, int STEPS, bool KEEP = true>
    __device__ __forceinline__ Feed<T, STEPS * R / ROW, ROW / R, KEEP> mixed(const SeqRows &r, int states) const
    {
        const int n = n0 + j % R;
        return {r, z, (int64_t)g * states, j / R, n < states ? n : states - 1};
    }
    // false where the wave has no channel
    __device__ __forceinline__ bool set(const ScanArgs &a, const Plan &p, int waves)
    {
        const int lane = threadIdx.x % WAVE, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
        row = lane / ROW, j = lane % ROW;
        const unsigned block = blockIdx.x, cb = block % (unsigned)p.across, rest = block / (unsigned)p.across;
        seg = (int)(rest % (unsigned)p.segments);
        z = rest / (unsigned)p.segments;
        g = (int)(cb / (unsigned)p.per_group);
        const int per = (int)((unsigned)a.dim / (unsigned)a.groups);
        const int at = ((int)(cb % (unsigned)p.per_group) * waves + wave) * ROW;
        real = at + j < per;
        first = g * per + (at < per ? at : per - 1);
        c = g * per + (real ? at + j : per - 1);
        n0 = R * row;
        from = seg * p.segment;
        to = (int)min((int64_t)from + p.segment, a.len);
        return at < per;
    }
};

// R states of a lane in an array [.., states]
template <int R> __device__ __forceinline__ void load_states(const float *p, int n0, int states, float (&x)[R])
{
#pragma unroll
    for (int i = 0; i < R; i += 4) {
        const vec<float, 4> v = load_some<float, 4>(p + n0 + i, (int64_t)states - n0 - i);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[i + k] = v[k];
    }
}
template <int R> __device__ __forceinline__ void store_states(float *p, int n0, int states, const float (&x)[R])
{
#pragma unroll
    for (int i = 0; i < R; i += 4) {
        vec<float, 4> v;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = x[i + k];
        store_some<float, 4>(p + n0 + i, (int64_t)states - n0 - i, v);
    }
}

// A of -inf, under which exp(dt A) is 0, as the lowest number, under which it is 0 for any dt above
// 2^-120.  So it is 1 for dt = 0 (steps past the end, lanes without a channel), where 0 times -inf
// would be NaN, and what A multiplies in the gradients is 0.  NaN stays one.
__device__ __forceinline__ float finite_rate(float A) { return A < -__FLT_MAX__ ? -__FLT_MAX__ : A; }
// log2(e) A, for a base of 2.
__device__ __forceinline__ float base2_rate(float A) { return finite_rate(A * LOG2E); }

// A segment's map, for the walk that composes them: Q of every state, the steps' sum.
struct Maps {
    float *Q, *sum;
    const ScanArgs &a;
    __device__ __forceinline__ Maps(const ScanArgs &args, float *ws, int segments)
        : Q(ws), sum(ws + (int64_t)segments * args.batch * args.dim * args.states), a(args)
    {
    }
    __device__ __forceinline__ int64_t at(int seg, int64_t z, int c) const { return (seg * a.batch + z) * a.dim + c; }
    // x through the maps of `count` segments from `seg` on, `step` apart; a few are on
    // their way together (16384 x 256 bf16 with 64 segments 67 -> 53 us)
    template <int R>
    __device__ __forceinline__ void apply(float (&x)[R], int seg, int count, int step, int64_t z, int c, int n0,
                                          const float (&A2)[R]) const
    {
        constexpr int AT_ONCE = 32 / R;
        for (int s = 0; s < count; s += AT_ONCE) {
            float total[AT_ONCE], q[AT_ONCE][R];
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) {
                const int64_t m = at(seg + (s + k < count ? s + k : count - 1) * step, z, c);
                total[k] = sum[m];
                load_states<R>(Q + m * a.states, n0, a.states, q[k]);
            }
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k)
                if (s + k < count)
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        x[i] = fmaf(__builtin_amdgcn_exp2f(total[k] * A2[i]), x[i], q[k][i]);
        }
    }
};

// A step's length.  (Both forms and a choice: a branch would part the block of steps.)
template <typename T> __device__ __forceinline__ float step_of(T raw, float bias, bool softplus)
{
    const float x = (float)raw + bias, s = softplus_of(x);
    return softplus ? s : x;
}

constexpr int WAVES = 4, STEPS = 16; // of a workgroup; of a block
// Steps between two saved states, and those that the adjoint holds in registers at a time.
template <int R> constexpr int block_steps = 256 / R;
template <int R> constexpr int part_steps = R < 16 ? 32 / R : 4;

// An empty sequence's states and gradients: the given ones, or zero.
__global__ void __launch_bounds__(256) k_scan_copy(const float *from, float *to, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n)
        to[i] = from ? from[i] : 0.f;
}

int rows_of(int states) { return states <= 16 ? 4 : states <= 32 ? 8 : 16; } // R

Plan plan_of(const ScanArgs &a, bool adjoint)
{
    Plan p;
    const int64_t per = a.dim / a.groups, wave_count = (per + ROW - 1) / ROW, block = scan_block(a.states);
    // Waves of a workgroup lie along a group's channels; the adjoint's idle ones would wait
    // at its barriers, so it takes one or two where a group has no more (27 x 1863 x 16 of 4
    // groups of 64 states 1250 -> 490 us, 27 x 2530 x 76 of 4 groups of 11 366 -> 271).  Beyond
    // that it has four, up to three of them idle in a group's last workgroup.
    const int waves = p.waves = adjoint && wave_count <= 2 ? (int)wave_count : WAVES;
    p.per_group = (int)((wave_count + waves - 1) / waves);
    p.across = (int64_t)p.per_group * a.groups;
    // A first walk costs a step of the forward about as much again, and less of the adjoint,
    // which also needs two waves a SIMD more: 4 x 2048 x 4096 bf16 (1024 waves, one a
    // SIMD) forward 178 us whole, 219 in 4 segments, adjoint 900 and 721; 2 x 2048 x 4096 forward
    // 160 in 2 segments, 126 in 8, adjoint 576 and 368.  Beyond 32 states a SIMD holds one wave,
    // and segments only fill it (4 x 2048 x 4096 of 64 states adjoint 2790 us whole, 3100 in 4 at the time;
    // 16 x 416 x 71 forward 43 us in 7, 73 in 26, adjoint 118 in 7, 162 in 9).  More than 64 segments cost more to put together than they save (16384 x 256
    // forward 68 us, with 256 116).
    // (waves, with the idle ones: they hold a place)
    const int64_t all = a.batch * p.across * waves, blocks = std::max<int64_t>(1, (a.len + block - 1) / block);
    const bool two = a.states <= 32;
    const int64_t want = all >= (adjoint && two ? 1536 : 768) ? 1 : std::min<int64_t>({blocks, 64, (two ? 4096 : 1024) / all});
    const int64_t each = (blocks + want - 1) / want;
    p.segment = (int)std::min<int64_t>(each * block, INT32_MAX);
    p.segments = (int)((blocks + each - 1) / each);
    return p;
}

int64_t maps_size(const ScanArgs &a, const Plan &p)
{
    return p.segments > 1 ? p.segments * a.batch * a.dim * (int64_t)(a.states + 1) : 0;
}

template <typename F> chol_status with_rows(int states, F f)
{
    return states <= 16 ? f(index<4>()) : states <= 32 ? f(index<8>()) : f(index<16>());
}

int64_t ceil_of(int64_t a, int64_t b) { return (a + b - 1) / b; }

chol_status copy(const float *from, float *to, int64_t n, hipStream_t st)
{
    if (n > 0 && to && from != to) {
        hipLaunchKernelGGL(k_scan_copy, dim3((unsigned)ceil_of(n, 256)), dim3(256), 0, st, from, to, n);
        CHOL_LAUNCH_CHECK();
    }
    return CHOL_OK;
}

bool grid_ok(double threads) { return threads <= 4294967295.0; }

} // namespace

} // namespace chol
