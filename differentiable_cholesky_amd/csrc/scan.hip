// The selective state space scan and its adjoint.
//
//   dt_t = softplus(delta_t + bias) (or delta_t + bias),
//   h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t          (N states a channel)
//   y_t = (sum_n C_t h_t + D u_t) silu(z_t)           (without z: the sum)
//
// and with a_t the gradient of the sum, from the last step,
//
//   g_t = C_t a_t + mu_{t+1},  mu_t = exp(dt_t A) g_t
//   adj_C = sum_c a h,  adj_B = sum_c g dt u          (over the channels of the group)
//   s_t = sum_n g B,  adj_u = dt s + D a,  adj_dt = u s + sum_n A mu h_{t-1}
//   adj_A = sum dt mu h_{t-1},  adj_D = sum a u,  adj_h0 = mu_0
//
// An exponential and four more operations a state and step forward: 8 + 16 cycles of a
// SIMD a wave, more than the channel's four 16-bit numbers cost in memory for 16 states.
// So the vector units bound it, and the layout serves them.  A wave holds 16 channels:
// lane l has channel l % 16 and R consecutive states, those of row l / 16 of the wave
// (16 lanes).  Then B and C are the same along a row: one register holds them for 16 / R
// steps and an operand of the multiplication broadcasts a lane of it (DPP).  Sums over
// the states are within the lane and over four rows; four steps' sums at once take
// three swaps of rows and leave each lane the sum of one step and channel, which is also
// how u, delta and z are loaded and y is stored: nothing of a step and channel is
// computed twice.  Only dt and dt u go from the lane that has them to the others, in LDS
// of the wave's own.
//
// Where batch and channels give too few waves, sequences are cut into segments.  A first
// launch walks each from a state of zero to its end, whose state, with the sum of its
// steps, is a map x -> exp(A sum dt) x + Q; the segments' own walks compose the maps
// before them.  No workgroup waits for another, and every sum has one order.
//
// The adjoint starts from states that the forward saved every `scan_block` steps, walks
// a part of a block forward in registers (R * T states and their exponentials a lane)
// and then back.  Sums over the channels take the lanes of a row, the waves of the
// workgroup, and by a second launch the workgroups.
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
// Lane j of a row gets the sum over the row's lanes of x[j].  Halves of the row, then of
// those, exchange what they do not keep: x[k] + its exchange goes to all lanes, and that of
// x[k + 8] (k + 4) over the upper half (the bank mask names groups of four lanes whose
// result is written).  Written with selections the compiler takes 47 instructions, this 35.
// An operand of an exchange has to be two instructions old: s_nop 1 sees to it for what
// comes in, and the order below has it for the rest.
__device__ __forceinline__ float over_lanes(const float (&in)[16], int lane)
{
    float x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k)
        x[k] = in[k];
#define EXCHANGE(k, from, ctrl, mask) "v_add_f32_dpp %" #k ", %" #from ", %" #from " " ctrl " row_mask:0xf bank_mask:" mask "\n\t"
#define BOTH(k, far, ctrl, mask) EXCHANGE(k, k, ctrl, "0xf") EXCHANGE(k, far, ctrl, mask)
#define FAR(k, far) BOTH(k, far, "row_ror:8", "0xc")         // lanes l and l + 8
#define MID(k, far) BOTH(k, far, "row_half_mirror", "0xa")   // l and l ^ 7
    asm("s_nop 1\n\t"
        FAR(0, 8) FAR(1, 9) FAR(2, 10) FAR(3, 11) FAR(4, 12) FAR(5, 13) FAR(6, 14) FAR(7, 15)
        MID(0, 4) MID(1, 5) MID(2, 6) MID(3, 7)
        EXCHANGE(0, 0, "quad_perm:[2,3,0,1]", "0xf") EXCHANGE(1, 1, "quad_perm:[2,3,0,1]", "0xf")
        EXCHANGE(2, 2, "quad_perm:[2,3,0,1]", "0xf") EXCHANGE(3, 3, "quad_perm:[2,3,0,1]", "0xf")
        EXCHANGE(0, 0, "quad_perm:[1,0,3,2]", "0xf") EXCHANGE(1, 1, "quad_perm:[1,0,3,2]", "0xf")
        EXCHANGE(2, 2, "quad_perm:[1,0,3,2]", "0xf") EXCHANGE(3, 3, "quad_perm:[1,0,3,2]", "0xf")
        : "+v"(x[0]), "+v"(x[1]), "+v"(x[2]), "+v"(x[3]), "+v"(x[4]), "+v"(x[5]), "+v"(x[6]), "+v"(x[7])
        : "v"(x[8]), "v"(x[9]), "v"(x[10]), "v"(x[11]), "v"(x[12]), "v"(x[13]), "v"(x[14]), "v"(x[15]));
#undef MID
#undef FAR
#undef BOTH
#undef EXCHANGE
    const float lo = lane & 1 ? x[1] : x[0], hi = lane & 1 ? x[3] : x[2];
    return lane & 2 ? hi : lo;
}

// log(1 + exp(x)): the larger of x and 0, and log(1 + w) with w = exp(-|x|).  Where
// u = 1 + w is rounded, what it lost is added (the logarithm's slope there is 1 / u; w
// is small where it matters).  The hardware's logarithm is within 1.2e-7 on all of (1, 2).
__device__ __forceinline__ float softplus_of(float x)
{
    // exp(-|x|) with its product's low part (expf_of); at -110, where it is 0, and below
    const float v = fmaxf(-fabsf(x), -110.f), y = v * LOG2E, e = __builtin_amdgcn_exp2f(y);
    const float low = fmaf(v, (float)(1.4426950408889634074 - LOG2E), fmaf(v, LOG2E, -y));
    const float w = fmaf(e * LN2, low, e), u = 1.f + w;
    return fmaxf(x, 0.f) + fmaf(__builtin_amdgcn_logf(u), LN2, w - (u - 1.f));
}

struct Plan {
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

constexpr int FWD_WAVES = 4, STEPS = 16;
// Steps between two saved states, and those that the adjoint holds in registers at a time.
template <int R> constexpr int block_steps = 256 / R;
template <int R> constexpr int part_steps = R < 16 ? 32 / R : 4;

// ENDS: only walks to the end of a segment from zero and writes its map.
template <typename T, int R, bool ENDS, bool GATED>
__global__ void __launch_bounds__(FWD_WAVES *WAVE, R > 4 ? 1 : 3) k_scan(ScanArgs a, Plan p, float *ws)
{
    constexpr bool FULL = sizeof(T) == 4;
    constexpr int Q = STEPS / 4, PER = ROW / R, REGS = R, BLOCK = block_steps<R>;
    // (two of each: the next block's is written while this one's is read)
    __shared__ float2 s_step[2][FWD_WAVES][STEPS][ROW];
    __shared__ vec<float, 4> s_mixed[2][FWD_WAVES][STEPS][R]; // C; on a first walk B
    Place<R> at;
    if (!at.set(a, p, FWD_WAVES))
        return;
    const int wave = threadIdx.x / WAVE, row = at.row, j = at.j;
    float A2[R], h[R];
    load_states<R>(a.A + (int64_t)at.c * a.states, at.n0, a.states, A2);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        A2[i] *= LOG2E;
        h[i] = 0.f;
    }
    const float bias = a.bias ? a.bias[at.c] : 0.f, D = a.D ? a.D[at.c] : 0.f;
    const Maps maps(a, ws, p.segments);
    // hlast may replace h0, so that where there are segments the first launch copies h0,
    // in the place of the last segment's map, which nobody needs
    if constexpr (ENDS) {
        if (at.seg == p.segments - 1) {
            if (a.h0)
                load_states<R>(a.h0 + (at.z * a.dim + at.c) * a.states, at.n0, a.states, h);
            at.to = at.from;
        }
    } else {
        if (p.segments > 1)
            load_states<R>(maps.Q + maps.at(p.segments - 1, at.z, at.c) * a.states, at.n0, a.states, h);
        else if (a.h0)
            load_states<R>(a.h0 + (at.z * a.dim + at.c) * a.states, at.n0, a.states, h);
        maps.template apply<R>(h, 0, at.seg, 1, at.z, at.c, at.n0, A2);
    }
    const auto ru = at.template column<T, STEPS>(a.u), rdelta = at.template column<T, STEPS>(a.delta);
    const auto rz = at.template column<T, STEPS>(a.z), ry = at.template column<T, STEPS>(a.y);
    const auto rB = at.template mixed<T, STEPS>(a.B, a.states), rC = at.template mixed<T, STEPS>(a.C, a.states);
    const bool no_state = at.n0 + j % R >= a.states;
    float total = 0.f;
    // of the block that is walked, the one after it, and the one on its way
    T u[Q], z[Q], next_u[Q], next_z[Q], far_u[Q], far_delta[Q], far_z[Q], far_B[REGS], far_C[REGS];
    float B[REGS], next_B[REGS];
    const auto fetch = [&](int t, auto whole) {
        constexpr bool W = whole;
        ru.template load<W>(far_u, t, at.to - t);
        rdelta.template load<W>(far_delta, t, at.to - t);
        rB.template load<W>(far_B, t, at.to - t);
        if constexpr (!ENDS)
            rC.template load<W>(far_C, t, at.to - t);
        if constexpr (GATED)
            rz.template load<W>(far_z, t, at.to - t);
    };
    // what arrived, into LDS
    const auto stage = [&](int t, int half, auto whole) {
        float dt[Q], x[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            dt[q] = step_of(far_delta[q], bias, a.softplus);
            x[q] = dt[q] * (float)far_u[q];
        }
        if (!whole && at.to - t < STEPS) // steps past the end leave the state as it is
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (!ru.inside(q, at.to - t))
                    dt[q] = x[q] = 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            s_step[half][wave][4 * q + row][j] = make_float2(dt[q], x[q]);
            next_u[q] = far_u[q];
            if constexpr (GATED)
                next_z[q] = far_z[q];
            if constexpr (ENDS)
                total += dt[q];
        }
#pragma unroll
        for (int k = 0; k < REGS; ++k) {
            next_B[k] = no_state ? 0.f : (float)far_B[k];
            ((float *)&s_mixed[half][wave][k * PER + j / R][0])[R * row + j % R] = ENDS ? next_B[k] : no_state ? 0.f : (float)far_C[k];
        }
    };
    float *start = nullptr;
    if (!ENDS && a.starts)
        start = a.starts + ((at.z * ((a.len + BLOCK - 1) / BLOCK) + at.from / BLOCK) * a.dim + at.c) * a.states;
    int half = 0;
    if (at.from < at.to) {
        fetch(at.from, std::false_type());
        stage(at.from, 0, std::false_type());
        if (at.from + STEPS < at.to)
            fetch(at.from + STEPS, std::false_type());
    }
    // One block; `whole`: it and the two after it are, so that nothing parts its instructions
    // (4 x 2048 x 4096 bf16, one wave a SIMD: 245 -> 180 us).
    const auto walk = [&](int t, auto whole) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            u[q] = next_u[q];
            if constexpr (GATED)
                z[q] = next_z[q];
        }
#pragma unroll
        for (int k = 0; k < REGS; ++k)
            B[k] = next_B[k];
        if constexpr (!ENDS)
            if (a.starts && t % BLOCK == 0) {
                if (at.real)
                    store_states<R>(start, at.n0, a.states, h);
                start += a.dim * a.states;
            }
        wave_sync();
        // the steps' operands are read a group ahead of their use
        constexpr int AHEAD = R > 8 ? 2 : 4;
        struct {
            float2 v[AHEAD];
            vec<float, 4> c[AHEAD][R / 4];
        } now, next;
        const auto read = [&](int step) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                next.v[k] = s_step[half][wave][step + k][j];
#pragma unroll
                for (int i = 0; i < R / 4; ++i)
                    next.c[k][i] = s_mixed[half][wave][step + k][row * (R / 4) + i];
            }
        };
        read(0);
        if (whole || at.to - t > STEPS) {
            stage(t + STEPS, half ^ 1, whole);
            if (whole || at.to - t > 2 * STEPS)
                fetch(t + 2 * STEPS, whole);
        }
        float y[Q][4];
        each<STEPS / AHEAD>([&](auto gg) {
            constexpr int g = gg;
            now = next;
            if constexpr ((g + 1) * AHEAD < STEPS)
                read((g + 1) * AHEAD);
            __builtin_amdgcn_sched_barrier(0); // (the reads stay ahead of a group's work)
            each<AHEAD>([&](auto kk) {
                constexpr int k = kk, step = g * AHEAD + k;
                const float2 v = now.v[k];
                float sum = 0.f;
                each<R>([&](auto ii) {
                    constexpr int i = ii;
                    const float e = __builtin_amdgcn_exp2f(v.x * A2[i]);
                    if constexpr (ENDS)
                        h[i] = fmaf(e, h[i], v.y * now.c[k][i / 4][i % 4]);
                    else
                        h[i] = fmaf(e, h[i], v.y * of_row<step % PER * R + i>(B[step / PER]));
                    if constexpr (!ENDS)
                        sum = i ? fmaf(now.c[k][i / 4][i % 4], h[i], sum) : now.c[k][0][0] * h[0];
                });
                y[step / 4][step % 4] = sum;
            });
        });
        if constexpr (!ENDS) {
            T out[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                float s = fmaf(D, (float)u[q], over_rows(y[q]));
                if constexpr (GATED) {
                    const float gate = (float)z[q];
                    s *= gate * sigmoid_of<FULL>(gate);
                }
                out[q] = (T)s;
            }
            if (at.real) {
                if (whole || at.to - t >= STEPS) {
#pragma unroll
                    for (int q = 0; q < Q; ++q)
                        ry.store(t, q, out[q]);
                } else {
#pragma unroll
                    for (int q = 0; q < Q; ++q)
                        if (ry.inside(q, at.to - t))
                            ry.store(t, q, out[q]);
                }
            }
        }
        half ^= 1;
    };
    int t = at.from;
    if constexpr (ENDS)
        for (; at.to - t >= 3 * STEPS; t += STEPS)
            walk(t, std::true_type());
    else
        for (; at.to - t >= 4 * STEPS; t += 2 * STEPS) { // (two, so that what is kept for the next need not move)
            walk(t, std::true_type());
            walk(t + STEPS, std::true_type());
        }
    for (; t < at.to; t += STEPS)
        walk(t, std::false_type());
    if constexpr (ENDS) {
        total = over_rows(total);
        if (at.real) {
            const int64_t m = maps.at(at.seg, at.z, at.c);
            store_states<R>(maps.Q + m * a.states, at.n0, a.states, h);
            if (row == 0)
                maps.sum[m] = total;
        }
    } else if (at.seg == p.segments - 1 && at.real) {
        store_states<R>(a.hlast + (at.z * a.dim + at.c) * a.states, at.n0, a.states, h);
    }
}

// ---------------------------------------------------------------- one step ----
//
// A token's work is its states, read and written once: four of a channel a lane, S lanes
// a channel, so that a wave's states are contiguous.
template <typename T, int S>
__global__ void __launch_bounds__(256) k_scan_step(ScanArgs a)
{
    constexpr bool FULL = sizeof(T) == 4;
    const unsigned one = (blockIdx.x * 256 + threadIdx.x) / S, dim = (unsigned)a.dim; // (the states are fewer than 2^31)
    if (one >= (unsigned)a.batch * dim)
        return;
    const int64_t at = one, z = one / dim;
    const int c = (int)(one % dim), g = a.groups == 1 ? 0 : c / (int)(dim / (unsigned)a.groups), n0 = (threadIdx.x % S) * 4;
    const int64_t left = a.states - n0;
    const vec<float, 4> A = load_some<float, 4>(a.A + (int64_t)c * a.states + n0, left);
    vec<float, 4> h = {0.f, 0.f, 0.f, 0.f};
    if (a.h0)
        h = load_some<float, 4>(a.h0 + at * a.states + n0, left);
    const vec<T, 4> B = load_some<T, 4>((const T *)a.B.p + z * a.B.stride + (int64_t)g * a.states + n0, left);
    const vec<T, 4> C = load_some<T, 4>((const T *)a.C.p + z * a.C.stride + (int64_t)g * a.states + n0, left);
    const float dt = step_of(((const T *)a.delta.p)[z * a.delta.stride + c], a.bias ? a.bias[c] : 0.f, a.softplus);
    const float u = (float)((const T *)a.u.p)[z * a.u.stride + c], x = dt * u;
    const float gate = a.z.p ? (float)((const T *)a.z.p)[z * a.z.stride + c] : 0.f;
    if (a.starts)
        store_some<float, 4>(a.starts + at * a.states + n0, left, h);
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(__builtin_amdgcn_exp2f(dt * (A[i] * LOG2E)), h[i], x * (float)B[i]);
        y = fmaf((float)C[i], h[i], y);
    }
    store_some<float, 4>(a.hlast + at * a.states + n0, left, h);
#pragma unroll
    for (int o = 1; o < S; o *= 2)
        y += __shfl_xor(y, o);
    if (n0 == 0) {
        y = fmaf(a.D ? a.D[c] : 0.f, u, y);
        if (a.z.p)
            y *= gate * sigmoid_of<FULL>(gate);
        ((T *)a.y.p)[z * a.y.stride + c] = (T)y;
    }
}

// ----------------------------------------------------------------- adjoint ----

constexpr int BWD_WAVES = 4;

// ENDS: walks a segment back from mu = 0 and writes its map.
template <typename T, int R>
__global__ void __launch_bounds__(FWD_WAVES *WAVE) k_scan_adjoint_ends(ScanArgs a, Plan p, float *ws)
{
    constexpr bool FULL = sizeof(T) == 4;
    constexpr int Q = STEPS / 4, PER = ROW / R, REGS = R;
    __shared__ float2 s_step[2][FWD_WAVES][STEPS][ROW];
    __shared__ vec<float, 4> s_C[2][FWD_WAVES][STEPS][R];
    Place<R> at;
    if (!at.set(a, p, FWD_WAVES))
        return;
    const int wave = threadIdx.x / WAVE, row = at.row, j = at.j;
    float A2[R], mu[R];
    load_states<R>(a.A + (int64_t)at.c * a.states, at.n0, a.states, A2);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        A2[i] *= LOG2E;
        mu[i] = 0.f;
    }
    const float bias = a.bias ? a.bias[at.c] : 0.f;
    // (the gradient of the end in the place of the first segment's map: adj_h0 may replace it)
    if (at.seg == 0) {
        if (a.adj_hlast)
            load_states<R>(a.adj_hlast + (at.z * a.dim + at.c) * a.states, at.n0, a.states, mu);
        if (at.real)
            store_states<R>(Maps(a, ws, p.segments).Q + Maps(a, ws, p.segments).at(0, at.z, at.c) * a.states, at.n0,
                            a.states, mu);
        return;
    }
    float total = 0.f;
    const bool gated = a.z.p, no_state = at.n0 + j % R >= a.states;
    const auto rdelta = at.template column<T, STEPS>(a.delta), radj = at.template column<T, STEPS>(a.adj);
    const auto rz = at.template column<T, STEPS>(gated ? a.z : a.adj);
    const auto rC = at.template mixed<T, STEPS>(a.C, a.states);
    T far_delta[Q], far_z[Q], far_adj[Q], far_C[REGS];
    const auto fetch = [&](int t, auto whole) {
        constexpr bool W = whole;
        rdelta.template load<W>(far_delta, t, at.to - t);
        radj.template load<W>(far_adj, t, at.to - t);
        rz.template load<W>(far_z, t, at.to - t);
        rC.template load<W>(far_C, t, at.to - t);
    };
    // what arrived, into LDS; steps past the end leave mu as it is
    const auto stage = [&](int t, int half) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const bool counts = rdelta.inside(q, at.to - t);
            const float gate = (float)far_z[q], sg = sigmoid_of<FULL>(gate);
            const float dy = (float)far_adj[q] * (gated ? gate * sg : 1.f);
            const float dt = counts ? step_of(far_delta[q], bias, a.softplus) : 0.f;
            s_step[half][wave][4 * q + row][j] = make_float2(dt, counts ? dy : 0.f);
            total += dt;
        }
#pragma unroll
        for (int k = 0; k < REGS; ++k)
            ((float *)&s_C[half][wave][k * PER + j / R][0])[R * row + j % R] = no_state ? 0.f : (float)far_C[k];
    };
    int half = 0;
    const int last = at.from + (at.to - 1 - at.from) / STEPS * STEPS;
    fetch(last, std::false_type());
    stage(last, 0);
    if (last > at.from)
        fetch(last - STEPS, std::true_type());
    for (int t = last; t >= at.from; t -= STEPS, half ^= 1) {
        wave_sync();
        // the steps' operands are read a group ahead of their use
        constexpr int AHEAD = R > 8 ? 2 : R > 4 ? 4 : 8;
        struct {
            float2 v[AHEAD];
            vec<float, 4> c[AHEAD][R / 4];
        } now, next;
        const auto read = [&](int step) { // and those before it
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                next.v[k] = s_step[half][wave][step - k][j];
#pragma unroll
                for (int i = 0; i < R / 4; ++i)
                    next.c[k][i] = s_C[half][wave][step - k][row * (R / 4) + i];
            }
        };
        read(STEPS - 1);
        if (t > at.from) {
            stage(t - STEPS, half ^ 1);
            if (t - STEPS > at.from)
                fetch(t - 2 * STEPS, std::true_type());
        }
        each<STEPS / AHEAD>([&](auto gg) {
            constexpr int g = gg;
            now = next;
            if constexpr ((g + 1) * AHEAD < STEPS)
                read(STEPS - 1 - (g + 1) * AHEAD);
            __builtin_amdgcn_sched_barrier(0); // (the reads stay ahead of a group's work)
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
#pragma unroll
                for (int i = 0; i < R; ++i)
                    mu[i] = __builtin_amdgcn_exp2f(now.v[k].x * A2[i]) * fmaf(now.c[k][i / 4][i % 4], now.v[k].y, mu[i]);
        });
    }
    total = over_rows(total);
    if (at.real) {
        const Maps maps(a, ws, p.segments);
        const int64_t m = maps.at(at.seg, at.z, at.c);
        store_states<R>(maps.Q + m * a.states, at.n0, a.states, mu);
        if (row == 0)
            maps.sum[m] = total;
    }
}

template <typename T, int R, bool GATED>
__global__ void __launch_bounds__(BWD_WAVES *WAVE, R < 16 ? 2 : 1)
    k_scan_adjoint(ScanArgs a, Plan p, float *ws, float *sums, float *own)
{
    constexpr bool FULL = sizeof(T) == 4;
    constexpr int TS = part_steps<R>, Q = TS / 4, PER = ROW / R, REGS = TS / PER, BLOCK = block_steps<R>, PARTS = BLOCK / TS;
    __shared__ vec<float, 4> s_step[BWD_WAVES][TS][ROW];
    __shared__ vec<float, 4> s_B[BWD_WAVES][TS][R], s_C[BWD_WAVES][TS][R];
    __shared__ float s_sum[2][BWD_WAVES][2][REGS][WAVE];
    __shared__ vec<float, 4> s_state[BWD_WAVES][PARTS - 2][R / 4][WAVE]; // (but for the first and the last)
    __shared__ float2 s_up[BWD_WAVES][PARTS - 1][TS][ROW]; // (dt, dt u) of the way up, for the way down
    Place<R> at;
    const bool some = at.set(a, p, BWD_WAVES);
    const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE, row = at.row, j = at.j;
    float A[R], A2[R], mu[R], dA[R];
    load_states<R>(a.A + (int64_t)at.c * a.states, at.n0, a.states, A);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        A2[i] = A[i] * LOG2E;
        mu[i] = dA[i] = 0.f;
    }
    const float bias = a.bias ? a.bias[at.c] : 0.f, D = a.D ? a.D[at.c] : 0.f;
    if (p.segments == 1) {
        if (a.adj_hlast)
            load_states<R>(a.adj_hlast + (at.z * a.dim + at.c) * a.states, at.n0, a.states, mu);
    } else {
        const Maps maps(a, ws, p.segments);
        load_states<R>(maps.Q + maps.at(0, at.z, at.c) * a.states, at.n0, a.states, mu);
        maps.template apply<R>(mu, p.segments - 1, p.segments - 1 - at.seg, -1, at.z, at.c, at.n0, A2);
    }
    // lanes without a channel add nothing to the sums over the channels
    if (!at.real)
#pragma unroll
        for (int i = 0; i < R; ++i)
            mu[i] = 0.f;
    const bool no_state = at.n0 + j % R >= a.states;
    const auto ru = at.template column<T, TS, false>(a.u), rdelta = at.template column<T, TS, false>(a.delta);
    const auto radj = at.template column<T, TS, false>(a.adj), rz = at.template column<T, TS, false>(a.z);
    const auto rB = at.template mixed<T, TS, false>(a.B, a.states), rC = at.template mixed<T, TS, false>(a.C, a.states);
    const auto wu = at.template column<T, TS, false>(a.adj_u), wdelta = at.template column<T, TS, false>(a.adj_delta);
    const auto wz = at.template column<T, TS, false>(a.adj_z);
    // the workgroup's sums over its channels: [batch, groups * per_group, len, 2, 4 R]
    sums += (at.z * p.across + blockIdx.x % (unsigned)p.across) * a.len * (8 * R);
    float dD = 0.f, dbias = 0.f;
    int turn = 0;
    // The waves' sums of a part.  (The other half is written while this one is read: a wave
    // reaches the next barrier only after it has read.)
    const auto add_up = [&](int t) {
#pragma unroll
        for (int i = threadIdx.x; i < 2 * REGS * WAVE; i += BWD_WAVES * WAVE) {
            const int which = i / (REGS * WAVE), reg = i / WAVE % REGS, l = i % WAVE;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < BWD_WAVES; ++w)
                s += s_sum[turn][w][which][reg][l];
            const int step = t + reg * PER + l % ROW / R;
            if (step < at.to)
                sums[(int64_t)step * (8 * R) + which * 4 * R + R * (l / ROW) + l % R] = s;
        }
        turn ^= 1;
    };
    // a part's inputs are on their way while the one before it is walked
    T far_u[Q], far_delta[Q], far_z[Q], far_adj[Q], far_B[REGS], far_C[REGS];
    float far_start[R];
    const auto fetch_start = [&](int t) {
        load_states<R>(a.starts + ((at.z * ((a.len + BLOCK - 1) / BLOCK) + t / BLOCK) * a.dim + at.c) * a.states, at.n0,
                       a.states, far_start);
    };
    const auto fetch_up = [&](int t) { // (a part that another follows is whole)
        ru.template load<true>(far_u, t, TS);
        rdelta.template load<true>(far_delta, t, TS);
        rB.template load<true>(far_B, t, TS);
    };
    const auto fetch_down = [&](int t) {
        const int left = at.to - t;
        ru.load(far_u, t, left);
        rdelta.load(far_delta, t, left);
        radj.load(far_adj, t, left);
        if constexpr (GATED)
            rz.load(far_z, t, left);
        rB.load(far_B, t, left);
        rC.load(far_C, t, left);
    };
    const int last = at.from + (at.to - 1 - at.from) / BLOCK * BLOCK;
    if (!some) { // a wave without channels adds zeros, and its share of the sums over the waves
#pragma unroll
        for (int k = 0; k < 2 * 2 * REGS; ++k)
            s_sum[k / (2 * REGS)][wave][k / REGS % 2][k % REGS][lane] = 0.f;
    } else {
        fetch_start(last);
        at.to - last > TS ? fetch_up(last) : fetch_down(last);
    }
    for (int b0 = last; b0 >= at.from; b0 -= BLOCK) {
        float start[R];
#pragma unroll
        for (int i = 0; i < R; ++i)
            start[i] = at.real ? far_start[i] : 0.f;
        const int parts = (min(at.to - b0, BLOCK) + TS - 1) / TS;
        if (!some) {
            for (int part = parts - 1; part >= 0; --part) {
                __syncthreads();
                add_up(b0 + part * TS);
            }
            continue;
        }
        // the states that the parts start from
        float h0[R];
#pragma unroll
        for (int i = 0; i < R; ++i)
            h0[i] = start[i];
        for (int part = 0; part + 1 < parts; ++part) {
            float B[REGS], dt[Q], x[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                dt[q] = at.real ? step_of(far_delta[q], bias, a.softplus) : 0.f;
                x[q] = at.real ? dt[q] * (float)far_u[q] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < REGS; ++k)
                B[k] = no_state ? 0.f : (float)far_B[k];
            if (part + 2 < parts)
                fetch_up(b0 + (part + 1) * TS);
            else
                fetch_down(b0 + (part + 1) * TS);
#pragma unroll
            for (int q = 0; q < Q; ++q)
                s_up[wave][part][4 * q + row][j] = make_float2(dt[q], x[q]);
            wave_sync();
            float2 v[TS];
#pragma unroll
            for (int k = 0; k < TS; ++k)
                v[k] = s_up[wave][part][k][j];
            each<TS>([&](auto tt) {
                constexpr int step = tt;
                each<R>([&](auto ii) {
                    constexpr int i = ii;
                    h0[i] = fmaf(__builtin_amdgcn_exp2f(v[step].x * A2[i]), h0[i],
                                 v[step].y * of_row<step % PER * R + i>(B[step / PER]));
                });
            });
            if (part + 2 < parts)
#pragma unroll
                for (int k = 0; k < R / 4; ++k) {
                    const vec<float, 4> w = {h0[4 * k], h0[4 * k + 1], h0[4 * k + 2], h0[4 * k + 3]};
                    s_state[wave][part][k][lane] = w;
                }
        }
        // (the last part starts where that walk ended: h0)
        for (int part = parts - 1; part >= 0; --part) {
            const int t = b0 + part * TS, left = at.to - t;
            float dt[Q], dy[Q], u[Q], raw[Q], slope[Q], B[REGS], C[REGS];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const bool counts = ru.inside(q, left) && at.real;
                u[q] = counts ? (float)far_u[q] : 0.f;
                raw[q] = (float)far_delta[q] + bias;
                if (part + 1 < parts)
                    dt[q] = s_up[wave][part][4 * q + row][j].x;
                else
                    dt[q] = counts ? step_of(far_delta[q], bias, a.softplus) : 0.f;
                dy[q] = counts ? (float)far_adj[q] : 0.f;
                slope[q] = 0.f;
                if constexpr (GATED) {
                    const float gate = counts ? (float)far_z[q] : 0.f, sg = sigmoid_of<FULL>(gate);
                    slope[q] = dy[q] * (sg * fmaf(gate, 1.f - sg, 1.f));
                    dy[q] *= gate * sg;
                }
            }
#pragma unroll
            for (int k = 0; k < REGS; ++k) {
                B[k] = no_state ? 0.f : (float)far_B[k];
                C[k] = no_state ? 0.f : (float)far_C[k];
            }
            if (part > 0) {
                fetch_down(t - TS);
            } else if (b0 > at.from) {
                fetch_start(b0 - BLOCK);
                fetch_up(b0 - BLOCK);
            }
            float first[R];
#pragma unroll
            for (int i = 0; i < R; ++i)
                first[i] = part == 0 ? start[i] : h0[i];
            if (part > 0 && part < parts - 1)
#pragma unroll
                for (int i = 0; i < R; ++i)
                    first[i] = s_state[wave][part - 1][i / 4][lane][i % 4];
            wave_sync();
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const vec<float, 4> v = {dt[q], dt[q] * u[q], dy[q], 0.f};
                s_step[wave][4 * q + row][j] = v;
            }
#pragma unroll
            for (int k = 0; k < REGS; ++k) {
                ((float *)&s_B[wave][k * PER + j / R][0])[R * row + j % R] = B[k];
                ((float *)&s_C[wave][k * PER + j / R][0])[R * row + j % R] = C[k];
            }
            wave_sync();
            // up, keeping the states and (but for many) their exponentials
            constexpr bool KEEP = R < 16;
            float h[TS][R], e[KEEP ? TS : 1][R];
            {
                float2 v[TS];
#pragma unroll
                for (int k = 0; k < TS; ++k)
                    v[k] = *(const float2 *)&s_step[wave][k][j];
                each<TS>([&](auto tt) {
                    constexpr int step = tt;
                    each<R>([&](auto ii) {
                        constexpr int i = ii;
                        const float x = __builtin_amdgcn_exp2f(v[step].x * A2[i]);
                        if constexpr (KEEP)
                            e[step][i] = x;
                        h[step][i] = fmaf(x, step ? h[step ? step - 1 : 0][i] : first[i],
                                          v[step].y * of_row<step % PER * R + i>(B[step / PER]));
                    });
                });
            }
            if constexpr (!KEEP)
#pragma unroll
                for (int i = 0; i < R; ++i)
                    asm volatile("" : "+v"(A2[i])); // (so that the compiler does not keep them either)
            // and down; a step's operands are on their way while the one after it is walked
            float(*const out)[REGS][WAVE] = s_sum[turn][wave];
            struct {
                vec<float, 4> v, b[R / 4], c[R / 4];
            } now, next;
            const auto read = [&](int step) {
                next.v = s_step[wave][step][j];
#pragma unroll
                for (int k = 0; k < R / 4; ++k) {
                    next.b[k] = s_B[wave][step][row * (R / 4) + k];
                    next.c[k] = s_C[wave][step][row * (R / 4) + k];
                }
            };
            read(TS - 1);
            T out_u[Q], out_delta[Q], out_z[Q];
            each<Q>([&](auto qq) {
                constexpr int q = Q - 1 - qq;
                float y[4] = {}, s1[4] = {}, s2[4] = {};
                each<R / 4>([&](auto rr) { // registers of 16 sums: PER steps
                    constexpr int reg = R / 4 - 1 - rr;
                    float pB[16], pC[16];
                    each<PER>([&](auto kk) {
                        constexpr int at_k = PER - 1 - kk, k = reg * PER + at_k, step = 4 * q + k;
                        now = next;
                        if constexpr (step > 0)
                            read(step - 1);
                        __builtin_amdgcn_sched_barrier(0);
                        const vec<float, 4> v = now.v;
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            const float bb = now.b[i / 4][i % 4], cc = now.c[i / 4][i % 4];
                            const float g = fmaf(cc, v[2], mu[i]);
                            if constexpr (GATED)
                                y[k] = fmaf(cc, h[step][i], y[k]);
                            pC[at_k * R + i] = v[2] * h[step][i];
                            pB[at_k * R + i] = g * v[1];
                            s1[k] = fmaf(g, bb, s1[k]);
                            mu[i] = g * (KEEP ? e[KEEP ? step : 0][i] : __builtin_amdgcn_exp2f(v[0] * A2[i]));
                            const float w = mu[i] * (step ? h[step ? step - 1 : 0][i] : first[i]);
                            s2[k] = fmaf(A[i], w, s2[k]);
                            dA[i] = fmaf(v[0], w, dA[i]);
                        }
                    });
                    out[0][q * (R / 4) + reg][lane] = over_lanes(pB, j);
                    out[1][q * (R / 4) + reg][lane] = over_lanes(pC, j);
                });
                const float along = over_rows(s1), back = over_rows(s2);
                float ddelta = fmaf(u[q], along, back);
                const float sg = sigmoid_of<true>(raw[q]);
                ddelta *= a.softplus ? sg : 1.f;
                dD = fmaf(dy[q], u[q], dD);
                out_u[q] = (T)fmaf(dt[q], along, D * dy[q]);
                out_delta[q] = (T)ddelta;
                if constexpr (GATED)
                    out_z[q] = (T)(slope[q] * fmaf(D, u[q], over_rows(y)));
                dbias += ru.inside(q, left) ? ddelta : 0.f;
            });
            if (at.real) {
#pragma unroll
                for (int q = 0; q < Q; ++q)
                    if (ru.inside(q, left)) {
                        wu.store(t, q, out_u[q]);
                        wdelta.store(t, q, out_delta[q]);
                        if constexpr (GATED)
                            wz.store(t, q, out_z[q]);
                    }
            }
            __syncthreads();
            add_up(t);
        }
    }
    dD = over_rows(dD), dbias = over_rows(dbias);
    if (!some || !at.real)
        return;
    if (at.seg == 0 && a.adj_h0)
        store_states<R>(a.adj_h0 + (at.z * a.dim + at.c) * a.states, at.n0, a.states, mu);
    float *o = own + ((at.z * p.segments + at.seg) * a.dim + at.c) * (a.states + 2);
    store_states<R>(o, at.n0, a.states, dA);
    if (row == 0)
        o[a.states] = dD, o[a.states + 1] = dbias;
}

// The first `mixed` workgroups: adj_B and adj_C, over a group's workgroups, a thread a
// (step, group, state) of one.  The others: adj_A, adj_D and adj_bias, over batch and
// segments, a column a lane, sixteen waves' sums of every sixteenth row joined.
constexpr int SUM_THREADS = 1024, SUM_WAVES = SUM_THREADS / WAVE;

template <typename T>
__global__ void __launch_bounds__(SUM_THREADS) k_scan_sums(ScanArgs a, Plan p, const float *sums, int wide, unsigned mixed,
                                                           const float *own)
{
    __shared__ float s_sum[SUM_WAVES][WAVE];
    float s = 0.f;
    if (blockIdx.x < mixed) {
        const int64_t i = (int64_t)blockIdx.x * SUM_THREADS + threadIdx.x, count = a.batch * a.len * a.groups * 2 * a.states;
        if (i >= count)
            return;
        const int n = (int)(i % a.states), which = (int)(i / a.states % 2);
        const int64_t rest = i / a.states / 2, t = rest % a.len;
        const int g = (int)(rest / a.len % a.groups);
        const int64_t z = rest / a.len / a.groups;
        const float *x = sums + ((z * p.across + (int64_t)g * p.per_group) * a.len + t) * (2 * wide) + which * wide + n;
        const int64_t step = a.len * 2 * wide;
#pragma unroll 8 // (loads together: 4 x 2048 x 4096 30 -> 12 us)
        for (int k = 0; k < p.per_group; ++k)
            s += x[k * step];
        const SeqRows &r = which ? a.adj_C : a.adj_B;
        ((T *)r.p)[z * r.stride + t * r.ld + (int64_t)g * a.states + n] = (T)s;
        return;
    }
    const int lane = threadIdx.x % WAVE, slot = threadIdx.x / WAVE;
    const int64_t i = (int64_t)(blockIdx.x - mixed) * WAVE + lane, cols = a.dim * (a.states + 2), rows = a.batch * p.segments;
    if (i < cols)
        for (int64_t r = slot; r < rows; r += SUM_WAVES)
            s += own[r * cols + i];
    s_sum[slot][lane] = s;
    __syncthreads();
    if (slot > 0 || i >= cols)
        return;
#pragma unroll
    for (int k = 1; k < SUM_WAVES; ++k)
        s += s_sum[k][lane];
    const int64_t c = i / (a.states + 2);
    const int n = (int)(i % (a.states + 2));
    float *out = n < a.states    ? a.adj_A + c * a.states + n
                 : n == a.states ? (a.adj_D ? a.adj_D + c : nullptr)
                                 : (a.adj_bias ? a.adj_bias + c : nullptr);
    if (out)
        *out = a.accumulate ? *out + s : s;
}

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
    const int waves = adjoint ? BWD_WAVES : FWD_WAVES, block = scan_block(a.states);
    const int64_t per = a.dim / a.groups, wave_count = (per + ROW - 1) / ROW;
    p.per_group = (int)((wave_count + waves - 1) / waves);
    p.across = (int64_t)p.per_group * a.groups;
    // A first walk costs a step of the forward about as much again, and less of the adjoint,
    // which also needs two waves a SIMD more: 4 x 2048 x 4096 bf16 (1024 waves, one a
    // SIMD) forward 178 us whole, 219 in 4 segments, adjoint 900 and 721; 2 x 2048 x 4096 forward
    // 160 in 2 segments, 126 in 8, adjoint 576 and 368.  Beyond 32 states a SIMD holds one wave
    // of the adjoint, and segments only fill it (4 x 2048 x 4096 of 64 states 2790 us whole,
    // 3100 in 4).  More than 64 segments cost more to put together than they save (16384 x 256
    // forward 68 us, with 256 116).
    const int64_t all = a.batch * a.groups * wave_count, blocks = std::max<int64_t>(1, (a.len + block - 1) / block);
    const bool two = !adjoint || a.states <= 32;
    const int64_t want = all >= (adjoint && two ? 1536 : 768) ? 1 : std::min<int64_t>({blocks, 64, (two ? 4096 : 1024) / all});
    const int64_t each = (blocks + want - 1) / want;
    p.segment = (int)std::min<int64_t>(each * block, INT32_MAX);
    p.segments = (int)((blocks + each - 1) / each);
    return p;
}
// where the adjoint's waves along the channels are put together in other workgroups
Plan ends_plan(const ScanArgs &a, Plan p)
{
    const Plan f = plan_of(a, false);
    p.per_group = f.per_group, p.across = f.across;
    return p;
}

int64_t maps_size(const ScanArgs &a, const Plan &p)
{
    return p.segments > 1 ? p.segments * a.batch * a.dim * (int64_t)(a.states + 1) : 0;
}
int64_t sums_size(const ScanArgs &a, const Plan &p) { return a.batch * p.across * a.len * 8 * rows_of(a.states); }
int64_t own_size(const ScanArgs &a, const Plan &p) { return a.batch * p.segments * a.dim * (int64_t)(a.states + 2); }

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

int step_lanes(int states)
{
    int s = 1;
    while (4 * s < states)
        s *= 2;
    return s;
}

bool grid_ok(double threads) { return threads <= 4294967295.0; }

} // namespace

int scan_block(int states) { return 256 / rows_of(states); }

int64_t scan_workspace(const ScanArgs &a)
{
    const Plan p = plan_of(a, false);
    if (!grid_ok((double)a.batch * p.across * p.segments * FWD_WAVES * WAVE) ||
        !grid_ok((double)a.batch * a.dim * std::max(step_lanes(a.states), a.states) + 256))
        return -1;
    return a.len > 1 ? maps_size(a, p) * (int64_t)sizeof(float) : 0;
}

int64_t scan_adjoint_workspace(const ScanArgs &a)
{
    const Plan p = plan_of(a, true);
    if (!grid_ok((double)a.batch * p.across * p.segments * BWD_WAVES * WAVE) ||
        !grid_ok((double)a.batch * a.len * a.groups * 2 * a.states + (double)a.dim * (a.states + 2) * SUM_WAVES + 4096) ||
        !grid_ok((double)a.batch * a.dim * a.states + 256))
        return -1;
    return a.len > 0 ? (maps_size(a, p) + sums_size(a, p) + own_size(a, p)) * (int64_t)sizeof(float) : 0;
}

chol_status scan(chol_dtype dt, const ScanArgs &a, void *ws, hipStream_t st)
{
    if (a.len == 0)
        return copy(a.h0, a.hlast, a.batch * a.dim * a.states, st);
    return with_lowp(dt, [&](auto *e) {
        typedef std::remove_pointer_t<decltype(e)> T;
        if (a.len == 1) {
            const int s = step_lanes(a.states);
            const dim3 grid((unsigned)ceil_of(a.batch * a.dim * s, 256));
            const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, a); };
            s == 1   ? launch(k_scan_step<T, 1>)
            : s == 2 ? launch(k_scan_step<T, 2>)
            : s == 4 ? launch(k_scan_step<T, 4>)
            : s == 8 ? launch(k_scan_step<T, 8>)
                     : launch(k_scan_step<T, 16>);
            CHOL_LAUNCH_CHECK();
            return CHOL_OK;
        }
        return with_rows(a.states, [&](auto r) {
            constexpr int R = r;
            const Plan p = plan_of(a, false);
            const dim3 grid((unsigned)(a.batch * p.across * p.segments));
            const auto launch = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, grid, dim3(FWD_WAVES * WAVE), 0, st, a, p, (float *)ws);
            };
            if (p.segments > 1) {
                launch(k_scan<T, R, true, false>);
                CHOL_LAUNCH_CHECK();
            }
            a.z.p ? launch(k_scan<T, R, false, true>) : launch(k_scan<T, R, false, false>);
            CHOL_LAUNCH_CHECK();
            return CHOL_OK;
        });
    });
}

chol_status scan_adjoint(chol_dtype dt, const ScanArgs &a, void *ws, hipStream_t st)
{
    if (a.len == 0 || a.batch == 0) {
        const chol_status s = copy(a.adj_hlast, a.adj_h0, a.batch * a.dim * a.states, st);
        if (s != CHOL_OK || a.accumulate)
            return s;
        for (const auto &[to, n] : {std::pair{a.adj_A, a.dim * a.states}, std::pair{a.adj_D, a.dim}, std::pair{a.adj_bias, a.dim}}) {
            const chol_status c = copy(nullptr, to, n, st);
            if (c != CHOL_OK)
                return c;
        }
        return CHOL_OK;
    }
    return with_lowp(dt, [&](auto *e) {
        typedef std::remove_pointer_t<decltype(e)> T;
        return with_rows(a.states, [&](auto r) {
            constexpr int R = r;
            const Plan p = plan_of(a, true);
            float *maps = (float *)ws, *sums = maps + maps_size(a, p), *own = sums + sums_size(a, p);
            if (p.segments > 1) {
                const Plan f = ends_plan(a, p);
                hipLaunchKernelGGL((k_scan_adjoint_ends<T, R>), dim3((unsigned)(a.batch * f.across * f.segments)),
                                   dim3(FWD_WAVES * WAVE), 0, st, a, f, maps);
                CHOL_LAUNCH_CHECK();
            }
            const auto launch = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, dim3((unsigned)(a.batch * p.across * p.segments)), dim3(BWD_WAVES * WAVE), 0, st,
                                   a, p, maps, sums, own);
            };
            a.z.p ? launch(k_scan_adjoint<T, R, true>) : launch(k_scan_adjoint<T, R, false>);
            CHOL_LAUNCH_CHECK();
            const unsigned mixed = (unsigned)ceil_of(a.batch * a.len * a.groups * 2 * a.states, SUM_THREADS);
            const unsigned rest = (unsigned)ceil_of(a.dim * (a.states + 2), WAVE);
            hipLaunchKernelGGL((k_scan_sums<T>), dim3(mixed + rest), dim3(SUM_THREADS), 0, st, a, p, (const float *)sums, 4 * R,
                               mixed, (const float *)own);
            CHOL_LAUNCH_CHECK();
            return CHOL_OK;
        });
    });
}

} // namespace chol
