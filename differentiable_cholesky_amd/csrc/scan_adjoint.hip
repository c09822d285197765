// The adjoint of the selective state space scan.  With a_t the gradient of the sum that
// the gate multiplies, from the last step,
//
//   g_t = C_t a_t + mu_{t+1},  mu_t = exp(dt_t A) g_t
//   adj_C = sum_c a h,  adj_B = sum_c g dt u          (over the channels of the group)
//   s_t = sum_n g B,  adj_u = dt s + D a,  adj_dt = u s + sum_n A mu h_{t-1}
//   adj_A = sum dt mu h_{t-1},  adj_D = sum a u,  adj_h0 = mu_0
//
// It starts from states that the forward saved every `block_steps` steps, walks up a block
// to the states of its parts, and then each part, the last one first, up and down: up in
// registers (R * part_steps states of a lane and their exponentials), down with the sums.
// Sums over the channels take the lanes of a row, the waves of the workgroup, and by a last
// launch the workgroups.
//
// Vector instructions bound it (900 a wave and 8 steps of 16 states, of which 160 walk up
// to the parts, 500 walk down, half of that the sums over lanes and rows), with two waves a
// SIMD, which 225 registers a lane and 74 KB of LDS a workgroup leave room for.  4 x 2048 x 4096
// bf16 of 16 states 630 us: first walks 95, walks 520, sums 12; 8 x 2048 x 4096 1090 us.
#include "scan_lanes.hpp"

namespace chol {

namespace {

// ENDS: walks a segment back from mu = 0 and writes its map.
template <typename T, int R>
__global__ void __launch_bounds__(WAVES *WAVE) k_scan_adjoint_ends(ScanArgs a, Plan p, float *ws)
{
    constexpr bool FULL = sizeof(T) == 4;
    constexpr int Q = STEPS / 4, PER = ROW / R, REGS = R;
    __shared__ float2 s_step[2][WAVES][STEPS][ROW];
    __shared__ vec<float, 4> s_C[2][WAVES][STEPS][R];
    Place<R> at;
    if (!at.set(a, p, p.waves))
        return;
    const int wave = threadIdx.x / WAVE, row = at.row, j = at.j;
    float A2[R], mu[R];
    load_states<R>(a.A + (int64_t)at.c * a.states, at.n0, a.states, A2);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        A2[i] = base2_rate(A2[i]);
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
    // what arrived, into LDS; steps past the end (none in a `whole` block) leave mu as it is: their C too
    // is 0, for 0 times an infinite one would be NaN
    const auto stage = [&](int t, int half, auto whole) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const bool counts = whole || rdelta.inside(q, at.to - t);
            const float gate = (float)far_z[q], sg = sigmoid_of<FULL>(gate);
            const float dy = (float)far_adj[q] * (gated ? gate * sg : 1.f);
            const float dt = counts ? step_of(far_delta[q], bias, a.softplus) : 0.f;
            s_step[half][wave][4 * q + row][j] = make_float2(dt, counts ? dy : 0.f);
            total += dt;
        }
#pragma unroll
        for (int k = 0; k < REGS; ++k)
            ((float *)&s_C[half][wave][k * PER + j / R][0])[R * row + j % R] =
                no_state || (!whole && !rC.inside(k, at.to - t)) ? 0.f : (float)far_C[k];
    };
    int half = 0;
    const int last = at.from + (at.to - 1 - at.from) / STEPS * STEPS;
    fetch(last, std::false_type());
    stage(last, 0, std::false_type());
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
            stage(t - STEPS, half ^ 1, std::true_type());
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

template <typename T, int R, bool GATED, int W>
__global__ void __launch_bounds__(W *WAVE, R < 16 ? 2 : 1)
    k_scan_adjoint(ScanArgs a, Plan p, float *ws, float *sums, float *own)
{
    constexpr bool FULL = sizeof(T) == 4;
    constexpr int TS = part_steps<R>, Q = TS / 4, PER = ROW / R, REGS = TS / PER, BLOCK = block_steps<R>, PARTS = BLOCK / TS;
    __shared__ vec<float, 4> s_step[W][TS][ROW];
    __shared__ vec<float, 4> s_B[W][TS][R], s_C[W][TS][R];
    __shared__ float s_sum[2][W][2][REGS][WAVE];
    __shared__ vec<float, 4> s_state[W][PARTS - 2][R / 4][WAVE]; // (but for the first and the last)
    __shared__ float2 s_up[W][PARTS - 1][TS][ROW]; // (dt, dt u) of the way up, for the way down
    Place<R> at;
    const bool some = at.set(a, p, W);
    const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE, row = at.row, j = at.j;
    float A[R], A2[R], mu[R], dA[R];
    load_states<R>(a.A + (int64_t)at.c * a.states, at.n0, a.states, A);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        A2[i] = base2_rate(A[i]);
        A[i] = finite_rate(A[i]);
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
    const auto between = [] {
        if constexpr (W > 1)
            __syncthreads();
        else
            wave_sync();
    };
    const auto add_up = [&](int t) {
#pragma unroll
        for (int i = threadIdx.x; i < 2 * REGS * WAVE; i += W * WAVE) {
            const int which = i / (REGS * WAVE), reg = i / WAVE % REGS, l = i % WAVE;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w)
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
                between();
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
                // (steps past the end too: 0 times an infinite B or C would be NaN)
                const bool none = no_state || !rB.inside(k, left);
                B[k] = none ? 0.f : (float)far_B[k];
                C[k] = none ? 0.f : (float)far_C[k];
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
            between();
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

int64_t sums_size(const ScanArgs &a, const Plan &p) { return a.batch * p.across * a.len * 8 * rows_of(a.states); }
int64_t own_size(const ScanArgs &a, const Plan &p) { return a.batch * p.segments * a.dim * (int64_t)(a.states + 2); }

} // namespace

int64_t scan_adjoint_workspace(const ScanArgs &a)
{
    const Plan p = plan_of(a, true);
    if (!grid_ok((double)a.batch * p.across * p.segments * WAVES * WAVE) ||
        !grid_ok((double)a.batch * a.len * a.groups * 2 * a.states + (double)a.dim * (a.states + 2) * SUM_WAVES + 4096) ||
        !grid_ok((double)a.batch * a.dim * a.states + 256))
        return -1;
    return a.len > 0 ? (maps_size(a, p) + sums_size(a, p) + own_size(a, p)) * (int64_t)sizeof(float) : 0;
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
                hipLaunchKernelGGL((k_scan_adjoint_ends<T, R>), dim3((unsigned)(a.batch * p.across * p.segments)),
                                   dim3(p.waves * WAVE), 0, st, a, p, maps);
                CHOL_LAUNCH_CHECK();
            }
            const auto launch = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, dim3((unsigned)(a.batch * p.across * p.segments)), dim3(p.waves * WAVE), 0, st,
                                   a, p, maps, sums, own);
            };
            if (p.waves == 1)
                a.z.p ? launch(k_scan_adjoint<T, R, true, 1>) : launch(k_scan_adjoint<T, R, false, 1>);
            else if (p.waves == 2)
                a.z.p ? launch(k_scan_adjoint<T, R, true, 2>) : launch(k_scan_adjoint<T, R, false, 2>);
            else
                a.z.p ? launch(k_scan_adjoint<T, R, true, WAVES>) : launch(k_scan_adjoint<T, R, false, WAVES>);
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
