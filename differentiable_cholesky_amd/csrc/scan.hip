// The selective state space scan.
//
//   dt_t = softplus(delta_t + bias) (or delta_t + bias),
//   h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t          (N states a channel)
//   y_t = (sum_n C_t h_t + D u_t) silu(z_t)           (without z: the sum)
//
// An exponential and four more operations a state and step: 25 cycles of a SIMD a wave
// (measured), 93 us for 4 x 2048 x 4096 of 16 states, where the channels' four 16-bit
// numbers take 52 of memory.  So the vector units bound it, and the layout (scan_lanes.hpp)
// serves them.  4 x 2048 x 4096 bf16 of 16 states, saving states: 182 us, one wave a SIMD,
// whose vector instructions take 69 of 100 cycles: of 480 vector instructions a wave and 16
// steps 320 are the walk, 90 softplus, 80 the gate, the sums over rows and the stores.  8 x 4096 x
// 4096 574 us.  1 x 16384 x 4096 442 us: 16 segments, of which a first walk takes 40 % (traced by
// themselves 213 and 314 us).
#include "scan_lanes.hpp"

namespace chol {

namespace {

// ENDS: only walks to the end of a segment from zero and writes its map.
template <typename T, int R, bool ENDS, bool GATED>
__global__ void __launch_bounds__(WAVES *WAVE, R > 4 ? 1 : 3) k_scan(ScanArgs a, Plan p, float *ws)
{
    constexpr bool FULL = sizeof(T) == 4;
    constexpr int Q = STEPS / 4, PER = ROW / R, REGS = R, BLOCK = block_steps<R>;
    // (two of each: the next block's is written while this one's is read)
    __shared__ float2 s_step[2][WAVES][STEPS][ROW];
    __shared__ vec<float, 4> s_mixed[2][WAVES][STEPS][R]; // C; on a first walk B
    Place<R> at;
    if (!at.set(a, p, WAVES))
        return;
    const int wave = threadIdx.x / WAVE, row = at.row, j = at.j;
    float A2[R], h[R];
    load_states<R>(a.A + (int64_t)at.c * a.states, at.n0, a.states, A2);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        A2[i] = base2_rate(A2[i]);
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
            const bool none = no_state || (!whole && !rB.inside(k, at.to - t)); // (0 times a B of inf would be NaN)
            next_B[k] = none ? 0.f : (float)far_B[k];
            ((float *)&s_mixed[half][wave][k * PER + j / R][0])[R * row + j % R] = ENDS ? next_B[k] : none ? 0.f : (float)far_C[k];
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
        h[i] = fmaf(__builtin_amdgcn_exp2f(dt * base2_rate(A[i])), h[i], x * (float)B[i]);
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

int step_lanes(int states)
{
    int s = 1;
    while (4 * s < states)
        s *= 2;
    return s;
}

} // namespace

int scan_block(int states) { return 256 / rows_of(states); }

int64_t scan_workspace(const ScanArgs &a)
{
    const Plan p = plan_of(a, false);
    if (!grid_ok((double)a.batch * p.across * p.segments * WAVES * WAVE) ||
        !grid_ok((double)a.batch * a.dim * std::max(step_lanes(a.states), a.states) + 256))
        return -1;
    return a.len > 1 ? maps_size(a, p) * (int64_t)sizeof(float) : 0;
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
                hipLaunchKernelGGL(kernel, grid, dim3(WAVES * WAVE), 0, st, a, p, (float *)ws);
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

} // namespace chol
