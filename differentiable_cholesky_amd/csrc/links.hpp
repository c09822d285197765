// How the workgroups of a recurrence's chain pass the state along the sequence.
//
// Workgroup k of a chain holds the composition x -> P x + Q of its steps and needs
// the state before them.  Each publishes one word: the first of the chain and the
// last of every group of LINKS the state after their steps, as (0, state), the
// others their (P, Q).  A workgroup composes the words before it in its group and
// applies that to the state its group starts from.
//
// The state that the chain starts from may share its memory with the one it ends
// with, which the last workgroup writes.  So it is read by the first workgroup
// alone, whose word is made of what it read: whatever follows from that word,
// that write among it, comes after the read.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>

namespace chol {

constexpr unsigned LINKS = 8, WINDOW = 4; // workgroups of a chain's group; words read at once

// x: the state before workgroup `chunk` of `chunks` (two or more), V channels.
// Chain: start(v), the chain's start; publish(k, v, P, Q), peek(k, v), which gives
// workgroup k's word or an empty one, and arrived(k, v, word), which waits until it
// is there and gives (P, Q).
template <int V, typename Chain>
__host__ __device__ __forceinline__ void state_before(Chain &chain, unsigned chunk, unsigned chunks,
                                                      const float (&P)[V], const float (&Q)[V], float (&x)[V])
{
    if (chunk == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = chain.start(v);
            chain.publish(0, v, 0.f, fmaf(P[v], x[v], Q[v]));
        }
        return;
    }
    typedef decltype(chain.peek(0u, 0)) Word;
    const unsigned first = chunk / LINKS * LINKS;
    const bool last = chunk % LINKS == LINKS - 1, read = chunk + 1 < chunks;
    if (!last && read)
#pragma unroll
        for (int v = 0; v < V; ++v)
            chain.publish(chunk, v, P[v], Q[v]);
    float bp[V], bq[V]; // of the group's workgroups before this one
    Word base[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bp[v] = 1.f, bq[v] = 0.f;
        base[v] = first ? chain.peek(first - 1, v) : Word{};
    }
    for (unsigned at = first; at < chunk; at += WINDOW) {
        Word w[WINDOW][V];
#pragma unroll
        for (unsigned k = 0; k < WINDOW; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (at + k < chunk)
                    w[k][v] = chain.peek(at + k, v);
#pragma unroll
        for (unsigned k = 0; k < WINDOW; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (at + k < chunk) {
                    const float2 n = chain.arrived(at + k, v, w[k][v]);
                    bq[v] = fmaf(n.x, bq[v], n.y);
                    bp[v] *= n.x;
                }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (first == 0) { // the first workgroup's word is a state
            x[v] = bq[v];
        } else {
            const float from = chain.arrived(first - 1, v, base[v]).y;
            x[v] = chunk == first ? from : fmaf(bp[v], from, bq[v]);
        }
        if (last && read)
            chain.publish(chunk, v, 0.f, fmaf(P[v], x[v], Q[v]));
    }
}

} // namespace chol
