// C-ABI of the operators of a selective state space language model: the causal
// convolution, the selective scan and the log probabilities of given tokens.  Every
// check runs on the host before anything is launched; a failed check launches nothing.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/libchol.h"
#include "checks.hpp"
#include "conv.hpp"
#include "logprob.hpp"
#include "profile.hpp"
#include "scan.hpp"

using namespace chol;

namespace {

// Most elements between two rows or batch elements.
const int64_t MAX_EXTENT = (int64_t)1 << 40;

// A [batch, rows, cols] array of a call; p NULL is one that the call does not have.
struct Array {
    const void *p;
    int64_t batch, rows, cols, ld, stride;
    size_t es;

    bool empty() const { return !p || batch == 0 || rows == 0 || cols == 0; }
    Extent extent() const { return empty() ? Extent{0, 0} : rect_extent(p, rows, cols, ld, batch, stride, es); }
    bool valid() const
    {
        return empty() || ((uintptr_t)p % es == 0 && ld <= MAX_EXTENT && stride <= MAX_EXTENT &&
                      layout_ok(rows, cols, ld, batch, stride));
    }
};

Array flat(const void *p, int64_t n, size_t es) { return {p, 1, 1, n, n, 0, es}; }
Array sequence(const SeqRows &r, int64_t batch, int64_t len, int64_t cols, size_t es)
{
    return {len > 0 ? r.p : nullptr, batch, len, cols, r.ld, r.stride, es};
}

bool same(const Array &a, const Array &b)
{
    return a.p == b.p && a.es == b.es && a.cols == b.cols && a.rows == b.rows && a.batch == b.batch &&
           (a.rows <= 1 || a.ld == b.ld) && (a.batch <= 1 || a.stride == b.stride);
}

// Whether two arrays share no element.  Where their address ranges interleave (slices
// of one buffer, of any widths) both need the same distances: rows of one lie i * outer
// + j * inner from rows of the other, and what the inner distances reach is less than
// `outer`, so two values of i and of j come into question.
bool apart(const Array &a, const Array &b)
{
    if (!overlap(a.extent(), b.extent()))
        return true;
    if (a.es != b.es || a.rows != b.rows || a.batch != b.batch || (a.rows > 1 && a.ld != b.ld) ||
        (a.batch > 1 && a.stride != b.stride))
        return false;
    const Array &low = (uintptr_t)a.p <= (uintptr_t)b.p ? a : b, &high = &low == &a ? b : a;
    const int64_t d = (int64_t)(((uintptr_t)high.p - (uintptr_t)low.p) / a.es);
    // (a coordinate of one value has no distance: one that nothing reaches stands for it)
    const int64_t none = (int64_t)1 << 60;
    int64_t inner = a.rows > 1 ? a.ld : none, outer = a.batch > 1 ? a.stride : none;
    int64_t inners = a.rows, outers = a.batch;
    if (inner > outer) {
        std::swap(inner, outer);
        std::swap(inners, outers);
    }
    for (int64_t i = d / outer; i <= d / outer + 1 && i < outers; ++i) {
        const int64_t left = d - i * outer, down = left >= 0 ? left / inner : -((-left + inner - 1) / inner);
        for (int64_t j = down; j <= down + 1; ++j) {
            const int64_t r = left - j * inner;
            if (j > -inners && j < inners && r < low.cols && r > -high.cols)
                return false;
        }
    }
    return true;
}

struct Pair {
    const Array *out, *in;
};

// Whether the arrays are valid, every output is apart from every input (or is one that
// `may` names with it) and from the other outputs, and the workspace from all.
template <int NI, int NO, int NP>
chol_status arrays_ok(const Array (&in)[NI], const Array (&out)[NO], const Pair (&may)[NP], const void *ws, size_t need)
{
    for (const Array &a : in)
        if (!a.valid())
            return CHOL_ERR_INVALID_VALUE;
    for (const Array &a : out)
        if (!a.valid())
            return CHOL_ERR_INVALID_VALUE;
    const Extent w = ws && need ? Extent{(uintptr_t)ws, (uintptr_t)ws + need} : Extent{0, 0};
    for (int o = 0; o < NO; ++o) {
        if (out[o].empty())
            continue;
        for (const Array &a : in) {
            if (a.empty())
                continue;
            bool allowed = false;
            for (const Pair &p : may)
                allowed = allowed || (p.out == &out[o] && p.in == &a && same(a, out[o]));
            if (!allowed && !apart(a, out[o]))
                return CHOL_ERR_INVALID_VALUE;
        }
        for (int k = 0; k < o; ++k)
            if (!out[k].empty() && !apart(out[k], out[o]))
                return CHOL_ERR_INVALID_VALUE;
        if (overlap(w, out[o].extent()))
            return CHOL_ERR_INVALID_VALUE;
    }
    for (const Array &a : in)
        if (overlap(w, a.extent()))
            return CHOL_ERR_INVALID_VALUE;
    return CHOL_OK;
}

chol_status workspace_ok(const void *ws, size_t bytes, size_t need, size_t align)
{
    if (need && (!ws || bytes < need))
        return CHOL_ERR_WORKSPACE;
    return need && (uintptr_t)ws % align ? CHOL_ERR_INVALID_VALUE : CHOL_OK;
}

// ------------------------------------------------------------ convolution ----

chol_status conv_sizes(chol_dtype dt, int64_t batch, int64_t len, int64_t dim, int64_t width)
{
    if (!lowp_dtype(dt) || batch < 0 || len < 0 || dim < 0 || width < 1)
        return CHOL_ERR_INVALID_VALUE;
    if (width < CHOL_CONV_MIN_WIDTH || width > CHOL_CONV_MAX_WIDTH || batch > INT32_MAX || len > INT32_MAX ||
        dim > INT32_MAX || batch * dim > INT32_MAX)
        return CHOL_ERR_NOT_SUPPORTED;
    return CHOL_OK;
}

// What the convolution and its adjoint check alike.
struct ConvArrays {
    Array x, w, bias, state;
    ConvArrays(const ConvArgs &a, size_t es)
        : x(sequence(a.x, a.batch, a.len, a.dim, es)), w(flat(a.w, a.dim * a.width, es)),
          bias(flat(a.bias, a.dim, es)), state(flat(a.state, a.batch * (a.width - 1) * a.dim, es))
    {
    }
};

} // namespace

extern "C" {

chol_status chol_causal_conv(chol_dtype dt, int silu, int64_t batch, int64_t len, int64_t dim, int64_t width,
                             const void *x, int64_t ldx, int64_t strideX, const void *w, const void *bias,
                             const void *state, void *last, void *y, int64_t ldy, int64_t strideY, void *stream)
{
    const chol_status s = conv_sizes(dt, batch, len, dim, width);
    if (s != CHOL_OK)
        return s;
    if (batch == 0 || dim == 0)
        return CHOL_OK;
    ConvArgs a{};
    a.batch = batch, a.len = len, a.dim = dim, a.width = (int)width, a.silu = silu != 0;
    a.x = {(void *)x, ldx, strideX};
    a.y = {y, ldy, strideY};
    a.w = w, a.bias = bias, a.state = state, a.last = last;
    if (!conv_fits(dt, a))
        return CHOL_ERR_NOT_SUPPORTED;
    if (!w || (len > 0 && (!x || !y)))
        return CHOL_ERR_INVALID_VALUE;
    const size_t es = lowp_size(dt);
    const ConvArrays c(a, es);
    const Array in[] = {c.x, c.w, c.bias, c.state};
    const Array out[] = {sequence(a.y, batch, len, dim, es), flat(last, batch * (width - 1) * dim, es)};
    const Pair may[] = {{&out[1], &in[3]}};
    const chol_status r = arrays_ok(in, out, may, nullptr, 0);
    if (r != CHOL_OK || (len == 0 && !last))
        return r;
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    prof::Scope ps(CHOL_K_CONV, st, 2.0 * batch * len * dim * es);
    return conv(dt, a, st);
}

chol_status chol_causal_conv_adjoint_workspace_size(chol_dtype dt, int64_t batch, int64_t len, int64_t dim,
                                                    int64_t width, size_t *bytes)
{
    if (!bytes)
        return CHOL_ERR_INVALID_VALUE;
    *bytes = 0;
    const chol_status s = conv_sizes(dt, batch, len, dim, width);
    if (s != CHOL_OK || dim == 0)
        return s;
    ConvArgs a{};
    a.batch = batch, a.len = len, a.dim = dim, a.width = (int)width;
    const int64_t need = conv_adjoint_workspace(dt, a);
    if (need < 0)
        return CHOL_ERR_NOT_SUPPORTED;
    *bytes = (size_t)need;
    return CHOL_OK;
}

chol_status chol_causal_conv_adjoint(chol_dtype dt, int silu, int64_t batch, int64_t len, int64_t dim, int64_t width,
                                     const void *x, int64_t ldx, int64_t strideX, const void *w, const void *bias,
                                     const void *state, const void *adj, int64_t lda, int64_t strideA,
                                     const void *adjLast, void *adjX, int64_t ldax, int64_t strideAX, float *adjW,
                                     float *adjBias, int accumulate, void *adjState, void *workspace,
                                     size_t workspace_bytes, void *stream)
{
    size_t need;
    const chol_status s = chol_causal_conv_adjoint_workspace_size(dt, batch, len, dim, width, &need);
    if (s != CHOL_OK)
        return s;
    if (dim == 0)
        return CHOL_OK;
    if (!w || !adjW || (batch > 0 && len > 0 && (!x || !adj || !adjX)))
        return CHOL_ERR_INVALID_VALUE;
    ConvArgs a{};
    a.batch = batch, a.len = len, a.dim = dim, a.width = (int)width, a.silu = silu != 0;
    a.x = {(void *)x, ldx, strideX};
    a.y = {adjX, ldax, strideAX};
    a.adj = {(void *)adj, lda, strideA};
    a.w = w, a.bias = bias, a.state = state, a.adj_last = adjLast, a.last = adjState;
    a.adj_w = adjW, a.adj_bias = adjBias, a.accumulate = accumulate != 0;
    const size_t es = lowp_size(dt);
    const int64_t kept = batch * (width - 1) * dim;
    const ConvArrays c(a, es);
    const Array in[] = {c.x, c.w, c.bias, c.state, sequence(a.adj, batch, len, dim, es), flat(adjLast, kept, es)};
    const Array out[] = {sequence(a.y, batch, len, dim, es), flat(adjState, kept, es), flat(adjW, dim * width, 4),
                         flat(adjBias, dim, 4)};
    const Pair may[] = {{nullptr, nullptr}};
    const chol_status r = arrays_ok(in, out, may, workspace, need);
    if (r != CHOL_OK)
        return r;
    const chol_status q = workspace_ok(workspace, workspace_bytes, need, 4);
    if (q != CHOL_OK)
        return q;
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    prof::Scope ps(CHOL_K_CONV_ADJOINT, st, 3.0 * batch * len * dim * es);
    return conv_adjoint(dt, a, workspace, st);
}

} // extern "C"

// ------------------------------------------------------------------- scan ----

namespace {

// The kernels count steps in 32 bits, and reach 16 rows on by offsets of 32 bits in bytes.
const int64_t MAX_LEN = (int64_t)1 << 30, MAX_ROW = (int64_t)1 << 25;

template <int N> bool rows_near(const Array (&arrays)[N])
{
    for (const Array &a : arrays)
        if (!a.empty() && a.rows > 1 && a.ld > MAX_ROW)
            return false;
    return true;
}

chol_status scan_sizes(int64_t batch, int64_t len, int64_t dim, int64_t groups, int64_t states)
{
    if (batch < 0 || len < 0 || dim < 0 || groups < 1 || states < 1 || dim % groups != 0)
        return CHOL_ERR_INVALID_VALUE;
    if (states > CHOL_SCAN_MAX_STATES || batch > INT32_MAX || len > MAX_LEN || dim > INT32_MAX ||
        (__int128)std::max<int64_t>(batch, 1) * dim * states > INT32_MAX)
        return CHOL_ERR_NOT_SUPPORTED;
    return CHOL_OK;
}

SeqRows rows_of(const chol_rows &r) { return {r.p, r.ld, r.stride}; }

ScanArgs scan_args(const chol_scan_args &g)
{
    ScanArgs a{};
    a.batch = g.batch, a.len = g.len, a.dim = g.dim, a.groups = (int)g.groups, a.states = (int)g.states;
    a.softplus = g.softplus != 0, a.accumulate = g.accumulate != 0;
    a.u = rows_of(g.u), a.delta = rows_of(g.delta), a.B = rows_of(g.B), a.C = rows_of(g.C), a.z = rows_of(g.z), a.y = rows_of(g.y);
    a.A = g.A, a.D = g.D, a.bias = g.bias, a.h0 = g.h0, a.hlast = g.hlast, a.starts = g.starts;
    a.adj = rows_of(g.adj), a.adj_u = rows_of(g.adj_u), a.adj_delta = rows_of(g.adj_delta);
    a.adj_B = rows_of(g.adj_B), a.adj_C = rows_of(g.adj_C), a.adj_z = rows_of(g.adj_z);
    a.adj_hlast = g.adj_hlast, a.adj_A = g.adj_A, a.adj_D = g.adj_D, a.adj_bias = g.adj_bias, a.adj_h0 = g.adj_h0;
    return a;
}

int64_t starts_size(const ScanArgs &a)
{
    const int64_t block = scan_block(a.states);
    return a.batch * ((a.len + block - 1) / block) * a.dim * a.states;
}

} // namespace

extern "C" {

int64_t chol_selective_scan_block(int64_t states)
{
    return states < 1 || states > CHOL_SCAN_MAX_STATES ? -1 : scan_block((int)states);
}

chol_status chol_selective_scan_workspace_size(int adjoint, int64_t batch, int64_t len, int64_t dim, int64_t groups,
                                               int64_t states, size_t *bytes)
{
    if (!bytes)
        return CHOL_ERR_INVALID_VALUE;
    *bytes = 0;
    const chol_status s = scan_sizes(batch, len, dim, groups, states);
    if (s != CHOL_OK || batch == 0 || dim == 0)
        return s;
    ScanArgs a{};
    a.batch = batch, a.len = len, a.dim = dim, a.groups = (int)groups, a.states = (int)states;
    const int64_t need = adjoint ? scan_adjoint_workspace(a) : scan_workspace(a);
    if (need < 0)
        return CHOL_ERR_NOT_SUPPORTED;
    *bytes = (size_t)need;
    return CHOL_OK;
}

chol_status chol_selective_scan(chol_dtype dt, const chol_scan_args *args, void *workspace, size_t workspace_bytes,
                                void *stream)
{
    if (!args || !lowp_dtype(dt))
        return CHOL_ERR_INVALID_VALUE;
    const chol_scan_args &g = *args;
    size_t need;
    const chol_status s = chol_selective_scan_workspace_size(0, g.batch, g.len, g.dim, g.groups, g.states, &need);
    if (s != CHOL_OK || g.batch == 0 || g.dim == 0)
        return s;
    const ScanArgs a = scan_args(g);
    if (!a.hlast || !a.A || (a.len > 0 && (!a.u.p || !a.delta.p || !a.B.p || !a.C.p || !a.y.p)))
        return CHOL_ERR_INVALID_VALUE;
    const size_t es = lowp_size(dt);
    const int64_t b = a.batch, l = a.len, d = a.dim, mixed = g.groups * g.states;
    const Array in[] = {sequence(a.u, b, l, d, es),     sequence(a.delta, b, l, d, es), sequence(a.z, b, l, d, es),
                        sequence(a.B, b, l, mixed, es), sequence(a.C, b, l, mixed, es), flat(a.h0, b * d * a.states, 4),
                        flat(a.A, d * a.states, 4),     flat(a.D, d, 4),                flat(a.bias, d, 4)};
    const Array out[] = {sequence(a.y, b, l, d, es), flat(a.hlast, b * d * a.states, 4),
                         flat(l > 0 ? a.starts : nullptr, starts_size(a), 4)};
    const Pair may[] = {{&out[0], &in[0]}, {&out[0], &in[1]}, {&out[0], &in[2]}, {&out[1], &in[5]}};
    const chol_status r = arrays_ok(in, out, may, workspace, need);
    if (r != CHOL_OK)
        return r;
    if (!rows_near(in) || !rows_near(out))
        return CHOL_ERR_NOT_SUPPORTED;
    const chol_status q = workspace_ok(workspace, workspace_bytes, need, 4);
    if (q != CHOL_OK)
        return q;
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    prof::Scope ps(CHOL_K_SCAN, st, (a.z.p ? 4.0 : 3.0) * b * l * d * es);
    return scan(dt, a, workspace, st);
}

chol_status chol_selective_scan_adjoint(chol_dtype dt, const chol_scan_args *args, void *workspace,
                                        size_t workspace_bytes, void *stream)
{
    if (!args || !lowp_dtype(dt))
        return CHOL_ERR_INVALID_VALUE;
    const chol_scan_args &g = *args;
    size_t need;
    const chol_status s = chol_selective_scan_workspace_size(1, g.batch, g.len, g.dim, g.groups, g.states, &need);
    if (s != CHOL_OK || g.dim == 0)
        return s;
    const ScanArgs a = scan_args(g);
    const bool work = a.batch > 0 && a.len > 0;
    if (!a.adj_A || (work && (!a.u.p || !a.delta.p || !a.A || !a.B.p || !a.C.p || !a.starts || !a.adj.p || !a.adj_u.p ||
                              !a.adj_delta.p || !a.adj_B.p || !a.adj_C.p || (a.z.p && !a.adj_z.p))))
        return CHOL_ERR_INVALID_VALUE;
    const size_t es = lowp_size(dt);
    const int64_t b = a.batch, l = a.len, d = a.dim, mixed = g.groups * g.states, state = b * d * a.states;
    const Array in[] = {sequence(a.u, b, l, d, es),     sequence(a.delta, b, l, d, es), sequence(a.z, b, l, d, es),
                        sequence(a.B, b, l, mixed, es), sequence(a.C, b, l, mixed, es), sequence(a.adj, b, l, d, es),
                        flat(a.adj_hlast, state, 4),    flat(a.A, d * a.states, 4),     flat(a.D, d, 4),
                        flat(a.bias, d, 4),             flat(work ? a.starts : nullptr, starts_size(a), 4)};
    SeqRows adj_z = a.adj_z;
    if (!a.z.p)
        adj_z.p = nullptr;
    const Array out[] = {sequence(a.adj_u, b, l, d, es),     sequence(a.adj_delta, b, l, d, es),
                         sequence(adj_z, b, l, d, es),       sequence(a.adj_B, b, l, mixed, es),
                         sequence(a.adj_C, b, l, mixed, es), flat(a.adj_h0, state, 4),
                         flat(a.adj_A, d * a.states, 4),     flat(a.adj_D, d, 4),
                         flat(a.adj_bias, d, 4)};
    const Pair may[] = {{&out[0], &in[0]}, {&out[1], &in[1]}, {&out[2], &in[2]}, {&out[3], &in[3]}, {&out[4], &in[4]},
                        {&out[0], &in[5]}, {&out[1], &in[5]}, {&out[2], &in[5]}, {&out[5], &in[6]}};
    const chol_status r = arrays_ok(in, out, may, workspace, need);
    if (r != CHOL_OK)
        return r;
    if (!rows_near(in) || !rows_near(out))
        return CHOL_ERR_NOT_SUPPORTED;
    const chol_status q = workspace_ok(workspace, workspace_bytes, need, 4);
    if (q != CHOL_OK)
        return q;
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    prof::Scope ps(CHOL_K_SCAN_ADJOINT, st, (a.z.p ? 7.0 : 5.0) * b * l * d * es);
    return scan_adjoint(dt, a, workspace, st);
}

} // extern "C"

// ------------------------------------------------------ log probabilities ----

namespace {

chol_status logprob_sizes(chol_dtype dt, int64_t rows, int64_t vocab)
{
    if (!lowp_dtype(dt) || rows < 0 || vocab < 0 || (vocab == 0 && rows > 0))
        return CHOL_ERR_INVALID_VALUE;
    if (rows > INT32_MAX || vocab > CHOL_LOGPROB_MAX_VOCAB || (rows > 0 && !logprob_fits(dt, rows, vocab)))
        return CHOL_ERR_NOT_SUPPORTED;
    return CHOL_OK;
}

// (the kernels multiply half distances by twice the scale and log2(e))
bool scale_ok(float scale) { return scale > 0.f && scale <= 0x1p126f; }

} // namespace

extern "C" {

chol_status chol_token_logprob_workspace_size(chol_dtype dt, int64_t rows, int64_t vocab, int64_t top, size_t *bytes)
{
    if (!bytes)
        return CHOL_ERR_INVALID_VALUE;
    *bytes = 0;
    const chol_status s = logprob_sizes(dt, rows, vocab);
    if (s != CHOL_OK)
        return s;
    if (top < 0 || (rows > 0 && top > std::min<int64_t>(vocab, CHOL_LOGPROB_MAX_TOP)))
        return CHOL_ERR_INVALID_VALUE;
    if (rows > 0)
        *bytes = logprob_workspace(dt, rows, vocab, (int)top);
    return CHOL_OK;
}

chol_status chol_token_logprob(chol_dtype dt, int64_t rows, int64_t vocab, const void *x, int64_t ldx,
                               const int64_t *tokens, float scale, float *logp, float *lse, float *entropy, int64_t top,
                               float *top_logp, int64_t *top_ids, void *workspace, size_t workspace_bytes, void *stream)
{
    size_t need;
    const chol_status s = chol_token_logprob_workspace_size(dt, rows, vocab, top, &need);
    if (s != CHOL_OK)
        return s;
    if (!scale_ok(scale))
        return CHOL_ERR_INVALID_VALUE;
    if (rows == 0)
        return CHOL_OK;
    if (!x || !tokens || !logp || !lse || (top > 0 && (!top_logp || !top_ids)))
        return CHOL_ERR_INVALID_VALUE;
    const Array in[] = {{x, 1, rows, vocab, ldx, 0, lowp_size(dt)}, flat(tokens, rows, 8)};
    const Array out[] = {flat(logp, rows, 4), flat(lse, rows, 4), flat(entropy, rows, 4),
                         flat(top > 0 ? top_logp : nullptr, rows * top, 4), flat(top > 0 ? top_ids : nullptr, rows * top, 8)};
    const Pair may[] = {{nullptr, nullptr}};
    const chol_status r = arrays_ok(in, out, may, workspace, need);
    if (r != CHOL_OK)
        return r;
    const chol_status q = workspace_ok(workspace, workspace_bytes, need, 8);
    if (q != CHOL_OK)
        return q;
    const LogprobArgs a{rows, vocab, x, ldx, tokens, scale, logp, lse, entropy, (int)top, top_logp, top_ids};
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    prof::Scope ps(CHOL_K_LOGPROB, st, 1.0 * rows * vocab * lowp_size(dt));
    return logprob(dt, a, workspace, st);
}

chol_status chol_token_logprob_adjoint(chol_dtype dt, int64_t rows, int64_t vocab, const void *x, int64_t ldx,
                                       const int64_t *tokens, float scale, const float *lse, const float *entropy,
                                       const float *adjLogp, const float *adjEntropy, void *adjX, int64_t ldax,
                                       void *stream)
{
    const chol_status s = logprob_sizes(dt, rows, vocab);
    if (s != CHOL_OK)
        return s;
    if (!scale_ok(scale))
        return CHOL_ERR_INVALID_VALUE;
    if (rows == 0)
        return CHOL_OK;
    if (!x || !tokens || !lse || !adjX || (adjEntropy && !entropy))
        return CHOL_ERR_INVALID_VALUE;
    const size_t es = lowp_size(dt);
    const Array in[] = {{x, 1, rows, vocab, ldx, 0, es}, flat(tokens, rows, 8),   flat(lse, rows, 4),
                        flat(entropy, rows, 4),          flat(adjLogp, rows, 4), flat(adjEntropy, rows, 4)};
    const Array out[] = {{adjX, 1, rows, vocab, ldax, 0, es}};
    const Pair may[] = {{&out[0], &in[0]}};
    const chol_status r = arrays_ok(in, out, may, nullptr, 0);
    if (r != CHOL_OK)
        return r;
    const LogprobAdjArgs a{rows, vocab, x, ldx, tokens, scale, lse, entropy, adjLogp, adjEntropy, adjX, ldax};
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    prof::Scope ps(CHOL_K_LOGPROB_ADJOINT, st, 2.0 * rows * vocab * es);
    return logprob_adjoint(dt, a, st);
}

} // extern "C"
