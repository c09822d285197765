// C-ABI of the operators of a recurrent model's training and decoding steps:
// the gated linear recurrence, the RMS norm and the AdamW step.  Every check
// runs on the host before anything is launched; a failed check launches
// nothing.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "../../include/libchol.h"
#include "adamw.hpp"
#include "checks.hpp"
#include "lowp.hpp"
#include "profile.hpp"
#include "recurrence.hpp"
#include "rmsnorm.hpp"

using namespace chol;

namespace {

// Most elements of a tensor, and of the distance between two rows.
const int64_t MAX_EXTENT = (int64_t)1 << 40;

} // namespace

extern "C" {

// -------------------------------------------------------------- recurrence ----

chol_status chol_recurrence_workspace_size(chol_dtype dt, int64_t batch, int64_t len, int64_t dim, size_t *bytes)
{
    if (!bytes || !lowp_dtype(dt) || batch < 0 || len < 0 || dim < 0)
        return CHOL_ERR_INVALID_VALUE;
    *bytes = 0;
    if (batch == 0 || dim == 0)
        return CHOL_OK;
    if (batch > INT32_MAX || len > INT32_MAX || dim > INT32_MAX || batch * dim > INT32_MAX)
        return CHOL_ERR_NOT_SUPPORTED;
    const int64_t need = recurrence_workspace(dt, batch, len, dim);
    if (need < 0)
        return CHOL_ERR_NOT_SUPPORTED;
    *bytes = (size_t)need;
    return CHOL_OK;
}

} // extern "C"

namespace {

// Checks shared by the recurrence and its adjoint; CHOL_OK with *noop for an
// empty state.
chol_status recurrence_args(chol_dtype dt, int gate, const RecArgs &r, bool adjoint, void *ws, size_t ws_bytes,
                            bool *noop)
{
    *noop = false;
    size_t need;
    if (gate != CHOL_GATE_LINEAR && gate != CHOL_GATE_LOG)
        return CHOL_ERR_INVALID_VALUE;
    const chol_status s = chol_recurrence_workspace_size(dt, r.batch, r.len, r.dim, &need);
    if (s != CHOL_OK)
        return s;
    if (r.batch == 0 || r.dim == 0) {
        *noop = true;
        return CHOL_OK;
    }
    const size_t es = lowp_size(dt);
    const RecRows *in[3] = {&r.a, &r.b, &r.h}, *out[2] = {&r.out, &r.adj_a};
    const int nin = adjoint ? 3 : 2, nout = adjoint ? 2 : 1;
    if (!r.end)
        return CHOL_ERR_INVALID_VALUE;
    if (r.len > 0) {
        for (int i = 0; i < nin + nout; ++i) {
            const RecRows &x = i < nin ? *in[i] : *out[i - nin];
            if (!x.p || x.ld > MAX_EXTENT || x.stride > MAX_EXTENT ||
                !layout_ok(r.len, r.dim, x.ld, r.batch, x.stride))
                return CHOL_ERR_INVALID_VALUE;
        }
        // an output may be one of the inputs, except that the adjoint reads the
        // states a step ahead of what it writes
        for (int o = 0; o < nout; ++o)
            for (int i = 0; i < nin; ++i)
                if (i == 2 ? !apart(in[i]->p, in[i]->ld, in[i]->stride, out[o]->p, out[o]->ld, out[o]->stride, r.len,
                                    r.dim, r.batch, es)
                           : !same_or_apart(in[i]->p, in[i]->ld, in[i]->stride, out[o]->p, out[o]->ld, out[o]->stride,
                                            r.len, r.dim, r.batch, es))
                    return CHOL_ERR_INVALID_VALUE;
        if (adjoint && !apart(r.out.p, r.out.ld, r.out.stride, r.adj_a.p, r.adj_a.ld, r.adj_a.stride, r.len, r.dim,
                              r.batch, es))
            return CHOL_ERR_INVALID_VALUE;
    }
    // the states: contiguous [batch, dim] fp32; the end may replace the start
    const Extent start = rect_extent(r.start, r.start ? r.batch : 0, r.dim, r.dim, 1, 0, 4);
    const Extent h0 = rect_extent(r.h0, r.h0 ? r.batch : 0, r.dim, r.dim, 1, 0, 4);
    const Extent end = rect_extent(r.end, r.batch, r.dim, r.dim, 1, 0, 4);
    if ((r.start != r.end && overlap(start, end)) || (adjoint && overlap(h0, end)))
        return CHOL_ERR_INVALID_VALUE;
    const Extent w{(uintptr_t)ws, (uintptr_t)ws + need};
    for (int i = 0; r.len > 0 && i < nin + nout; ++i) {
        const RecRows &x = i < nin ? *in[i] : *out[i - nin];
        const Extent e = rect_extent(x.p, r.len, r.dim, x.ld, r.batch, x.stride, es);
        if (overlap(e, end) || (i >= nin && (overlap(e, start) || overlap(e, h0))))
            return CHOL_ERR_INVALID_VALUE;
        if (need && ws && overlap(e, w))
            return CHOL_ERR_INVALID_VALUE;
    }
    if (need && (!ws || ws_bytes < need))
        return CHOL_ERR_WORKSPACE;
    if (need && ((uintptr_t)ws % 8 || overlap(w, start) || overlap(w, h0) || overlap(w, end)))
        return CHOL_ERR_INVALID_VALUE;
    return CHOL_OK;
}

} // namespace

extern "C" {

chol_status chol_recurrence(chol_dtype dt, int gate, int64_t batch, int64_t len, int64_t dim, const void *a,
                            int64_t lda, int64_t strideA, const void *b, int64_t ldb, int64_t strideB,
                            const float *h0, float *hlast, void *h, int64_t ldh, int64_t strideH, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    RecArgs r{};
    r.batch = batch, r.len = len, r.dim = dim;
    r.a = {(void *)a, lda, strideA};
    r.b = {(void *)b, ldb, strideB};
    r.out = {h, ldh, strideH};
    r.h0 = r.start = h0;
    r.end = hlast;
    bool noop;
    const chol_status s = recurrence_args(dt, gate, r, false, workspace, workspace_bytes, &noop);
    if (s != CHOL_OK || noop)
        return s;
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    prof::Scope ps(CHOL_K_RECURRENCE, st, 3.0 * batch * len * dim * lowp_size(dt));
    return recurrence(dt, gate == CHOL_GATE_LOG, false, r, workspace, st);
}

chol_status chol_recurrence_adjoint(chol_dtype dt, int gate, int64_t batch, int64_t len, int64_t dim, const void *a,
                                    int64_t lda, int64_t strideA, const void *h, int64_t ldh, int64_t strideH,
                                    const void *adjH, int64_t ldah, int64_t strideAH, const float *h0,
                                    const float *adjHlast, void *adjA, int64_t ldaa, int64_t strideAA, void *adjB,
                                    int64_t ldab, int64_t strideAB, float *adjH0, void *workspace,
                                    size_t workspace_bytes, void *stream)
{
    RecArgs r{};
    r.batch = batch, r.len = len, r.dim = dim;
    r.a = {(void *)a, lda, strideA};
    r.b = {(void *)adjH, ldah, strideAH};
    r.h = {(void *)h, ldh, strideH};
    r.out = {adjB, ldab, strideAB};
    r.adj_a = {adjA, ldaa, strideAA};
    r.h0 = h0;
    r.start = adjHlast;
    r.end = adjH0;
    bool noop;
    const chol_status s = recurrence_args(dt, gate, r, true, workspace, workspace_bytes, &noop);
    if (s != CHOL_OK || noop)
        return s;
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    prof::Scope ps(CHOL_K_RECURRENCE_ADJOINT, st, 5.0 * batch * len * dim * lowp_size(dt));
    return recurrence(dt, gate == CHOL_GATE_LOG, true, r, workspace, st);
}

} // extern "C"

// ------------------------------------------------------------------ norm ----

namespace {

// One [rows, cols] array of a norm call.
struct Rows2 {
    const void *p;
    int64_t ld;
    size_t es;
    int64_t cols;
    Extent extent(int64_t rows) const { return rect_extent(p, rows, cols, ld, 1, 0, es); }
};

chol_status norm_sizes(chol_dtype dt, int64_t rows, int64_t cols)
{
    if (!lowp_dtype(dt) || rows < 0 || cols < 0)
        return CHOL_ERR_INVALID_VALUE;
    if (rows > INT32_MAX || cols > CHOL_RMSNORM_MAX_COLS)
        return CHOL_ERR_NOT_SUPPORTED;
    return CHOL_OK;
}

bool rows_ok(const Rows2 &a, int64_t rows)
{
    return a.p && a.ld <= MAX_EXTENT && (rows <= 1 ? a.ld >= 0 : a.ld >= a.cols) && span_ok(rows, a.cols, a.ld, 1, 0);
}

// A row is read whole before any of it is written, by the threads that read
// it: an output may be an input itself.
bool rows_apart(const Rows2 &in, const Rows2 &out, int64_t rows, bool may_be_same)
{
    if (in.es == out.es && in.cols == out.cols)
        return may_be_same ? same_or_apart(in.p, in.ld, 0, out.p, out.ld, 0, rows, in.cols, 1, in.es)
                           : apart(in.p, in.ld, 0, out.p, out.ld, 0, rows, in.cols, 1, in.es);
    return !overlap(in.extent(rows), out.extent(rows));
}

chol_status norm_args(chol_dtype dt, const NormArgs &a, bool quantise, bool *noop)
{
    *noop = false;
    const chol_status s = norm_sizes(dt, a.rows, a.cols);
    if (s != CHOL_OK)
        return s;
    if (!(a.eps >= 0.f) || (quantise && a.group != 0 && a.group != 32 && a.group != 64 && a.group != 128 && a.group != 256))
        return CHOL_ERR_INVALID_VALUE;
    if (a.rows == 0 || a.cols == 0) {
        *noop = true;
        return CHOL_OK;
    }
    const size_t es = lowp_size(dt);
    const int64_t groups = quantise && a.group ? (a.cols + a.group - 1) / a.group : 1;
    const Rows2 x{a.x, a.ldx, es, a.cols}, r{a.residual, a.ldr, es, a.cols}, h{a.h, a.ldh, es, a.cols};
    const Rows2 y{a.y, a.ldy, quantise ? 1 : es, a.cols}, sc{a.scale, a.lds, 4, groups};
    const Extent w = rect_extent(a.w, 1, a.cols, a.cols, 1, 0, es);
    if (!a.w || !rows_ok(x, a.rows) || !rows_ok(y, a.rows) || (a.residual && (!rows_ok(r, a.rows) || !rows_ok(h, a.rows))) ||
        (quantise && !rows_ok(sc, a.rows)))
        return CHOL_ERR_INVALID_VALUE;
    const Rows2 *out[3] = {&y, a.residual ? &h : nullptr, quantise ? &sc : nullptr};
    for (int o = 0; o < 3; ++o) {
        if (!out[o])
            continue;
        if (!rows_apart(x, *out[o], a.rows, true) || (a.residual && !rows_apart(r, *out[o], a.rows, true)) ||
            overlap(w, out[o]->extent(a.rows)))
            return CHOL_ERR_INVALID_VALUE;
        for (int p = 0; p < o; ++p)
            if (out[p] && !rows_apart(*out[p], *out[o], a.rows, false))
                return CHOL_ERR_INVALID_VALUE;
    }
    return CHOL_OK;
}

} // namespace

extern "C" {

chol_status chol_rmsnorm(chol_dtype dt, int64_t rows, int64_t cols, const void *x, int64_t ldx, const void *residual,
                         int64_t ldr, const void *w, float eps, void *y, int64_t ldy, void *h, int64_t ldh,
                         void *stream)
{
    const NormArgs a{rows, cols, x, residual, w, ldx, ldr, eps, y, ldy, h, ldh, nullptr, 0, 0};
    bool noop;
    const chol_status s = norm_args(dt, a, false, &noop);
    if (s != CHOL_OK || noop)
        return s;
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    prof::Scope ps(CHOL_K_RMSNORM, st, (residual ? 4.0 : 2.0) * rows * cols * lowp_size(dt));
    return rmsnorm(dt, false, a, st);
}

chol_status chol_rmsnorm_quant(chol_dtype dt, int64_t rows, int64_t cols, int64_t group, const void *x, int64_t ldx,
                               const void *residual, int64_t ldr, const void *w, float eps, void *q, int64_t ldq,
                               float *scale, int64_t lds, void *h, int64_t ldh, void *stream)
{
    if (group < 0 || group > 256)
        return CHOL_ERR_INVALID_VALUE;
    const NormArgs a{rows, cols, x, residual, w, ldx, ldr, eps, q, ldq, h, ldh, scale, lds, (int)group};
    bool noop;
    const chol_status s = norm_args(dt, a, true, &noop);
    if (s != CHOL_OK || noop)
        return s;
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    prof::Scope ps(CHOL_K_RMSNORM, st, ((residual ? 3.0 : 1.0) * lowp_size(dt) + 1.0) * rows * cols);
    return rmsnorm(dt, true, a, st);
}

chol_status chol_rmsnorm_adjoint_workspace_size(chol_dtype dt, int64_t rows, int64_t cols, size_t *bytes)
{
    if (!bytes)
        return CHOL_ERR_INVALID_VALUE;
    *bytes = 0;
    const chol_status s = norm_sizes(dt, rows, cols);
    if (s == CHOL_OK && rows > 0 && cols > 0)
        *bytes = rmsnorm_adjoint_workspace(dt, rows, cols);
    return s;
}

chol_status chol_rmsnorm_adjoint(chol_dtype dt, int64_t rows, int64_t cols, const void *h, int64_t ldh, const void *w,
                                 const void *adj, int64_t lda, const void *adjH, int64_t ldah, float eps, void *adjX,
                                 int64_t ldax, float *adjW, int accumulate, void *workspace, size_t workspace_bytes,
                                 void *stream)
{
    size_t need;
    const chol_status s = chol_rmsnorm_adjoint_workspace_size(dt, rows, cols, &need);
    if (s != CHOL_OK)
        return s;
    if (!(eps >= 0.f))
        return CHOL_ERR_INVALID_VALUE;
    if (cols == 0)
        return CHOL_OK;
    const size_t es = lowp_size(dt);
    const Rows2 in[3] = {{h, ldh, es, cols}, {adj, lda, es, cols}, {adjH, ldah, es, cols}}, x{adjX, ldax, es, cols};
    const Extent we = rect_extent(w, 1, cols, cols, 1, 0, es), aw = rect_extent(adjW, 1, cols, cols, 1, 0, 4);
    if (!adjW)
        return CHOL_ERR_INVALID_VALUE;
    if (rows > 0) {
        if (!w || !rows_ok(x, rows) || overlap(we, x.extent(rows)) || overlap(we, aw) || overlap(aw, x.extent(rows)))
            return CHOL_ERR_INVALID_VALUE;
        const Extent ws{(uintptr_t)workspace, (uintptr_t)workspace + need};
        for (int i = 0; i < (adjH ? 3 : 2); ++i)
            if (!rows_ok(in[i], rows) || !rows_apart(in[i], x, rows, true) || overlap(in[i].extent(rows), aw) ||
                (need && workspace && overlap(ws, in[i].extent(rows))))
                return CHOL_ERR_INVALID_VALUE;
        if (need && (!workspace || workspace_bytes < need))
            return CHOL_ERR_WORKSPACE;
        if (need && ((uintptr_t)workspace % 4 || overlap(ws, x.extent(rows)) || overlap(ws, aw) || overlap(ws, we)))
            return CHOL_ERR_INVALID_VALUE;
    }
    const NormAdjArgs a{rows, cols, h, w, adj, adjH, ldh, lda, ldah, eps, adjX, ldax, adjW, accumulate};
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    prof::Scope ps(CHOL_K_RMSNORM_ADJOINT, st, (adjH ? 4.0 : 3.0) * rows * cols * es);
    return rmsnorm_adjoint(dt, a, workspace, st);
}

} // extern "C"

// ----------------------------------------------------------------- AdamW ----

namespace {

chol_status adamw_list(chol_dtype dt, int bits, int64_t count, const chol_adamw_tensor *tensors, void *table,
                       size_t table_bytes, int64_t *chunks, size_t *bytes)
{
    if (!lowp_dtype(dt) || (bits != 32 && bits != 8) || count < 0 || (count > 0 && !tensors) || !chunks || !bytes)
        return CHOL_ERR_INVALID_VALUE;
    struct Range {
        Extent e;
        bool written;
    };
    std::vector<Range> ranges;
    int64_t total = 0;
    bool with_master = false, without = false;
    const size_t es = lowp_size(dt), ss = bits == 8 ? 1 : 4;
    for (int64_t i = 0; i < count; ++i) {
        const chol_adamw_tensor &t = tensors[i];
        if (t.n < 0 || t.n > MAX_EXTENT)
            return CHOL_ERR_INVALID_VALUE;
        if (t.n == 0)
            continue;
        (t.master ? with_master : without) = true;
        if (!t.p || !t.g || !t.m || !t.v || (bits == 8 && (!t.m_scale || !t.v_scale)) || (uintptr_t)t.p % es ||
            (uintptr_t)t.g % es || (uintptr_t)t.m % ss || (uintptr_t)t.v % ss || (uintptr_t)t.master % 4 ||
            (uintptr_t)t.m_scale % 4 || (uintptr_t)t.v_scale % 4)
            return CHOL_ERR_INVALID_VALUE;
        const int64_t tiles = (t.n + ADAMW_TILE - 1) / ADAMW_TILE;
        const auto add = [&](const void *p, int64_t n, size_t size, bool written) {
            if (p)
                ranges.push_back({rect_extent(p, 1, n, n, 1, 0, size), written});
        };
        add(t.p, t.n, es, true);
        add(t.g, t.n, es, false);
        add(t.m, t.n, ss, true);
        add(t.v, t.n, ss, true);
        add(t.master, t.n, 4, true);
        if (bits == 8) {
            add(t.m_scale, tiles, 4, true);
            add(t.v_scale, tiles, 4, true);
        }
        total += (t.n + ADAMW_CHUNK - 1) / ADAMW_CHUNK;
    }
    if (with_master && without)
        return CHOL_ERR_INVALID_VALUE;
    if (total > INT32_MAX)
        return CHOL_ERR_NOT_SUPPORTED;
    // nothing that is written may be shared
    std::sort(ranges.begin(), ranges.end(), [](const Range &a, const Range &b) { return a.e.lo < b.e.lo; });
    uintptr_t read_to = 0, written_to = 0;
    for (const Range &r : ranges) {
        if (r.e.lo < written_to || (r.written && r.e.lo < read_to))
            return CHOL_ERR_INVALID_VALUE;
        uintptr_t &to = r.written ? written_to : read_to;
        to = std::max(to, r.e.hi);
    }
    *chunks = total;
    *bytes = (size_t)total * sizeof(AdamwChunk);
    if (!table)
        return CHOL_OK;
    if (table_bytes < *bytes)
        return CHOL_ERR_WORKSPACE;
    AdamwChunk *c = (AdamwChunk *)table;
    for (int64_t i = 0; i < count; ++i) {
        const chol_adamw_tensor &t = tensors[i];
        for (int64_t at = 0; at < t.n; at += ADAMW_CHUNK, ++c) {
            c->p = (char *)t.p + at * es;
            c->g = (const char *)t.g + at * es;
            c->m = (char *)t.m + at * ss;
            c->v = (char *)t.v + at * ss;
            c->master = t.master ? t.master + at : nullptr;
            c->m_scale = bits == 8 ? t.m_scale + at / ADAMW_TILE : nullptr;
            c->v_scale = bits == 8 ? t.v_scale + at / ADAMW_TILE : nullptr;
            c->n = (uint32_t)std::min<int64_t>(ADAMW_CHUNK, t.n - at);
            c->first = (uint32_t)(t.first + at);
        }
    }
    return CHOL_OK;
}

} // namespace

extern "C" {

chol_status chol_adamw_list(chol_dtype dt, int bits, int64_t count, const chol_adamw_tensor *tensors, void *table,
                            size_t table_bytes, int64_t *chunks, size_t *bytes)
{
    try {
        return adamw_list(dt, bits, count, tensors, table, table_bytes, chunks, bytes);
    } catch (...) { // host memory for the ranges
        return CHOL_ERR_NOT_SUPPORTED;
    }
}

chol_status chol_adamw(chol_dtype dt, int bits, int master, int64_t chunks, const void *table, const float *grad_scale,
                       double lr, double beta1, double beta2, double eps, double weight_decay, int64_t step,
                       uint32_t seed, void *stream)
{
    if (!lowp_dtype(dt) || (bits != 32 && bits != 8) || chunks < 0 || chunks > INT32_MAX || step < 1 ||
        !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) || !std::isfinite(eps) ||
        !std::isfinite(lr) || !std::isfinite(weight_decay))
        return CHOL_ERR_INVALID_VALUE;
    if (chunks == 0)
        return CHOL_OK;
    if (!table || (uintptr_t)table % 8 || (uintptr_t)grad_scale % 4)
        return CHOL_ERR_INVALID_VALUE;
    AdamwHyper k;
    k.beta1 = (float)beta1, k.one_beta1 = (float)(1 - beta1);
    k.beta2 = (float)beta2, k.one_beta2 = (float)(1 - beta2);
    k.decay = (float)(lr * weight_decay);
    k.rate = (float)(lr / (1 - std::pow(beta1, (double)step)));
    k.inv_root = (float)(1 / std::sqrt(1 - std::pow(beta2, (double)step)));
    k.eps = (float)eps;
    k.grad_scale = grad_scale;
    k.key = adamw_mix(seed);
    hipStream_t st = (hipStream_t)stream;
    clear_stale_status();
    const double element = 2.0 * lowp_size(dt) + (master ? 8 : lowp_size(dt)) + (bits == 8 ? 4 : 16);
    prof::Scope ps(CHOL_K_ADAMW, st, element * chunks * ADAMW_CHUNK);
    return adamw(dt, bits, master != 0, chunks, (const AdamwChunk *)table, k, st);
}

} // extern "C"
