// C-ABI of the operators a training or decoding step runs next to the factor:
// the gated linear recurrence, the RMS norm and the AdamW step.  Every check
// runs on the host before anything is launched; a failed check launches
// nothing.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/libchol.h"
#include "checks.hpp"
#include "lowp.hpp"
#include "profile.hpp"
#include "recurrence.hpp"

using namespace chol;

namespace {

// Sizes whose products stay far inside 64 bits.
const int64_t MAX_EXTENT = (int64_t)1 << 40;

bool size_ok(int64_t n) { return n >= 0 && n <= MAX_EXTENT; }

} // namespace

extern "C" {

// -------------------------------------------------------------- recurrence ----

chol_status chol_recurrence_workspace_size(chol_dtype dt, int64_t batch, int64_t len, int64_t dim, size_t *bytes)
{
    if (!bytes || !lowp_dtype(dt) || batch < 0 || len < 0 || dim < 0)
        return CHOL_ERR_INVALID_VALUE;
    *bytes = 0;
    if (batch == 0 || len == 0 || dim == 0)
        return CHOL_OK;
    if (batch > INT32_MAX || len > INT32_MAX || dim > INT32_MAX || batch * dim > INT32_MAX)
        return CHOL_ERR_NOT_SUPPORTED;
    *bytes = recurrence_workspace(batch, len, dim);
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
