// Arguments of the gated linear recurrence and its adjoint (recurrence.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/libchol.h"

namespace chol {

struct RecRows {          // one [batch, len, dim] array
    void *p;
    int64_t ld, stride;
};

struct RecArgs {
    int64_t batch, len, dim;
    RecRows a;            // gates
    RecRows b;            // forward: inputs; adjoint: adj_h
    RecRows h;            // adjoint: the states the forward gave
    RecRows out;          // forward: h; adjoint: adj_b
    RecRows adj_a;        // adjoint only
    const float *h0;      // state before the first step, or NULL for zero
    const float *start;   // state the walk starts from: forward h0, adjoint adj_hlast (or NULL)
    float *end;           // state it ends with: forward hlast, adjoint adj_h0
};

int64_t recurrence_workspace(chol_dtype dt, int64_t batch, int64_t len, int64_t dim);
chol_status recurrence(chol_dtype dt, bool log_gate, bool adjoint, const RecArgs &args, void *ws, hipStream_t st);

} // namespace chol
