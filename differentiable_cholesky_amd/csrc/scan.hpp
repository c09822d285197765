// Launchers of the selective state space scan (scan.hip).
#pragma once

#include "rows.hpp"

namespace chol {

struct ScanArgs {
    int64_t batch, len, dim;
    int groups, states;
    bool softplus;
    SeqRows u, delta, B, C, z, y;            // z.p may be null; y: what the forward writes
    const float *A, *D, *bias, *h0;          // D, bias, h0 may be null
    float *hlast, *starts;                   // starts: written by the forward (may be null), read by the adjoint
    // the adjoint's
    SeqRows adj, adj_u, adj_delta, adj_B, adj_C, adj_z;
    const float *adj_hlast;
    float *adj_A, *adj_D, *adj_bias, *adj_h0; // adj_D, adj_bias, adj_h0 may be null
    bool accumulate;
};

// steps between two saved states
int scan_block(int states);
// bytes, or -1 where the threads are more than a grid holds
int64_t scan_workspace(const ScanArgs &a);
int64_t scan_adjoint_workspace(const ScanArgs &a);
chol_status scan(chol_dtype dt, const ScanArgs &a, void *ws, hipStream_t st);
chol_status scan_adjoint(chol_dtype dt, const ScanArgs &a, void *ws, hipStream_t st);

} // namespace chol
