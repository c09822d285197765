// Launcher of the short causal convolution (conv.hip).
#pragma once

#include "rows.hpp"

namespace chol {

struct ConvArgs {
    int64_t batch, len, dim;
    int width;
    bool silu;
    SeqRows x, y;                // y: adj_x in the adjoint
    SeqRows adj;                 // adjoint only
    const void *w, *bias, *state;
    const void *adj_last;        // adjoint only
    void *last;                  // adj_state in the adjoint
    float *adj_w, *adj_bias;     // adjoint only
    bool accumulate;
};

// bytes, or -1 where the threads are more than a grid holds
int64_t conv_adjoint_workspace(chol_dtype dt, const ConvArgs &a);
bool conv_fits(chol_dtype dt, const ConvArgs &a);
chol_status conv(chol_dtype dt, const ConvArgs &a, hipStream_t st);
chol_status conv_adjoint(chol_dtype dt, const ConvArgs &a, void *ws, hipStream_t st);

} // namespace chol
