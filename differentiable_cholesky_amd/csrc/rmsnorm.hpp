// Arguments of the RMS norm and its adjoint (rmsnorm.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/libchol.h"

namespace chol {

struct NormArgs {
    int64_t rows, cols;
    const void *x, *residual, *w; // residual may be NULL
    int64_t ldx, ldr;
    float eps;
    void *y;                      // same type, or e4m3 codes
    int64_t ldy;
    void *h;                      // x + residual, rounded; not written without a residual
    int64_t ldh;
    float *scale;                 // e4m3 only
    int64_t lds;
    int group;                    // columns that share a scale, 0: the row
};

struct NormAdjArgs {
    int64_t rows, cols;
    const void *h, *w, *adj, *adj_h; // adj_h may be NULL
    int64_t ldh, lda, ldah;
    float eps;
    void *adj_x;
    int64_t ldax;
    float *adj_w;
    int accumulate;
};

chol_status rmsnorm(chol_dtype dt, bool quantise, const NormArgs &a, hipStream_t st);
size_t rmsnorm_adjoint_workspace(chol_dtype dt, int64_t rows, int64_t cols);
chol_status rmsnorm_adjoint(chol_dtype dt, const NormAdjArgs &a, void *ws, hipStream_t st);

} // namespace chol
