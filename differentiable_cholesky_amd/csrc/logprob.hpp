// Launchers of the token log probabilities (logprob.hip).
#pragma once

#include "lowp.hpp"

namespace chol {

struct LogprobArgs {
    int64_t rows, vocab;
    const void *x;
    int64_t ld;
    const int64_t *tokens;
    float scale;
    float *logp, *lse, *entropy; // entropy may be null
    int top;
    float *top_logp;             // [rows, top]
    int64_t *top_ids;
};

struct LogprobAdjArgs {
    int64_t rows, vocab;
    const void *x;
    int64_t ld;
    const int64_t *tokens;
    float scale;
    const float *lse, *entropy, *adj_logp, *adj_entropy; // the last may be null, with entropy
    void *adj;
    int64_t lda;
};

size_t logprob_workspace(chol_dtype dt, int64_t rows, int64_t vocab, int top);
// false where the threads are more than a grid holds
bool logprob_fits(chol_dtype dt, int64_t rows, int64_t vocab);
chol_status logprob(chol_dtype dt, const LogprobArgs &a, void *ws, hipStream_t st);
chol_status logprob_adjoint(chol_dtype dt, const LogprobAdjArgs &a, hipStream_t st);

} // namespace chol
