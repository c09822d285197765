// Work list and constants of the AdamW step (adamw.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/libchol.h"

namespace chol {

constexpr int ADAMW_TILE = 256;            // elements that share a scale of an 8-bit state
constexpr int ADAMW_CHUNK = 4096;          // elements of a table entry, 16 workgroups of a tile each

// A piece of one tensor, stepped by ADAMW_CHUNK / ADAMW_TILE workgroups of one wave; the
// device table is an array of these.
struct AdamwChunk {
    void *p;
    const void *g;
    void *m, *v;
    float *master, *m_scale, *v_scale;
    uint32_t n, first;                     // elements; position of the first one in the random sequence
};
static_assert(sizeof(AdamwChunk) == 64, "one cache line's half");

struct AdamwHyper {
    float beta1, one_beta1, beta2, one_beta2; // beta and 1 - beta
    float decay;                              // lr * weight_decay
    float rate;                               // lr / (1 - beta1^step)
    float inv_root;                           // (1 - beta2^step)^(-1/2)
    float eps;
    const float *grad_scale;                  // NULL: 1
    uint32_t key;                             // mixed seed
};

uint32_t adamw_mix(uint32_t x);
chol_status adamw(chol_dtype dt, int bits, bool master, int64_t chunks, const AdamwChunk *table, const AdamwHyper &k,
                  hipStream_t st);

} // namespace chol
