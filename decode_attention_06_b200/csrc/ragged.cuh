// ragged.cuh -- ragged batches of new tokens: rows q_starts[b] .. q_starts[b + 1] of the
// call's row tensors belong to sequence b and are the last of its seqlens[b] cached tokens.
#pragma once

#include "common.cuh"

namespace gqla {

// New tokens n, cached tokens L and first row of a sequence; n = 0 for a sequence without
// new tokens and for one whose numbers are inconsistent (`bad`).
struct RaggedSeq {
    int n, L;
    int64_t q0;
    bool bad;
};

__device__ __forceinline__ RaggedSeq ragged_seq(const int32_t *q_starts, const int32_t *seqlens, int b,
                                                int64_t total, int max_pages) {
    const int a = q_starts[b], e = q_starts[b + 1], L = seqlens[b];
    RaggedSeq s;
    s.bad = a < 0 || e < a || (int64_t)e > total || (e > a && L < e - a) || (int64_t)L > (int64_t)max_pages * kPage;
    s.n = s.bad ? 0 : e - a;
    s.L = L;
    s.q0 = a;
    return s;
}

}  // namespace gqla
