// What the kernels of drafted tokens share: a sequence's length, its drafted
// tokens' rows, and their checks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pkv_tree.h"

namespace pkv {

struct TreeBatch {
    const int32_t *offs, *lens;
    int T, N;                // rows, drafted tokens of a sequence at most
    int M, lb, cap;          // table columns, block size 1 << lb, tokens of a row
    unsigned *err;
};

// n drafted tokens at rows o.. of a context of L; a sequence left out has n 0.
struct TreeSeq {
    int L, n, o;
    int raw;                 // the length as it was given
    bool ok;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeBatch &b, int s, bool tell) {
    TreeSeq q;
    q.raw = q.L = __ldg(b.lens + s);
    q.o = __ldg(b.offs + s);
    const int e = __ldg(b.offs + s + 1);
    unsigned bad = 0;
    if (q.L < 0 || q.L > b.cap) bad = PKV_DEVERR_CONTEXT;
    if (q.o < 0 || e < q.o || e > b.T || e - q.o > b.N || (!bad && e - q.o > q.L)) bad |= PKV_DEVERR_TOKENS;
    q.n = e - q.o;
    q.ok = bad == 0;
    if (bad) {
        if (tell) atomicOr(b.err, bad);
        q.n = q.L = q.o = 0;
    }
    return q;
}

}  // namespace pkv
