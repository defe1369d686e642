// The decode over short selections of a 16-bit cache (decode_rows.cu), used by
// the block-sparse decode.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pkv.h"

namespace pkv {

constexpr int kRowsMaxSeqs = 2048;       // contexts of one launch: 256 sequences of 8 kv heads

// Workspace bytes for `heads` q heads a kv head (0: no device).
size_t rows_workspace_bytes(int heads, int head_dim);

// pkv_decode_attention's contract, for fp16 / bf16 caches; the arguments are
// the caller's to check but for sizes of one launch.
pkv_status decode_rows(const pkv_cache_desc *cache, const void *q, int S, int Hq, const void *k_pool,
                       const void *v_pool, const int32_t *tables, int M, const int32_t *lens, float scale,
                       void *out, int out_dtype, void *ws, cudaStream_t stream);

}  // namespace pkv
