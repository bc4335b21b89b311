// cache.cuh -- layout of the paged, block-quantized key/value cache.
//
// A cache is n_pages pages of P tokens.  A page holds, for each of H heads, one chunk: [P][D] codes
// (Q8_0: int8; Q4_0: [P][D/2] bytes, byte 16b + j holding element 32b + j in its low nibble and element
// 32b + j + 16 in its high nibble) and then [P][D/32] fp16 scales.  So the tokens of a page that one
// head's attention reads are one contiguous piece of memory, codes and scales each contiguous by
// token.  P is a power of two from 16 to 256, so every piece is a multiple of 16 bytes.
#pragma once

#include "qmm_internal.cuh"

namespace qmm {

__host__ __device__ __forceinline__ int cache_code_bytes(int type, int D) { return type == QMM_Q8_0 ? D : D / 2; }
__host__ __device__ __forceinline__ int cache_token_bytes(int type, int D) { return cache_code_bytes(type, D) + D / 32 * 2; }

// Where head h's chunk of a page starts.
__host__ __device__ __forceinline__ int64_t cache_chunk(int type, int H, int D, int P, int64_t page, int h) {
    return (page * H + h) * ((int64_t)P * cache_token_bytes(type, D));
}

}  // namespace qmm
