// kvq_chunk.cuh -- what the two forms of kvq_attend_chunk (chunk.cu: few query
// rows; prefill.cu: many) share.
#pragma once

#include <cuda.h>

#include "kvq_rows.cuh"

namespace kvq {

struct ChunkArgs {
    rows::View v;
    __nv_bfloat16* out;
    float* lse;              // or nullptr
    float* part;             // [outer][row][split][C + 4]: y, m, l
    int32_t nsplit, ntiles;
};

rows::View cache_view(const CacheArgs& x);

// out and lse from the splits' partial results, in split order
void launch_merge_rows(const ChunkArgs& A, int64_t outer, int64_t C, cudaStream_t st);

bool chunk_uses_tc(int64_t T, int64_t rows);
size_t chunk_tc_workspace(int64_t outer, int64_t C, int64_t tmax, int64_t rows);
cudaError_t launch_attend_tc(const ChunkArgs& A, int bits, int64_t C, int64_t outer, void* ws, cudaStream_t st);

// the same for kvq_attend_weights (weights_tc.cu)
bool weights_use_tc(int64_t rows);
size_t weights_tc_workspace(int64_t outer, int64_t C, int64_t rows);
cudaError_t launch_weights_tc(const rows::View& v, const float* lse, const float* in, float* out, int64_t stride,
                              int bits, int64_t C, int64_t outer, void* ws, cudaStream_t st);

// [rows, C] bf16 as boxes of 64 channels x 128 rows, 128-byte swizzle (prefill.cu)
bool encode_rows_tile_map(const void* x, int64_t rows, int64_t C, CUtensorMap* map);

}  // namespace kvq
