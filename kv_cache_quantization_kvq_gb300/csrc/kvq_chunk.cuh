// kvq_chunk.cuh -- what the two forms of kvq_attend_chunk (chunk.cu: few query
// rows; prefill.cu: many) share.
#pragma once

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

}  // namespace kvq
