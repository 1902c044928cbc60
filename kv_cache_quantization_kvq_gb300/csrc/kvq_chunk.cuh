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
    float* part;             // [row][split][C + 4]: y, m, l
    int32_t nsplit, ntiles, cluster;
};

rows::View cache_view(const CacheArgs& x);

// One warp joins the splits' (y, m, l) of query row r of slice o, in split order.
template <int C>
__device__ __forceinline__ void merge_row(const ChunkArgs& A, int64_t o, int r, const float* p, int lane) {
    using namespace rows;
    float M = -INFINITY;
    for (int s = lane; s < A.nsplit; s += 32) M = fmaxf(M, p[(int64_t)s * (C + 4) + C]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, x));
    constexpr int N = C / 32;
    float L = 0.0f, v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    if (M != -INFINITY) {
#pragma unroll 4
        for (int s = 0; s < A.nsplit; ++s) {
            const float* ps = p + (int64_t)s * (C + 4);
            const float2 ml = *reinterpret_cast<const float2*>(ps + C);
            const float f = ex2(__fsub_rn(ml.x, M));
            L = __fmaf_rn(ml.y, f, L);
            float x[N];
            if constexpr (N == 4) {
                const float4 t = *reinterpret_cast<const float4*>(ps + 4 * lane);
                x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
            } else {
                const float2 t = *reinterpret_cast<const float2*>(ps + 2 * lane);
                x[0] = t.x; x[1] = t.y;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __fmaf_rn(x[i], f, v[i]);
        }
    }
    const int64_t at = row_index(A.v, o, r);
    const float inv = L > 0.0f ? __fdiv_rn(1.0f, L) : 0.0f;
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2(__fmul_rn(v[2 * i], inv), __fmul_rn(v[2 * i + 1], inv));
    if constexpr (N == 4) *reinterpret_cast<uint2*>(A.out + at * C + 4 * lane) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(A.out + at * C + 2 * lane) = w[0];
    if (A.lse && lane == 0)
        A.lse[at] = L > 0.0f ? __fmul_rn(__fadd_rn(M, log2f(L)), 0.6931471805599453f) : -INFINITY;
}

bool chunk_uses_tc(int64_t rows);
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
