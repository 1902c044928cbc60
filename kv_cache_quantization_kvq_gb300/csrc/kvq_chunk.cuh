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
    // What each split counts is worked out a split per lane, and the outputs are loaded kJoin splits at a time: as a
    // plain loop over the splits the loads wait for one another (one token of 8 slices x 4 heads over 131263 tokens:
    // 73.3 us with it, 66.6 so).
    constexpr int kJoin = 8;
    for (int s0 = 0; s0 < A.nsplit; s0 += 32) {
        const int n = min(32, A.nsplit - s0);
        const float* ps = p + (int64_t)s0 * (C + 4);
        float l = 0.0f, f = 0.0f;
        if (lane < n) {
            const float2 ml = *reinterpret_cast<const float2*>(ps + (int64_t)lane * (C + 4) + C);
            l = ml.y;
            f = part_scale(ml.x, M);
        }
        for (int i0 = 0; i0 < n; i0 += kJoin) {
            float x[kJoin][N];
#pragma unroll
            for (int i = 0; i < kJoin; ++i) {
#pragma unroll
                for (int k = 0; k < N; ++k) x[i][k] = 0.0f;
                if (i0 + i >= n) continue;
                const float* py = ps + (int64_t)(i0 + i) * (C + 4) + N * lane;
                if constexpr (N == 4) {
                    const float4 t = *reinterpret_cast<const float4*>(py);
                    x[i][0] = t.x; x[i][1] = t.y; x[i][2] = t.z; x[i][3] = t.w;
                } else {
                    const float2 t = *reinterpret_cast<const float2*>(py);
                    x[i][0] = t.x; x[i][1] = t.y;
                }
            }
#pragma unroll
            for (int i = 0; i < kJoin; ++i) {    // splits past the last: all zeros
                const float fi = __shfl_sync(0xFFFFFFFFu, f, i0 + i);
                L = __fmaf_rn(__shfl_sync(0xFFFFFFFFu, l, i0 + i), fi, L);
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] = __fmaf_rn(x[i][k], fi, v[k]);
            }
        }
    }
    const int64_t at = row_index(A.v, o, r);
    const float inv = row_scale(L);
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2(row_value(v[2 * i], inv), row_value(v[2 * i + 1], inv));
    if constexpr (N == 4) *reinterpret_cast<uint2*>(A.out + at * C + 4 * lane) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(A.out + at * C + 2 * lane) = w[0];
    if (A.lse && lane == 0)
        A.lse[at] = row_lse(M, L);
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
