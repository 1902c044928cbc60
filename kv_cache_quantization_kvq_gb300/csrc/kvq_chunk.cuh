// kvq_chunk.cuh -- what the two forms of kvq_attend_chunk (chunk.cu: few query
// rows; prefill.cu: many) share.
#pragma once

#include <cuda.h>

#include "kvq_rows.cuh"

namespace kvq {

// JOIN in the kernels' templates: the launch is one of several whose results meet,
// and only then are `sums`, `shared` and the rows' own places looked at.
struct ChunkArgs {
    rows::View v;
    __nv_bfloat16* out;
    float* lse;              // or nullptr
    float* part;             // [row][split][C + 4]: y, m, l
    float* sums;             // [row_index][C + 4]: the same of whole rows, in place of out and lse; or nullptr
    int32_t nsplit, ntiles, cluster;
    int32_t share;           // batches of a split, or 0: a slice has as many splits as its tokens need, of at most nsplit
    // shared: a launch over tokens that every row sees, to be joined with what the rows
    // have seen elsewhere: own_sums as `sums` holds it, own_part as `part` does (of the rows
    // kernel over `own`, own_nsplit and own_share), or (own_out, own_lse), or nothing
    int32_t shared;
    const float* own_sums;
    const float* own_part;
    rows::View own;
    int32_t own_nsplit, own_share;
    const __nv_bfloat16* own_out;
    const float* own_lse;
};

rows::View cache_view(const CacheArgs& x);

// The visible batches [b0, b0 + len) of slice o, and how many splits of `share` batches they are.
__device__ __forceinline__ int splits_seen(const rows::View& a, int64_t o, int share, int& b0, int& len) {
    const int first = rows::padding(a, o), last = a.T - 1;
    b0 = len = 0;
    if (first <= last) {
        const rows::Span sp = rows::span_of(a);
        b0 = rows::batch_of(a, sp, first);
        len = rows::batch_of(a, sp, last) + 1 - b0;
    }
    return share ? max(1, (len + share - 1) / share) : 1;
}

// One warp takes the largest m of a row's splits, and adds up the splits' y
// (channels N lane + i) and l, scaled to the maximum M of the whole, in split order.
template <int C>
__device__ __forceinline__ float parts_max(const float* p, int nsplit, int lane) {
    float M = -INFINITY;
    for (int s = lane; s < nsplit; s += 32) M = fmaxf(M, p[(int64_t)s * (C + 4) + C]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, x));
    return M;
}
template <int C>
__device__ __forceinline__ void add_parts(const float* p, int nsplit, int lane, float M, float& L, float (&v)[C / 32]) {
    using namespace rows;
    constexpr int N = C / 32;
    // What each split counts is worked out a split per lane, and the outputs are loaded kJoin splits at a time: as a
    // plain loop over the splits the loads wait for one another (one token of 8 slices x 4 heads over 131263 tokens:
    // 73.3 us with it, 66.6 so).
    constexpr int kJoin = 8;
    for (int s0 = 0; s0 < nsplit; s0 += 32) {
        const int n = min(32, nsplit - s0);
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
}
// the row with maximum M and sums L and v: out and lse
template <int C>
__device__ __forceinline__ void write_joined(__nv_bfloat16* out, float* lse, int64_t at, int lane, float M, float L,
                                             const float (&v)[C / 32]) {
    using namespace rows;
    constexpr int N = C / 32;
    const float inv = row_scale(L);
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2(row_value(v[2 * i], inv), row_value(v[2 * i + 1], inv));
    if constexpr (N == 4) *reinterpret_cast<uint2*>(out + at * C + 4 * lane) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(out + at * C + 2 * lane) = w[0];
    if (lse && lane == 0)
        lse[at] = row_lse(M, L);
}

// One warp joins the splits' (y, m, l) of query row r of slice o.
template <int C, bool JOIN>
__device__ __forceinline__ void merge_row(const ChunkArgs& A, int64_t o, int r, const float* p, int lane) {
    constexpr int N = C / 32;
    float M = parts_max<C>(p, A.nsplit, lane), L = 0.0f, v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    const int64_t at = rows::row_index<JOIN>(A.v, o, r);
    if (JOIN && A.own_sums) {
        const float* own = A.own_sums + at * (C + 4);
        M = fmaxf(M, own[C]);
        add_parts<C>(own, 1, lane, M, L, v);
    } else if (JOIN && A.own_part) {
        // row r of KV head o is row r % own.rows of a request's slice
        const int b = r / A.own.rows;
        const int64_t so = (int64_t)b * A.own.kv_heads + o;
        int b0, len;
        const int n = splits_seen(A.own, so, A.own_share, b0, len);
        const float* own = A.own_part + ((so * A.own.rows + (r - b * A.own.rows)) * A.own_nsplit) * (C + 4);
        M = fmaxf(M, parts_max<C>(own, n, lane));
        add_parts<C>(own, n, lane, M, L, v);
    } else if (JOIN && A.own_lse) {
        // weights that sum to 1 at the maximum lse; -inf: nothing was seen, NaN: nothing else comes out
        const float lse = A.own_lse[at], m = __fmul_rn(lse, rows::kLog2e);
        M = fmaxf(M, m);
        if (lse != -INFINITY) {
            const float f = rows::part_scale(m, M);
            L = lse != lse ? lse : f;
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(A.own_out + at * C + N * lane + i);
                v[i] = __fmul_rn(rows::bf_lo(w), f);
                v[i + 1] = __fmul_rn(rows::bf_hi(w), f);
            }
        }
    }
    add_parts<C>(p, A.nsplit, lane, M, L, v);
    if (JOIN && A.sums) {
        float* dst = A.sums + at * (C + 4);
#pragma unroll
        for (int i = 0; i < C / 32; i += 2)
            *reinterpret_cast<float2*>(dst + C / 32 * lane + i) = make_float2(v[i], v[i + 1]);
        if (lane == 0) *reinterpret_cast<float2*>(dst + C) = make_float2(M, L);
    } else {
        write_joined<C>(A.out, A.lse, at, lane, M, L, v);
    }
}

bool chunk_uses_tc(int64_t rows);
size_t chunk_tc_workspace(int64_t outer, int64_t C, int64_t tmax, int64_t rows, bool shared);
cudaError_t launch_attend_tc(const ChunkArgs& A, int bits, int64_t C, int64_t outer, void* ws, cudaStream_t st);

// A launch that starts while the one before it ends; its kernel waits for that one
// itself (griddepcontrol.wait).
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned threads, cudaStream_t st, bool early, const A&... args) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = early ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// The rows kernel (at most 32 rows a slice) over slices that need not be equally long. Its
// results are left in A.part; nsplit and share are returned in A.
size_t rows_parts_workspace(int64_t outer, int64_t C, int64_t tmax, int64_t rows);
cudaError_t launch_rows_parts(ChunkArgs& A, int bits, int64_t C, int64_t outer, cudaStream_t st);
// The attention of kvq_attend_chunk over a cache: its rows into A.out and A.lse, joined with what they
// have seen elsewhere (A.shared), or into A.sums (tensor-core forms alone).
cudaError_t launch_chunk(ChunkArgs A, int bits, int64_t C, int64_t outer, void* ws, cudaStream_t st);

// Rows that all see every token on pairs of SMs (prefix.cu), and the launch that
// joins the splits of part [slice][row][split] (chunk.cu).
bool prefix_uses_pairs(int64_t C, int64_t rows);
size_t prefix_workspace(int64_t outer, int64_t tmax, int64_t rows);
cudaError_t launch_attend_prefix(ChunkArgs A, int bits, int64_t outer, void* ws, cudaStream_t st);
cudaError_t launch_merge_rows(const ChunkArgs& A, int64_t C, int64_t outer, cudaStream_t st);

// the same for kvq_attend_weights (weights_tc.cu)
bool weights_use_tc(int64_t rows);
size_t weights_tc_workspace(int64_t outer, int64_t C, int64_t rows);
cudaError_t launch_weights_tc(const rows::View& v, const float* lse, const float* in, float* out, int64_t stride,
                              int bits, int64_t C, int64_t outer, void* ws, cudaStream_t st);

// [rows, C] bf16 as boxes of 64 channels x 128 rows, 128-byte swizzle (prefill.cu)
bool encode_rows_tile_map(const void* x, int64_t rows, int64_t C, CUtensorMap* map);

}  // namespace kvq
