// shared.cu -- attention of a batch over a quantized prefix that all its requests
// share (kvq_attend_shared).
//
// "KV cache 压缩：把历史装得更小" §"让 kernel 接住收益" (the attention kernel reads the
// low-bit cache).  Softmax over the union of two token sets A and B needs each
// set's maximum m, sum l and weighted values y only (the online softmax): with
// M = max(m_A, m_B), l = l_A 2^(m_A - M) + l_B 2^(m_B - M), y alike, out = y / l.
// So the prefix is one launch of the streaming attention (chunk.cu, prefill.cu)
// in which a KV head's rows are the query rows of all requests, batch x n x group
// of them, that see every token: its codes are read, and unpacked, once for all.
// The requests' own tokens are another launch over their caches, which leaves
// (y, m, l) in float32, and the launch that joins the prefix's splits joins that too.
// The prefix's launch starts while the last CTAs of that one run: it reads nothing of theirs.
//
// Measured on one GB300: 64 requests of 50 to 1500 tokens, 8 KV heads x 8, behind a prefix of 8192 tokens 63 us, of which
// 28 are their own tokens'; reading the prefix once for each request, as kvq_attend_chunk would, has 64 times its bytes.
#include "kvq_chunk.cuh"

namespace kvq {

namespace {

size_t padded(size_t b) { return (b + 255) / 256 * 256; }

// The workspace: the own rows' sums, then what each launch needs.
struct SharedPlan { size_t sums, own, prefix; };

SharedPlan shared_plan(int64_t prefix_tmax, int64_t own_tmax, bool own, int64_t C, int64_t batch, int64_t n, int64_t group,
                       int64_t kv_heads)
{
    SharedPlan p = {0, 0, 0};
    if (own) {
        const int64_t outer = batch * kv_heads, rows = n * group;
        if (chunk_uses_tc(rows)) {
            p.sums = padded((size_t)(outer * rows * (C + 4)) * sizeof(float));
            p.own = padded(chunk_workspace(outer, C, own_tmax, n, group));
        } else {
            p.own = padded(rows_parts_workspace(outer, C, own_tmax, rows));
        }
    }
    p.prefix = prefix_uses_pairs(C, batch * n * group) ? prefix_workspace(kv_heads, prefix_tmax, batch * n * group)
                                                       : chunk_workspace(kv_heads, C, prefix_tmax, batch * n, group, true);
    return p;
}

}  // namespace

size_t shared_workspace(int64_t prefix_tmax, int64_t own_tmax, bool own, int64_t C, int64_t batch, int64_t n, int64_t group,
                        int64_t kv_heads)
{
    if (batch == 0 || n == 0) return 0;
    const SharedPlan p = shared_plan(prefix_tmax, own_tmax, own, C, batch, n, group, kv_heads);
    return p.sums + p.own + p.prefix;
}

cudaError_t launch_attend_shared(const CacheArgs& prefix, const CacheArgs* own, const void* own_out, const float* own_lse,
                                 int64_t batch, int64_t n, void* out, float* lse, void* ws, cudaStream_t st)
{
    if (batch == 0 || n == 0) return cudaSuccess;
    const SharedPlan p = shared_plan(prefix.cap + prefix.rrows, own ? own->cap + own->rrows : 0, own != nullptr, prefix.C,
                                     batch, n, prefix.group, prefix.kv_heads);
    unsigned char* w = static_cast<unsigned char*>(ws);
    ChunkArgs A = {};
    if (own) {
        ChunkArgs B = {};
        B.v = A.own = cache_view(*own);
        cudaError_t e;
        if (chunk_uses_tc(B.v.rows)) {
            B.sums = reinterpret_cast<float*>(w);
            e = launch_chunk(B, own->bits, own->C, own->outer, w + p.sums, st);
            A.own_sums = B.sums;
        } else {
            B.part = reinterpret_cast<float*>(w);
            e = launch_rows_parts(B, own->bits, own->C, own->outer, st);
            A.own_part = B.part;
            A.own_nsplit = B.nsplit;
            A.own_share = B.share;
        }
        if (e != cudaSuccess) return e;
    } else {
        A.own_out = static_cast<const __nv_bfloat16*>(own_out);
        A.own_lse = own_lse;
    }
    A.v = cache_view(prefix);
    A.v.n = 1;                       // every row sees every token
    A.v.group = A.v.rows;
    A.out = static_cast<__nv_bfloat16*>(out);
    A.lse = lse;
    A.shared = 1;
    w += p.sums + p.own;
    if (prefix_uses_pairs(prefix.C, A.v.rows)) return launch_attend_prefix(A, prefix.bits, prefix.outer, w, st);
    return launch_chunk(A, prefix.bits, prefix.C, prefix.outer, w, st);
}

}  // namespace kvq
