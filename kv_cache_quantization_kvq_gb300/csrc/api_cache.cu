// api_cache.cu -- the extern "C" entry points declared in include/kvq_cache.h.
//
// As in api.cu, every argument is validated on the host before anything is
// launched; a rejected call has no side effect, and the workspace queries
// never touch the CUDA runtime.
#include <algorithm>

#include "kvq_cache.h"
#include "kvq_internal.h"

namespace {

#define KVQ_FAIL(status, ...) return (kvq::set_last_error(__VA_ARGS__), (status))

constexpr int64_t kMaxElems = int64_t(1) << 50;  // keeps every index product in int64
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 256;       // token and query row numbers are 32-bit

bool mul_ok(int64_t a, int64_t b, int64_t c = 1)
{
    if (a == 0 || b == 0 || c == 0) return true;
    return a <= kMaxElems / b && a * b <= kMaxElems / c;
}

kvq_status need(const void* p, bool used, size_t align, const char* name)
{
    if (!used) return KVQ_OK;
    if (!p) KVQ_FAIL(KVQ_EINVAL, "%s must not be NULL", name);
    if ((uintptr_t)p % align != 0) KVQ_FAIL(KVQ_EINVAL, "%s must be %zu-byte aligned", name, align);
    return KVQ_OK;
}

kvq_status cuda_result(cudaError_t e, const char* what)
{
    if (e == cudaSuccess) return KVQ_OK;
    KVQ_FAIL(KVQ_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

// A store's format: as validate_format, over all T_cap tokens.
kvq_status store_format(const kvq_shape* shape, const kvq_qparams* p, kvq::QSpec& q)
{
    if (!p) KVQ_FAIL(KVQ_EINVAL, "qparams must not be NULL");
    kvq_qparams sp = *p;
    sp.residual = 0;
    return kvq::validate_format(shape, KVQ_BF16, &sp, q);
}

// What the attention calls need of one format.
kvq_status attend_format(const kvq::QSpec& q, int64_t group, bool keys)
{
    const char* who = keys ? "K" : "V";
    if (q.bits != 2 && q.bits != 4) KVQ_FAIL(KVQ_EUNSUPPORTED, "the streaming attention reads 2- and 4-bit codes (%s has %d)", who, q.bits);
    if (q.scale_dt != KVQ_BF16 || (q.mode == KVQ_ASYM && q.zero_dt != KVQ_BF16))
        KVQ_FAIL(KVQ_EUNSUPPORTED, "the streaming attention needs bf16 scales and zero points (%s)", who);
    if (keys) {
        if (q.axis != KVQ_GROUP_ALONG_T || group < 32 || group % 32 != 0)
            KVQ_FAIL(KVQ_EUNSUPPORTED, "the streaming attention needs K groups along T of a multiple of 32 tokens (got %lld, axis %d)",
                     (long long)group, q.axis);
        if (group > kMaxTokens) KVQ_FAIL(KVQ_EUNSUPPORTED, "K group too long");
    } else if (q.axis != KVQ_GROUP_ALONG_C || (q.g != 32 && q.g != 64 && q.g != 128) || q.C % q.g != 0) {
        KVQ_FAIL(KVQ_EUNSUPPORTED, "the streaming attention needs V groups along C of 32, 64 or 128 channels (got %lld, axis %d)",
                 (long long)q.g, q.axis);
    }
    return KVQ_OK;
}

// The counters of a cache over its shape.
kvq_status counters(const kvq_cache* c, const kvq_shape* shape)
{
    if (c->tq < 0 || c->tq > shape->T)
        KVQ_FAIL(KVQ_EINVAL, "tq (%lld) must be in [0, T_cap = %lld]", (long long)c->tq, (long long)shape->T);
    if (c->resid_rows < 0 || c->nres < 0 || c->nres > c->resid_rows)
        KVQ_FAIL(KVQ_EINVAL, "nres (%lld) must be in [0, resid_rows = %lld]", (long long)c->nres, (long long)c->resid_rows);
    if (!mul_ok(shape->outer, c->resid_rows, std::max<int64_t>(shape->C, 1))) KVQ_FAIL(KVQ_EINVAL, "buffer too large");
    if (c->tq > kMaxTokens || c->nres > kMaxTokens - c->tq) KVQ_FAIL(KVQ_EUNSUPPORTED, "a cache of 2^31 tokens or more");
    return KVQ_OK;
}

kvq_status queries(const kvq_shape* shape, int64_t n, int64_t group)
{
    if (!shape) KVQ_FAIL(KVQ_EINVAL, "shape must not be NULL");
    if (shape->outer < 0 || shape->T < 0 || shape->C < 0) KVQ_FAIL(KVQ_EINVAL, "negative extent");
    if (!mul_ok(shape->outer, shape->T, shape->C)) KVQ_FAIL(KVQ_EINVAL, "tensor too large");
    if (shape->C != 64 && shape->C != 128)
        KVQ_FAIL(KVQ_EUNSUPPORTED, "the streaming attention supports head_dim 64 and 128 (got %lld)", (long long)shape->C);
    if (n < 0) KVQ_FAIL(KVQ_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
    if (group < 1) KVQ_FAIL(KVQ_EINVAL, "group must be >= 1 (got %lld)", (long long)group);
    if (group > 64) KVQ_FAIL(KVQ_EUNSUPPORTED, "the streaming attention supports up to 64 query heads per KV head (got %lld)", (long long)group);
    if (n > kMaxTokens / group) KVQ_FAIL(KVQ_EUNSUPPORTED, "too many queries (%lld)", (long long)n);
    if (!mul_ok(shape->outer, n * group, shape->C)) KVQ_FAIL(KVQ_EINVAL, "q too large");
    return KVQ_OK;
}

// Everything the two attention calls have in common.
kvq_status attend_args(const void* q, int64_t n, int64_t group, int64_t kv_heads, const kvq_cache* c,
                       const kvq_qparams* kp, const kvq_qparams* vp, bool values, const kvq_shape* shape,
                       kvq::CacheArgs& a)
{
    if (!c) KVQ_FAIL(KVQ_EINVAL, "cache must not be NULL");
    kvq_status s = queries(shape, n, group);
    if (s != KVQ_OK) return s;
    kvq::QSpec k, v = {};
    if ((s = store_format(shape, kp, k)) || (s = attend_format(k, kp->group, true))) return s;
    if (values) {
        if ((s = store_format(shape, vp, v)) || (s = attend_format(v, v.g, false))) return s;
        if (v.bits != k.bits) KVQ_FAIL(KVQ_EUNSUPPORTED, "the streaming attention needs K and V of the same bit width");
    }
    if (kv_heads < 1 || kv_heads > kMaxTokens || shape->outer % kv_heads != 0)
        KVQ_FAIL(KVQ_EINVAL, "kv_heads (%lld) must divide outer (%lld)", (long long)kv_heads, (long long)shape->outer);
    if ((s = counters(c, shape))) return s;
    const bool st = shape->outer > 0 && c->tq > 0, bu = shape->outer > 0 && c->nres > 0;
    if ((s = need(q, shape->outer > 0 && n > 0, 16, "q")) || (s = need(c->k_codes, st, 16, "k_codes")) ||
        (s = need(c->k_scale, st, 16, "k_scale")) || (s = need(c->k_zero, st && k.mode == KVQ_ASYM, 16, "k_zero")) ||
        (s = need(c->k_resid, bu, 16, "k_resid")))
        return s;
    if (values && ((s = need(c->v_codes, st, 16, "v_codes")) || (s = need(c->v_scale, st, 2, "v_scale")) ||
                   (s = need(c->v_zero, st && v.mode == KVQ_ASYM, 2, "v_zero")) || (s = need(c->v_resid, bu, 16, "v_resid"))))
        return s;
    if ((s = need(c->first, c->first != nullptr, 4, "first"))) return s;
    a = kvq::CacheArgs{};
    a.q = q;
    a.k_codes = c->k_codes;
    a.k_scale = c->k_scale;
    a.k_zero = c->k_zero;
    a.k_resid = c->k_resid;
    a.v_codes = c->v_codes;
    a.v_scale = c->v_scale;
    a.v_zero = c->v_zero;
    a.v_resid = c->v_resid;
    a.first = c->first;
    a.outer = shape->outer;
    a.cap = shape->T;
    a.C = shape->C;
    a.tq = c->tq;
    a.nres = c->nres;
    a.rrows = c->resid_rows;
    a.n = n;
    a.group = group;
    a.kv_heads = kv_heads;
    a.bits = k.bits;
    a.gk = (int32_t)kp->group;
    a.gv = values ? (int32_t)v.g : 0;
    a.k_asym = k.mode == KVQ_ASYM;
    a.v_asym = values && v.mode == KVQ_ASYM;
    a.k_signed = k.is_signed;
    a.v_signed = values && v.is_signed;
    return KVQ_OK;
}

kvq_status workspace_args(const kvq_shape* shape, int64_t resid_rows, int64_t n, int64_t group, size_t* workspace_B)
{
    kvq_status s = queries(shape, n, group);
    if (s != KVQ_OK) return s;
    if (!workspace_B) KVQ_FAIL(KVQ_EINVAL, "workspace_B must not be NULL");
    if (resid_rows < 0 || resid_rows > kMaxTokens || shape->T > kMaxTokens) KVQ_FAIL(KVQ_EINVAL, "bad resid_rows or T_cap");
    return KVQ_OK;
}

kvq_status check_workspace(const void* ws, size_t have, size_t want, size_t align, const char* who)
{
    if (want && (!ws || have < want)) KVQ_FAIL(KVQ_EWORKSPACE, "%s needs %zu workspace bytes (got %zu)", who, want, have);
    return need(ws, want > 0, align, "workspace");
}

bool partly_overlap(const void* a, const void* b, size_t bytes)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x != y && (x < y ? y - x : x - y) < bytes;
}

}  // namespace

extern "C" {

kvq_status kvq_attend_chunk_workspace(const kvq_shape* shape, int64_t resid_rows, int64_t n, int64_t group,
                                      size_t* workspace_B)
{
    kvq_status s = workspace_args(shape, resid_rows, n, group, workspace_B);
    if (s != KVQ_OK) return s;
    *workspace_B = kvq::chunk_workspace(shape->outer, shape->C, shape->T + resid_rows, n, group);
    return KVQ_OK;
}

kvq_status kvq_attend_chunk(const void* q, int64_t n, int64_t group, int64_t kv_heads, const kvq_cache* cache,
                            const kvq_qparams* k_params, const kvq_qparams* v_params, const kvq_shape* shape,
                            void* out, float* lse, void* workspace, size_t workspace_B, void* stream)
{
    kvq::CacheArgs a;
    kvq_status s = attend_args(q, n, group, kv_heads, cache, k_params, v_params, true, shape, a);
    if (s != KVQ_OK) return s;
    if ((s = need(out, shape->outer > 0 && n > 0, 16, "out")) || (s = need(lse, lse != nullptr, 4, "lse"))) return s;
    // in place each row is read before it is written; shifted, another row's query would be gone
    if (a.outer > 0 && n > 0 && partly_overlap(q, out, (size_t)(a.outer * n * group * a.C) * 2))
        KVQ_FAIL(KVQ_EINVAL, "q and out overlap without being the same buffer");
    const size_t want = kvq::chunk_workspace(a.outer, a.C, a.cap + a.rrows, n, group);
    if ((s = check_workspace(workspace, workspace_B, want, 256, "kvq_attend_chunk"))) return s;
    return cuda_result(kvq::launch_attend_chunk(a, out, lse, workspace, (cudaStream_t)stream), "kvq_attend_chunk launch");
}

kvq_status kvq_attend_weights_workspace(const kvq_shape* shape, int64_t resid_rows, int64_t n, int64_t group,
                                        size_t* workspace_B)
{
    kvq_status s = workspace_args(shape, resid_rows, n, group, workspace_B);
    if (s != KVQ_OK) return s;
    *workspace_B = kvq::weights_workspace(shape->outer, shape->C, n, group);
    return KVQ_OK;
}

kvq_status kvq_attend_weights(const void* q, const float* lse, int64_t n, int64_t group, int64_t kv_heads,
                              const kvq_cache* cache, const kvq_qparams* k_params, const kvq_shape* shape,
                              const float* scores_in, float* scores_out, int64_t score_stride, void* workspace,
                              size_t workspace_B, void* stream)
{
    kvq::CacheArgs a;
    kvq_status s = attend_args(q, n, group, kv_heads, cache, k_params, nullptr, false, shape, a);
    if (s != KVQ_OK) return s;
    const int64_t T = a.tq + a.nres;
    if (score_stride < T) KVQ_FAIL(KVQ_EINVAL, "score_stride (%lld) must hold the cache's %lld tokens", (long long)score_stride, (long long)T);
    if (!mul_ok(a.outer, score_stride)) KVQ_FAIL(KVQ_EINVAL, "scores too large");
    const bool any = a.outer > 0 && T > 0;
    if ((s = need(lse, any && n > 0, 4, "lse")) || (s = need(scores_out, any, 4, "scores_out")) ||
        (s = need(scores_in, scores_in != nullptr, 4, "scores_in")))
        return s;
    if (any && scores_in && partly_overlap(scores_in, scores_out, ((a.outer - 1) * score_stride + T) * sizeof(float)))
        KVQ_FAIL(KVQ_EINVAL, "scores_in and scores_out overlap without being the same buffer");
    const size_t want = kvq::weights_workspace(a.outer, a.C, n, group);
    if ((s = check_workspace(workspace, workspace_B, want, 256, "kvq_attend_weights"))) return s;
    return cuda_result(kvq::launch_attend_weights(a, lse, scores_in, scores_out, score_stride, workspace,
                                                  (cudaStream_t)stream),
                       "kvq_attend_weights launch");
}

kvq_status kvq_evict_blocks_workspace(const kvq_shape* shape, int64_t block, size_t* workspace_B)
{
    if (!shape || !workspace_B) KVQ_FAIL(KVQ_EINVAL, "shape and workspace_B must not be NULL");
    if (shape->outer < 0 || shape->T < 0 || !mul_ok(shape->outer, shape->T)) KVQ_FAIL(KVQ_EINVAL, "bad extents");
    if (block < 1) KVQ_FAIL(KVQ_EINVAL, "block must be >= 1 (got %lld)", (long long)block);
    *workspace_B = kvq::evict_workspace(shape->outer, shape->T / block);
    return KVQ_OK;
}

kvq_status kvq_evict_blocks(const kvq_cache* src, kvq_cache* dst, const kvq_qparams* k_params,
                            const kvq_qparams* v_params, const kvq_shape* shape, int64_t block, int64_t budget,
                            int64_t window, const float* scores_in, float* scores_out, int64_t score_stride,
                            int32_t* keep, void* workspace, size_t workspace_B, void* stream)
{
    if (!src || !dst) KVQ_FAIL(KVQ_EINVAL, "src and dst must not be NULL");
    kvq::QSpec f[2];
    const kvq_qparams* ps[2] = {k_params, v_params};
    kvq_status s;
    if (block < 1) KVQ_FAIL(KVQ_EINVAL, "block must be >= 1 (got %lld)", (long long)block);
    for (int i = 0; i < 2; ++i) {
        if ((s = store_format(shape, ps[i], f[i])) != KVQ_OK) return s;
        if (ps[i]->axis == KVQ_GROUP_ALONG_T && (ps[i]->group <= 0 || block % ps[i]->group != 0))
            KVQ_FAIL(KVQ_EINVAL, "groups along T need block (%lld) to be a multiple of the group (%lld > 0)",
                     (long long)block, (long long)ps[i]->group);
    }
    if ((s = counters(src, shape))) return s;
    // what dst must hold whatever moves: the buffered tokens' rows, and what is left of the padding
    if (dst->resid_rows < src->nres)
        KVQ_FAIL(KVQ_EINVAL, "dst's resid_rows (%lld) must hold the %lld buffered tokens", (long long)dst->resid_rows, (long long)src->nres);
    if (src->first && !dst->first) KVQ_FAIL(KVQ_EINVAL, "dst needs first: the source is padded");
    if (src->tq % block != 0) KVQ_FAIL(KVQ_EINVAL, "tq (%lld) must be a multiple of block (%lld)", (long long)src->tq, (long long)block);
    if (budget < 1) KVQ_FAIL(KVQ_EINVAL, "budget must be >= 1");
    if (window < 0 || window > budget) KVQ_FAIL(KVQ_EINVAL, "window must be in [0, budget]");
    const int64_t outer = shape->outer, T = src->tq + src->nres, nb = src->tq / block, kept = std::min(budget, nb);
    if (outer > kMaxTokens) KVQ_FAIL(KVQ_EUNSUPPORTED, "too many slices");
    if (score_stride < T) KVQ_FAIL(KVQ_EINVAL, "score_stride (%lld) must hold the cache's %lld tokens", (long long)score_stride, (long long)T);
    if (!mul_ok(outer, score_stride)) KVQ_FAIL(KVQ_EINVAL, "scores too large");
    const bool any = outer > 0 && nb > 0, sc = outer > 0 && T > 0;

    kvq::EvictArgs a = {};
    const void* from[2][3] = {{src->k_codes, src->k_scale, src->k_zero}, {src->v_codes, src->v_scale, src->v_zero}};
    void* to[2][3] = {{dst->k_codes, dst->k_scale, dst->k_zero}, {dst->v_codes, dst->v_scale, dst->v_zero}};
    static const char* const names[2][3] = {{"k_codes", "k_scale", "k_zero"}, {"v_codes", "v_scale", "v_zero"}};
    for (int i = 0; i < 2; ++i) {
        const kvq::QSpec& q = f[i];
        const bool along_t = q.axis == KVQ_GROUP_ALONG_T;
        const int64_t units = along_t ? q.ngroups * q.C : shape->T * q.ngroups;      // metadata elements of a slice
        const int64_t block_units = along_t ? block / q.g * q.C : block * q.ngroups;
        for (int m = 0; m < 3; ++m) {
            if (m == 2 && q.mode != KVQ_ASYM) continue;
            const int dt = m == 1 ? q.scale_dt : q.zero_dt;
            const int64_t es = m == 0 ? 1 : dt == KVQ_F32 ? 4 : dt == KVQ_BF16 ? 2 : 1;
            kvq::EvictBuf b;
            b.src = static_cast<const char*>(from[i][m]);
            b.dst = static_cast<char*>(to[i][m]);
            b.slice_B = m == 0 ? shape->T * (q.C * q.bits / 8) : units * es;
            b.block_B = m == 0 ? block * (q.C * q.bits / 8) : block_units * es;
            if ((s = need(b.src, any && b.block_B > 0, (size_t)es, names[i][m])) ||
                (s = need(b.dst, any && b.block_B > 0, (size_t)es, names[i][m])))
                return s;
            if (any && b.block_B > 0 && partly_overlap(b.src, b.dst, (size_t)(outer * b.slice_B)))
                KVQ_FAIL(KVQ_EINVAL, "%s of src and dst overlap without being the same buffer", names[i][m]);
            if (any && b.block_B > 0) a.buf[a.nbuf++] = b;
        }
    }
    if ((s = need(scores_in, sc, 4, "scores_in")) || (s = need(scores_out, sc, 4, "scores_out")) ||
        (s = need(keep, any, 4, "keep")) || (s = need(src->first, src->first != nullptr, 4, "first")) ||
        (s = need(dst->first, dst->first != nullptr, 4, "first")))
        return s;
    if (src->first && partly_overlap(src->first, dst->first, (size_t)outer * sizeof(int32_t)))
        KVQ_FAIL(KVQ_EINVAL, "first of src and dst overlap without being the same buffer");
    if (sc && partly_overlap(scores_in, scores_out, ((outer - 1) * score_stride + T) * sizeof(float)))
        KVQ_FAIL(KVQ_EINVAL, "scores_in and scores_out overlap without being the same buffer");
    const size_t want = kvq::evict_workspace(outer, shape->T / block);
    if ((s = check_workspace(workspace, workspace_B, want, 16, "kvq_evict_blocks"))) return s;
    a.outer = outer;
    a.block = block;
    a.nb = nb;
    a.kept = kept;
    a.window = window;
    a.nres = src->nres;
    a.stride = score_stride;
    a.scores_in = scores_in;
    a.scores_out = scores_out;
    a.first_in = src->first;
    a.first_out = dst->first;
    a.keep = keep;
    a.ws = workspace;
    if (!kvq::evict_fits(a)) KVQ_FAIL(KVQ_EUNSUPPORTED, "blocks of %lld tokens over %lld slices are more than a grid holds", (long long)block, (long long)outer);
    s = cuda_result(kvq::launch_evict(a, (cudaStream_t)stream), "kvq_evict_blocks launch");
    if (s != KVQ_OK) return s;
    dst->nres = src->nres;
    dst->tq = kept * block;
    return KVQ_OK;
}

}  // extern "C"
