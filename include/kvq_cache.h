/*
 * kvq_cache.h -- C ABI of the streaming quantized cache: attention over it for
 * any number of new tokens, the attention weight it gives every token, and
 * eviction from it by accumulated weight; and what serving a batch of requests
 * needs beside it: attention over packed prompts, filling a cache from them, and
 * attention over a prefix that the requests share.
 *
 * The first three calls work on the cache that kvq_append_kv fills (kvq.h): a store
 * of quantized tokens and a bf16 buffer of the newest ones.  A serving loop
 * runs them in this order, per layer and step:
 *     kvq_append_kv        the new tokens' K and V enter the cache;
 *     kvq_attend_chunk     their queries attend to it;
 *     kvq_attend_weights   the weight given to every token is accumulated;
 *     kvq_evict_blocks     now and then, the blocks with the least weight go.
 * A batch of prompts of different lengths comes before that loop, per layer:
 *     kvq_attend_prompts   their causal attention, packed, from bf16 K and V;
 *     kvq_fill_prompts     their K and V become the cache's first tokens.
 * Where the requests share a prefix (a system prompt, a document), it is a cache
 * of its own, of kv_heads slices, and kvq_attend_shared takes kvq_attend_chunk's
 * place in the loop, and follows kvq_attend_prompts, joining its results.
 *
 * Sources, cited by page title and section:
 *  [KVC] "KV cache 压缩：把历史装得更小": §"让 kernel 接住收益" (the attention
 *        kernel reads the low-bit cache), §"K 的误差会改变权重，V 的误差会改变内容"
 *        (logit_t = q^T k_t / sqrt(d), y = sum_t a_t v_t), §"少存 token：合并，或淘汰"
 *        (eviction frees the dropped K/V).
 *  [FtC] "KV Compression 公式到源码对照": §3.1 cumulative attention score,
 *        §3.2 recent window union heavy hitters; §1.1 and §1.2 scales, zero points
 *        and codes.
 *
 * The conventions of kvq.h hold: device buffers owned by the caller, work
 * enqueued on `stream` of the current device, arguments checked on the host
 * before anything is launched, no allocation and no synchronisation.  A
 * workspace must not be shared by calls that may overlap on the GPU, two
 * captured graphs among them.  The counters tq and nres are read on the host
 * when the call is made: a captured call replays with the counters it was
 * captured with.
 */
#ifndef KVQ_CACHE_H
#define KVQ_CACHE_H

#include "kvq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One layer's streaming cache, read on the host during a call.
 *  - k_* / v_*: the store of each cache, laid out as kvq_quantize lays out a
 *    [outer, T_cap, C] tensor without residual (shape = {outer, T_cap, C} is
 *    passed beside this struct), and the bf16 buffer [outer][resid_rows][C].
 *  - tq: filled tokens of the store, 0 <= tq <= T_cap; nres: filled rows of
 *    the buffer, 0 <= nres <= resid_rows.  The cache holds T = tq + nres
 *    tokens in this order: token t < tq is store token t, the others are
 *    buffer rows t - tq.
 *    A cache written by one kvq_quantize call has T_cap = tq = Tq and
 *    resid_rows = nres = min(R, T).
 *  - first: device int32 [outer], or NULL for zeros: slice o's tokens before
 *    first[o] are left padding.  They are never seen, whatever they hold
 *    (NaN included); first[o] <= 0 hides nothing, first[o] >= T everything.
 * What lies behind the filled tokens of the store and of the buffer is never
 * used, whatever it holds. */
typedef struct {
    void *k_codes, *k_scale, *k_zero, *k_resid;
    void *v_codes, *v_scale, *v_zero, *v_resid;
    int64_t tq, nres, resid_rows;
    int32_t* first;
} kvq_cache;

/* Causal attention of n queries over the cache; query i is the token at
 * position T - n + i, so the last query sees every token ([KVC] logit and
 * output formulas; grouped-query attention: `group` query heads read a KV
 * slice).  outer = batch * kv_heads, slice o = b * kv_heads + h, C = head_dim:
 *     seen(o, i)  = { t : first[o] <= t <= T - n + i }
 *     lse[b][i][h*group+j]    = log sum_{t in seen} exp(q . k_t / sqrt(C))
 *     out[b][i][h*group+j][:] = sum_{t in seen} exp(q . k_t / sqrt(C) - lse) v_t
 * with q = q[b][i][h*group+j][:] and k_t, v_t the bf16 rows that
 * kvq_dequantize returns, s * (code - zero_point) rounded once to bf16, and
 * the buffer's rows as they are.  A query that sees nothing (T = 0, n > T, or
 * padding), or only logits of -inf, gets out = 0 and lse = -inf; one that sees
 * a logit of NaN or +inf gets NaN in all of out and in lse.
 * An infinity or NaN in v_t reaches its channel of the queries that see token t,
 * and no other query.  n = 0 does nothing.
 *  - q: bf16 [outer/kv_heads][n][kv_heads*group][C]; out: bf16, same shape, may
 *    be q itself and must not overlap it otherwise; lse: float32
 *    [outer/kv_heads][n][kv_heads*group], or NULL.
 *  - Logits, softmax statistics and sums are float32; the probabilities enter
 *    the value product in bf16 (relative error 2^-8 at most), out is rounded
 *    once more.  The sums are divided at the end and may carry 2^8 more than the
 *    weights, so 2^8 T |v| must stay within float32.  Equal calls give equal bits.
 *  - Formats: K groups along T of a multiple of 32 tokens, V groups along C of
 *    32, 64 or 128 channels, both of 2 or both of 4 bits, bf16 scales,
 *    symmetric or with bf16 zero points; C = 64 or 128; group 1 .. 64
 *    (KVQ_EUNSUPPORTED otherwise).  The formats' residual is not used.
 *  - Codes, the keys' scales and zero points, buffers, q and out 16-byte
 *    aligned.
 *  - workspace: at least kvq_attend_chunk_workspace(shape, resid_rows, n,
 *    group) bytes, 256-byte aligned; enough for every tq and nres.
 *  - Errors: KVQ_EINVAL, KVQ_EUNSUPPORTED, KVQ_EWORKSPACE, KVQ_ECUDA. */
KVQ_API kvq_status kvq_attend_chunk_workspace(const kvq_shape* shape, int64_t resid_rows, int64_t n, int64_t group,
                                              size_t* workspace_B);
KVQ_API kvq_status kvq_attend_chunk(const void* q, int64_t n, int64_t group, int64_t kv_heads, const kvq_cache* cache,
                                    const kvq_qparams* k_params, const kvq_qparams* v_params, const kvq_shape* shape,
                                    void* out, float* lse, void* workspace, size_t workspace_B, void* stream);

/* The attention weight that n queries give every token, added to the tokens'
 * scores ([FtC] §3.1 without a stored history; [FtC] §3.3's observation window
 * when q holds the last n queries only):
 *     scores_out[o][t] = scores_in[o][t]
 *                      + sum_{i < n, j < group, t in seen(o, i)} exp(q . k_t / sqrt(C) - lse[b][i][h*group+j])
 * for t < T; scores of other columns are left as they are.
 *  - q, lse: as kvq_attend_chunk takes and writes them.  A row whose lse is
 *    -inf gives nothing, whatever its q holds; one whose lse is NaN makes NaN of
 *    the score of every token it sees.  Only the K side of the cache is read (its v_* and
 *    v_params are not).
 *  - scores_in, scores_out: float32 [outer][score_stride], score_stride >= T;
 *    scores_in may be NULL (zeros) or scores_out itself; otherwise they must
 *    not overlap.
 *  - The sums are float32, taken in a fixed order: equal calls give equal bits.
 *  - Formats, workspace and errors as kvq_attend_chunk. */
KVQ_API kvq_status kvq_attend_weights_workspace(const kvq_shape* shape, int64_t resid_rows, int64_t n, int64_t group,
                                                size_t* workspace_B);
KVQ_API kvq_status kvq_attend_weights(const void* q, const float* lse, int64_t n, int64_t group, int64_t kv_heads,
                                      const kvq_cache* cache, const kvq_qparams* k_params, const kvq_shape* shape,
                                      const float* scores_in, float* scores_out, int64_t score_stride,
                                      void* workspace, size_t workspace_B, void* stream);

/* Eviction from the store by accumulated score, in whole blocks of `block`
 * tokens ([FtC] §3.2, [KVC] eviction).  A key group of g tokens shares its
 * scales, so a block of whole groups is the smallest piece that can leave
 * without being quantized again.  With nb = tq / block, W' = min(window, nb)
 * and k = min(budget, nb), per slice:
 *     block score = sum of its tokens' scores, held as three float32 whose
 *                   additions are error-free, so it is exact as long as the sum
 *                   of magnitudes is less than 2^63 of the numbers' last place
 *                   (else off by less than block 2^-63 of it), then rounded to a
 *                   pair of float32 (48 bits at least): equal sums
 *                   tie, in whatever order their numbers come; a sum beyond
 *                   float32 is an infinity
 *     keep        = the newest W' blocks and the k - W' best of the others by
 *                   (score descending, index ascending), ascending
 * (a NaN score ranks below every other).  The kept blocks become blocks
 * 0 .. k-1 of dst, in order, K and V:
 * codes, scales and zero points move as they are.  The scores move with their
 * tokens, those of the nres buffered tokens behind them, and the columns
 * between the new and the old number of tokens become 0.  first counts what is
 * left of the padding.
 *  - src, dst: two caches of the same shape and formats; dst may be src, or
 *    share any of its buffers (in place); buffers that are not shared must not
 *    overlap.  The bf16 buffers are neither read nor written.  src->tq must be
 *    a multiple of block.  On success dst->tq = k * block, dst->nres = src->nres
 *    (host counters).  dst->resid_rows must be at least src->nres.
 *    dst->first is written unless NULL, which only a source without first allows
 *    (src->first NULL counts as zeros).  What dst holds behind its k blocks is left as it is.
 *  - block: a multiple of k_params->group when keys are grouped along T, and of
 *    v_params->group when values are; >= 1.
 *  - scores_in: float32 [outer][score_stride], score_stride >= tq + nres, read;
 *    scores_out: same shape, may be scores_in; must not overlap it otherwise.
 *  - keep: device int32 [outer][k], the kept blocks' indices in src.
 *  - budget >= 1, 0 <= window <= budget; scores must not be NULL.
 *  - formats: any that kvq_append takes; no shape limits but 2^31 tokens or slices,
 *    and that a grid holds a thread for every piece of 1 to 16 bytes of a block
 *    (KVQ_EUNSUPPORTED otherwise).
 *  - workspace: at least kvq_evict_blocks_workspace bytes, 16-byte aligned.
 *  - Errors: KVQ_EINVAL, KVQ_EUNSUPPORTED, KVQ_EWORKSPACE, KVQ_ECUDA. */
KVQ_API kvq_status kvq_evict_blocks_workspace(const kvq_shape* shape, int64_t block, size_t* workspace_B);
KVQ_API kvq_status kvq_evict_blocks(const kvq_cache* src, kvq_cache* dst, const kvq_qparams* k_params,
                                    const kvq_qparams* v_params, const kvq_shape* shape, int64_t block, int64_t budget,
                                    int64_t window, const float* scores_in, float* scores_out, int64_t score_stride,
                                    int32_t* keep, void* workspace, size_t workspace_B, void* stream);

/* Attention of a batch over a prefix that all its requests share and over tokens
 * of their own ([KVC] as kvq_attend_chunk):
 *     seen(b, i) = all tokens of the prefix that are not padding, and
 *                  { t : first[o] <= t <= T - n + i } of `cache`'s slice o = b * kv_heads + h
 *     lse, out   as kvq_attend_chunk defines them over that union.
 * The prefix is read once for all batch * n * group query rows of a KV head.
 *  - prefix, shape: a cache of kv_heads slices (shape->outer = kv_heads).
 *  - The requests' own tokens, one of:
 *      cache, cache_shape: their cache, batch * kv_heads slices, whose newest n
 *        tokens are the queries'; its formats may differ from the prefix's;
 *      own_out, own_lse: what the same queries saw elsewhere, as kvq_attend_chunk
 *        or kvq_attend_prompts wrote it (out's and lse's shapes); a row whose
 *        own_lse is -inf saw nothing, whatever own_out holds;
 *      neither (all NULL): the prefix alone.
 *  - q, out: bf16 [batch][n][kv_heads*group][C]; out may be q or own_out itself and
 *    must not overlap them otherwise; lse: float32 [batch][n][kv_heads*group], or
 *    NULL, may be own_lse itself.
 *  - Arithmetic, numbers that are not finite, formats, alignment and errors as
 *    kvq_attend_chunk.  The own cache's part stays in float32 until it is joined;
 *    own_out has been rounded to bf16 before.
 *  - workspace: at least kvq_attend_shared_workspace(shape, resid_rows, cache_shape,
 *    cache's resid_rows, batch, n, group) bytes, 256-byte aligned (cache_shape NULL
 *    where there is no cache); enough for every tq and nres. */
KVQ_API kvq_status kvq_attend_shared_workspace(const kvq_shape* shape, int64_t resid_rows, const kvq_shape* cache_shape,
                                               int64_t cache_resid_rows, int64_t batch, int64_t n, int64_t group,
                                               size_t* workspace_B);
KVQ_API kvq_status kvq_attend_shared(const void* q, int64_t batch, int64_t n, int64_t group, int64_t kv_heads,
                                     const kvq_cache* prefix, const kvq_qparams* k_params, const kvq_qparams* v_params,
                                     const kvq_shape* shape, const kvq_cache* cache, const kvq_qparams* cache_k_params,
                                     const kvq_qparams* cache_v_params, const kvq_shape* cache_shape,
                                     const void* own_out, const float* own_lse, void* out, float* lse, void* workspace,
                                     size_t workspace_B, void* stream);

/* Causal attention over packed prompts, from bf16 keys and values ([KVC] as
 * kvq_attend_chunk, before anything is quantized).  Prompt s is tokens
 * starts[s] .. starts[s + 1] - 1 of q, k and v; token t of it sees
 * starts[s] .. t, and query head h * group + j reads KV head h:
 *     lse[t][h*group+j]    = log sum_u exp(q_t . k_u / sqrt(C))
 *     out[t][h*group+j][:] = sum_u exp(q_t . k_u / sqrt(C) - lse) v_u
 *  - q: bf16, token t's kv_heads*group heads of C channels at q + t * q_stride
 *    (elements); k, v alike with kv_heads heads and their strides, so views of one
 *    projection's output are taken as they are.  16-byte aligned, strides
 *    multiples of 8 that hold a token's heads.
 *  - starts: device int32 [prompts + 1], ascending, 0 <= starts[s] <= total, read on
 *    the GPU: a captured call replays with the lengths it finds.  A prompt may be empty.
 *    Whatever starts holds, nothing outside of the tensors is read or written;
 *    prompts that are not in order or overlap give unspecified results.
 *  - out: bf16 [total][kv_heads*group][C], may be q itself (of q_stride = kv_heads*group*C)
 *    and must not overlap q, k or v otherwise; lse: float32 [total][kv_heads*group],
 *    or NULL.  Rows of tokens in no prompt are left as they are.
 *  - Arithmetic and numbers that are not finite as kvq_attend_chunk.  Equal calls
 *    give equal bits.
 *  - C = 64 or 128, group 1 .. 64 (KVQ_EUNSUPPORTED otherwise).
 *  - workspace: at least kvq_attend_prompts_workspace bytes, 256-byte aligned.
 *  - Errors: KVQ_EINVAL, KVQ_EUNSUPPORTED, KVQ_EWORKSPACE, KVQ_ECUDA. */
KVQ_API kvq_status kvq_attend_prompts_workspace(int64_t prompts, int64_t total, int64_t group, int64_t kv_heads, int64_t C,
                                                size_t* workspace_B);
KVQ_API kvq_status kvq_attend_prompts(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                      int64_t v_stride, const int32_t* starts, int64_t prompts, int64_t total,
                                      int64_t group, int64_t kv_heads, int64_t C, void* out, float* lse, void* workspace,
                                      size_t workspace_B, void* stream);

/* Packed prompts' keys and values become the tokens of a streaming cache ([FtC]
 * §1.1, §1.2; the layout of kvq_append_kv).  With T = tq + nres, the length the
 * cache then has, and L_s = starts[s + 1] - starts[s], slice o = s * kv_heads + h gets
 * the newest min(L_s, T) tokens of prompt s at positions T - L_s .. T - 1, and
 *     first[o] = max(T - L_s, 0).
 * Groups count the tokens that are there: a key group of which first[o] cuts off a
 * part has its scale and zero point from the rest.  Codes, scales and zero points
 * are those of kvq_quantize over each group's tokens.  What lies before first[o]
 * (whole key groups, value groups, rows of codes, buffer rows) is left as it is, as
 * is everything behind the cache's T tokens.
 *  - k, v, strides, starts, total: as kvq_attend_prompts; no workspace.
 *  - cache: the buffers of shape = {prompts * kv_heads, T_cap, C}; tq (a multiple of
 *    the key group, at most T_cap) and nres (at most resid_rows) say how long it
 *    becomes; first must not be NULL (but where there are no prompts), it is written.
 *    Neither it nor a buffer may overlap k, v or starts.
 *  - A cache that kvq_append_kv goes on with needs tq = block * max(0, (T - R) / block)
 *    and nres = T - tq.
 *  - Formats and alignment as kvq_attend_chunk.
 *  - Errors: KVQ_EINVAL, KVQ_EUNSUPPORTED, KVQ_ECUDA. */
KVQ_API kvq_status kvq_fill_prompts(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                    const int32_t* starts, int64_t prompts, int64_t total, int64_t kv_heads,
                                    const kvq_cache* cache, const kvq_qparams* k_params, const kvq_qparams* v_params,
                                    const kvq_shape* shape, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_CACHE_H */
