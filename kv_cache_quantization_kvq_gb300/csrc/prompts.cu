// prompts.cu -- causal attention over packed prompts in bf16 (kvq_attend_prompts).
//
// "KV cache 压缩：把历史装得更小" §"K 的误差会改变权重，V 的误差会改变内容" (logit_t = q^T k_t /
// sqrt(d), y = sum_t a_t v_t), before anything is compressed: prompt s is the rows
// starts[s] .. starts[s + 1] of q, k and v.
//
// A warp per (token, query head): 32 keys at a time, a key per lane, with the running
// maximum and sum of the softmax in base 2, then a share of the channels per lane.
#include "kvq_rows.cuh"

namespace kvq {

namespace {

using namespace rows;

constexpr int kWarps = 4;

// [begin, end) of prompt s, whatever starts holds
__device__ __forceinline__ void prompt_range(const PromptArgs& a, int64_t s, int& begin, int& end) {
    begin = min(max(a.starts[s], 0), (int)a.total);
    end = min(max(a.starts[s + 1], begin), (int)a.total);
}

template <int C>
__global__ void __launch_bounds__(kWarps * 32)
prompts_kernel(const PromptArgs a, int64_t heads)
{
    constexpr int N = C / 32;
    __shared__ float qs[kWarps][C];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * kWarps + warp;
    if (id >= a.total * heads) return;
    const int t = (int)(id / heads), head = (int)(id % heads), h = head / (int)a.group;
    int64_t lo = 0, hi = a.prompts;                     // the last prompt that starts at or before t
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (a.starts[mid] <= t) lo = mid;
        else hi = mid;
    }
    int begin, end;
    prompt_range(a, lo, begin, end);
    if (t < begin || t >= end) return;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_stride + head * C;
    for (int c = lane; c < C; c += 32) qs[warp][c] = __bfloat162float(q[c]);
    __syncwarp();
    const float scale2 = (float)(1.4426950408889634 / (C == 128 ? 11.313708498984761 : 8.0));
    float m = -INFINITY, l = 0.0f, y[N] = {};
    for (int k0 = begin; k0 <= t; k0 += 32) {
        float x = -INFINITY;
        const int k = k0 + lane;
        if (k <= t) {
            const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(a.k) + k * a.k_stride + h * C;
            float d = 0.0f;
            for (int c = 0; c < C; c += 8) {
                Raw8<__nv_bfloat16> raw;
                float v[8];
                load_raw8(kr + c, raw);
                widen8(raw, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) d = __fmaf_rn(qs[warp][c + i], v[i], d);
            }
            x = __fmul_rn(d, scale2);
        }
        float top = x;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
        top = fmaxf(top, m);
        const float f = m == top ? 1.0f : ex2(__fsub_rn(m, top));
        const float p = k > t ? 0.0f : ex2(__fsub_rn(x, top == -INFINITY ? 0.0f : top));
        m = top;
        l = __fmaf_rn(l, f, p);
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = __fmul_rn(y[i], f);
        const int n = min(32, t + 1 - k0);
        for (int j = 0; j < n; ++j) {
            const float w = __shfl_sync(0xFFFFFFFFu, p, j);
            const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(a.v) + (k0 + j) * a.v_stride + h * C + lane * N;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float v = __bfloat162float(vr[i]);
                y[i] = isfinite(v) ? __fmaf_rn(w, v, y[i]) : __fadd_rn(y[i], v);
            }
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) l = __fadd_rn(l, __shfl_xor_sync(0xFFFFFFFFu, l, s));
    const float inv = row_scale(l);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + id * C + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = __float2bfloat16_rn(row_value(y[i], inv));
    if (a.lse && lane == 0) a.lse[id] = row_lse(m, l);
}

}  // namespace

size_t prompts_workspace(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_attend_prompts(const PromptArgs& a, void*, cudaStream_t st)
{
    const int64_t heads = a.kv_heads * a.group, ctas = (a.total * heads + kWarps - 1) / kWarps;
    if (a.total == 0 || a.prompts == 0) return cudaSuccess;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    if (a.C == 128) prompts_kernel<128><<<(unsigned)ctas, kWarps * 32, 0, st>>>(a, heads);
    else prompts_kernel<64><<<(unsigned)ctas, kWarps * 32, 0, st>>>(a, heads);
    return cudaGetLastError();
}

}  // namespace kvq
