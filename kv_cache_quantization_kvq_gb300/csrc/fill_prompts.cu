// fill_prompts.cu -- packed prompts' keys and values into a streaming cache
// (kvq_fill_prompts).
//
// "KV Compression 公式到源码对照" §1.1 and §1.2 (group scales and zero points, codes), in the
// KIVI layout: keys grouped along tokens, values along channels.  Slice (b, h) of
// the cache gets the newest min(L_b, T) tokens of prompt b at its positions
// T - L_b .. T - 1, T = tq + nres; what lies before is padding, which no group counts
// and nothing writes.
//
// A thread makes one byte column of a key group, or one value group of a token, or
// moves eight channels of a buffered token.
#include <algorithm>

#include "kvq_elem.cuh"

namespace kvq {

namespace {

struct Place { int first, shift; };              // position t of the slice holds row t + shift, from t = first on

__device__ __forceinline__ Place place_of(const FillArgs& a, int64_t b) {
    const int T = (int)(a.tq + a.nres);
    const int begin = min(max(a.starts[b], 0), (int)a.total), end = min(max(a.starts[b + 1], begin), (int)a.total);
    return {max(T - (end - begin), 0), end - T};
}

template <bool ASYM>
__device__ __forceinline__ Meta group_meta(float mn, float mx, const QSpec& q) {
    return ASYM ? meta_asym(mn, mx, q) : meta_sym(fmaxf(-mn, mx), q);
}

template <bool ASYM>
__global__ void __launch_bounds__(256) fill_keys_kernel(const FillArgs a, int64_t total)
{
    const QSpec& q = a.k.q;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= total) return;
    const int per = 8 / q.bits, rowB = (int)(a.C / per);
    const int64_t groups = a.tq / q.g;
    const int byte = (int)(id % rowB);
    const int64_t gi = id / rowB % groups, o = id / rowB / groups, b = o / a.kv_heads, h = o % a.kv_heads;
    const Place p = place_of(a, b);
    const int64_t t0 = max(gi * q.g, (int64_t)p.first), t1 = (gi + 1) * q.g;
    if (t0 >= t1) return;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.k.x) + h * a.C + byte * per;
    uint8_t* codes = static_cast<uint8_t*>(a.k.codes) + o * a.cap * rowB + byte;
    const int64_t mi = (o * q.ngroups + gi) * a.C + byte * per;
    Meta m[4];
    for (int c = 0; c < per; ++c) {
        float mn = INFINITY, mx = -INFINITY;
        for (int64_t t = t0; t < t1; ++t) {
            const float v = __bfloat162float(x[(t + p.shift) * a.k.stride + c]);
            mn = fminf(mn, v);
            mx = fmaxf(mx, v);
        }
        m[c] = group_meta<ASYM>(mn, mx, q);
        store_scale(a.k.scale, q.scale_dt, mi + c, m[c].s);
        if (ASYM) store_zero(a.k.zero, q.zero_dt, mi + c, m[c].z);
    }
    for (int64_t t = t0; t < t1; ++t) {
        uint32_t w = 0;
        for (int c = 0; c < per; ++c)
            w |= ((uint32_t)quant_code<ASYM>(__bfloat162float(x[(t + p.shift) * a.k.stride + c]), m[c], q.lo, q.hi) &
                  ((1u << q.bits) - 1)) << (c * q.bits);
        codes[t * rowB] = (uint8_t)w;
    }
}

template <bool ASYM>
__global__ void __launch_bounds__(256) fill_values_kernel(const FillArgs a, int64_t total)
{
    const QSpec& q = a.v.q;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= total) return;
    const int64_t gi = id % q.ngroups, t = id / q.ngroups % a.tq, o = id / q.ngroups / a.tq, b = o / a.kv_heads, h = o % a.kv_heads;
    const Place p = place_of(a, b);
    if (t < p.first) return;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.v.x) + (t + p.shift) * a.v.stride + h * a.C + gi * q.g;
    float mn = INFINITY, mx = -INFINITY;
    for (int c = 0; c < q.g; ++c) {
        mn = fminf(mn, __bfloat162float(x[c]));
        mx = fmaxf(mx, __bfloat162float(x[c]));
    }
    const Meta m = group_meta<ASYM>(mn, mx, q);
    const int64_t mi = (o * a.cap + t) * q.ngroups + gi;
    store_scale(a.v.scale, q.scale_dt, mi, m.s);
    if (ASYM) store_zero(a.v.zero, q.zero_dt, mi, m.z);
    const int per = 8 / q.bits;
    uint8_t* codes = static_cast<uint8_t*>(a.v.codes) + (o * a.cap + t) * (a.C / per) + gi * q.g / per;
    for (int c = 0; c < q.g; c += per) {
        uint32_t w = 0;
        for (int i = 0; i < per; ++i)
            w |= ((uint32_t)quant_code<ASYM>(__bfloat162float(x[c + i]), m, q.lo, q.hi) & ((1u << q.bits) - 1)) << (i * q.bits);
        codes[c / per] = (uint8_t)w;
    }
}

__global__ void __launch_bounds__(256) fill_buffer_kernel(const FillArgs a, int64_t total)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int P = (int)(a.C / 8);
    if (id < a.prompts * a.kv_heads) a.first[id] = place_of(a, id / a.kv_heads).first;
    if (id >= total) return;
    const int64_t r = id / P % a.nres, o = id / P / a.nres, b = o / a.kv_heads, h = o % a.kv_heads;
    const Place p = place_of(a, b);
    if (a.tq + r < p.first) return;
    const FillStore& s = blockIdx.y ? a.v : a.k;
    Raw8<__nv_bfloat16> w;
    load_raw8(static_cast<const __nv_bfloat16*>(s.x) + (a.tq + r + p.shift) * s.stride + h * a.C + id % P * 8, w);
    store_raw8(static_cast<__nv_bfloat16*>(s.resid) + (o * a.rrows + r) * a.C + id % P * 8, w);
}

}  // namespace

cudaError_t launch_fill_prompts(const FillArgs& a, cudaStream_t st)
{
    const int64_t outer = a.prompts * a.kv_heads;
    if (outer == 0) return cudaSuccess;
    auto ctas = [](int64_t n) { return (unsigned)((n + 255) / 256); };
    const int64_t nk = a.tq ? outer * (a.tq / a.k.q.g) * (a.C * a.k.q.bits / 8) : 0, nv = outer * a.tq * a.v.q.ngroups;
    const int64_t nb = outer * a.nres * (a.C / 8);
    if (std::max(nk, std::max(nv, nb)) / 256 > 0x7FFFFFF0) return cudaErrorInvalidConfiguration;
    if (nk && a.k.q.mode == KVQ_ASYM) fill_keys_kernel<true><<<ctas(nk), 256, 0, st>>>(a, nk);
    else if (nk) fill_keys_kernel<false><<<ctas(nk), 256, 0, st>>>(a, nk);
    if (nv && a.v.q.mode == KVQ_ASYM) fill_values_kernel<true><<<ctas(nv), 256, 0, st>>>(a, nv);
    else if (nv) fill_values_kernel<false><<<ctas(nv), 256, 0, st>>>(a, nv);
    fill_buffer_kernel<<<dim3(ctas(std::max(nb, outer)), 2), 256, 0, st>>>(a, nb);
    return cudaGetLastError();
}

}  // namespace kvq
