// fill_prompts.cu -- packed prompts' keys and values into a streaming cache
// (kvq_fill_prompts).
//
// "KV Compression 公式到源码对照" §1.1 and §1.2 (group scales and zero points, codes), in the
// KIVI layout: keys grouped along tokens, values along channels.  Slice (b, h) of
// the cache gets the newest min(L_b, T) tokens of prompt b at its positions
// T - L_b .. T - 1, T = tq + nres; what lies before is padding, which no group counts
// and nothing writes.
//
// One launch, bound by memory (4 C bytes in and about C out a token and KV head).  A
// warp takes a few units of one slice, of those that hold tokens, so that padding
// costs nothing:
//  * keys: a group of 64 channels.  Lane (lr, lc) = (lane / 8, lane % 8) has eight
//    channels of every fourth token, up to 64 tokens in registers (longer groups are
//    read twice, the second time from L2); the extremes meet in two shuffles, each lane
//    derives two channels' constants and writes them;
//  * values: the rows of 16 KB / 4 C tokens.  A lane has eight channels of eight tokens;
//    the lanes of a group each derive one token's constants;
//  * buffered tokens: the same rows, copied.
// The arithmetic is that of the quantize kernels (kvq_elem.cuh), bit for bit.
#include <algorithm>

#include "kvq_elem.cuh"

namespace kvq {

namespace {

using namespace elem;

constexpr int kWarps = 4;
constexpr int kRows = 16;                        // rows of a lane that are in flight, keys
constexpr int kRowsV = 8;                        // values and buffer

struct Place { int first, shift; };              // position t of the slice holds row t + shift, from t = first on

__device__ __forceinline__ Place place_of(const FillArgs& a, int64_t b) {
    const int T = (int)(a.tq + a.nres);
    const int begin = min(max(a.starts[b], 0), (int)a.total), end = min(max(a.starts[b + 1], begin), (int)a.total);
    return {max(T - (end - begin), 0), end - T};
}

struct FillPlan {
    int64_t kwarps, vwarps, rwarps;              // warps of a slice for keys, values and buffer rows
    int64_t kblocks, vblocks;                    // blocks of the launch; the buffer's follow
};

// units [u0, u1) of a warp, the part-th of `parts`, of units [lo, hi)
__device__ __forceinline__ void share(int64_t lo, int64_t hi, int64_t part, int64_t parts, int64_t& u0, int64_t& u1) {
    const int64_t n = hi > lo ? hi - lo : 0;
    u0 = lo + n * part / parts;
    u1 = lo + n * (part + 1) / parts;
}

__device__ __forceinline__ void store_meta16(void* buf, int64_t i, float v) {
    static_cast<__nv_bfloat16*>(buf)[i] = __float2bfloat16_rn(v);
}

template <int BITS, bool ASYM>
__device__ __forceinline__ typename CodeWord<BITS>::T codes_of(const uint4& w, const QuotK (&kq)[4], const int32_t (&zo)[8],
                                                               const float (&s)[8], const QSpec& q, int off, bool fast) {
    uint32_t c[8];
    if (fast) {
        codes8_fast<ASYM>(w, kq, zo, q.qmin + off, q.qmax + off, c);
    } else {
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = __int_as_float(zo[i]);           // the zero points themselves
        codes8_slow<ASYM>(w, s, z, q, off, c);
    }
    return finish_word<BITS>(c, q.is_signed);
}

template <int BITS, int C, bool ASYM>
__device__ __forceinline__ void fill_keys(const FillArgs& a, const FillPlan& p, int64_t warp, int lane)
{
    const QSpec& q = a.k.q;
    constexpr int kParts = C / 64;               // groups of 64 channels
    const int64_t o = warp / p.kwarps, b = o / a.kv_heads, h = o - b * a.kv_heads;
    if (o >= a.prompts * a.kv_heads) return;
    const Place at = place_of(a, b);
    const int g = (int)q.g, lr = lane >> 3, lc = lane & 7, off = q.is_signed ? 1 << (BITS - 1) : 0;
    int64_t u0, u1;
    share(at.first / g * kParts, a.tq / g * kParts, warp - o * p.kwarps, p.kwarps, u0, u1);
    const int passes = (g + 4 * kRows - 1) / (4 * kRows);
    for (int64_t u = u0; u < u1; ++u) {
        const int64_t gi = u / kParts;
        const int c0 = (int)(u - gi * kParts) * 64 + lc * 8;
        const int t0 = (int)(gi * g), from = max(at.first, t0);
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.k.x) + (int64_t)(t0 + at.shift) * a.k.stride + h * C + c0;
        uint4 w[kRows];
        auto load = [&](int pass) {
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int r = pass * 4 * kRows + 4 * j + lr;
                w[j] = make_uint4(0, 0, 0, 0);
                if (r < g && t0 + r >= from) w[j] = __ldcg(reinterpret_cast<const uint4*>(x + (int64_t)r * a.k.stride));
            }
        };
        uint32_t mn[4], mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mn[i] = kBfPosInf2;
            mx[i] = ASYM ? kBfNegInf2 : 0u;
        }
        for (int pass = 0; pass < passes; ++pass) {
            load(pass);
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int r = pass * 4 * kRows + 4 * j + lr;
                if (r >= g || t0 + r < from) continue;
                const uint32_t ws[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (ASYM) mn[i] = bmin2(mn[i], ws[i]);
                    mx[i] = bmax2(mx[i], ASYM ? ws[i] : babs2(ws[i]));
                }
            }
        }
#pragma unroll
        for (int s = 8; s < 32; s <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (ASYM) mn[i] = bmin2(mn[i], __shfl_xor_sync(0xFFFFFFFFu, mn[i], s));
                mx[i] = bmax2(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], s));
            }
        // channels 2 lr and 2 lr + 1 of the lane's eight
        uint32_t wn = mn[0], wx = mx[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            if (lr == i) {
                wn = mn[i];
                wx = mx[i];
            }
        }
        const GroupC g0 = make_group<ASYM>(lo_f(wn), lo_f(wx), q, off), g1 = make_group<ASYM>(hi_f(wn), hi_f(wx), q, off);
        const int64_t mi = (o * q.ngroups + gi) * C + c0 + 2 * lr;
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.k.scale) + mi) = pack_bf16x2(g0.s, g1.s);
        if (ASYM) *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.k.zero) + mi) = pack_bf16x2(g0.zp, g1.zp);
        const bool fast = __all_sync(0xFFFFFFFFu, g0.fast && g1.fast);
        float s8[8];
        int32_t zo[8];
        QuotK kq[4];
        const int32_t z0 = fast ? g0.zoff : __float_as_int(g0.zp), z1 = fast ? g1.zoff : __float_as_int(g1.zp);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int src = 8 * i + lc;
            s8[2 * i] = __shfl_sync(0xFFFFFFFFu, g0.s, src);
            s8[2 * i + 1] = __shfl_sync(0xFFFFFFFFu, g1.s, src);
            zo[2 * i] = __shfl_sync(0xFFFFFFFFu, z0, src);
            zo[2 * i + 1] = __shfl_sync(0xFFFFFFFFu, z1, src);
            kq[i].ns = pk(-s8[2 * i], -s8[2 * i + 1]);
            kq[i].inv = pk(__shfl_sync(0xFFFFFFFFu, g0.inv, src), __shfl_sync(0xFFFFFFFFu, g1.inv, src));
        }
        uint8_t* codes = static_cast<uint8_t*>(a.k.codes) + (o * a.cap + t0) * (C * BITS / 8) + c0 / 8 * BITS;
        for (int pass = 0; pass < passes; ++pass) {
            if (passes > 1) load(pass);
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int r = pass * 4 * kRows + 4 * j + lr;
                if (r < g && t0 + r >= from)
                    store_codes<BITS>(codes + (int64_t)r * (C * BITS / 8), codes_of<BITS, ASYM>(w[j], kq, zo, s8, q, off, fast));
            }
        }
    }
}

template <int BITS, int C, bool ASYM>
__device__ __forceinline__ void fill_values(const FillArgs& a, const FillPlan& p, int64_t warp, int lane)
{
    const QSpec& q = a.v.q;
    constexpr int kLanes = C / 8, kAcross = 32 / kLanes, kUnit = kRowsV * kAcross;    // lanes of a row, rows of a load
    const int64_t o = warp / p.vwarps, b = o / a.kv_heads, h = o - b * a.kv_heads;
    if (o >= a.prompts * a.kv_heads) return;
    const Place at = place_of(a, b);
    const int lr = lane / kLanes, lc = lane % kLanes, off = q.is_signed ? 1 << (BITS - 1) : 0;
    const int gl = (int)q.g / 8, mine = lc & (gl - 1);              // 4, 8 or 16 lanes a group
    int64_t u0, u1;
    share(at.first / kUnit, (a.tq + kUnit - 1) / kUnit, warp - o * p.vwarps, p.vwarps, u0, u1);
    for (int64_t u = u0; u < u1; ++u) {
        const int t0 = (int)u * kUnit + lr;      // the lane's rows: t0 + k kAcross
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.v.x) + (int64_t)(t0 + at.shift) * a.v.stride + h * C + lc * 8;
        auto live = [&](int k) { return t0 + k * kAcross >= at.first && t0 + k * kAcross < a.tq; };
        uint4 w[kRowsV];
#pragma unroll
        for (int k = 0; k < kRowsV; ++k) {
            w[k] = make_uint4(0, 0, 0, 0);
            if (live(k)) w[k] = __ldcs(reinterpret_cast<const uint4*>(x + (int64_t)k * kAcross * a.v.stride));
        }
        // a group's (min, -max), or (0, -max |x|), as one pair: they meet in log2(gl) shuffles
        uint32_t ext[kRowsV];
#pragma unroll
        for (int k = 0; k < kRowsV; ++k) {
            uint32_t mn = kBfPosInf2, mx = ASYM ? kBfNegInf2 : 0u;
            if (ASYM) fold_minmax(w[k], mn, mx);
            else fold_absmax(w[k], mx);
            mn = bmin2(mn, __byte_perm(mn, mn, 0x1032));
            mx = bmax2(mx, __byte_perm(mx, mx, 0x1032)) ^ 0x80008000u;
            ext[k] = __byte_perm(mn, mx, 0x5410);
        }
        for (int s = 1; s < gl; s <<= 1)
#pragma unroll
            for (int k = 0; k < kRowsV; ++k) ext[k] = bmin2(ext[k], __shfl_xor_sync(0xFFFFFFFFu, ext[k], s));
        // lane `mine` of a group derives the constants of rows mine and, where a group has four lanes, mine + 4
        GroupC gc[2];
        bool fast = true;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = i == 0 ? mine & 7 : (mine & 3) + 4;
            uint32_t e = ext[0];
#pragma unroll
            for (int k = 1; k < kRowsV; ++k)
                if (row == k) e = ext[k];
            if (i == 0 || gl == 4) {
                gc[i] = make_group<ASYM>(lo_f(e), -hi_f(e), q, off);
                fast = fast && gc[i].fast;
                const int t = t0 + row * kAcross;
                if (mine < 8 && t >= at.first && t < a.tq) {
                    const int64_t mi = (o * a.cap + t) * q.ngroups + lc / gl;
                    store_meta16(a.v.scale, mi, gc[i].s);
                    if (ASYM) store_meta16(a.v.zero, mi, gc[i].zp);
                }
            } else {
                gc[i] = gc[0];
            }
        }
        fast = __all_sync(0xFFFFFFFFu, fast);
        const int lane0 = lane - mine;
        uint8_t* codes = static_cast<uint8_t*>(a.v.codes) + (o * a.cap + t0) * (C * BITS / 8) + lc * BITS;
#pragma unroll
        for (int k = 0; k < kRowsV; ++k) {
            const int src = lane0 + (gl == 4 ? k & 3 : k);
            const bool second = k >= 4 && gl == 4;
            const float s = __shfl_sync(0xFFFFFFFFu, second ? gc[1].s : gc[0].s, src);
            const float inv = __shfl_sync(0xFFFFFFFFu, second ? gc[1].inv : gc[0].inv, src);
            const GroupC& gk = second ? gc[1] : gc[0];
            const int32_t z = __shfl_sync(0xFFFFFFFFu, fast ? gk.zoff : __float_as_int(gk.zp), src);
            float s8[8];
            int32_t zo[8];
            QuotK kq[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s8[i] = s;
                zo[i] = z;
                kq[i / 2].ns = pk(-s, -s);
                kq[i / 2].inv = pk(inv, inv);
            }
            const auto word = codes_of<BITS, ASYM>(w[k], kq, zo, s8, q, off, fast);
            if (live(k)) store_codes<BITS>(codes + (int64_t)k * kAcross * (C * BITS / 8), word);
        }
    }
}

template <int C>
__device__ __forceinline__ void fill_buffers(const FillArgs& a, const FillPlan& p, int64_t warp, int lane)
{
    constexpr int kLanes = C / 8, kAcross = 32 / kLanes, kUnit = kRowsV * kAcross;
    const int64_t o = warp / p.rwarps, b = o / a.kv_heads, h = o - b * a.kv_heads, part = warp - o * p.rwarps;
    if (o >= a.prompts * a.kv_heads) return;
    const Place at = place_of(a, b);
    if (part == 0 && lane == 0) a.first[o] = at.first;
    const int64_t half = p.rwarps / 2;           // keys, then values
    if (half == 0) return;
    const FillStore& s = part < half ? a.k : a.v;
    int64_t u0, u1;
    share(max(at.first - a.tq, (int64_t)0) / kUnit, (a.nres + kUnit - 1) / kUnit, part < half ? part : part - half, half, u0, u1);
    const int lr = lane / kLanes, lc = lane % kLanes;
    for (int64_t u = u0; u < u1; ++u) {
        const int r0 = (int)u * kUnit + lr;
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(s.x) + (a.tq + r0 + at.shift) * s.stride + h * C + lc * 8;
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(s.resid) + (o * a.rrows + r0) * C + lc * 8;
        auto live = [&](int k) { return a.tq + r0 + k * kAcross >= at.first && r0 + k * kAcross < a.nres; };
        uint4 w[kRowsV];
#pragma unroll
        for (int k = 0; k < kRowsV; ++k)
            if (live(k)) w[k] = __ldcs(reinterpret_cast<const uint4*>(x + (int64_t)k * kAcross * s.stride));
#pragma unroll
        for (int k = 0; k < kRowsV; ++k)
            if (live(k)) *reinterpret_cast<uint4*>(y + (int64_t)k * kAcross * C) = w[k];
    }
}

template <int BITS, int C>
__global__ void __launch_bounds__(kWarps * 32, 4)
fill_kernel(const FillArgs a, const FillPlan p)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t block = blockIdx.x;
    if (block < p.kblocks) {
        if (a.k.q.mode == KVQ_ASYM) fill_keys<BITS, C, true>(a, p, block * kWarps + warp, lane);
        else fill_keys<BITS, C, false>(a, p, block * kWarps + warp, lane);
        return;
    }
    block -= p.kblocks;
    if (block < p.vblocks) {
        if (a.v.q.mode == KVQ_ASYM) fill_values<BITS, C, true>(a, p, block * kWarps + warp, lane);
        else fill_values<BITS, C, false>(a, p, block * kWarps + warp, lane);
        return;
    }
    fill_buffers<C>(a, p, (block - p.vblocks) * kWarps + warp, lane);
}

// Units for a warp: enough warps to fill the GPU twice, but at most eight units.
int64_t warps_of(int64_t units, int64_t outer)
{
    const int64_t each = std::min<int64_t>(8, std::max<int64_t>(1, units * outer / (2 * 152 * 16)));
    return (units + each - 1) / each;
}

template <int BITS, int C>
cudaError_t launch(const FillArgs& a, int64_t outer, cudaStream_t st)
{
    constexpr int kUnit = kRowsV * 32 / (C / 8);
    FillPlan p;
    p.kwarps = a.tq ? warps_of(a.tq / a.k.q.g * (C / 64), outer) : 0;
    p.vwarps = a.tq ? warps_of((a.tq + kUnit - 1) / kUnit, outer) : 0;
    p.rwarps = std::max<int64_t>(1, 2 * warps_of((a.nres + kUnit - 1) / kUnit, outer));
    auto blocks = [&](int64_t warps) { return (outer * warps + kWarps - 1) / kWarps; };
    p.kblocks = blocks(p.kwarps);
    p.vblocks = blocks(p.vwarps);
    const int64_t grid = p.kblocks + p.vblocks + blocks(p.rwarps);
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    fill_kernel<BITS, C><<<(unsigned)grid, kWarps * 32, 0, st>>>(a, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fill_prompts(const FillArgs& a, cudaStream_t st)
{
    const int64_t outer = a.prompts * a.kv_heads;
    if (outer == 0) return cudaSuccess;
    if (a.k.q.bits == 4) return a.C == 128 ? launch<4, 128>(a, outer, st) : launch<4, 64>(a, outer, st);
    return a.C == 128 ? launch<2, 128>(a, outer, st) : launch<2, 64>(a, outer, st);
}

}  // namespace kvq
