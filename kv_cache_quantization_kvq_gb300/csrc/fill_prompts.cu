// fill_prompts.cu -- packed prompts' keys and values into a streaming cache
// (kvq_fill_prompts).
//
// "KV Compression 公式到源码对照" §1.1 and §1.2 (group scales and zero points, codes), in the
// KIVI layout: keys grouped along tokens, values along channels.  Slice (b, h) of
// the cache gets the newest min(L_b, T) tokens of prompt b at its positions
// T - L_b .. T - 1, T = tq + nres; what lies before is padding, which no group counts
// and nothing writes.
//
// One launch, bound by memory (4 C bytes in and about C out a token and KV head) and
// by the instructions that make the codes.  A warp takes a few units of one slice, of
// those that hold tokens, so that padding costs nothing:
//  * keys: a group of 64 channels.  Lane (lr, lc) = (lane / 8, lane % 8) has eight
//    channels of every fourth token; the extremes meet in two shuffles, each lane
//    derives two channels' constants and writes them;
//  * values: eight tokens a lane, eight channels of each; the lanes of a group each
//    derive a token's constants;
//  * buffered tokens: the same rows, copied.
// A unit is read twice, for the extremes and for the codes, the second time from L1:
// with the rows kept in registers the loops had to be unrolled over all of them, and
// missed the instruction cache at 16 warps a SM (64 prompts of 26422 tokens: 55 us).
// The arithmetic is that of the quantize kernels (kvq_elem.cuh), bit for bit.
//
// Measured on one GB300, 8 KV heads of 128 channels: 64 prompts of 16 to 2000 tokens at 4 bits 49 us (3.2 TB/s), 4 of
// 9000 to 32768 at 2 bits 138 us (3.3 TB/s): 54 % of the issue slots, 31 to 39 % of DRAM busy, so that neither bounds it
// but a warp's way from loads to extremes, constants, loads again and codes.
// Six CTAs an SM leave a thread 80 registers, which spill (132 bytes at C = 128, 156 at 64); five, at 96 without a spill, are
// slower: 69892 tokens in 64 prompts 105.4 and 108.7 us at 4 bits, at C = 64 60.5 and 64.3; 83768 in 4 at 2 bits 127.4 and 134.0.
#include <algorithm>
#include <type_traits>

#include "kvq_elem.cuh"

namespace kvq {

namespace {

using namespace elem;

constexpr int kWarps = 4;
constexpr int kRows = 8;                         // rows of a lane that are in flight

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

// The line that p lies in, into L2 (64 ragged prompts 49.7 -> 48.5 us, long ones 141.6 -> 136.9).
__device__ __forceinline__ void fetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The codes of eight channels by the IEEE division, out of line: the groups that need it are few.
template <int BITS, bool ASYM>
__device__ __noinline__ uint32_t slow_codes(const uint4& w, const float* s, const float* z, const QSpec& q, int off) {
    float s8[8], z8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        s8[i] = s[i];
        z8[i] = z[i];
    }
    uint32_t c[8];
    codes8_slow<ASYM>(w, s8, z8, q, off, c);
    return finish_word<BITS>(c, q.is_signed);
}

template <int BITS, int C, bool ASYM>
__device__ __forceinline__ void fill_keys(const FillArgs& a, const FillPlan& p, int64_t warp, int lane)
{
    const QSpec& q = a.k.q;
    constexpr int kParts = C / 64;               // groups of 64 channels
    constexpr int kRowB = C * BITS / 8;
    const int64_t o = warp / p.kwarps, b = o / a.kv_heads, h = o - b * a.kv_heads;
    if (o >= a.prompts * a.kv_heads) return;
    const Place at = place_of(a, b);
    const int g = (int)q.g, lr = lane >> 3, lc = lane & 7, off = q.is_signed ? 1 << (BITS - 1) : 0;
    int64_t u0, u1;
    share(at.first / g * kParts, a.tq / g * kParts, warp - o * p.kwarps, p.kwarps, u0, u1);
#pragma unroll 1
    for (int64_t u = u0; u < u1; ++u) {
        const int64_t gi = u / kParts;
        const int c0 = (int)(u - gi * kParts) * 64 + lc * 8;
        const int t0 = (int)(gi * g), from = max(at.first - t0, 0);         // rows from .. g - 1 are there
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.k.x) + (int64_t)(t0 + at.shift) * a.k.stride + h * C + c0;
        if (u + 1 < u1) {                        // the next unit's rows, a 128-byte line a lane
            const int64_t gn = (u + 1) / kParts;
            const int tn = (int)(gn * g);
            const __nv_bfloat16* xn = static_cast<const __nv_bfloat16*>(a.k.x) + (int64_t)(tn + at.shift) * a.k.stride + h * C +
                                      (u + 1 - gn * kParts) * 64;
#pragma unroll 1
            for (int r = lane; r < g; r += 32)
                if (tn + r >= at.first) fetch(xn + (int64_t)r * a.k.stride);
        }
        uint32_t mn[4], mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mn[i] = kBfPosInf2;
            mx[i] = ASYM ? kBfNegInf2 : 0u;
        }
#pragma unroll 1
        for (int r = lr; r < g; r += 4 * kRows) {
            uint4 w[kRows];
#pragma unroll
            for (int j = 0; j < kRows; ++j)
                if (r + 4 * j >= from && r + 4 * j < g) w[j] = *reinterpret_cast<const uint4*>(x + (int64_t)(r + 4 * j) * a.k.stride);
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                if (r + 4 * j < from || r + 4 * j >= g) continue;
                const uint32_t ws[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (ASYM) mn[i] = bmin2(mn[i], ws[i]);
                    mx[i] = bmax2(mx[i], ASYM ? ws[i] : babs2(ws[i]));
                }
            }
        }
        __syncwarp();
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
        uint8_t* codes = static_cast<uint8_t*>(a.k.codes) + (o * a.cap + t0) * kRowB + c0 / 8 * BITS;
        if (__all_sync(0xFFFFFFFFu, g0.fast && g1.fast)) {
            int32_t zo[8];
            QuotK kq[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int src = 8 * i + lc;
                zo[2 * i] = __shfl_sync(0xFFFFFFFFu, g0.zoff, src);
                zo[2 * i + 1] = __shfl_sync(0xFFFFFFFFu, g1.zoff, src);
                kq[i].ns = pk(-__shfl_sync(0xFFFFFFFFu, g0.s, src), -__shfl_sync(0xFFFFFFFFu, g1.s, src));
                kq[i].inv = pk(__shfl_sync(0xFFFFFFFFu, g0.inv, src), __shfl_sync(0xFFFFFFFFu, g1.inv, src));
            }
            const int lo = q.qmin + off, hi = q.qmax + off;
            const uint4* px = reinterpret_cast<const uint4*>(x + (int64_t)lr * a.k.stride);
            const int64_t step = a.k.stride / 2;                    // four rows, in pieces of eight channels
            uint8_t* pc = codes + lr * kRowB;
            auto rows = [&](auto clip) {
#pragma unroll 2
                for (int r = lr; r < g; r += 4) {
                    if (r >= from) {
                        uint32_t c[8];
                        codes8_fast<ASYM, decltype(clip)::value>(*px, kq, zo, lo, hi, c);
                        store_codes<BITS>(pc, finish_word<BITS>(c, q.is_signed));
                    }
                    px += step;
                    pc += 4 * kRowB;
                }
            };
            if (__all_sync(0xFFFFFFFFu, g0.lo_ok && g1.lo_ok)) rows(std::false_type{});
            else rows(std::true_type{});
        } else {
            float s8[8], z8[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int src = 8 * i + lc;
                s8[2 * i] = __shfl_sync(0xFFFFFFFFu, g0.s, src);
                s8[2 * i + 1] = __shfl_sync(0xFFFFFFFFu, g1.s, src);
                z8[2 * i] = __shfl_sync(0xFFFFFFFFu, g0.zp, src);
                z8[2 * i + 1] = __shfl_sync(0xFFFFFFFFu, g1.zp, src);
            }
#pragma unroll 1
            for (int r = lr; r < g; r += 4)
                if (r >= from)
                    store_codes<BITS>(codes + (int64_t)r * kRowB, (typename CodeWord<BITS>::T)slow_codes<BITS, ASYM>(
                                          *reinterpret_cast<const uint4*>(x + (int64_t)r * a.k.stride), s8, z8, q, off));
        }
        __syncwarp();
    }
}

template <int BITS, int C, bool ASYM>
__device__ __forceinline__ void fill_values(const FillArgs& a, const FillPlan& p, int64_t warp, int lane)
{
    const QSpec& q = a.v.q;
    constexpr int kLanes = C / 8, kAcross = 32 / kLanes, kUnit = kRows * kAcross;     // lanes of a row, rows of a load
    constexpr int kRowB = C * BITS / 8;
    const int64_t o = warp / p.vwarps, b = o / a.kv_heads, h = o - b * a.kv_heads;
    if (o >= a.prompts * a.kv_heads) return;
    const Place at = place_of(a, b);
    const int lr = lane / kLanes, lc = lane % kLanes, off = q.is_signed ? 1 << (BITS - 1) : 0;
    const int gl = (int)q.g / 8, mine = lc & (gl - 1);              // 4, 8 or 16 lanes a group
    int64_t u0, u1;
    share(at.first / kUnit, (a.tq + kUnit - 1) / kUnit, warp - o * p.vwarps, p.vwarps, u0, u1);
#pragma unroll 1
    for (int64_t u = u0; u < u1; ++u) {
        const int t0 = (int)u * kUnit + lr;      // the lane's rows: t0 + k kAcross
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.v.x) + (int64_t)(t0 + at.shift) * a.v.stride + h * C + lc * 8;
        auto live = [&](int k) { return t0 + k * kAcross >= at.first && t0 + k * kAcross < a.tq; };
        if (u + 1 < u1) {
            const int tn = (int)(u + 1) * kUnit + lane / (C / 64);
            if (tn >= at.first && tn < a.tq)
                fetch(static_cast<const __nv_bfloat16*>(a.v.x) + (int64_t)(tn + at.shift) * a.v.stride + h * C + lane % (C / 64) * 64);
        }
        // a group's (min, -max), or (0, -max |x|), as one pair: they meet in log2(gl) shuffles
        uint32_t ext[kRows];
        {
            uint4 w[kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                w[k] = make_uint4(0, 0, 0, 0);
                if (live(k)) w[k] = *reinterpret_cast<const uint4*>(x + (int64_t)k * kAcross * a.v.stride);
            }
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                uint32_t mn = kBfPosInf2, mx = ASYM ? kBfNegInf2 : 0u;
                if (ASYM) fold_minmax(w[k], mn, mx);
                else fold_absmax(w[k], mx);
                mn = bmin2(mn, __byte_perm(mn, mn, 0x1032));
                mx = bmax2(mx, __byte_perm(mx, mx, 0x1032)) ^ 0x80008000u;
                ext[k] = __byte_perm(mn, mx, 0x5410);
            }
        }
#pragma unroll 1
        for (int s = 1; s < gl; s <<= 1)
#pragma unroll
            for (int k = 0; k < kRows; ++k) ext[k] = bmin2(ext[k], __shfl_xor_sync(0xFFFFFFFFu, ext[k], s));
        // lane `mine` of a group derives the constants of rows mine and, where a group has four lanes, mine + 4
        float gs[2], gi[2], gz[2];
        int32_t zoff[2];
        bool fast = true, lo_ok = true;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i == 1 && gl != 4) {             // not looked at
                gs[1] = gi[1] = gz[1] = 0.0f;
                zoff[1] = 0;
                break;
            }
            const int row = i == 0 ? mine & 7 : mine + 4;
            uint32_t e = ext[0];
#pragma unroll
            for (int k = 1; k < kRows; ++k)
                if (row == k) e = ext[k];
            const GroupC gc = make_group<ASYM>(lo_f(e), -hi_f(e), q, off);
            gs[i] = gc.s;
            gi[i] = gc.inv;
            gz[i] = gc.zp;
            zoff[i] = gc.zoff;
            fast = fast && gc.fast;
            lo_ok = lo_ok && gc.lo_ok;
            const int t = t0 + row * kAcross;
            if (mine < 8 && t >= at.first && t < a.tq) {
                const int64_t mi = (o * a.cap + t) * q.ngroups + lc / gl;
                store_meta16(a.v.scale, mi, gc.s);
                if (ASYM) store_meta16(a.v.zero, mi, gc.zp);
            }
        }
        const int lane0 = lane - mine;
        uint8_t* codes = static_cast<uint8_t*>(a.v.codes) + (o * a.cap + t0) * kRowB + lc * BITS;
        if (__all_sync(0xFFFFFFFFu, fast)) {
            const int lo = q.qmin + off, hi = q.qmax + off;
            const uint4* px = reinterpret_cast<const uint4*>(x);
            const int64_t step = kAcross * a.v.stride / 8;
            uint8_t* pc = codes;
            auto rows = [&](auto clip) {
#pragma unroll 2
                for (int k = 0; k < kRows; ++k) {
                    const bool second = k >= 4 && gl == 4;
                    const int src = lane0 + (second ? k - 4 : k);
                    const float s = __shfl_sync(0xFFFFFFFFu, second ? gs[1] : gs[0], src);
                    const float inv = __shfl_sync(0xFFFFFFFFu, second ? gi[1] : gi[0], src);
                    const int32_t z = __shfl_sync(0xFFFFFFFFu, second ? zoff[1] : zoff[0], src);
                    if (live(k)) {
                        const int32_t zo[8] = {z, z, z, z, z, z, z, z};
                        const QuotK one = {pk(-s, -s), pk(inv, inv)};
                        const QuotK kq[4] = {one, one, one, one};
                        uint32_t c[8];
                        codes8_fast<ASYM, decltype(clip)::value>(*px, kq, zo, lo, hi, c);
                        store_codes<BITS>(pc, finish_word<BITS>(c, q.is_signed));
                    }
                    px += step;
                    pc += kAcross * kRowB;
                }
            };
            if (__all_sync(0xFFFFFFFFu, lo_ok)) rows(std::false_type{});
            else rows(std::true_type{});
        } else {
#pragma unroll 1
            for (int k = 0; k < kRows; ++k) {
                const bool second = k >= 4 && gl == 4;
                const int src = lane0 + (second ? k - 4 : k);
                const float s = __shfl_sync(0xFFFFFFFFu, second ? gs[1] : gs[0], src);
                const float z = __shfl_sync(0xFFFFFFFFu, second ? gz[1] : gz[0], src);
                if (!live(k)) continue;
                const float s8[8] = {s, s, s, s, s, s, s, s}, z8[8] = {z, z, z, z, z, z, z, z};
                store_codes<BITS>(codes + (int64_t)k * kAcross * kRowB, (typename CodeWord<BITS>::T)slow_codes<BITS, ASYM>(
                                      *reinterpret_cast<const uint4*>(x + (int64_t)k * kAcross * a.v.stride), s8, z8, q, off));
            }
        }
        __syncwarp();
    }
}

template <int C>
__device__ __forceinline__ void fill_buffers(const FillArgs& a, const FillPlan& p, int64_t warp, int lane)
{
    constexpr int kLanes = C / 8, kAcross = 32 / kLanes, kUnit = kRows * kAcross;
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
        uint4 w[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (live(k)) w[k] = __ldcs(reinterpret_cast<const uint4*>(x + (int64_t)k * kAcross * s.stride));
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (live(k)) *reinterpret_cast<uint4*>(y + (int64_t)k * kAcross * C) = w[k];
    }
}

template <int BITS, int C>
__global__ void __launch_bounds__(kWarps * 32, 6)
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
    const int64_t each = std::min<int64_t>(8, std::max<int64_t>(1, units * outer / (2 * 152 * 28)));
    return (units + each - 1) / each;
}

template <int BITS, int C>
cudaError_t launch(const FillArgs& a, int64_t outer, cudaStream_t st)
{
    constexpr int kUnit = kRows * 32 / (C / 8);
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
