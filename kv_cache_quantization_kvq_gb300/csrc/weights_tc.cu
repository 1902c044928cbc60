// weights_tc.cu -- the attention weights of many query rows, on tcgen05 tensor
// cores (kvq_attend_weights with enough rows).
//
// As in weights.cu the keys stay and the queries stream, with the product
// transposed: S^T = K Q^T puts a token in each lane of tensor memory and the
// query rows in its columns, so a token's sum over the rows is a sum over one
// thread's registers: no shuffles, no atomics, a fixed order.
//  1. pack_rows_kernel writes the query rows of every slice densely (rows
//     padded to 128 with zeros) with their base-2 log-sum-exp (+inf where a row
//     gives nothing, so that 2^(x - inf) = 0);
//  2. weights_tc_kernel, a CTA per (slice, 256 tokens, split of the rows): its
//     keys are unpacked from the codes into two swizzled M = 128 tiles once;
//     warp 8 loads tiles of 128 query rows by TMA into a ring, warps 9
//     and 10 issue the products of a key tile each into two tensor-memory
//     buffers, four groups of four warps, one per buffer, turn them into sums
//     of 2^(x - lse), a token per thread.
//  3. with several splits of the rows, join_kernel adds their sums in order.
#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kvq_chunk.cuh"
#include "kvq_fast.cuh"
#include "kvq_tc.cuh"

namespace kvq {

namespace {

using namespace rows;

constexpr int kTile = 128;
constexpr int kSumWarps = 16;                    // four per scheduler: one warp's exponentials cover another's loads
constexpr int kThreadsW = (kSumWarps + 4) * 32;

struct WtArgs {
    View v;
    const float* lse;
    const float* in;
    float* out;
    int64_t stride, R;                           // R: rows padded to 128
    const float* row;                            // [outer][R / 128][2][128]: -lse in base 2; last token seen (int bits)
    float* part;                                 // [outer][split][Tp]
    int32_t nsplit, ntok;                        // row splits, 256-token CTAs of a slice
};

__global__ void __launch_bounds__(256)
pack_rows_kernel(const View a, const float* lse, int64_t R, int C, int64_t total, __nv_bfloat16* qx, float* rows2)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= total) return;
    const int P = C / 8;
    const int64_t row = id / P;
    const int p = (int)(id - row * P);
    const int64_t o = row / R;
    const int r = (int)(row - o * R);
    uint4 x = make_uint4(0, 0, 0, 0);
    float l = -INFINITY;                         // 2^(x - inf) = 0: no weight
    int last = -1;
    if (r < a.rows) {
        const int64_t at = row_index(a, o, r);
        x = *reinterpret_cast<const uint4*>(a.q + at * C + p * 8);
        if (p == 0) {
            l = lse[at];
            l = l == -INFINITY ? -INFINITY : -__fmul_rn(l, kLog2e);
            last = a.T - a.n + r / a.group;
        }
    }
    reinterpret_cast<uint4*>(qx)[id] = x;
    if (p == 0) {
        float* at = rows2 + row / kTile * (2 * kTile) + row % kTile;
        at[0] = l;
        at[kTile] = __int_as_float(last);
    }
}

template <int C>
struct SmemW {
    static constexpr int kTileB = kTile * C * 2;
    static constexpr int kSlots = 4;
    static constexpr int kK = 0, kRing = 2 * kTileB, kLse = kRing + kSlots * kTileB, kBars = kLse + kSlots * kTile * 8;
    static constexpr int kBytes = kBars + 256 + 1024;
};

template <int BITS, int C>
__global__ void __launch_bounds__(kThreadsW, 1)
weights_tc_kernel(const WtArgs A, const __grid_constant__ CUtensorMap qmap)
{
    using S = SmemW<C>;
    using W = typename CodeWord<BITS>::T;
    constexpr int kSlots = S::kSlots, kHalves = C / 64, P = C / 8;
    __shared__ float half_sum[2][2 * kTile];
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    float4* srow = reinterpret_cast<float4*>(sm + S::kLse);        // [slot][2][32]: four rows' -lse; their last tokens
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::kBars);
    uint64_t* empty = full + kSlots;             // slot free: products done (2) and row data read (2 x 4 warps)
    uint64_t* dfull = empty + kSlots;            // [2 tiles][2 buffers]
    uint64_t* dfree = dfull + 4;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dfree + 4);
    volatile int* gone = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const View& a = A.v;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t blk = blockIdx.x;
    const int split = (int)(blk % A.nsplit);
    blk /= A.nsplit;
    const int tb = (int)(blk % A.ntok);
    const int64_t o = blk / A.ntok;
    const int t0 = tb * 2 * kTile;
    const int first = a.first ? max(a.first[o], 0) : 0;
    const int base = a.T - a.n;

    // ---- the row tiles that see any of these tokens
    const int see = max(t0, first);              // the first token that can be seen
    const int i0 = max(0, see - base);           // by query i0 and later ones
    int n0 = (int)((int64_t)i0 * a.group / kTile), n1 = (a.rows + kTile - 1) / kTile;
    if (see >= min(t0 + 2 * kTile, a.T) || i0 >= a.n) n1 = n0;
    {
        const int64_t len = max(n1 - n0, 0);
        const int e = n0 + (int)(len * (split + 1) / A.nsplit);
        n0 += (int)(len * split / A.nsplit);
        n1 = e;
    }
    const int n = n1 - n0;

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 10);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&dfull[i], 1);
            mbar_init(&dfree[i], 4);
        }
        *gone = 0;
        mbar_init_fence();
    }
    if (warp == kSumWarps + 1) tc::alloc(tmem_slot, 512);
    // ---- the keys: row = token, 16-byte pieces of 8 channels; hidden tokens are zeros
    if (n > 0) {
#pragma unroll 4
        for (int k = tid; k < 2 * kTile * P; k += kThreadsW) {
            const int row = k / P, p = k % P, t = t0 + row;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (t >= first && t < a.T) {
                if (t >= a.tq) {
                    x = *reinterpret_cast<const uint4*>(a.kr + ((uint64_t)o * a.rrows + (t - a.tq)) * C + p * 8);
                } else {
                    const int64_t at = (o * a.ngk + t / a.gk) * C + p * 8;
                    Raw8<__nv_bfloat16> rs, rz;
                    load_raw8(a.ks + at, rs);
                    float s[8], z[8], v[8];
                    widen8(rs, s);
                    if (a.kz) {
                        load_raw8(a.kz + at, rz);
                        widen8(rz, z);
                    }
                    W w = *reinterpret_cast<const W*>(a.kc + ((uint64_t)o * a.cap + t) * (C * BITS / 8) + p * BITS);
                    w ^= (W)a.kflip;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float c = __fsub_rn((float)((w >> (BITS * i)) & ((1 << BITS) - 1)), a.koff);
                        v[i] = __fmul_rn(a.kz ? __fsub_rn(c, z[i]) : c, s[i]);
                    }
                    store8(reinterpret_cast<__nv_bfloat16*>(&x), v);
                }
            }
            *reinterpret_cast<uint4*>(sm + S::kK + (row / kTile) * S::kTileB + (p / 8) * (kTile * 128) +
                                      tc::swizzled(row % kTile, p % 8)) = x;
        }
        tc::async_fence();
    }
    tc::before_sync();
    __syncthreads();
    tc::after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp == kSumWarps) {
        int it = 0;
        for (; it < n; ++it) {
            const int s = it % kSlots;
            if (it >= kSlots && !__all_sync(0xFFFFFFFFu, tc::wait(&empty[s], ((it / kSlots) - 1) & 1, gone))) break;
            if (tc::elect()) {
                mbar_expect_tx(&full[s], S::kTileB + kTile * 8);
                const int64_t row = o * A.R + (int64_t)(n0 + it) * kTile;
                for (int h = 0; h < kHalves; ++h)
                    tma_load_2d(sm + S::kRing + s * S::kTileB + h * (kTile * 128), &qmap, h * 64, (int)row, &full[s]);
                bulk_g2s(srow + s * (kTile / 2), A.row + row * 2, kTile * 8, &full[s]);
            }
            __syncwarp();
        }
        // every copy issued lands before the CTA's shared memory goes
        for (int i = max(0, it - kSlots); i < it; ++i) tc::drain(&full[i % kSlots], (i / kSlots) & 1);
    } else if (warp == kSumWarps + 1 || warp == kSumWarps + 2) {
        // ---- products of key tile t
        const int t = warp - kSumWarps - 1;
        constexpr uint32_t kDesc = tc::instr_desc(kTile, kTile, false);
        const uint32_t k_at = smem_u32(sm + S::kK) + t * S::kTileB, ring = smem_u32(sm + S::kRing);
        auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, tc::wait(bar, parity, gone)) != 0; };
        for (int it = 0; it < n; ++it) {
            const int s = it % kSlots, b = it & 1;
            if (!ready(&full[s], (it / kSlots) & 1)) break;
            if (it >= 2 && !ready(&dfree[2 * t + b], ((it >> 1) - 1) & 1)) break;
            tc::after_sync();
            if (tc::elect()) {
#pragma unroll
                for (int k = 0; k < C / 16; ++k) {
                    const uint32_t at = (k / 4) * (kTile * 128) + (k % 4) * 32;
                    tc::mma_ss(tmem + (2 * t + b) * kTile, tc::smem_desc(k_at + at, 16),
                               tc::smem_desc(ring + s * S::kTileB + at, 16), kDesc, k > 0);
                }
                tc::commit(&dfull[2 * t + b]);
                tc::commit(&empty[s]);
            }
            __syncwarp();
        }
    } else if (warp < kSumWarps) {
        // ---- a thread per token of tile t and buffer b (every second row tile): sum of 2^(x - lse)
        const int t = (warp >> 2) & 1, b = warp >> 3;
        const int tok = t0 + t * kTile + (warp & 3) * 32 + lane;
        const int tile_hi = t0 + t * kTile + kTile - 1;
        const uint32_t d_at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (2 * t + b) * kTile;
        const u64 sc2 = pk(a.scale2, a.scale2);
        float sum = 0.0f;
        for (int it = b; it < n; it += 2) {
            const int s = it % kSlots;
            bool ok = tc::wait(&full[s], (it / kSlots) & 1, gone) && tc::wait(&dfull[2 * t + b], (it >> 1) & 1, gone);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc::after_sync();
            const int row0 = (n0 + it) * kTile;
            const bool cut = tile_hi > base + row0 / a.group;       // some row does not see some token
            const float4* rp = srow + s * (kTile / 2);
            u64 acc0 = 0, acc1 = 0;
            if (!cut) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t y[32];
                    tc::ld32(d_at + 32 * h, y);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 l = rp[8 * h + i];
                        const u64 e0 = fma2(pk(__uint_as_float(y[4 * i]), __uint_as_float(y[4 * i + 1])), sc2, pk(l.x, l.y));
                        const u64 e1 = fma2(pk(__uint_as_float(y[4 * i + 2]), __uint_as_float(y[4 * i + 3])), sc2, pk(l.z, l.w));
                        acc0 = add2(acc0, pk(ex2(lo_of(e0)), ex2(hi_of(e0))));
                        acc1 = add2(acc1, pk(ex2(lo_of(e1)), ex2(hi_of(e1))));
                    }
                }
            } else {
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {
                    uint32_t y[32];
                    tc::ld32(d_at + 32 * h, y);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 l = rp[8 * h + i], z = rp[kTile / 4 + 8 * h + i];
                        const u64 e0 = fma2(pk(__uint_as_float(y[4 * i]), __uint_as_float(y[4 * i + 1])), sc2, pk(l.x, l.y));
                        const u64 e1 = fma2(pk(__uint_as_float(y[4 * i + 2]), __uint_as_float(y[4 * i + 3])), sc2, pk(l.z, l.w));
                        acc0 = add2(acc0, pk(tok <= __float_as_int(z.x) ? ex2(lo_of(e0)) : 0.0f,
                                             tok <= __float_as_int(z.y) ? ex2(hi_of(e0)) : 0.0f));
                        acc1 = add2(acc1, pk(tok <= __float_as_int(z.z) ? ex2(lo_of(e1)) : 0.0f,
                                             tok <= __float_as_int(z.w) ? ex2(hi_of(e1)) : 0.0f));
                    }
                }
            }
            tc::before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&dfree[2 * t + b]);
                mbar_arrive(&empty[s]);
            }
            const u64 acc = add2(acc0, acc1);
            sum = __fadd_rn(sum, __fadd_rn(lo_of(acc), hi_of(acc)));
        }
        half_sum[b][t * kTile + (warp & 3) * 32 + lane] = sum;
    }
    __syncwarp();
    tc::before_sync();
    __syncthreads();
    tc::after_sync();
    if (warp == kSumWarps + 1) tc::dealloc(tmem, 512);
    if (tid < 2 * kTile && t0 + tid < a.T && !*gone) {
        const int tok = t0 + tid;
        const float sum = tok < first ? 0.0f : __fadd_rn(half_sum[0][tid], half_sum[1][tid]);
        if (A.nsplit > 1) {
            A.part[(o * A.nsplit + split) * ((int64_t)A.ntok * 2 * kTile) + tok] = sum;
        } else {
            const int64_t at = o * A.stride + tok;
            A.out[at] = A.in ? __fadd_rn(A.in[at], sum) : sum;
        }
    }
}

__global__ void __launch_bounds__(256)
join_kernel(const WtArgs A, int64_t total)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= total) return;
    const int64_t o = id / A.v.T, t = id - o * A.v.T, Tp = (int64_t)A.ntok * 2 * kTile;
    float s = 0.0f;
    for (int k = 0; k < A.nsplit; ++k) s = __fadd_rn(s, A.part[(o * A.nsplit + k) * Tp + t]);
    const int64_t at = o * A.stride + t;
    A.out[at] = A.in ? __fadd_rn(A.in[at], s) : s;
}

constexpr int64_t kMaxCtas = 8 * 152;             // more CTAs than this are not split further

struct WtPlan { int64_t R, ntok, nsplit; };

WtPlan wt_plan(int64_t outer, int64_t T, int64_t rows)
{
    WtPlan p;
    p.R = (rows + kTile - 1) / kTile * kTile;
    p.ntok = (T + 2 * kTile - 1) / (2 * kTile);
    // Splits of the rows that leave the least idle at the end: waves of 152 CTAs,
    // each the row tiles of a split and the time of about three to lay out its keys.
    const int64_t ctas = std::max<int64_t>(outer * p.ntok, 1), tiles = p.R / kTile;
    p.nsplit = 1;
    int64_t best = INT64_MAX;
    for (int64_t s = 1; s == 1 || (s <= tiles && ctas * s <= kMaxCtas); ++s) {
        const int64_t cost = ((ctas * s + 151) / 152) * ((tiles + s - 1) / s + 3);
        if (cost < best) {
            best = cost;
            p.nsplit = s;
        }
    }
    return p;
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

template <int BITS, int C>
cudaError_t launch_wt(WtArgs A, int64_t outer, void* ws, cudaStream_t st)
{
    const WtPlan p = wt_plan(outer, A.v.T, A.v.rows);
    char* at = static_cast<char*>(ws);
    __nv_bfloat16* qx = reinterpret_cast<__nv_bfloat16*>(at);
    at += round256((size_t)(outer * p.R * C) * 2);
    float* rows2 = reinterpret_cast<float*>(at);
    at += round256((size_t)(outer * p.R) * 8);
    A.R = p.R;
    A.row = rows2;
    A.part = reinterpret_cast<float*>(at);
    A.nsplit = (int32_t)p.nsplit;
    A.ntok = (int32_t)p.ntok;
    const int64_t packs = outer * p.R * (C / 8), grid = outer * p.ntok * p.nsplit;
    if (outer * p.R > 0x7FFFFFFF || grid > 0x7FFFFFFF || packs / 256 >= 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    CUtensorMap qm;
    if (!encode_rows_tile_map(qx, outer * p.R, C, &qm)) return cudaErrorNotSupported;
    cudaError_t e = ensure_kernel_attrs(reinterpret_cast<const void*>(weights_tc_kernel<BITS, C>), SmemW<C>::kBytes);
    if (e != cudaSuccess) return e;
    pack_rows_kernel<<<(unsigned)((packs + 255) / 256), 256, 0, st>>>(A.v, A.lse, p.R, C, packs, qx, rows2);
    weights_tc_kernel<BITS, C><<<(unsigned)grid, kThreadsW, SmemW<C>::kBytes, st>>>(A, qm);
    if (p.nsplit > 1) {
        const int64_t total = outer * A.v.T;
        join_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(A, total);
    }
    return cudaGetLastError();
}

}  // namespace

bool weights_use_tc(int64_t rows) { return rows > 64; }

size_t weights_tc_workspace(int64_t outer, int64_t C, int64_t rows)
{
    const int64_t R = (rows + kTile - 1) / kTile * kTile;
    size_t b = round256((size_t)(outer * R * C) * 2) + round256((size_t)(outer * R) * 8);
    if (R > kTile) b += (size_t)kMaxCtas * 2 * kTile * 4;
    return b;
}

cudaError_t launch_weights_tc(const rows::View& v, const float* lse, const float* in, float* out, int64_t stride,
                              int bits, int64_t C, int64_t outer, void* ws, cudaStream_t st)
{
    WtArgs A = {};
    A.v = v;
    A.lse = lse;
    A.in = in;
    A.out = out;
    A.stride = stride;
    if (bits == 4) return C == 128 ? launch_wt<4, 128>(A, outer, ws, st) : launch_wt<4, 64>(A, outer, ws, st);
    return C == 128 ? launch_wt<2, 128>(A, outer, ws, st) : launch_wt<2, 64>(A, outer, ws, st);
}

}  // namespace kvq
