// weights_tc.cu -- the attention weights of many query rows, on tcgen05 tensor
// cores (kvq_attend_weights with enough rows).
//
// As in weights.cu the keys stay and the queries stream, with the product
// transposed: S^T = K Q^T puts a token in each lane of tensor memory and the
// query rows in its columns, so a token's sum over the rows is a sum over one
// thread's registers: no shuffles, no atomics, a fixed order.
//  1. pack_rows_kernel writes the query rows of every slice densely, with -lse in
//     base 2 and the last token a row sees (-1 where it gives nothing: a tile with
//     such a row takes the masked sums, for its scores may be NaN).  The last row is
//     repeated to a multiple of 128 rows, with -lse = -inf: zeros there would make
//     NaN of an infinite key that gives every real row a weight of 0;
//  2. weights_tc_kernel, one CTA a SM, walks jobs of 256 tokens (and a split of
//     the rows): eight fill warps unpack the next job's keys into two swizzled
//     M = 128 tiles (kvq_fill.cuh) while the current ones are in use; one warp loads tiles of 128
//     query rows by TMA into a ring, two issue the products of a key tile each
//     into two tensor-memory buffers, four groups of four warps, one per buffer,
//     turn them into sums of 2^(x - lse), a token per thread;
//  3. with several splits of the rows, join_kernel adds their sums in order.
// Measured on one GB300: 2048 queries x 4 heads over 16384 tokens and 8 slices 238
// us (1.08 PFLOP/s; tensor cores 52 % busy, issue slots 60 %: a value costs one
// exponential and two packed operations).  63 queries x 4 heads over 32774 tokens
// and 16 slices 80.5 us, bound by the latency of the fill; a CTA per job, its keys
// filled before its products, took 146.  At 72 registers the kernel spills 124 to 136
// bytes.
#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kvq_chunk.cuh"
#include "kvq_fill.cuh"

namespace kvq {

namespace {

using namespace rows;

using fill::interleave;
using fill::kTile;
using fill::Staged;
constexpr int kSumWarps = 16;                    // four per scheduler: one warp's exponentials cover another's loads
constexpr int kFillWarp = kSumWarps + 4;         // 16: query tiles, 17 and 18: products, 19: codes, 20-27: fill
constexpr int kThreadsW = (kFillWarp + 8) * 32;

struct WtArgs {
    View v;
    const float* lse;
    const float* in;
    float* out;
    int64_t stride, R;                           // R: rows padded to 128
    const float* row;                            // [outer][R / 128][2][128]: -lse in base 2; last token seen (int bits)
    float* part;                                 // [outer][split][Tp]
    int32_t nsplit, ntok;                        // row splits, 256-token jobs of a slice
    int64_t jobs, outer;                         // slices x splits x ntok; slices
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
    const int real = min(r, a.rows - 1);
    const int64_t at = row_index(a, o, real);
    const uint4 x = interleave(*reinterpret_cast<const uint4*>(a.q + at * C + p * 8));
    float l = -INFINITY;
    int last = -1;                               // gives nothing
    if (p == 0) {
        l = lse[at];
        l = l == -INFINITY ? -INFINITY : -__fmul_rn(l, kLog2e);
        if (l != -INFINITY) last = a.T - a.n + real / a.group;
        if (r > real) l = -INFINITY;
    }
    reinterpret_cast<uint4*>(qx)[id] = x;
    if (p == 0) {
        float* to = rows2 + row / kTile * (2 * kTile) + row % kTile;
        to[0] = l;
        to[kTile] = __int_as_float(last);
    }
}

template <int BITS, int C>
struct SmemW {
    static constexpr int kTileB = kTile * C * 2;
    static constexpr int kSlots = 2, kRowSlots = 4;                 // rings of query tiles and of their rows' data
    static constexpr int kK = 0, kRing = 4 * kTileB;                // two jobs' two key tiles
    static constexpr int kRows = kRing + kSlots * kTileB, kHalf = kRows + kRowSlots * kTile * 8;
    static constexpr int kRaw = kHalf + 2 * 2 * kTile * 4, kBars = kRaw + Staged<BITS, C, true>::kBytes;
    static constexpr int kBytes = kBars + 512 + 1024;
};

// A job: 256 tokens from t0 of slice o, row tiles [n0, n0 + n).  Each role walks
// its CTA's jobs by next(): worked out from the job's number every time, the
// divisions took longer than a row tile.
struct Job {
    int64_t o;
    int tb, t0, n0, n, split, first;
    __device__ __forceinline__ Job(const WtArgs& A, int64_t job) {
        tb = (int)(job % A.ntok);
        job /= A.ntok;
        split = (int)(job % A.nsplit);
        o = job / A.nsplit;
        slice(A);
        rows(A);
    }
    __device__ __forceinline__ void next(const WtArgs& A) {
        if (++tb == A.ntok) {
            tb = 0;
            if (++split == A.nsplit) {
                split = 0;
                if (++o < A.outer) slice(A);
            }
        }
        rows(A);
    }
    __device__ __forceinline__ void slice(const WtArgs& A) { first = padding(A.v, o); }
    __device__ __forceinline__ void rows(const WtArgs& A) {
        const View& a = A.v;
        t0 = tb * 2 * kTile;
        // the row tiles that see any of these tokens: from the first query that does
        const int see = max(t0, first), i0 = max(0, see - (a.T - a.n));
        int lo = (int)((int64_t)i0 * a.group / kTile), hi = (a.rows + kTile - 1) / kTile;
        if (see >= min(t0 + 2 * kTile, a.T) || i0 >= a.n) hi = lo;
        const int len = max(hi - lo, 0);
        n0 = lo;
        n = len;
        if (A.nsplit > 1) {
            n0 = lo + (int)((int64_t)len * split / A.nsplit);
            n = lo + (int)((int64_t)len * (split + 1) / A.nsplit) - n0;
        }
    }
};

template <int BITS, int C>
__global__ void __launch_bounds__(kThreadsW, 1)
weights_tc_kernel(const __grid_constant__ WtArgs A, const __grid_constant__ CUtensorMap qmap)
{
    using S = SmemW<BITS, C>;
    constexpr int kSlots = S::kSlots, kHalves = C / 64;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    float4* srow = reinterpret_cast<float4*>(sm + S::kRows);       // [slot][2][32]: four rows' -lse; their last tokens
    float* half = reinterpret_cast<float*>(sm + S::kHalf);         // [job parity][2 tiles][128]: sums of odd row tiles
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::kBars);   // [slot] a query tile has landed
    uint64_t* empty = full + kSlots;             // [slot] both products are done with it
    uint64_t* rfull = empty + kSlots;            // [row slot] the same for -lse and last tokens (2 x 4 warps read them)
    uint64_t* rempty = rfull + S::kRowSlots;
    uint64_t* kfull = rempty + S::kRowSlots;     // [job parity][2] a key tile is filled (8 warps)
    uint64_t* kfree = kfull + 4;                 // [job parity] both products are done with them
    uint64_t* dfull = kfree + 2;                 // [2 tiles][2 buffers]
    uint64_t* dfree = dfull + 4;
    uint64_t* hfull = dfree + 4;                 // [2 tiles][job parity] the odd groups' sums are there
    uint64_t* hfree = hfull + 4;
    uint64_t* raw_bars = hfree + 4;              // [full, free][3] of the staged codes
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(raw_bars + 6);
    volatile int* gone = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const View& a = A.v;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t job0 = A.jobs * blockIdx.x / gridDim.x, job1 = A.jobs * (blockIdx.x + 1) / gridDim.x;

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 2);
        }
        for (int i = 0; i < S::kRowSlots; ++i) {
            mbar_init(&rfull[i], 1);
            mbar_init(&rempty[i], 8);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&kfree[i], 2);
        for (int i = 0; i < 6; ++i) mbar_init(&raw_bars[i], i < 3 ? 1 : 4);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&kfull[i], 8);
            mbar_init(&dfull[i], 1);
            mbar_init(&dfree[i], 4);
            mbar_init(&hfull[i], 4);
            mbar_init(&hfree[i], 4);
        }
        *gone = 0;
        mbar_init_fence();
    }
    if (warp == kSumWarps + 1) tc::alloc(tmem_slot, 512);
    tc::before_sync();
    __syncthreads();
    tc::after_sync();
    const uint32_t tmem = *tmem_slot;
    auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, tc::wait(bar, parity, gone)) != 0; };
    // every role walks the jobs alike; `it` counts row tiles and `k` jobs with any, over the whole CTA

    if (warp >= kFillWarp - 1) {
        // ---- keys, and (warp 19) the copies of their codes: runs of jobs that go on in the same slice
        int k = 0, staged = 0;
        bool ok = true;
        Job J(A, job0);
        for (int64_t job = job0; ok && job < job1;) {
            const int64_t o = J.o;
            const int split = J.split, first = J.first, j0 = J.t0 / kTile;
            const bool any = J.n > 0;
            int tiles = 0;
            do {
                ++job;
                tiles += 2;
                J.next(A);
            } while (job < job1 && J.o == o && J.split == split && (J.n > 0) == any);
            if (!any) continue;
            Staged<BITS, C, true> f(a, o, first, j0, tiles, tid & 127, (warp - kFillWarp) >> 2 & 1, sm + S::kRaw, raw_bars,
                                    raw_bars + 3, staged);
            staged += f.staged();
            if (warp < kFillWarp) {
                ok = f.produce(ready);
                continue;
            }
            ok = f.run(j0, tiles, ready,
                       [&](int j) -> unsigned char* {
                           const int c = k + (j >> 1);              // the job's number among those with any row
                           if (!(j & 1) && c >= 2 && !ready(&kfree[c & 1], ((c >> 1) - 1) & 1)) return nullptr;
                           return sm + S::kK + (2 * (c & 1) + (j & 1)) * S::kTileB;
                       },
                       [&](int j) {
                           tc::async_fence();
                           __syncwarp();
                           if (lane == 0) mbar_arrive(&kfull[2 * ((k + (j >> 1)) & 1) + (j & 1)]);
                       });
            k += tiles >> 1;
        }
    } else if (warp == kSumWarps) {
        // ---- query tiles
        int it = 0;
        bool ok = true;
        Job J(A, job0);
        for (int64_t job = job0; ok && job < job1; ++job, J.next(A)) {
            for (int i = 0; i < J.n; ++i, ++it) {
                const int s = it % kSlots, rs = it % S::kRowSlots;
                if (it >= kSlots) ok = ready(&empty[s], ((it / kSlots) - 1) & 1);
                if (ok && it >= S::kRowSlots) ok = ready(&rempty[rs], ((it / S::kRowSlots) - 1) & 1);
                if (!ok) break;
                if (tc::elect()) {
                    const int64_t row = J.o * A.R + (int64_t)(J.n0 + i) * kTile;
                    mbar_expect_tx(&rfull[rs], kTile * 8);
                    bulk_g2s(srow + rs * (kTile / 2), A.row + row * 2, kTile * 8, &rfull[rs]);
                    mbar_expect_tx(&full[s], S::kTileB);
                    for (int h = 0; h < kHalves; ++h)
                        tma_load_2d(sm + S::kRing + s * S::kTileB + h * (kTile * 128), &qmap, h * 64, (int)row, &full[s]);
                }
                __syncwarp();
            }
        }
        // every copy issued lands before the CTA's shared memory goes
        for (int i = max(0, it - kSlots); i < it; ++i) tc::drain(&full[i % kSlots], (i / kSlots) & 1);
        for (int i = max(0, it - S::kRowSlots); i < it; ++i) tc::drain(&rfull[i % S::kRowSlots], (i / S::kRowSlots) & 1);
    } else if (warp == kSumWarps + 1 || warp == kSumWarps + 2) {
        // ---- products of key tile t
        const int t = warp - kSumWarps - 1;
        constexpr uint32_t kDesc = tc::instr_desc(kTile, kTile, false);
        const uint32_t ring = smem_u32(sm + S::kRing);
        int it = 0, k = 0;
        bool ok = true;
        Job J(A, job0);
        for (int64_t job = job0; ok && job < job1; ++job, J.next(A)) {
            if (J.n == 0) continue;
            const uint32_t k_at = smem_u32(sm + S::kK) + (2 * (k & 1) + t) * S::kTileB;
            ok = ready(&kfull[2 * (k & 1) + t], (k >> 1) & 1);
            for (int i = 0; ok && i < J.n; ++i, ++it) {
                const int s = it % kSlots, b = it & 1;
                ok = ready(&full[s], (it / kSlots) & 1) && (it < 2 || ready(&dfree[2 * t + b], ((it >> 1) - 1) & 1));
                if (!ok) break;
                tc::after_sync();
                if (tc::elect()) {
#pragma unroll
                    for (int c = 0; c < C / 16; ++c) {
                        const uint32_t at = (c / 4) * (kTile * 128) + (c % 4) * 32;
                        tc::mma_ss(tmem + (2 * t + b) * kTile, tc::smem_desc(k_at + at, 16),
                                   tc::smem_desc(ring + s * S::kTileB + at, 16), kDesc, c > 0);
                    }
                    tc::commit(&dfull[2 * t + b]);
                    tc::commit(&empty[s]);
                    if (i == J.n - 1) tc::commit(&kfree[k & 1]);
                }
                __syncwarp();
            }
            ++k;
        }
    } else if (warp < kSumWarps) {
        // ---- a thread per token of tile t and buffer b (every second row tile): sum of 2^(x - lse)
        const int t = (warp >> 2) & 1, b = warp >> 3, me = (warp & 3) * 32 + lane;
        const uint32_t d_at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (2 * t + b) * kTile;
        const u64 sc2 = pk(a.scale2, a.scale2);
        int it = 0, k = 0;
        bool ok = true;
        Job J(A, job0);
        for (int64_t job = job0; ok && job < job1; ++job, J.next(A)) {
            const int tok = J.t0 + t * kTile + me, tile_hi = J.t0 + t * kTile + kTile - 1;
            float sum = 0.0f;
            for (int i = 0; i < J.n; ++i, ++it) {
                if ((it & 1) != b) continue;
                const int s = it % S::kRowSlots;
                ok = ready(&rfull[s], (it / S::kRowSlots) & 1) && ready(&dfull[2 * t + b], (it >> 1) & 1);
                if (!ok) break;
                tc::after_sync();
                const float4* rp = srow + s * (kTile / 2);
                const float4 z4 = rp[kTile / 4 + lane];
                const int fewest = __reduce_min_sync(0xFFFFFFFFu, min(min(__float_as_int(z4.x), __float_as_int(z4.y)),
                                                                     min(__float_as_int(z4.z), __float_as_int(z4.w))));
                const bool cut = tile_hi > fewest;                  // some row does not see some token, or gives nothing
                u64 acc0 = 0, acc1 = 0;
                if (!cut) {
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
                        uint32_t y[32];
                        tc::ld32(d_at + 32 * h, y);
                        tc::wait_ld();
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float4 l = rp[8 * h + c];
                            const u64 e0 = fma2(pk(__uint_as_float(y[4 * c]), __uint_as_float(y[4 * c + 1])), sc2, pk(l.x, l.y));
                            const u64 e1 = fma2(pk(__uint_as_float(y[4 * c + 2]), __uint_as_float(y[4 * c + 3])), sc2, pk(l.z, l.w));
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
                        for (int c = 0; c < 8; ++c) {
                            const float4 l = rp[8 * h + c], z = rp[kTile / 4 + 8 * h + c];
                            const u64 e0 = fma2(pk(__uint_as_float(y[4 * c]), __uint_as_float(y[4 * c + 1])), sc2, pk(l.x, l.y));
                            const u64 e1 = fma2(pk(__uint_as_float(y[4 * c + 2]), __uint_as_float(y[4 * c + 3])), sc2, pk(l.z, l.w));
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
                    mbar_arrive(&rempty[s]);
                }
                const u64 acc = add2(acc0, acc1);
                sum = __fadd_rn(sum, __fadd_rn(lo_of(acc), hi_of(acc)));
            }
            if (!ok) break;
            // the odd group hands its sums to the even one, which writes
            const int hp = k & 1;
            float* hs = half + (hp * 2 + t) * kTile + me;
            if (b == 1) {
                if (k >= 2 && !(ok = ready(&hfree[2 * t + hp], ((k >> 1) - 1) & 1))) break;
                *hs = sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(&hfull[2 * t + hp]);
            } else {
                if (!(ok = ready(&hfull[2 * t + hp], (k >> 1) & 1))) break;
                sum = tok < J.first ? 0.0f : __fadd_rn(sum, *hs);
                __syncwarp();
                if (lane == 0) mbar_arrive(&hfree[2 * t + hp]);
                if (tok < a.T) {
                    if (A.nsplit > 1) {
                        A.part[(J.o * A.nsplit + J.split) * ((int64_t)A.ntok * 2 * kTile) + tok] = sum;
                    } else {
                        const int64_t at = J.o * A.stride + tok;
                        A.out[at] = A.in ? __fadd_rn(A.in[at], sum) : sum;
                    }
                }
            }
            ++k;                                 // counts every job here
        }
    }
    __syncwarp();
    tc::before_sync();
    __syncthreads();
    tc::after_sync();
    if (warp == kSumWarps + 1) tc::dealloc(tmem, 512);
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

constexpr int64_t kMaxCtas = 8 * 152;             // more jobs than this are not split further

struct WtPlan { int64_t R, ntok, nsplit; };

WtPlan wt_plan(int64_t outer, int64_t T, int64_t rows)
{
    WtPlan p;
    p.R = (rows + kTile - 1) / kTile * kTile;
    p.ntok = (T + 2 * kTile - 1) / (2 * kTile);
    // Splits of the rows that leave the least idle at the end: rounds of 152 jobs,
    // each its row tiles, or the time of about three to unpack the next job's keys.
    const int64_t jobs = std::max<int64_t>(outer * p.ntok, 1), tiles = p.R / kTile;
    p.nsplit = 1;
    int64_t best = INT64_MAX;
    for (int64_t s = 1; s == 1 || (s <= tiles && jobs * s <= kMaxCtas); ++s) {
        const int64_t cost = (jobs * s + 151) / 152 * std::max<int64_t>((tiles + s - 1) / s + 1, 3);
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
    const int64_t packs = outer * p.R * (C / 8);
    A.jobs = outer * p.ntok * p.nsplit;
    A.outer = outer;
    if (outer * p.R > 0x7FFFFFFF || packs / 256 >= 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    CUtensorMap qm;
    if (!encode_rows_tile_map(qx, outer * p.R, C, &qm)) return cudaErrorNotSupported;
    cudaError_t e = ensure_kernel_attrs(reinterpret_cast<const void*>(weights_tc_kernel<BITS, C>), (SmemW<BITS, C>::kBytes));
    if (e != cudaSuccess) return e;
    pack_rows_kernel<<<(unsigned)((packs + 255) / 256), 256, 0, st>>>(A.v, A.lse, p.R, C, packs, qx, rows2);
    weights_tc_kernel<BITS, C><<<(unsigned)std::min<int64_t>(A.jobs, 152), kThreadsW, (SmemW<BITS, C>::kBytes), st>>>(A, qm);
    if (p.nsplit > 1) {
        const int64_t total = outer * A.v.T;
        join_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(A, total);
    }
    return cudaGetLastError();
}

}  // namespace

// Rows from which this form is taken (64 slices of 32768 tokens: 64 rows 205 us on
// mma.sync and 268 here, where the time hardly moves up to 256 rows).
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
