// prompts.cu -- causal attention over packed prompts in bf16, on tcgen05 tensor
// cores (kvq_attend_prompts).
//
// "KV cache 压缩：把历史装得更小" §"K 的误差会改变权重，V 的误差会改变内容" (logit_t = q^T k_t /
// sqrt(d), y = sum_t a_t v_t), before anything is compressed: prompt s is the rows
// starts[s] .. starts[s + 1] of q, k and v.
//
// One pass over the keys with the running maximum and sum of the softmax in base 2
// (the online softmax of Milakov and Gimelshein, 2018), as in prefill.cu: the
// products of 256 query rows cost 4 * 256 C operations a key, its bytes are 4 C, so
// the tensor cores and the exponentials bound it, and memory does where prompts
// are short.
//  1. plan_kernel, one CTA, cuts the prompts into items of two row tiles, the
//     longest first.  A row tile is tpt = 128 / group whole tokens with their
//     `group` query heads, which read the same keys: rows lie token by token, so
//     a tile spans few tokens and little of the diagonal's key tile is wasted.
//  2. prompts_kernel, one CTA a SM, walks (item, KV head) pairs, those of a round
//     in turn forwards and backwards, so that long and short ones add up alike.
//     Warp 8 copies query, key and value tiles by TMA (straight from the packed
//     tensors: a box of 64 channels x group heads x tpt tokens is a row tile);
//     warps 9 and 10 issue the products of a row tile each; warps 0-3 and 4-7 are the
//     softmax of the row tiles, a thread per row: S from tensor memory into
//     registers, P in bf16 over the same columns, which the value product reads
//     from there; warp 11 looks through every value tile for numbers that are not
//     finite.  All of them run on into the next pair, whose queries and first
//     keys arrive while the last one's output is written.
//     The running maximum is moved (and the output rescaled) only when it grows by
//     more than 2^8: the weights are then at most 256, which costs float32 sums and
//     bf16 weights no relative precision.
// A tile's last rows of keys and values may be another prompt's, or tokens that a
// row does not see.  Their weights are 0, and values enter a product as 0 where they
// are not finite (0 times NaN would reach every row); what a row sees of them is
// added when it is written.
// The weights enter the value product as one bf16 (its operands are of one type): an
// error of 2^-8 of each weight at most, the size of out's own rounding.
//
// Measured on one GB300 (C = 128, 8 KV heads x 4): one prompt of 32768 tokens 5.6 ms (1.57 PFLOP/s, tensor cores
// bound), 64 prompts of 16 to 2000 tokens 263 us, one of 17 tokens 7.1 us (a launch's way through one tile).  At C = 64 no
// unit is half busy (5 prompts of 1501 to 4001 tokens x 12 heads 105 us: tensor pipe 34 %, issue slots 39 %, exponentials 34
// %): a row tile's chain scores -> weights -> values bounds it.
// Key tiles of 64 tokens: 6.6 ms | 262 us; the scores' halves handed over one by one: 6.06 ms.
#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kvq_fast.cuh"
#include "kvq_plan.cuh"
#include "kvq_rows.cuh"
#include "kvq_tc.cuh"

namespace kvq {

namespace {

using namespace rows;
using namespace plan;

constexpr int kThreads = 384;                    // 12 warps, 168 registers each at launch (64512 in all):
constexpr int kRegsSoftmax = 216;                // 8 softmax warps take 216 and the other four keep 56
constexpr int kRegsOther = 56;                   // (62464), so a row of 128 scores stays in registers
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "registers of the launch");
constexpr float kSlack = 8.0f;                   // base-2 growth of the maximum that is let pass

// ---------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 64 + 19 * 16;           // of numbers of key tiles: exact below 64, in sixteenths of powers of 2 above
constexpr int kAlone = 8;                        // items of a prompt that its thread makes; a warp shares the others

__device__ __forceinline__ int bucket_of(int keys) {                // larger numbers first
    int b = keys;
    if (keys >= 64) {
        const int e = 31 - __clz(keys);
        b = 64 + (e - 6) * 16 + ((keys >> (e - 4)) & 15);
    }
    return kBuckets - 1 - min(b, kBuckets - 1);
}

// What the prompts before this thread's ask for in this pass of the prompts, and in `all` what all of the pass do; n: its
// own.  Out of line: prompts in order never come here.
struct Asked { int64_t before, all; };
__device__ __noinline__ Asked asked_in_pass(int n, int64_t* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t upto = n;
#pragma unroll 1
    for (int d = 1; d < 32; d *= 2) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += x;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    Asked r = {upto - n, 0};
#pragma unroll 1
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) r.before += sums[w];
        r.all += sums[w];
    }
    __syncthreads();
    return r;
}

// The order of items in a bucket is not fixed, and nothing depends on it.  Starts in order make `cap` items at most.
// Others may ask for any number: of those the first `cap` are made, in the prompts' order, so that neither the counts
// nor the work grow beyond what a well-formed call has.
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const int32_t* starts, int64_t prompts, int64_t total, int tpt, int cap, Plan* plan)
{
    __shared__ int at[kBuckets];
    __shared__ int64_t sums[kPlanThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31;
    Item* items = reinterpret_cast<Item*>(plan + 1);
    int begin0 = 0, len0 = 0;                    // the thread's prompt of the first pass
    bool wild = false;
    if (tid < prompts) {
        prompt_range(starts, tid, total, begin0, len0);
        wild = starts[tid + 1] < starts[tid];
    }
#pragma unroll 4
    for (int64_t s = tid + kPlanThreads; s < prompts; s += kPlanThreads) wild |= starts[s + 1] < starts[s];
    auto each = [&](auto use) {                  // use(item) for every item
        int64_t before = 0;                      // wild: what the prompts before s0 ask for
        for (int64_t s0 = 0; s0 < prompts; s0 += kPlanThreads) {
            const int64_t s = s0 + tid;
            int begin = begin0, len = len0;
            if (s0 > 0) {
                begin = len = 0;
                if (s < prompts) prompt_range(starts, s, total, begin, len);
            }
            int n = items_of(len, tpt);
            if (__builtin_expect(wild, 0)) {
                const Asked x = asked_in_pass(n, sums);
                n = items_left(before + x.before, n, cap);
                before += x.all;
            }
            for (int i = 0; i < min(n, kAlone); ++i) use(item_at(begin, len, i, tpt));
            for (uint32_t more = __ballot_sync(0xFFFFFFFFu, n > kAlone); more; more &= more - 1) {
                const int from = __ffs(more) - 1;
                const int b = __shfl_sync(0xFFFFFFFFu, begin, from), l = __shfl_sync(0xFFFFFFFFu, len, from);
                const int m = __shfl_sync(0xFFFFFFFFu, n, from);
                for (int i = kAlone + lane; i < m; i += 32) use(item_at(b, l, i, tpt));
            }
            if (before >= cap) break;
        }
    };
    for (int i = tid; i < kBuckets; i += kPlanThreads) at[i] = 0;
    wild = __syncthreads_or(wild);
    each([&](const Item& x) { atomicAdd(&at[bucket_of(x.keys)], 1); });
    __syncthreads();
    if (tid < 32) {                              // exclusive sums
        constexpr int kPer = (kBuckets + 31) / 32;
        int mine = 0;
        for (int i = lane * kPer; i < min((lane + 1) * kPer, kBuckets); ++i) mine += at[i];
        int before = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int x = __shfl_up_sync(0xFFFFFFFFu, before, d);
            if (lane >= d) before += x;
        }
        if (lane == 31) plan->count = min(before, cap);
        before -= mine;
        for (int i = lane * kPer; i < min((lane + 1) * kPer, kBuckets); ++i) {
            const int n = at[i];
            at[i] = before;
            before += n;
        }
    }
    __syncthreads();
    each([&](const Item& x) {
        const int i = atomicAdd(&at[bucket_of(x.keys)], 1);
        if ((uint32_t)i < (uint32_t)cap) items[i] = x;              // also where starts change meanwhile
    });
}

// ---------------------------------------------------------------- attention
template <int C>
struct Smem {
    static constexpr int kTileB = kTile * C * 2; // one Q, K or V tile
    static constexpr int kQ = 0, kK = 2 * kTileB, kV = kK + 2 * kTileB, kOut = kV + 2 * kTileB;
    static constexpr int kOutB = 32 * 64;        // a warp's 32 rows, 32 channels at a time
    static constexpr int kBars = kOut + 8 * kOutB, kOdd = kBars + 512, kBytes = kOdd + 2 * (2 * C + 4) * 4 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
};

struct Args {
    __nv_bfloat16* out;
    float* lse;                                  // or nullptr
    const Plan* plan;                            // or nullptr: a CTA has at most one pair, and finds it itself
    const int32_t* starts;
    int64_t prompts, total;
    int32_t group, kv_heads, tpt;
    float scale2;                                // log2(e) / sqrt(C)
};

// The pairs of a CTA, and what a role needs of the current one.  The next one is
// read ahead: where a pair ends, nobody waits for that.
struct Walk {
    const Item* items;
    int64_t pairs;
    int kv_heads, round;
    Item x;
    int h;
    int4 next_x;
    int next_h;                                  // -1: there is none
    __device__ __forceinline__ explicit Walk(const Args& a) : items(reinterpret_cast<const Item*>(a.plan + 1)), kv_heads(a.kv_heads), round(0) {
        if (a.plan) {
            pairs = (int64_t)a.plan->count * a.kv_heads;
            ahead();
        } else {
            pairs = 0;
            find(a);
        }
    }
    __device__ __forceinline__ void ahead() {
        const int c = round & 1 ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
        const int64_t i = (int64_t)round * gridDim.x + c;
        ++round;
        next_h = -1;
        if (i >= pairs) return;
        const int64_t e = i >> 32 ? i / kv_heads : (int64_t)((uint32_t)i / (uint32_t)kv_heads);
        next_h = (int)(i - e * kv_heads);
        next_x = *reinterpret_cast<const int4*>(items + e);
    }
    // the item blockIdx.x / kv_heads of the prompts in their order, by a whole warp
    __device__ __forceinline__ void find(const Args& a) {
        const int lane = threadIdx.x & 31;
        int64_t e = blockIdx.x / kv_heads;
        next_h = -1;
        for (int64_t s0 = 0; s0 < a.prompts; s0 += 32) {
            int begin = 0, len = 0;
            if (s0 + lane < a.prompts) prompt_range(a.starts, s0 + lane, a.total, begin, len);
            const int n = items_of(len, a.tpt);
            int64_t upto = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
                if (lane >= d) upto += v;
            }
            const uint32_t beyond = __ballot_sync(0xFFFFFFFFu, upto > e);
            if (beyond) {
                const int at = __ffs(beyond) - 1;
                begin = __shfl_sync(0xFFFFFFFFu, begin, at);
                len = __shfl_sync(0xFFFFFFFFu, len, at);
                const Item it = item_at(begin, len, (int)(e - __shfl_sync(0xFFFFFFFFu, upto - n, at)), a.tpt);
                next_x = make_int4(it.begin, it.len, it.tok0, it.keys);
                next_h = (int)blockIdx.x % kv_heads;
                return;
            }
            e -= __shfl_sync(0xFFFFFFFFu, upto, 31);
        }
    }
    __device__ __forceinline__ bool next() {
        if (next_h < 0) return false;
        h = next_h;
        x = {next_x.x, next_x.y, next_x.z, next_x.w};
        ahead();                                 // without a plan pairs is 0
        return true;
    }
    // the key tiles that row tile t sees, 0: it has no rows
    __device__ __forceinline__ int keys(int t, int tpt) const {
        const int first = x.tok0 + t * tpt;
        return first >= x.len ? 0 : (min(first + tpt, x.len) + kTile - 1) / kTile;
    }
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Looks through a value tile of tokens [0, live) of which are the prompt's, from
// token u0 of it on; a whole warp.  Values that are not finite become 0, those of
// the prompt are noted by their token.
template <int C>
__device__ __noinline__ void clean_values(unsigned char* tile, int u0, int live, int* odd, int lane) {
    for (int k = lane; k < kTile * (C / 8); k += 32) {
        const int r = k / (C / 8), c = k % (C / 8);
        uint4* p = reinterpret_cast<uint4*>(tile + (c / 8) * (kTile * 128) + tc::swizzled(r, c % 8));
        const uint4 x = *p;
        if (!is_odd(x)) continue;
        if (r < live) {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll 1
            for (int i = 0; i < 8; ++i) note_odd(odd, C, c * 8 + i, (w[i / 2] >> (16 * (i & 1))) & 0xFFFFu, u0 + r);
            odd[2 * C] = 1;
        }
        *p = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
    }
    tc::async_fence();
    __syncwarp();
}

template <int C>
__global__ void __launch_bounds__(kThreads, 1)
prompts_kernel(const Args a, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap)
{
    using S = Smem<C>;
    constexpr int kHalves = C / 64;              // 64-channel halves of a tile, 16 KB each
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* qfull = reinterpret_cast<uint64_t*>(sm + S::kBars);  // [2] a row tile's queries are in shared memory
    uint64_t* qfree = qfull + 2;                 // [2] its last score product is done
    uint64_t* kfull = qfree + 2;                 // [2] a key tile is there
    uint64_t* kfree = kfull + 2;                 // [2] both row tiles are done with it
    uint64_t* vfull = kfree + 2;
    uint64_t* vfree = vfull + 2;
    uint64_t* vgood = vfree + 2;                 // [2] a value tile has been looked through
    uint64_t* sfull = vgood + 2;                 // [2] scores of a row tile are in tensor memory
    uint64_t* pfull = sfull + 2;                 // [2] its weights are
    uint64_t* odone = pfull + 2;                 // [2] its output is complete
    uint64_t* wrote = odone + 2;                 // [2] the softmax warps are done with a pair (pairs alternate)
    uint64_t* clear = wrote + 2;                 // [2] nothing is noted for a pair yet
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(clear + 2);
    volatile int* gone = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* odds = reinterpret_cast<int*>(sm + S::kOdd);              // [2][2 C + 4]: first tokens, and whether any is noted

    // the shuffle tells the compiler that a warp's number is uniform: the products' operands then are, too
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qfull[i], 1);
            mbar_init(&qfree[i], 1);
            mbar_init(&kfull[i], 1);
            mbar_init(&kfree[i], 2);
            mbar_init(&vfull[i], 1);
            mbar_init(&vfree[i], 2);
            mbar_init(&vgood[i], 1);
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);
            mbar_init(&odone[i], 2);
            mbar_init(&wrote[i], 8);
            mbar_init(&clear[i], 1);
        }
        *gone = 0;
        mbar_init_fence();
    }
    if (warp == 9) tc::alloc(tmem_slot, 512);
    tc::before_sync();
    __syncthreads();
    tc::after_sync();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");              // the plan
    auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, tc::wait(bar, parity & 1, gone)) != 0; };
    Walk w(a);

    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) {
        // ---- tiles by TMA, in the order the products take them: Q, K0, K1, V0, K2, V1, ...
        int nk = 0, nv = 0, nq[2] = {0, 0};      // tiles so far
        bool ok = true;
        auto load = [&](const CUtensorMap* map, uint64_t* full, uint64_t* free, unsigned char* tiles, int& it, int row) {
            const int s = it & 1;
            if (it >= 2) ok = ok && ready(&free[s], (it >> 1) - 1);
            if (!ok) return;
            if (tc::elect()) {
                mbar_expect_tx(&full[s], S::kTileB);
                for (int i = 0; i < kHalves; ++i)
                    tma_load_3d(tiles + s * S::kTileB + i * (kTile * 128), map, i * 64, w.h, row, &full[s]);
            }
            __syncwarp();
            ++it;
        };
        while (ok && w.next()) {
            for (int t = 0; t < 2; ++t) {
                if (w.keys(t, a.tpt) == 0) continue;
                if (nq[t] > 0) ok = ok && ready(&qfree[t], nq[t] - 1);
                if (!ok) break;
                if (tc::elect()) {
                    mbar_expect_tx(&qfull[t], (uint32_t)(kHalves * a.tpt * a.group * 128));
                    for (int i = 0; i < kHalves; ++i)
                        tma_load_3d(sm + S::kQ + t * S::kTileB + i * (kTile * 128), &qmap, i * 64, w.h * a.group,
                                    w.x.begin + w.x.tok0 + t * a.tpt, &qfull[t]);
                }
                __syncwarp();
                ++nq[t];
            }
            if (ok) load(&kmap, kfull, kfree, sm + S::kK, nk, w.x.begin);
            for (int j = 0; ok && j < w.x.keys; ++j) {
                if (j + 1 < w.x.keys) load(&kmap, kfull, kfree, sm + S::kK, nk, w.x.begin + (j + 1) * kTile);
                if (ok) load(&vmap, vfull, vfree, sm + S::kV, nv, w.x.begin + j * kTile);
            }
        }
        // every copy issued lands before the CTA's shared memory goes
        for (int t = 0; t < 2; ++t) {
            if (nq[t] > 0) tc::drain(&qfull[t], (nq[t] - 1) & 1);
            for (int i = max(0, nk - 2); i < nk; ++i) tc::drain(&kfull[i & 1], (i >> 1) & 1);
            for (int i = max(0, nv - 2); i < nv; ++i) tc::drain(&vfull[i & 1], (i >> 1) & 1);
        }
    } else if (warp <= 10) {
        // ---- products of row tile t
        const int t = warp - 9;
        constexpr uint32_t kScores = tc::instr_desc(kTile, kTile, false), kValues = tc::instr_desc(kTile, C, true);
        const uint32_t q_at = smem_u32(sm + S::kQ) + t * S::kTileB, k_at = smem_u32(sm + S::kK), v_at = smem_u32(sm + S::kV);
        const uint32_t s_at = tmem + t * kTile, o_at = tmem + 256 + t * C;
        int nk = 0, nv = 0, nq = 0, np = 0;      // key and value tiles, row tiles and weights so far
        bool ok = true;
        auto scores = [&](int s, bool last) {
#pragma unroll
            for (int k = 0; k < C / 16; ++k) {
                const uint32_t at = (k / 4) * (kTile * 128) + (k % 4) * 32;
                tc::mma_ss(s_at, tc::smem_desc(q_at + at, 16), tc::smem_desc(k_at + s * S::kTileB + at, 16), kScores, k > 0);
            }
            tc::commit(&sfull[t]);
            tc::commit(&kfree[s]);
            if (last) tc::commit(&qfree[t]);
        };
        while (ok && w.next()) {
            const int n = w.keys(t, a.tpt);
            if (n > 0) {
                ok = ready(&qfull[t], nq++) && ready(&kfull[nk & 1], nk >> 1);
                if (!ok) break;
                tc::after_sync();
                if (tc::elect()) scores(nk & 1, n == 1);
                __syncwarp();
                ++nk;
                for (int j = 0; j < n; ++j) {
                    if (j + 1 < n) ok = ready(&kfull[nk & 1], nk >> 1);
                    ok = ok && ready(&vgood[nv & 1], nv >> 1) && ready(&pfull[t], np++);
                    if (!ok) break;
                    tc::after_sync();
                    if (tc::elect()) {
                        const uint32_t v = v_at + (nv & 1) * S::kTileB;
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            tc::mma_ts(o_at, s_at + k * 8, tc::smem_desc(v + k * 2048, kTile * 128), kValues, j > 0 || k > 0);
                        tc::commit(&vfree[nv & 1]);
                        if (j + 1 < n) {
                            scores(nk & 1, j + 2 == n);
                        } else {
                            tc::commit(&odone[t]);
                            mbar_arrive(&odone[t]);                // what warp 11 noted is seen by who waits
                        }
                    }
                    __syncwarp();
                    ++nv;
                    if (j + 1 < n) ++nk;
                }
            }
            // tiles that the other row tile alone sees
            for (int j = n; ok && j < w.x.keys; ++j) {
                ok = ready(&kfull[nk & 1], nk >> 1);
                if (ok && lane == 0) mbar_arrive(&kfree[nk & 1]);
                ok = ok && ready(&vgood[nv & 1], nv >> 1);
                if (ok && lane == 0) mbar_arrive(&vfree[nv & 1]);
                ++nk;
                ++nv;
            }
        }
    } else {
        // ---- value tiles looked through
        int nv = 0, pair = 0;
        bool ok = true;
        while (ok && w.next()) {
            int* odd = odds + (pair & 1) * (2 * C + 4);
            if (pair >= 2) ok = ready(&wrote[pair & 1], (pair >> 1) - 1);
            for (int c = lane; c <= 2 * C; c += 32) odd[c] = c < 2 * C ? kNever : 0;
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&clear[pair & 1]);
            ++pair;
            for (int j = 0; ok && j < w.x.keys; ++j) {
                ok = ready(&vfull[nv & 1], nv >> 1);
                if (!ok) break;
                unsigned char* tile = sm + S::kV + (nv & 1) * S::kTileB;
                uint32_t bad[4] = {0u, 0u, 0u, 0u};
#pragma unroll 8
                for (int k = 0; k < S::kTileB / 512; ++k) {
                    const uint4 x = *reinterpret_cast<const uint4*>(tile + k * 512 + lane * 16);
                    bad[0] = add_if_odd(bad[0], x.x);
                    bad[1] = add_if_odd(bad[1], x.y);
                    bad[2] = add_if_odd(bad[2], x.z);
                    bad[3] = add_if_odd(bad[3], x.w);
                }
                if (__any_sync(0xFFFFFFFFu, (bad[0] | bad[1] | bad[2] | bad[3]) != 0u))
                    clean_values<C>(tile, j * kTile, w.x.len - j * kTile, odd, lane);
                if (lane == 0) mbar_arrive(&vgood[nv & 1]);
                ++nv;
            }
        }
    }
    } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ---- softmax of row tile t, a thread per row
    const int t = warp / 4, row = (warp & 3) * 32 + lane;
    const int token = row / a.group;             // of the row tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + t * kTile, o_at = tmem + lanes + 256 + t * C;
    unsigned char* stage = sm + S::kOut + warp * S::kOutB;
    // the rows that this lane writes a quarter of, four at a time: their tokens and their distance from row 0
    const int64_t heads = (int64_t)a.kv_heads * a.group;
    int to_token[4];
    int64_t to_row[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int R = (warp & 3) * 32 + 8 * i + lane / 4;
        to_token[i] = R / a.group;
        to_row[i] = to_token[i] * heads + (R - to_token[i] * a.group);
        if (to_token[i] >= a.tpt) to_token[i] = kNever;
    }
    int ns = 0, no = 0, pair = 0;                // score tiles, row tiles and pairs so far
    bool ok = true;
    while (ok && w.next()) {
        const int n = w.keys(t, a.tpt);
        if (n > 0) {
            const int tok = w.x.tok0 + t * a.tpt;                  // the first row's token, which sees the fewest
            const bool live = token < a.tpt && tok + token < w.x.len;
            const int last = live ? tok + token : w.x.len;         // rows that do not exist are not written
            float m = -INFINITY;
            u64 sum = 0;
            for (int j = 0; j < n; ++j) {
                ok = ready(&sfull[t], ns++);
                if (!ok) break;
                tc::after_sync();
                uint32_t s[kTile];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::ld32(s_at + 32 * c, s + 32 * c);
                tc::wait_ld();
                const int c0 = j * kTile;
                if (c0 + kTile - 1 > tok) {
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        if (c0 + c > last) s[c] = 0xFF800000u;     // -inf; selected: a hidden token's score may be NaN
                }
                float x0 = -INFINITY, x1 = -INFINITY, x2 = -INFINITY, x3 = -INFINITY;
#pragma unroll
                for (int c = 0; c < kTile; c += 4) {
                    x0 = fmaxf(x0, __uint_as_float(s[c]));
                    x1 = fmaxf(x1, __uint_as_float(s[c + 1]));
                    x2 = fmaxf(x2, __uint_as_float(s[c + 2]));
                    x3 = fmaxf(x3, __uint_as_float(s[c + 3]));
                }
                const float top = __fmul_rn(fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)), a.scale2);
                const bool grow = top > __fadd_rn(m, kSlack);       // m = -inf: whenever anything is seen
                if (__any_sync(0xFFFFFFFFu, grow)) {
                    const float f = grow ? ex2(__fsub_rn(m, top)) : 1.0f;
                    if (grow) m = top;
                    sum = mul2(sum, pk(f, f));
                    if (j > 0) {
                        // the scores' arrival says that the products before them are done too
#pragma unroll
                        for (int c = 0; c < C / 32; ++c) {
                            uint32_t y[32];
                            tc::ld32(o_at + 32 * c, y);
                            tc::wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__fmul_rn(__uint_as_float(y[i]), f));
                            tc::st32(o_at + 32 * c, y);
                        }
                    }
                }
                const float neg = m == -INFINITY ? 0.0f : -m;
                const u64 sc2 = pk(a.scale2, a.scale2), ng2 = pk(neg, neg);
#pragma unroll
                for (int i = 0; i < 2; ++i) {    // 64 scores -> 32 columns of weight pairs
                    uint32_t p[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const int c = 64 * i + 2 * k;
                        const u64 e = fma2(pk(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, ng2);
                        const float e0 = ex2(lo_of(e)), e1 = ex2(hi_of(e));
                        sum = add2(sum, pk(e0, e1));
                        p[k] = pack_bf16x2(e0, e1);
                    }
                    tc::st32(s_at + 32 * i, p);
                }
                tc::wait_st();
                tc::before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[t]);
            }
            // ---- output: 32 rows of a warp by way of shared memory, so that its lanes write rows' pieces side by side
            ok = ok && ready(&odone[t], no++);
            if (!ok) break;
            tc::after_sync();
            const float l = __fadd_rn(lo_of(sum), hi_of(sum)), inv = row_scale(l);
            const int64_t base = (int64_t)(w.x.begin + tok) * heads + w.h * a.group;          // of row 0
            const int* odd = odds + (pair & 1) * (2 * C + 4);
            const bool any_odd = odd[2 * C] != 0;
            if (live && a.lse) a.lse[base + token * heads + (row - token * a.group)] = row_lse(m, l);
            // a row that saw nothing has sums of 0, and inv = 0
            const u64 inv2 = pk(inv, inv);
            // rolled: unrolled it is as much code again as the loop above, and fetched anew for every pair
#pragma unroll 1
            for (int c = 0; c < C / 32; ++c) {
                uint32_t y[32];
                tc::ld32(o_at + 32 * c, y);
                tc::wait_ld();
                __syncwarp();                    // the piece before has been read
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t p[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const u64 v = mul2(pk(__uint_as_float(y[8 * i + 2 * k]), __uint_as_float(y[8 * i + 2 * k + 1])), inv2);
                        p[k] = pack_bf16x2(lo_of(v), hi_of(v));
                    }
                    *reinterpret_cast<uint4*>(stage + lane * 64 + ((i ^ (lane >> 1)) & 3) * 16) = make_uint4(p[0], p[1], p[2], p[3]);
                }
                if (any_odd && l != 0.0f) {      // what the row sees of values that are not finite
#pragma unroll 1
                    for (int i = 0; i < 32; ++i) {
                        const float x = odd_value(odd, C, 32 * c + i, last);
                        __nv_bfloat16* v = reinterpret_cast<__nv_bfloat16*>(stage + lane * 64 + ((i / 8 ^ (lane >> 1)) & 3) * 16) + i % 8;
                        if (x != 0.0f) *v = __float2bfloat16_rn(__fadd_rn(__bfloat162float(*v), x));
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {    // four lanes a row
                    const int r = 8 * i + lane / 4, q = lane & 3;
                    const uint4 x = *reinterpret_cast<const uint4*>(stage + r * 64 + ((q ^ (r >> 1)) & 3) * 16);
                    if (to_token[i] < w.x.len - tok) *reinterpret_cast<uint4*>(a.out + (base + to_row[i]) * C + 32 * c + 8 * q) = x;
                }
            }
            __syncwarp();
        }
        // warps of a row tile without rows have waited for nothing: they must not run ahead of the others, and arrive
        // for a pair whose barrier still counts the one before the last
        ok = ready(&clear[pair & 1], pair >> 1);
        if (ok && lane == 0) mbar_arrive(&wrote[pair & 1]);
        ++pair;
    }
    }
    __syncwarp();
    tc::before_sync();
    __syncthreads();
    tc::after_sync();
    if (warp == 9) tc::dealloc(tmem, 512);
}

// [total, heads, C] bf16 with a token every `stride` elements, as boxes of 64 channels x `across` heads x `tokens`
bool encode_map(const void* x, int64_t total, int64_t stride, int64_t heads, int64_t C, int across, int tokens, CUtensorMap* map)
{
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)C, (cuuint64_t)heads, (cuuint64_t)total};
    const cuuint64_t strides[2] = {(cuuint64_t)C * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)across, (cuuint32_t)tokens};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int C>
cudaError_t launch(const PromptArgs& p, Plan* plan, cudaStream_t st)
{
    CUtensorMap qm, km, vm;
    const int tpt = kTile / (int)p.group;
    if (!encode_map(p.q, p.total, p.q_stride, p.kv_heads * p.group, C, (int)p.group, tpt, &qm) ||
        !encode_map(p.k, p.total, p.k_stride, p.kv_heads, C, 1, kTile, &km) ||
        !encode_map(p.v, p.total, p.v_stride, p.kv_heads, C, 1, kTile, &vm))
        return cudaErrorNotSupported;
    cudaError_t e = ensure_kernel_attrs(reinterpret_cast<const void*>(prompts_kernel<C>), Smem<C>::kBytes);
    if (e != cudaSuccess) return e;
    const int64_t cap = most_items(p.prompts, p.total, p.group);
    if (cap > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const int64_t grid = std::min<int64_t>(sm_count(), cap * p.kv_heads);
    // else every CTA finds its pair by itself, one launch: a prompt of 17 | 600 | 2400 tokens 9.7 -> 7.1, 19.4 -> 16.4,
    // 39.6 -> 37.2 us in a graph.  It looks through the prompts for that, which takes longer than the launch from about 200
    // of them on: 1 | 64 | 128 | 256 | 1024 prompts, all but the last empty, 8.5 | 9.1 | 9.8 | 11.5 | 21.6 us for 100 tokens and
    // 7.0 | 7.3 | 8.1 | 9.7 | 19.8 us for 18 (of 1 and 8 KV heads), with the launch 10.7 to 10.9 and 9.7 to 9.9 us
    const bool planned = cap * p.kv_heads > grid || p.prompts > 192;
    if (planned) plan_kernel<<<1, kPlanThreads, 0, st>>>(p.starts, p.prompts, p.total, tpt, (int)cap, plan);
    Args a;
    a.out = static_cast<__nv_bfloat16*>(p.out);
    a.lse = p.lse;
    a.plan = planned ? plan : nullptr;
    a.starts = p.starts;
    a.prompts = p.prompts;
    a.total = p.total;
    a.group = (int32_t)p.group;
    a.kv_heads = (int32_t)p.kv_heads;
    a.tpt = tpt;
    a.scale2 = (float)(1.4426950408889634 / (C == 128 ? 11.313708498984761 : 8.0));
    // launched while the plan is made, and waits for it
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Smem<C>::kBytes;
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = planned ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, prompts_kernel<C>, a, qm, km, vm);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t prompts_workspace(int64_t prompts, int64_t total, int64_t group, int64_t, int64_t)
{
    return total == 0 || prompts == 0 ? 0 : sizeof(Plan) + (size_t)most_items(prompts, total, group) * sizeof(Item);
}

cudaError_t launch_attend_prompts(const PromptArgs& a, void* ws, cudaStream_t st)
{
    if (a.total == 0 || a.prompts == 0) return cudaSuccess;
    Plan* plan = static_cast<Plan*>(ws);
    return a.C == 128 ? launch<128>(a, plan, st) : launch<64>(a, plan, st);
}

}  // namespace kvq
