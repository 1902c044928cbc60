// evict.cu -- eviction from the streaming cache by accumulated score, in whole
// blocks (kvq_evict_blocks).
//
// "KV Compression 公式到源码对照" §3.2: keep = TopK(score, B - W) union the recent
// window; "KV cache 压缩：把历史装得更小" §"少存 token：合并，或淘汰": the dropped
// entries' K and V are freed.
//
// select_blocks_kernel, a CTA per slice: block scores as unevaluated sums of three
// float32 (error-free additions: 63 bits at least; in binary64, whose units are
// few here, the sums took 90 of 110 us for 128 slices of 32768 tokens), rounded to
// a pair, an order-preserving 64-bit key each, a radix search for the key of the last kept
// block (8 bits a pass, until the remaining bin is taken whole), ties by index,
// and an ordered scan that writes the ascending keep list; it also counts what
// is left of the padding.
//
// move_blocks_kernel: kept block j goes to place j <= keep[j].  A thread owns
// one piece (16 bytes where the alignment allows) at one place within the
// block, of one buffer of one slice, and takes the kept blocks in ascending
// order, a few loads ahead of their stores.  In place, a store to block j can
// only hit a block that the same thread has loaded before (keep[j'] > j for
// every later j'), and no other thread touches that piece: no barrier and no
// second buffer are needed.  Out of place the kept blocks are shared among more
// threads where there are few pieces.
//
// Measured on one GB300: 128 slices of 32768 tokens to a quarter, 16 us of selection
// (64 % of the issue slots) and 52 us of moves (290 MB: 5.6 TB/s, 82 % of a plain copy
// and 70 % of the DRAM's peak).  In place 70.4 us; with few slices and many blocks one
// thread a piece is slow: 8 slices of 131072 tokens to a quarter take 154 us in place
// and 54 out of place.
#include <algorithm>

#include "kvq_device.cuh"

namespace kvq {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSumAhead = 4;                     // blocks whose scores a warp has in flight
constexpr int kSharedKeys = 2048;                // block keys held in shared memory; more go through the workspace
constexpr int kMoveThreads = 256;
constexpr int kAhead = 8;                        // loads in flight per thread

// order_of: ascending unsigned order = ascending order of floats, -0 = +0
__device__ __forceinline__ uint32_t order_of(float x) {
    const int b = __float_as_int(__fadd_rn(x, 0.0f));
    return b < 0 ? ~(uint32_t)b : (uint32_t)b | 0x80000000u;
}

// ---- block scores.  A sum is hi + mid + lo, each addition error-free (Knuth's
// two-sum) down to lo.  A lane's mid is within 17 2^-24 of the sum S of magnitudes when
// it is renormalised every 16 numbers, what mid misses within 17 2^-48, so lo is within
// 2^-39 and is exact as long as S is less than 2^63 of the numbers' last place; else
// each addition is off by 2^-63 S at most.  (An infinity, a NaN or a partial sum beyond
// the range makes NaN of mid and lo: such blocks are added again, plainly.)
struct Sum { float hi, mid, lo; };

// a = RN(a + b), b = what that misses
__device__ __forceinline__ void two_sum(float& a, float& b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    b = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
    a = s;
}
__device__ __forceinline__ void add_to(Sum& s, float x) {
    two_sum(s.hi, x);
    two_sum(s.mid, x);
    s.lo = __fadd_rn(s.lo, x);
}
__device__ __forceinline__ void normalise(Sum& s) {
    two_sum(s.hi, s.mid);
    two_sum(s.mid, s.lo);
}
__device__ __forceinline__ void join_to(Sum& s, Sum r) {
    two_sum(s.hi, r.hi);
    two_sum(s.mid, r.hi);
    two_sum(s.mid, r.mid);
    s.lo = __fadd_rn(s.lo, __fadd_rn(__fadd_rn(r.hi, r.mid), r.lo));
}
__device__ __forceinline__ Sum shuffled(const Sum& s, int x) {
    return {__shfl_xor_sync(0xFFFFFFFFu, s.hi, x), __shfl_xor_sync(0xFFFFFFFFu, s.mid, x),
            __shfl_xor_sync(0xFFFFFFFFu, s.lo, x)};
}
// a + b + c rounded once: the low parts are added rounding to odd, after which the
// last rounding is right (Boldo and Melquiond).  What the first two steps leave, for a
// second call: a + b + c = th + b + c with the new b and c.
__device__ __forceinline__ float sum3(float& a, float& b, float& c) {
    two_sum(b, c);
    two_sum(a, b);
    float u = b, v = c;
    two_sum(u, v);
    const uint32_t w = __float_as_uint(u);
    if (v != 0.0f && !(w & 1u)) u = __uint_as_float((v > 0.0f) == (u > 0.0f) ? w + 1 : w - 1);
    return __fadd_rn(a, u);
}
// Ascending order of keys = ascending order of scores: the sum rounded to a pair of
// floats, RN(sum) and RN(what that misses), so equal sums have equal keys.  NaN lowest.
__device__ __forceinline__ unsigned long long key_of(float h, float m) {
    return h != h ? 0ull : ((unsigned long long)order_of(h) << 32) | order_of(m);
}

// exclusive prefix sum of one flag word per thread over the CTA; total in *sum
__device__ __forceinline__ int cta_scan(int v, int* warp_sums, int* sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
        const int s = warp_sums[w];
        before += w < warp ? s : 0;
        total += s;
    }
    __syncthreads();
    *sum = total;
    return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads)
select_blocks_kernel(const EvictArgs A)
{
    __shared__ unsigned long long near[kSharedKeys];
    __shared__ int hist[256];
    __shared__ int warp_sums[kSelThreads / 32];
    __shared__ int s_digit, s_need, s_done;
    __shared__ unsigned long long s_first;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t o = blockIdx.x;
    const int nb = (int)A.nb, kept = (int)A.kept;
    const int recent = (int)min(A.window, A.nb);
    const int cand = nb - recent;                // candidates [0, cand)
    int need = kept - recent;                    // to be taken of them (kept >= recent)
    unsigned long long* key = nb <= kSharedKeys ? near : reinterpret_cast<unsigned long long*>(A.ws) + o * A.nb;
    int32_t* keep = A.keep + o * kept;

    unsigned long long prefix = 0;
    int shift = 64;                              // key bits below `shift` are still open
    if (need > 0 && need < cand) {
        // ---- block scores: a warp takes kSumAhead blocks at a time, 32 tokens of each a step
        for (uint32_t b0 = warp * kSumAhead; b0 < (uint32_t)cand; b0 += kSelThreads / 32 * kSumAhead) {
            const float* p = A.scores_in + o * A.stride + (int64_t)b0 * A.block;
            Sum sum[kSumAhead];
            for (int64_t t = lane; t < A.block || t < 32; t += 64) {
                float x[kSumAhead][2];
#pragma unroll
                for (int i = 0; i < kSumAhead; ++i) {
                    const float* at = p + i * A.block + t;
                    x[i][0] = b0 + i < (uint32_t)cand && t < A.block ? at[0] : 0.0f;
                    x[i][1] = b0 + i < (uint32_t)cand && t + 32 < A.block ? at[32] : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < kSumAhead; ++i) {
                    if (t < 64) {                // the first two numbers of a lane
                        sum[i] = {x[i][0], x[i][1], 0.0f};
                        two_sum(sum[i].hi, sum[i].mid);
                    } else {
                        add_to(sum[i], x[i][0]);
                        add_to(sum[i], x[i][1]);
                        if ((t & 511) < 64) normalise(sum[i]);
                    }
                }
            }
            // the lanes' sums: every step halves the blocks that a lane goes on with, so four blocks take six
            // joins; eight lanes end with one of them each
            static_assert(kSumAhead == 4, "two halvings");
            const bool up = lane & 16, odd = lane & 8;
            Sum two[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                two[i] = up ? sum[i + 2] : sum[i];
                join_to(two[i], shuffled(up ? sum[i] : sum[i + 2], 16));
            }
            Sum one = odd ? two[1] : two[0];
            join_to(one, shuffled(odd ? two[0] : two[1], 8));
#pragma unroll
            for (int x = 4; x > 0; x >>= 1) join_to(one, shuffled(one, x));
            const int mine = (up ? 2 : 0) + (odd ? 1 : 0);
            float h = sum3(one.hi, one.mid, one.lo), rest = __fsub_rn(one.hi, h), m = sum3(rest, one.mid, one.lo);
            const bool fits = fabsf(h) < INFINITY && fabsf(m) < INFINITY;
            if (!__all_sync(0xFFFFFFFFu, fits)) {
#pragma unroll 1
                for (int i = 0; i < kSumAhead && b0 + i < (uint32_t)cand; ++i) {
                    float plain = 0.0f;
                    for (int64_t t = lane; t < A.block; t += 32) plain = __fadd_rn(plain, p[i * A.block + t]);
#pragma unroll
                    for (int x = 16; x > 0; x >>= 1) plain = __fadd_rn(plain, __shfl_xor_sync(0xFFFFFFFFu, plain, x));
                    if (mine == i && !fits) {
                        h = plain;
                        m = 0.0f;
                    }
                }
            }
            if ((lane & 7) == 0 && b0 + mine < (uint32_t)cand) key[b0 + mine] = key_of(h, m);
        }
        // ---- radix search, most significant digit first
        for (bool done = false; !done && shift > 0;) {
            for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            const int lo = shift - 8;
            for (uint32_t b = tid; b < (uint32_t)cand; b += kSelThreads) {
                const unsigned long long k = key[b];
                if (shift == 64 || (k >> shift) == (prefix >> shift)) atomicAdd(&hist[(int)(k >> lo) & 255], 1);
            }
            __syncthreads();
            if (tid < 32) {                      // the digit where the count from above reaches need
                int c[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) { c[i] = hist[255 - (8 * tid + i)]; sum += c[i]; }
                int x = sum;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
                    if (lane >= d) x += y;
                }
                int above = x - sum;
                if (above < need && need <= x) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (above < need && need <= above + c[i]) {
                            s_digit = 255 - (8 * tid + i);
                            s_need = need - above;
                            s_done = c[i] == need - above;
                        }
                        above += c[i];
                    }
                }
            }
            __syncthreads();
            prefix |= (unsigned long long)s_digit << lo;
            need = s_need;
            done = s_done;
            shift = lo;
            __syncthreads();
        }
    }
    // a candidate stays if its open key is above the prefix, or equal to it and
    // among the first `need` of those (all of them when the search ended early)
    const bool all = kept - recent >= cand, none = kept - recent <= 0;
    int base = 0, ties = 0;
    unsigned long long left = 0;                 // tokens of the padding that stay
    const long long pad = A.first_in ? max(A.first_in[o], 0) : 0;
    if (tid == 0) s_first = 0;
    __syncthreads();
    for (uint32_t b0 = 0; b0 < (uint32_t)nb; b0 += kSelThreads) {  // past 2^31 near the most blocks there may be
        const uint32_t b = b0 + tid;
        int above = 0, equal = 0;
        if (b < (uint32_t)nb) {
            if (b >= (uint32_t)cand || all) above = 1;
            else if (!none) {
                const unsigned long long k = key[b];
                const unsigned long long kh = shift == 64 ? 0ull : k >> shift, ph = shift == 64 ? 0ull : prefix >> shift;
                above = kh > ph;
                equal = kh == ph;
            }
        }
        int total;
        const int tie_rank = cta_scan(equal, warp_sums, &total);
        const int flag = above || (equal && ties + tie_rank < need);
        ties += total;
        const int at = base + cta_scan(flag, warp_sums, &total);
        base += total;
        if (flag) {
            keep[at] = (int32_t)b;
            left += (unsigned long long)min(max(pad - (long long)b * A.block, 0ll), (long long)A.block);
        }
    }
    if (A.first_out) {
        if (left) atomicAdd(&s_first, left);     // integers: any order gives the same sum
        __syncthreads();
        // a padding that reaches past the store keeps its part of the buffer
        const long long over = max(pad - (long long)nb * A.block, 0ll);
        if (tid == 0) A.first_out[o] = (int32_t)((long long)s_first + over);
    }
}

template <typename V>
__device__ __forceinline__ void move_pieces(const char* src, char* dst, int64_t block_B, const int32_t* keep, int kept, int part, int parts)
{
    const bool same = src == dst;
    if (same && part > 0) return;                // in place: one thread, in order
    const int from = same ? 0 : (int)((int64_t)kept * part / parts);
    if (!same) kept = (int)((int64_t)kept * (part + 1) / parts);
    for (int j0 = from; j0 < kept; j0 += kAhead) {                 // kept is at most 2^31 - 256
        V x[kAhead];
        int k[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int j = j0 + i;
            k[i] = j < kept ? keep[j] : -1;
            if (k[i] >= 0 && !(same && k[i] == j)) x[i] = *reinterpret_cast<const V*>(src + k[i] * block_B);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int j = j0 + i;
            if (k[i] >= 0 && !(same && k[i] == j)) *reinterpret_cast<V*>(dst + j * block_B) = x[i];
        }
    }
}

// threads of a slice: the pieces of every buffer's block, then one per score column of a block
struct MovePlan {
    int32_t first[kEvictBufs + 1];               // first thread of each buffer, and of the scores
    int32_t width[kEvictBufs];                   // bytes of a piece
    int32_t threads;                             // per slice
};

__global__ void __launch_bounds__(kMoveThreads)
move_blocks_kernel(const EvictArgs A, const MovePlan P, int64_t total)
{
    const int64_t id = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x;
    if (id >= total) return;
    const int64_t o = id / P.threads;
    const int w = (int)(id - o * P.threads);
    const int kept = (int)A.kept;
    const int32_t* keep = A.keep + o * kept;
    const int part = blockIdx.y, parts = gridDim.y;
    if (w >= P.first[kEvictBufs]) {
        // scores: a column of the store's blocks, then of the buffered tokens, then zeros
        const int64_t c = w - P.first[kEvictBufs];
        const float* in = A.scores_in + o * A.stride;
        float* out = A.scores_out + o * A.stride;
        const int64_t tq = A.nb * A.block, tk = (int64_t)kept * A.block;
        move_pieces<float>(reinterpret_cast<const char*>(in + c), reinterpret_cast<char*>(out + c), A.block * 4, keep, kept, part, parts);
        if (part > 0) return;
        for (int64_t r = c; r < A.nres; r += A.block) out[tk + r] = in[tq + r];
        // columns [tk + nres, tq + nres) that this thread owns: x = c (mod block)
        const int64_t z0 = tk + A.nres;
        for (int64_t x = z0 + ((c - z0) % A.block + A.block) % A.block; x < tq + A.nres; x += A.block) out[x] = 0.0f;
        return;
    }
    int i = 0;
#pragma unroll
    for (int k = 1; k < kEvictBufs; ++k)
        if (k < A.nbuf && w >= P.first[k]) i = k;
    const EvictBuf& B = A.buf[i];
    const int64_t at = o * B.slice_B + (int64_t)(w - P.first[i]) * P.width[i];
    const char* src = B.src + at;
    char* dst = B.dst + at;
    switch (P.width[i]) {
    case 16: move_pieces<uint4>(src, dst, B.block_B, keep, kept, part, parts); break;
    case 4: move_pieces<uint32_t>(src, dst, B.block_B, keep, kept, part, parts); break;
    case 2: move_pieces<uint16_t>(src, dst, B.block_B, keep, kept, part, parts); break;
    default: move_pieces<uint8_t>(src, dst, B.block_B, keep, kept, part, parts); break;
    }
}

}  // namespace

size_t evict_workspace(int64_t outer, int64_t nb_max) { return nb_max > kSharedKeys ? (size_t)(outer * nb_max) * 8 : 0; }

// The move's threads, and the CTAs that hold them; false: more than a grid does.
static bool plan_move(const EvictArgs& a, MovePlan& P, int64_t& total, int64_t& grid)
{
    int64_t n = 0;
    for (int i = 0; i < kEvictBufs; ++i) {
        P.first[i] = (int32_t)n;
        P.width[i] = 16;
        if (i >= a.nbuf) continue;
        const EvictBuf& b = a.buf[i];
        const uint64_t bits = (uint64_t)(uintptr_t)b.src | (uint64_t)(uintptr_t)b.dst | (uint64_t)b.slice_B | (uint64_t)b.block_B;
        P.width[i] = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
        n += b.block_B / P.width[i];
        if (n > 0x7FFFFFFF) return false;
    }
    P.first[kEvictBufs] = (int32_t)n;
    // a thread per score column of a block; a block may be longer than an empty store's buffer
    n += std::min(a.block, std::max<int64_t>(a.nb * a.block + a.nres, 1));
    if (n > 0x7FFFFFFF) return false;
    P.threads = (int32_t)n;
    total = a.outer * n;
    grid = (total + kMoveThreads - 1) / kMoveThreads;
    return grid <= 0x7FFFFFFF;
}

bool evict_fits(const EvictArgs& a)
{
    MovePlan P = {};
    int64_t total, grid;
    return plan_move(a, P, total, grid);
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st)
{
    if (a.outer == 0) return cudaSuccess;
    MovePlan P = {};
    int64_t total, grid;
    if (!plan_move(a, P, total, grid)) return cudaErrorInvalidConfiguration;
    select_blocks_kernel<<<(unsigned)a.outer, kSelThreads, 0, st>>>(a);
    // a full GPU of threads, each with eight blocks at least (64 slices, 112 of 128 blocks: 30 us in one part)
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>({152 * 2048 / total, a.kept / kAhead, 65535}));
    move_blocks_kernel<<<dim3((unsigned)grid, (unsigned)parts), kMoveThreads, 0, st>>>(a, P, total);
    return cudaGetLastError();
}

}  // namespace kvq
