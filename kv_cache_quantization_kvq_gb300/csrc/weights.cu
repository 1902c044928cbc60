// weights.cu -- the attention weight that n queries give every token of the
// streaming quantized cache (kvq_attend_weights).
//
// "KV Compression 公式到源码对照" §3.1: the cumulative attention score of a token
// is the sum of its attention weights over the steps.  With the log-sum-exp of
// every query row at hand, w_t = sum_r exp(q_r.k_t / sqrt(C) - lse_r) needs one
// pass over the keys and no history.
//
// A CTA takes the query rows of a slice, 16 at a time, as A fragments in shared
// memory; each of its warps walks a run of 32-token batches, turns their keys
// into B fragments of mma.sync.m16n8k16 (kvq_rows.cuh) and sums the weights of
// its columns over the rows.  Each token belongs to one warp, so no sum needs an
// atomic and its order is fixed.  Up to 64 rows; more take weights_tc.cu.
//
// Measured on one GB300: 64 slices x 8 heads over 8192 tokens 21.5 us (42 MB: 1.9
// TB/s; 26.7 us with cold caches); like chunk.cu bound by the latency of a warp's
// chain (52 % of the issue slots, 20 % of DRAM busy at 16 warps a SM).  Spills at 2
// bits: 92 bytes at head_dim 128, 12 at 64; at 4 bits 8 and none.
#include <algorithm>

#include "kvq_chunk.cuh"

namespace kvq {

namespace {

using namespace rows;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxTiles = 4;                     // row tiles of 16 held in shared memory

struct WeightArgs {
    View v;
    const float* lse;
    const float* in;                             // nullptr: zeros
    float* out;
    int64_t stride;
    int32_t ntiles, nrun;                        // row tiles; CTAs of a slice
};

template <int BITS, int C>
__global__ void __launch_bounds__(kThreads, 4)
weights_rows_kernel(const WeightArgs A)
{
    using G = Geo<BITS, C>;
    const View& a = A.v;
    __shared__ __align__(16) uint4 qf[kMaxTiles * G::kSteps * 32];
    __shared__ float nlse[kMaxTiles * 16];       // -lse in base 2; -inf: no weight
    __shared__ int lasts[kMaxTiles * 16];        // the last token a row sees
    __shared__ __align__(16) uint4 kcs[kWarps][C / 4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int64_t o = blockIdx.x / (uint32_t)A.nrun;
    const int run = (int)(blockIdx.x - (uint32_t)o * (uint32_t)A.nrun);
    const Span sp = span_of(a);
    const int first = padding(a, o);
    const int base = a.T - a.n;                  // token of query 0

    for (int t = 0; t < A.ntiles; ++t) stage_queries<BITS, C, 1>(a, o, 16 * t, qf + t * G::kSteps * 32, tid, kThreads);
    for (int r = tid; r < 16 * A.ntiles; r += kThreads) {
        float l = -INFINITY;
        if (r < a.rows) {
            l = A.lse[row_index(a, o, r)];
            l = l == -INFINITY ? -INFINITY : -__fmul_rn(l, kLog2e);
        }
        nlse[r] = l;
        lasts[r] = base + r / a.group;
    }
    // ---- this warp's run of batches
    const int k = run * kWarps + warp, of = A.nrun * kWarps;
    const int b0 = (int)((int64_t)sp.nb * k / of), b1 = (int)((int64_t)sp.nb * (k + 1) / of);
    const int bs = min(b1, sp.nsb);
    const uint8_t* kc = a.kc + (uint64_t)o * a.cap * G::kRowB + tig * (G::kRowB / 4);
    const uint32_t kmg = magic<BITS>(a.kflip);
    uint32_t kw[4][G::kWpl];
    auto load_k = [&](int b) {
        const uint8_t* p = kc + (int64_t)b * (kBatch * G::kRowB);
        const int cnt = a.tq - b * kBatch - 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) load_words<G::kWpl>(p + min(8 * j + g, cnt) * G::kRowB, kw[j]);
    };
    KRaw kr = {0u, 0u, 0u, 0u};
    int staged = -1, fetched = -1;
    bool kfast = true;
    if (b0 < bs) {
        fetched = b0 * kBatch / a.gk;
        load_k(b0);
        kr = fetch_k_group<BITS, C>(a, o, fetched, lane);
    }
    __syncthreads();

    for (int b = b0; b < b1; ++b) {
        int t0, t1;
        batch_at(a, sp, b, t0, t1);
        const bool seen = t1 > first;
        const bool store = b < sp.nsb;
        if (store && fetched != staged) {
            kfast = stage_k_group(kr, a.kbias, a.kz != nullptr, kcs[warp], lane, C / 4);
            staged = fetched;
        }
        float sum[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j][0] = sum[j][1] = 0.0f;
        // the old scores, in flight meanwhile: lane (g, tig) writes n-tile g
        const int wt = t0 + 8 * g + 2 * tig;
        const int64_t at = o * A.stride + wt;
        const float old0 = A.in && g < 4 && wt < t1 ? A.in[at] : 0.0f;
        const float old1 = A.in && g < 4 && wt + 1 < t1 ? A.in[at + 1] : 0.0f;

        auto add = [&](const float (&s)[1][4][4], int t) {
            const float la = nlse[16 * t + g], lb = nlse[16 * t + g + 8];
            const int ra = lasts[16 * t + g], rb = lasts[16 * t + g + 8];
            const bool whole = t0 >= first && t1 - t0 == kBatch && t1 - 1 <= lasts[16 * t];
            // rows that do not exist, or give nothing: selected, since their scores may be NaN all the same
            const bool da = la == -INFINITY, db = lb == -INFINITY;
            const bool two = 16 * t + 8 < a.rows;                   // rows g + 8 exist
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float wa = da ? 0.0f : ex2(__fmaf_rn(s[0][j][e], a.scale2, la));
                    float wb = two && !db ? ex2(__fmaf_rn(s[0][j][2 + e], a.scale2, lb)) : 0.0f;
                    if (!whole) {                // selected: a hidden token's score may be NaN
                        const int tok = t0 + 8 * j + 2 * tig + e;
                        const bool live = tok >= first && tok < t1;
                        wa = live && tok <= ra ? wa : 0.0f;
                        wb = live && tok <= rb ? wb : 0.0f;
                    }
                    sum[j][e] = __fadd_rn(sum[j][e], __fadd_rn(wa, wb));
                }
        };
        if (seen) {
            for (int t = 0; t < A.ntiles; ++t) {
                if (lasts[min(16 * t + 16, a.rows) - 1] < t0) continue;  // the tile sees none of the batch
                float s[1][4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) s[0][j][0] = s[0][j][1] = s[0][j][2] = s[0][j][3] = 0.0f;
                const uint4* qt = qf + t * G::kSteps * 32;
                if (!store) {
                    const __nv_bfloat16* krow[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        krow[j] = a.kr + ((uint64_t)o * a.rrows + (min(t0 + 8 * j + g, t1 - 1) - a.tq)) * C + tig * (C / 4);
                    scores_of_rows<BITS, C, 1>(s, krow, qt, lane);
                } else if (kfast) {
                    scores_of<BITS, C, 1, true>(s, kw, qt, kcs[warp], kmg, a.kbias, lane);
                } else {
                    scores_of<BITS, C, 1, false>(s, kw, qt, kcs[warp], kmg, a.kbias, lane);
                }
                add(s, t);
            }
        }
        if (b + 1 < bs) {
            load_k(b + 1);
            const int gk = (b + 1) * kBatch / a.gk;
            if (gk != fetched) {
                fetched = gk;
                kr = fetch_k_group<BITS, C>(a, o, gk, lane);
            }
        }
        // ---- sum the lanes of a column (rows g, g + 8 of every tile), add the old score
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1)
                    sum[j][e] = __fadd_rn(sum[j][e], __shfl_xor_sync(0xFFFFFFFFu, sum[j][e], x));
        if (g < 4) {
            float w0 = sum[0][0], w1 = sum[0][1];
#pragma unroll
            for (int j = 1; j < 4; ++j)
                if (g == j) { w0 = sum[j][0]; w1 = sum[j][1]; }
            if (wt < t1) A.out[at] = A.in ? __fadd_rn(old0, w0) : w0;
            if (wt + 1 < t1) A.out[at + 1] = A.in ? __fadd_rn(old1, w1) : w1;
        }
    }
}

template <int BITS, int C>
cudaError_t launch_rows(WeightArgs A, int64_t outer, cudaStream_t st)
{
    // one wave of four CTAs a SM, or a CTA per four batches where there are fewer
    const int64_t nb = (A.v.tq + kBatch - 1) / kBatch + (A.v.nres + kBatch - 1) / kBatch;
    A.ntiles = (A.v.rows + 15) / 16;
    A.nrun = (int32_t)std::max<int64_t>(1, std::min<int64_t>((152 * 4) / outer, (nb + kWarps - 1) / kWarps));
    const int64_t grid = outer * A.nrun;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    weights_rows_kernel<BITS, C><<<(unsigned)grid, kThreads, 0, st>>>(A);
    return cudaGetLastError();
}

}  // namespace

size_t weights_workspace(int64_t outer, int64_t C, int64_t n, int64_t group)
{
    return outer > 0 && weights_use_tc(n * group) ? weights_tc_workspace(outer, C, n * group) : 0;
}

cudaError_t launch_attend_weights(const CacheArgs& x, const float* lse, const float* scores_in, float* scores_out,
                                  int64_t stride, void* ws, cudaStream_t st)
{
    if (x.outer == 0 || x.tq + x.nres == 0) return cudaSuccess;
    WeightArgs A;
    A.v = cache_view(x);
    A.lse = lse;
    A.in = scores_in;
    A.out = scores_out;
    A.stride = stride;
    if (weights_use_tc(A.v.rows))
        return launch_weights_tc(A.v, lse, scores_in, scores_out, stride, x.bits, x.C, x.outer, ws, st);
    if (x.bits == 4) return x.C == 128 ? launch_rows<4, 128>(A, x.outer, st) : launch_rows<4, 64>(A, x.outer, st);
    return x.C == 128 ? launch_rows<2, 128>(A, x.outer, st) : launch_rows<2, 64>(A, x.outer, st);
}

}  // namespace kvq
