// weights.cu -- the attention weight that n queries give every token of the
// streaming quantized cache (kvq_attend_weights).
//
// "KV Compression 公式到源码对照" §3.1: the cumulative attention score of a token
// is the sum of its attention weights over the steps.  With the log-sum-exp of
// every query row at hand, w_t = sum_r exp(q_r.k_t / sqrt(C) - lse_r) needs one
// pass over the keys and no history.
//
// The keys stay and the queries stream: a warp turns the keys of a 32-token
// batch into B fragments of mma.sync.m16n8k16 once (kvq_rows.cuh), walks the
// row tiles (16 query rows each) that see the batch, and keeps the running sum
// of its columns' weights in registers.  Each token belongs to one warp, so no
// sum needs an atomic and its order is fixed.
#include <algorithm>

#include "kvq_chunk.cuh"

namespace kvq {

namespace {

using namespace rows;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRowTile = 16;
constexpr int kFold = 32;                        // row tiles summed before they join the total

struct WeightArgs {
    View v;
    const float* lse;
    const float* in;                             // nullptr: zeros
    float* out;
    int64_t stride;
};

template <int BITS, int C>
__global__ void __launch_bounds__(kThreads, 2)
weights_rows_kernel(const WeightArgs A, int nb, int64_t total)
{
    using G = Geo<BITS, C>;
    const View& a = A.v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int64_t job = (int64_t)blockIdx.x * kWarps + warp;
    if (job >= total) return;
    const int64_t o = job / nb;
    const int b = (int)(job - o * nb);
    const Span sp = span_of(a);
    int t0, t1;
    batch_at(a, sp, b, t0, t1);
    const int first = a.first ? max(a.first[o], 0) : 0;
    const int base = a.T - a.n;                  // token of query 0

    float sum[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j][0] = sum[j][1] = 0.0f;
    if (t1 > first) {
        // ---- the batch's keys
        uint32_t kb[4][C / 8];
        if (b < sp.nsb) {
            const uint8_t* kc = a.kc + (uint64_t)o * a.cap * G::kRowB + tig * (G::kRowB / 4);
            uint32_t kw[4][G::kWpl];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = min(t0 + 8 * j + g, t1 - 1);
                load_words<G::kWpl>(kc + (int64_t)t * G::kRowB, kw[j]);
#pragma unroll
                for (int i = 0; i < G::kWpl; ++i) kw[j][i] ^= a.kflip;
            }
            uint32_t ks[C / 8], kz[C / 8];
            const bool fast = load_k_group<BITS, C>(a, o, t0 / a.gk, tig, ks, kz);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (fast) keys_of<BITS, C, true>(kw[j], ks, kz, a.koff, kb[j]);
                else keys_of<BITS, C, false>(kw[j], ks, kz, a.koff, kb[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = min(t0 + 8 * j + g, t1 - 1) - a.tq;
                load_pairs<BITS, C>(a.kr + ((uint64_t)o * a.rrows + t) * C + tig * (C / 4), kb[j]);
            }
        }

        // ---- the rows that see any of it: from query t0 - base on
        const int i0 = max(0, max(t0, first) - base);
        float part[4][2];
        int fold = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) part[j][0] = part[j][1] = 0.0f;
        for (int r0 = (int)((int64_t)i0 * a.group / kRowTile) * kRowTile; r0 < a.rows; r0 += kRowTile) {
            const int ra = r0 + g, rb = ra + 8;
            uint32_t qa[C / 8], qb[C / 8];
            float xa = INFINITY, xb = INFINITY;  // a row past the last, or without weight, gives 2^-inf
            int la = -1, lb = -1;
#pragma unroll
            for (int p = 0; p < C / 8; ++p) qa[p] = qb[p] = 0u;
            if (ra < a.rows) {
                const int64_t at = row_index(a, o, ra);
                load_pairs<BITS, C>(a.q + at * C + tig * (C / 4), qa);
                const float l = A.lse[at];
                if (l != -INFINITY) { xa = __fmul_rn(l, kLog2e); la = base + ra / a.group; }
            }
            if (rb < a.rows) {
                const int64_t at = row_index(a, o, rb);
                load_pairs<BITS, C>(a.q + at * C + tig * (C / 4), qb);
                const float l = A.lse[at];
                if (l != -INFINITY) { xb = __fmul_rn(l, kLog2e); lb = base + rb / a.group; }
            }
            const bool whole = t0 >= first && t1 - t0 == kBatch && t1 - 1 <= base + r0 / a.group;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int kk = 0; kk < G::kSteps; ++kk) {
                    const uint32_t qf[4] = {qa[2 * kk], qb[2 * kk], qa[2 * kk + 1], qb[2 * kk + 1]};
                    mma16816(s, qf, kb[j][2 * kk], kb[j][2 * kk + 1]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float wa = ex2(__fmaf_rn(s[e], a.scale2, -xa)), wb = ex2(__fmaf_rn(s[2 + e], a.scale2, -xb));
                    if (!whole) {                // selected: a hidden token's score may be NaN
                        const int t = t0 + 8 * j + 2 * tig + e;
                        const bool live = t >= first && t < t1;
                        wa = live && t <= la ? wa : 0.0f;
                        wb = live && t <= lb ? wb : 0.0f;
                    }
                    part[j][e] = __fadd_rn(part[j][e], __fadd_rn(wa, wb));
                }
            }
            if (++fold == kFold) {
                fold = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        sum[j][e] = __fadd_rn(sum[j][e], part[j][e]);
                        part[j][e] = 0.0f;
                    }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) sum[j][e] = __fadd_rn(sum[j][e], part[j][e]);
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
        // lane (g, tig) writes n-tile j = g
        float w0 = sum[0][0], w1 = sum[0][1];
#pragma unroll
        for (int j = 1; j < 4; ++j)
            if (g == j) { w0 = sum[j][0]; w1 = sum[j][1]; }
        const int t = t0 + 8 * g + 2 * tig;
        const int64_t at = o * A.stride + t;
        if (t < t1) A.out[at] = A.in ? __fadd_rn(A.in[at], w0) : w0;
        if (t + 1 < t1) A.out[at + 1] = A.in ? __fadd_rn(A.in[at + 1], w1) : w1;
    }
}

template <int BITS, int C>
cudaError_t launch_rows(const WeightArgs& A, int64_t outer, cudaStream_t st)
{
    const int nb = (A.v.tq + kBatch - 1) / kBatch + (A.v.nres + kBatch - 1) / kBatch;
    const int64_t total = outer * nb, grid = (total + kWarps - 1) / kWarps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    weights_rows_kernel<BITS, C><<<(unsigned)grid, kThreads, 0, st>>>(A, nb, total);
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
