// chunk.cu -- causal attention of n queries over the streaming quantized cache
// (kvq_attend_chunk).
//
// "KV cache 压缩：把历史装得更小" §"让 kernel 接住收益" (the attention kernel reads
// the low-bit cache) and §"K 的误差会改变权重，V 的误差会改变内容" (logit_t = q^T k_t /
// sqrt(d), y = sum_t a_t v_t).
//
// One pass over the cache with the running maximum m and sum l of the softmax,
// in base 2: x_t = q.k_t log2(e) / sqrt(C); y <- y 2^(m - m') + sum 2^(x_t -
// m') v_t.  Query rows of a slice (token i, head j: row i * group + j) share
// its keys, so up to 16 rows are one m16 tile of mma.sync.m16n8k16; the score
// fragment of a lane is the A fragment of its value product, so the
// probabilities never leave registers, and the keys and values go from packed
// codes to B fragments in registers (kvq_rows.cuh).
//
// attend_rows_kernel: a CTA takes (slice, row tile, split of the visible
// batches); its four warps walk the split's 32-token batches in turn, each with
// its own m, l, y, merged through shared memory at the end.  With one split the
// CTA writes out and lse; otherwise merge_rows_kernel joins the splits' partial
// (m, l, y) in split order.
#include <algorithm>

#include "kvq_chunk.cuh"

namespace kvq {

namespace {

using namespace rows;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRowTile = 16;

// P.V of one 32-token batch of the store: this lane's code words of its eight
// tokens (w[2 ks + e / 2][...], tokens 16 ks + {2 tig, 2 tig + 1, 8 + 2 tig,
// 9 + 2 tig}), their scale pairs and zero pairs.
template <int BITS, int C, bool FAST>
__device__ __forceinline__ void values_of(float (&y)[C / 8][4], const uint32_t (&p)[2][4],
                                          const uint32_t (&w)[8][Geo<BITS, C>::kVW], const uint32_t (&s)[4],
                                          const uint32_t (&z)[4], float off) {
    using G = Geo<BITS, C>;
    constexpr int FH = 16 / BITS;                // fields of a half word: n-tiles per half
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int h = 0; h < G::kVB / 2; ++h) {
            const uint32_t sel = (h & 1) ? 0x7632 : 0x5410;
            const uint32_t x0 = __byte_perm(w[4 * ks][h / 2], w[4 * ks + 1][h / 2], sel);
            const uint32_t x1 = __byte_perm(w[4 * ks + 2][h / 2], w[4 * ks + 3][h / 2], sel);
#pragma unroll
            for (int i = 0; i < FH; ++i) {
                const uint32_t b0 = value_pair<BITS, FAST>(x0, BITS * i, s[2 * ks], z[2 * ks], off);
                const uint32_t b1 = value_pair<BITS, FAST>(x1, BITS * i, s[2 * ks + 1], z[2 * ks + 1], off);
                mma16816(y[h * FH + i], p[ks], b0, b1);
            }
        }
}

template <int BITS, int C>
__global__ void __launch_bounds__(kThreads, 2)
attend_rows_kernel(const ChunkArgs A)
{
    using G = Geo<BITS, C>;
    const View& a = A.v;
    __shared__ float sm[kWarps][kRowTile], sl[kWarps][kRowTile];
    __shared__ __align__(16) float sy[kWarps][kRowTile][C];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, tig = lane & 3;
    int64_t blk = blockIdx.x;
    const int split = (int)(blk % A.nsplit);
    blk /= A.nsplit;
    const int tile = (int)(blk % A.ntiles);
    const int64_t o = blk / A.ntiles;
    const int r0 = tile * kRowTile;

    // ---- this lane's two query rows and the last token each sees
    const int ra = r0 + g, rb = r0 + g + 8;
    uint32_t qa[C / 8], qb[C / 8];
#pragma unroll
    for (int p = 0; p < C / 8; ++p) qa[p] = qb[p] = 0u;
    if (ra < a.rows) load_pairs<BITS, C>(a.q + row_index(a, o, ra) * C + tig * (C / 4), qa);
    if (rb < a.rows) load_pairs<BITS, C>(a.q + row_index(a, o, rb) * C + tig * (C / 4), qb);
    const int base = a.T - a.n;                  // token of query 0
    const int last_a = base + ra / a.group, last_b = base + rb / a.group;      // rows past the last are not written
    const int last_hi = base + (min(r0 + kRowTile, a.rows) - 1) / a.group;     // of the tile's rows
    const int last_lo = base + r0 / a.group;
    const int first = a.first ? max(a.first[o], 0) : 0;

    // ---- the visible batches, cut into splits
    const Span sp = span_of(a);
    int b0 = 0, b1 = 0;
    if (first <= last_hi) {                      // first <= last_hi < T
        b0 = batch_of(a, sp, first);
        b1 = batch_of(a, sp, last_hi) + 1;
    }
    const int64_t len = b1 - b0;
    const int e1 = b0 + (int)(len * (split + 1) / A.nsplit);
    b0 += (int)(len * split / A.nsplit);
    b1 = e1;

    float y[C / 8][4];
#pragma unroll
    for (int nt = 0; nt < C / 8; ++nt) y[nt][0] = y[nt][1] = y[nt][2] = y[nt][3] = 0.0f;
    float ma = -INFINITY, mb = -INFINITY, la = 0.0f, lb = 0.0f;
    uint32_t ks[C / 8], kz[C / 8];
    int cur = -1;
    bool kfast = true;

    const uint8_t* kc = a.kc + (uint64_t)o * a.cap * G::kRowB + tig * (G::kRowB / 4);
    const uint8_t* vc = a.vc + (uint64_t)o * a.cap * G::kRowB + g * G::kVB;
    const int vg = g * (C / 8) / a.gv;           // this lane's V group (its C/8 channels lie in one)

    for (int b = b0 + warp; b < b1; b += kWarps) {
        int t0, t1;
        batch_at(a, sp, b, t0, t1);
        const bool store = b < sp.nsb;
        const bool whole = t0 >= first && t1 - t0 == kBatch && t1 - 1 <= last_lo;

        // ---- scores: n-tile j, token t0 + 8 j + {2 tig, 2 tig + 1}
        float s[4][4];
        if (store) {
            uint32_t kw[4][G::kWpl];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = min(t0 + 8 * j + g, t1 - 1);
                load_words<G::kWpl>(kc + (int64_t)t * G::kRowB, kw[j]);
#pragma unroll
                for (int i = 0; i < G::kWpl; ++i) kw[j][i] ^= a.kflip;
            }
            const int gk = t0 / a.gk;
            if (gk != cur) {
                cur = gk;
                kfast = load_k_group<BITS, C>(a, o, gk, tig, ks, kz);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t kb[C / 8];
                if (kfast) keys_of<BITS, C, true>(kw[j], ks, kz, a.koff, kb);
                else keys_of<BITS, C, false>(kw[j], ks, kz, a.koff, kb);
                s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
#pragma unroll
                for (int kk = 0; kk < G::kSteps; ++kk) {
                    const uint32_t qf[4] = {qa[2 * kk], qb[2 * kk], qa[2 * kk + 1], qb[2 * kk + 1]};
                    mma16816(s[j], qf, kb[2 * kk], kb[2 * kk + 1]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = min(t0 + 8 * j + g, t1 - 1) - a.tq;
                uint32_t kb[C / 8];
                load_pairs<BITS, C>(a.kr + ((uint64_t)o * a.rrows + t) * C + tig * (C / 4), kb);
                s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
#pragma unroll
                for (int kk = 0; kk < G::kSteps; ++kk) {
                    const uint32_t qf[4] = {qa[2 * kk], qb[2 * kk], qa[2 * kk + 1], qb[2 * kk + 1]};
                    mma16816(s[j], qf, kb[2 * kk], kb[2 * kk + 1]);
                }
            }
        }
        if (!whole) {
            // selected, not multiplied: a hidden token's score may be NaN
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = t0 + 8 * j + 2 * tig + e;
                    const bool live = t >= first && t < t1;
                    if (!live || t > last_a) s[j][e] = -INFINITY;
                    if (!live || t > last_b) s[j][2 + e] = -INFINITY;
                }
        }

        // ---- running maximum and sum (the four lanes of a quad share a row)
        float na = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])),
                         fmaxf(fmaxf(s[2][0], s[2][1]), fmaxf(s[3][0], s[3][1])));
        float nb = fmaxf(fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3])),
                         fmaxf(fmaxf(s[2][2], s[2][3]), fmaxf(s[3][2], s[3][3])));
        na = fmaxf(na, __shfl_xor_sync(0xFFFFFFFFu, na, 1));
        nb = fmaxf(nb, __shfl_xor_sync(0xFFFFFFFFu, nb, 1));
        na = fmaxf(na, __shfl_xor_sync(0xFFFFFFFFu, na, 2));
        nb = fmaxf(nb, __shfl_xor_sync(0xFFFFFFFFu, nb, 2));
        na = fmaxf(ma, __fmul_rn(na, a.scale2));
        nb = fmaxf(mb, __fmul_rn(nb, a.scale2));
        if (__any_sync(0xFFFFFFFFu, na != ma || nb != mb)) {
            const float fa = na == -INFINITY ? 1.0f : ex2(__fsub_rn(ma, na));
            const float fb = nb == -INFINITY ? 1.0f : ex2(__fsub_rn(mb, nb));
            la = __fmul_rn(la, fa);
            lb = __fmul_rn(lb, fb);
#pragma unroll
            for (int nt = 0; nt < C / 8; ++nt) {
                y[nt][0] = __fmul_rn(y[nt][0], fa);
                y[nt][1] = __fmul_rn(y[nt][1], fa);
                y[nt][2] = __fmul_rn(y[nt][2], fb);
                y[nt][3] = __fmul_rn(y[nt][3], fb);
            }
            ma = na;
            mb = nb;
        }
        const float xa = ma == -INFINITY ? 0.0f : -ma, xb = mb == -INFINITY ? 0.0f : -mb;
        uint32_t p[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[j][e] = ex2(__fmaf_rn(s[j][e], a.scale2, xa));
                s[j][2 + e] = ex2(__fmaf_rn(s[j][2 + e], a.scale2, xb));
                la = __fadd_rn(la, s[j][e]);
                lb = __fadd_rn(lb, s[j][2 + e]);
            }
            p[j / 2][2 * (j & 1)] = pack_bf16x2(s[j][0], s[j][1]);
            p[j / 2][2 * (j & 1) + 1] = pack_bf16x2(s[j][2], s[j][3]);
        }

        // ---- values: tokens t0 + 16 ks + {2 tig, 2 tig + 1, 8 + 2 tig, 9 + 2 tig}
        if (store) {
            uint32_t vw[8][G::kVW], vs[4], vz[4];
            bool vfast = true;
#pragma unroll
            for (int k = 0; k < 4; ++k) {        // pairs of tokens
                const int tp = t0 + 8 * k + 2 * tig;
                uint32_t sb[2], zb[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = min(tp + e, t1 - 1);
                    const bool dead = tp + e < first || tp + e >= t1;     // its scale may be NaN
                    if constexpr (G::kVB >= 4) {
                        load_words<G::kVW>(vc + (int64_t)t * G::kRowB, vw[2 * k + e]);
                        vw[2 * k + e][0] ^= a.vflip;
                        if constexpr (G::kVW == 2) vw[2 * k + e][1] ^= a.vflip;
                    } else {
                        vw[2 * k + e][0] = __ldcs(reinterpret_cast<const uint16_t*>(vc + (int64_t)t * G::kRowB)) ^
                                           (a.vflip & 0xFFFFu);
                    }
                    const int64_t at = (o * a.cap + t) * a.ngv + vg;
                    sb[e] = dead ? 0u : bits_of(a.vs + at);
                    zb[e] = dead || !a.vz ? 0u : bits_of(a.vz + at);
                }
                vs[k] = sb[0] | (sb[1] << 16);
                vz[k] = zb[0] | (zb[1] << 16);
                vfast = vfast && zero_exact(bf_lo(vz[k])) && zero_exact(bf_hi(vz[k]));
            }
            vfast = __all_sync(0xFFFFFFFFu, vfast);
            if (vfast) {
                const float off = 128.0f + a.voff;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    vz[k] = pack_bf16x2(__fadd_rn(off, bf_lo(vz[k])), __fadd_rn(off, bf_hi(vz[k])));
                values_of<BITS, C, true>(y, p, vw, vs, vz, a.voff);
            } else {
                values_of<BITS, C, false>(y, p, vw, vs, vz, a.voff);
            }
        } else {
            // bf16 rows: this lane's C/8 channels of its tokens, paired by token
#pragma unroll
            for (int ks2 = 0; ks2 < 2; ++ks2) {
                uint32_t r[4][C / 16];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = t0 + 16 * ks2 + 8 * (e >> 1) + 2 * tig + (e & 1);
                    if (t >= first && t < t1) {
                        const uint4* src = reinterpret_cast<const uint4*>(
                            a.vr + ((uint64_t)o * a.rrows + (t - a.tq)) * C + g * (C / 8));
#pragma unroll
                        for (int i = 0; i < C / 64; ++i) {
                            const uint4 x = src[i];
                            r[e][4 * i] = x.x; r[e][4 * i + 1] = x.y; r[e][4 * i + 2] = x.z; r[e][4 * i + 3] = x.w;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < C / 16; ++i) r[e][i] = 0u;
                    }
                }
#pragma unroll
                for (int nt = 0; nt < C / 8; ++nt) {
                    const uint32_t sel = (nt & 1) ? 0x7632 : 0x5410;
                    mma16816(y[nt], p[ks2], __byte_perm(r[0][nt / 2], r[1][nt / 2], sel),
                             __byte_perm(r[2][nt / 2], r[3][nt / 2], sel));
                }
            }
        }
    }

    // ---- merge the warps; channel of (nt, column e of lane tig) = (2 tig + e) C/8 + nt
    la = __fadd_rn(la, __shfl_xor_sync(0xFFFFFFFFu, la, 1));
    lb = __fadd_rn(lb, __shfl_xor_sync(0xFFFFFFFFu, lb, 1));
    la = __fadd_rn(la, __shfl_xor_sync(0xFFFFFFFFu, la, 2));
    lb = __fadd_rn(lb, __shfl_xor_sync(0xFFFFFFFFu, lb, 2));
    if (tig == 0) {
        sm[warp][g] = ma;
        sm[warp][g + 8] = mb;
        sl[warp][g] = la;
        sl[warp][g + 8] = lb;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int q4 = 0; q4 < C / 32; ++q4) {
            *reinterpret_cast<float4*>(&sy[warp][g][(2 * tig + e) * (C / 8) + 4 * q4]) =
                make_float4(y[4 * q4][e], y[4 * q4 + 1][e], y[4 * q4 + 2][e], y[4 * q4 + 3][e]);
            *reinterpret_cast<float4*>(&sy[warp][g + 8][(2 * tig + e) * (C / 8) + 4 * q4]) =
                make_float4(y[4 * q4][2 + e], y[4 * q4 + 1][2 + e], y[4 * q4 + 2][2 + e], y[4 * q4 + 3][2 + e]);
        }
    __syncthreads();
    for (int k = tid; k < kRowTile * (C / 4); k += kThreads) {
        const int row = k / (C / 4), c4 = (k % (C / 4)) * 4, r = r0 + row;
        if (r >= a.rows) break;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w][row]);
        float L = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (M != -INFINITY) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(__fsub_rn(sm[w][row], M));
                L = __fmaf_rn(sl[w][row], f, L);
                const float4 x = *reinterpret_cast<const float4*>(&sy[w][row][c4]);
                v[0] = __fmaf_rn(x.x, f, v[0]);
                v[1] = __fmaf_rn(x.y, f, v[1]);
                v[2] = __fmaf_rn(x.z, f, v[2]);
                v[3] = __fmaf_rn(x.w, f, v[3]);
            }
        }
        if (A.nsplit > 1) {
            float* dst = A.part + ((o * a.rows + r) * A.nsplit + split) * (C + 4);
            *reinterpret_cast<float4*>(dst + c4) = make_float4(v[0], v[1], v[2], v[3]);
            if (c4 == 0) *reinterpret_cast<float2*>(dst + C) = make_float2(M, L);
        } else {
            const int64_t at = row_index(a, o, r);
            const float inv = L > 0.0f ? __fdiv_rn(1.0f, L) : 0.0f;
            *reinterpret_cast<uint2*>(A.out + at * C + c4) =
                make_uint2(pack_bf16x2(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv)),
                           pack_bf16x2(__fmul_rn(v[2], inv), __fmul_rn(v[3], inv)));
            if (A.lse && c4 == 0)
                A.lse[at] = L > 0.0f ? __fmul_rn(__fadd_rn(M, log2f(L)), 0.6931471805599453f) : -INFINITY;
        }
    }
}

template <int C>
__global__ void __launch_bounds__(kThreads)
merge_rows_kernel(const ChunkArgs A, int64_t total)
{
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= total) return;
    const int64_t o = row / A.v.rows;
    merge_row<C>(A, o, (int)(row - o * A.v.rows), A.part + row * A.nsplit * (C + 4), threadIdx.x & 31);
}

constexpr int64_t kSlots = 152 * 2;              // resident CTAs (two per SM)

// Splits of the visible batches: enough CTAs for two waves of the GPU, at
// least two batches per warp and split, and no more than the cache has.
int64_t splits_of(int64_t outer, int64_t T, int64_t rows)
{
    const int64_t ctas = outer * ((rows + kRowTile - 1) / kRowTile);
    const int64_t nb = (T + kBatch - 1) / kBatch;
    return std::max<int64_t>(1, std::min<int64_t>((2 * kSlots + ctas - 1) / ctas, nb / (2 * kWarps)));
}

template <int BITS, int C>
cudaError_t launch_rows(const ChunkArgs& A, int64_t outer, cudaStream_t st)
{
    const int64_t grid = outer * A.ntiles * A.nsplit;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    attend_rows_kernel<BITS, C><<<(unsigned)grid, kThreads, 0, st>>>(A);
    if (A.nsplit > 1) {
        const int64_t total = outer * A.v.rows;
        merge_rows_kernel<C><<<(unsigned)((total + kWarps - 1) / kWarps), kThreads, 0, st>>>(A, total);
    }
    return cudaGetLastError();
}

}  // namespace

size_t chunk_workspace(int64_t outer, int64_t C, int64_t tmax, int64_t n, int64_t group)
{
    const int64_t rows = n * group;
    if (outer == 0 || rows == 0) return 0;
    if (chunk_uses_tc(tmax, rows)) return chunk_tc_workspace(outer, C, tmax, rows);
    const int64_t ns = splits_of(outer, tmax, rows);
    return ns > 1 ? (size_t)(outer * rows * ns * (C + 4)) * sizeof(float) : 0;
}

rows::View cache_view(const CacheArgs& x)
{
    rows::View v = {};
    v.q = static_cast<const __nv_bfloat16*>(x.q);
    v.kc = static_cast<const uint8_t*>(x.k_codes);
    v.ks = static_cast<const __nv_bfloat16*>(x.k_scale);
    v.kz = x.k_asym ? static_cast<const __nv_bfloat16*>(x.k_zero) : nullptr;
    v.kr = static_cast<const __nv_bfloat16*>(x.k_resid);
    v.vc = static_cast<const uint8_t*>(x.v_codes);
    v.vs = static_cast<const __nv_bfloat16*>(x.v_scale);
    v.vz = x.v_asym ? static_cast<const __nv_bfloat16*>(x.v_zero) : nullptr;
    v.vr = static_cast<const __nv_bfloat16*>(x.v_resid);
    v.first = x.first;
    v.cap = x.cap;
    v.rrows = x.rrows;
    v.tq = (int32_t)x.tq;
    v.nres = (int32_t)x.nres;
    v.T = (int32_t)(x.tq + x.nres);
    v.n = (int32_t)x.n;
    v.group = (int32_t)x.group;
    v.rows = (int32_t)(x.n * x.group);
    v.kv_heads = (int32_t)x.kv_heads;
    v.gk = x.gk;
    v.ngk = (int32_t)((x.cap + x.gk - 1) / x.gk);
    v.gv = x.gv > 0 ? x.gv : (int32_t)x.C;
    v.ngv = (int32_t)(x.C / v.gv);
    const uint32_t flip = x.bits == 4 ? 0x88888888u : 0xAAAAAAAAu;
    v.kflip = x.k_signed ? flip : 0u;
    v.vflip = x.v_signed ? flip : 0u;
    v.koff = x.k_signed ? (float)(1 << (x.bits - 1)) : 0.0f;
    v.voff = x.v_signed ? (float)(1 << (x.bits - 1)) : 0.0f;
    v.scale2 = (float)(1.4426950408889634 / (x.C == 128 ? 11.313708498984761 : 8.0));
    return v;
}

cudaError_t launch_attend_chunk(const CacheArgs& x, void* out, float* lse, void* ws, cudaStream_t st)
{
    if (x.outer == 0 || x.n == 0) return cudaSuccess;
    ChunkArgs A;
    A.v = cache_view(x);
    A.out = static_cast<__nv_bfloat16*>(out);
    A.lse = lse;
    A.part = static_cast<float*>(ws);
    if (chunk_uses_tc(A.v.T, A.v.rows)) return launch_attend_tc(A, x.bits, x.C, x.outer, ws, st);
    A.ntiles = (A.v.rows + kRowTile - 1) / kRowTile;
    A.nsplit = (int32_t)splits_of(x.outer, x.tq + x.nres, A.v.rows);
    if (x.bits == 4) return x.C == 128 ? launch_rows<4, 128>(A, x.outer, st) : launch_rows<4, 64>(A, x.outer, st);
    return x.C == 128 ? launch_rows<2, 128>(A, x.outer, st) : launch_rows<2, 64>(A, x.outer, st);
}

}  // namespace kvq
