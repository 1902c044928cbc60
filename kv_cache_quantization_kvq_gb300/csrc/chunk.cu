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
// attend_rows_kernel: a CTA takes (slice, split of the visible batches) for
// the slice's up to 8, 16 or 32 query rows; each of its four warps walks its run of the split's
// 32-token batches with its own m, l, y, merged through shared memory at the
// end.  The query fragments and the key group's constants stay in shared memory
// (12 warps a SM instead of 8), the next batch's codes are loaded as soon as the
// current ones are used.  m is moved only when it grows by more than 2^8: until
// then the weights are at most 256, which costs float32 sums and bf16 weights no
// relative precision, and the output is seldom rescaled.  With one split the CTA
// writes out and lse; up to eight splits are a thread-block cluster that joins
// its partial (m, l, y) through distributed shared memory (one launch); more go
// through the workspace and merge_rows_kernel.  Both join in split order.
//
// Measured on one GB300, 4-bit codes: 64 slices x 8 heads over 8192 tokens 35.4 us
// (79 MB: 2.2 TB/s), 8 x 4 over 131263 tokens 67 us.  At 16 warps a SM (128
// registers) 49 % of the issue slots, 28 % of DRAM and 17 % of the tensor pipe are
// busy: each warp waits on its chain codes -> unpacking -> scores -> weights -> values.
// At head_dim 128 the kernels spill: 4 bits 12, 4 and 42 bytes (8, 16, 32 rows), 2 bits
// 80, 52 and 124; at 64 none.
#include <algorithm>

#include "kvq_chunk.cuh"
#include "kvq_bulk.cuh"

namespace kvq {

namespace {

using namespace rows;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kAhead = 3;                         // batches that the codes are fetched into L2 ahead
constexpr float kSlack = 8.0f;                   // base-2 growth of the maximum that is let pass

// What a number of query rows takes: MT tiles of 16 rows of the score product, H
// halves of a tile in use.  Up to 8 rows the value product is transposed, Y^T[C x 8]
// = V^T[C x tokens] P^T[tokens x 8]: a lane's score fragment of row g is just the B
// fragment of P^T and two value B fragments are the A fragment of V^T, and the
// output takes half the registers and half the products (16 warps a SM instead of
// 12).
template <int ROWS, int C>
struct Rows {
    static constexpr int MT = (ROWS + 15) / 16, H = ROWS == 8 ? 1 : 2;
    static constexpr int NT = ROWS == 8 ? C / 16 : C / 8;          // output fragments of a tile
    static constexpr int kCtas = ROWS == 8 ? 4 : ROWS == 16 ? 3 : 2;
    static constexpr int kOut = ROWS == 8 ? 8 : 16;                // rows merged at a time
};

// y += P.V for 16 tokens: b0, b1: the value fragments of n-tiles nt and nt + 1 (tokens 2 tig + {0, 1} and + 8)
template <int ROWS, int C>
__device__ __forceinline__ void add_values(float (&y)[Rows<ROWS, C>::MT][Rows<ROWS, C>::NT][4], int nt,
                                           const uint4 (&p)[Rows<ROWS, C>::MT], uint32_t b0, uint32_t b1, uint32_t c0,
                                           uint32_t c1) {
    if constexpr (ROWS == 8) {
        mma16816(y[0][nt / 2], make_uint4(b0, c0, b1, c1), p[0].x, p[0].z);
    } else {
#pragma unroll
        for (int m = 0; m < Rows<ROWS, C>::MT; ++m) {
            mma16816(y[m][nt], p[m], b0, b1);
            mma16816(y[m][nt + 1], p[m], c0, c1);
        }
    }
}

// a pair of values; where they are not known to be finite, 0 in place of those that are not
template <int BITS, bool FAST>
__device__ __forceinline__ uint32_t value_of(uint32_t w, int sh, uint32_t mg, uint32_t s, uint32_t z, float bias) {
    const uint32_t x = value_pair<BITS, FAST>(w, sh, mg, s, z, bias);
    return FAST ? x : finite_or_zero(x);
}

// P.V of one 32-token batch of the store: this lane's code words of its eight
// tokens, 16 ks + {2 tig, 2 tig + 1, 8 + 2 tig, 9 + 2 tig}; vm: (scale, zero
// point) of each token and V group.
template <int BITS, int C, int ROWS, bool FAST>
__device__ __forceinline__ void values_of(float (&y)[Rows<ROWS, C>::MT][Rows<ROWS, C>::NT][4],
                                          const uint4 (&p)[2][Rows<ROWS, C>::MT],
                                          const uint32_t (&w)[8][Geo<BITS, C>::kVW], const uint32_t* vm, uint32_t mg,
                                          float bias, int tig) {
    using G = Geo<BITS, C>;
    constexpr int FH = 16 / BITS;                // fields of a half word: n-tiles per half
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        const uint2 m0 = *reinterpret_cast<const uint2*>(vm + 16 * ks + 2 * tig);
        const uint2 m1 = *reinterpret_cast<const uint2*>(vm + 16 * ks + 8 + 2 * tig);
        const uint32_t s0 = __byte_perm(m0.x, m0.y, 0x5410), z0 = __byte_perm(m0.x, m0.y, 0x7632);
        const uint32_t s1 = __byte_perm(m1.x, m1.y, 0x5410), z1 = __byte_perm(m1.x, m1.y, 0x7632);
#pragma unroll
        for (int h = 0; h < G::kVB / 2; ++h) {
            const uint32_t sel = (h & 1) ? 0x7632 : 0x5410;
            const uint32_t x0 = __byte_perm(w[4 * ks][h / 2], w[4 * ks + 1][h / 2], sel);
            const uint32_t x1 = __byte_perm(w[4 * ks + 2][h / 2], w[4 * ks + 3][h / 2], sel);
#pragma unroll
            for (int i = 0; i < FH; i += 2)
                add_values<ROWS, C>(y, h * FH + i, p[ks], value_of<BITS, FAST>(x0, BITS * i, mg, s0, z0, bias),
                                    value_of<BITS, FAST>(x1, BITS * i, mg, s1, z1, bias),
                                    value_of<BITS, FAST>(x0, BITS * (i + 1), mg, s0, z0, bias),
                                    value_of<BITS, FAST>(x1, BITS * (i + 1), mg, s1, z1, bias));
        }
    }
}

// ---- thread-block clusters
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float remote_f(const void* p, int rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float4 remote_f4(const void* p, int rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(remote(p, rank)) : "memory");
    return v;
}

// out (4 channels) and, with the row's first channels, lse
template <int C>
__device__ __forceinline__ void write_row(const ChunkArgs& A, int64_t o, int r, int c4, float M, float L, const float (&v)[4]) {
    const int64_t at = row_index(A.v, o, r);
    const float inv = row_scale(L);
    *reinterpret_cast<uint2*>(A.out + at * C + c4) =
        make_uint2(pack_bf16x2(row_value(v[0], inv), row_value(v[1], inv)),
                   pack_bf16x2(row_value(v[2], inv), row_value(v[3], inv)));
    if (A.lse && c4 == 0)
        A.lse[at] = row_lse(M, L);
}

// Softmax state of a lane's rows (g, and g + 8 of each tile unless there are at most 8).
template <int MT, int H>
struct Running { float m[MT][H], l[MT][H]; };

// Masks (unless `whole`), moves the maximum if it must, and turns scores into
// the weights' fragments.
template <int C, int ROWS, class R = Rows<ROWS, C>>
__device__ __forceinline__ void softmax_of(const View& a, float (&s)[R::MT][4][4], float (&y)[R::MT][R::NT][4],
                                           Running<R::MT, R::H>& st, uint4 (&p)[2][R::MT], bool whole, int t0, int t1,
                                           int first, const int (&last)[R::MT][R::H], int tig) {
#pragma unroll
    for (int m = 0; m < R::MT; ++m) {
        if (!whole) {
            // selected, not multiplied: a hidden token's score may be NaN
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 2 * R::H; ++e) {
                    const int t = t0 + 8 * j + 2 * tig + (e & 1);
                    if (t < first || t >= t1 || t > last[m][e >> 1]) s[m][j][e] = -INFINITY;
                }
        }
        float top[R::H];
        bool grow[R::H], any = false;
#pragma unroll
        for (int h = 0; h < R::H; ++h) {
            float x = fmaxf(fmaxf(fmaxf(s[m][0][2 * h], s[m][0][2 * h + 1]), fmaxf(s[m][1][2 * h], s[m][1][2 * h + 1])),
                            fmaxf(fmaxf(s[m][2][2 * h], s[m][2][2 * h + 1]), fmaxf(s[m][3][2 * h], s[m][3][2 * h + 1])));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
            top[h] = __fmul_rn(x, a.scale2);
            grow[h] = top[h] > __fadd_rn(st.m[m][h], kSlack);
            any = any || grow[h];
        }
        if (__any_sync(0xFFFFFFFFu, any)) {
            float f[R::H];
#pragma unroll
            for (int h = 0; h < R::H; ++h) {
                f[h] = grow[h] ? ex2(__fsub_rn(st.m[m][h], top[h])) : 1.0f;
                if (grow[h]) st.m[m][h] = top[h];
                st.l[m][h] = __fmul_rn(st.l[m][h], f[h]);
            }
            // columns of a fragment: rows g and g + 8 of the tile, or (transposed) rows 2 tig and 2 tig + 1
            float f0 = f[0], f1 = f[R::H - 1];
            if constexpr (ROWS == 8) {
                f0 = __shfl_sync(0xFFFFFFFFu, f[0], 8 * tig);
                f1 = __shfl_sync(0xFFFFFFFFu, f[0], 8 * tig + 4);
            }
#pragma unroll
            for (int nt = 0; nt < R::NT; ++nt) {
                y[m][nt][0] = __fmul_rn(y[m][nt][0], f0);
                y[m][nt][1] = __fmul_rn(y[m][nt][1], ROWS == 8 ? f1 : f0);
                y[m][nt][2] = __fmul_rn(y[m][nt][2], ROWS == 8 ? f0 : f1);
                y[m][nt][3] = __fmul_rn(y[m][nt][3], f1);
            }
        }
        uint32_t w[4][2] = {};
#pragma unroll
        for (int h = 0; h < R::H; ++h) {
            const float neg = st.m[m][h] == -INFINITY ? 0.0f : -st.m[m][h];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e0 = ex2(__fmaf_rn(s[m][j][2 * h], a.scale2, neg));
                const float e1 = ex2(__fmaf_rn(s[m][j][2 * h + 1], a.scale2, neg));
                st.l[m][h] = __fadd_rn(st.l[m][h], __fadd_rn(e0, e1));
                // one bf16 for the value product, whose operands are of one type: hi + lo would be a second product
                // a fragment, for an error (2^-8 of each weight at most) of the size of out's own rounding
                w[j][h] = pack_bf16x2(e0, e1);
            }
        }
        p[0][m] = make_uint4(w[0][0], w[0][1], w[1][0], w[1][1]);
        p[1][m] = make_uint4(w[2][0], w[2][1], w[3][0], w[3][1]);
    }
}

template <int BITS, int C, int ROWS>
__global__ void __launch_bounds__(kThreads, (Rows<ROWS, C>::kCtas))
attend_rows_kernel(const ChunkArgs A)
{
    using G = Geo<BITS, C>;
    using R = Rows<ROWS, C>;
    constexpr int MT = R::MT, H = R::H;
    const View& a = A.v;
    __shared__ float sm[kWarps][16], sl[kWarps][16], gm[16], gl[16];
    __shared__ __align__(16) float sy[kWarps][R::kOut][C];
    __shared__ __align__(16) uint4 qf[MT * G::kSteps * 32];
    __shared__ __align__(16) uint4 kcs[kWarps][C / 4];
    __shared__ __align__(16) uint32_t vms[kWarps][4][kBatch];
    __shared__ __align__(16) int odd[2 * C];     // the first tokens with values that are not finite

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int split = (int)(blockIdx.x % (uint32_t)A.nsplit);
    const int64_t o = blockIdx.x / (uint32_t)A.nsplit;
    stage_queries<BITS, C, MT>(a, o, 0, qf, tid, kThreads);
    for (int c = tid; c < 2 * C; c += kThreads) odd[c] = kNever;

    // ---- the last token each of this lane's rows sees
    const int base = a.T - a.n;                  // token of query 0
    int last[MT][H];
#pragma unroll
    for (int m = 0; m < MT; ++m)                 // rows past the last are not written
#pragma unroll
        for (int h = 0; h < H; ++h) last[m][h] = base + (16 * m + g + 8 * h) / a.group;
    const int last_hi = a.T - 1, last_lo = base;                   // of the last and of the first row
    const int first = padding(a, o);

    // ---- the visible batches, cut into splits, and a run of the split for each warp
    const Span sp = span_of(a);
    int b0 = 0, b1 = 0;
    if (first <= last_hi) {                      // first <= last_hi < T
        b0 = batch_of(a, sp, first);
        b1 = batch_of(a, sp, last_hi) + 1;
    }
    {
        const int64_t len = b1 - b0;
        const int k = split * kWarps + warp, of = A.nsplit * kWarps;
        b1 = b0 + (int)(len * (k + 1) / of);
        b0 += (int)(len * k / of);
    }
    const int bs = min(b1, sp.nsb);              // the run's store batches: [b0, bs)

    float y[MT][R::NT][4];
    Running<MT, H> st;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int nt = 0; nt < R::NT; ++nt) y[m][nt][0] = y[m][nt][1] = y[m][nt][2] = y[m][nt][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            st.m[m][h] = -INFINITY;
            st.l[m][h] = 0.0f;
        }
    }
    const int64_t row0 = o * a.cap;              // the slice's first row: one register pair, not a pointer for each buffer
    const uint32_t kmg = magic<BITS>(a.kflip), vmg = magic<BITS>(a.vflip);
    const uint32_t* vm = &vms[warp][g * (C / 8) / a.gv][0];         // this lane's V group (its C/8 channels lie in one)

    // a batch's codes: whole batches at fixed offsets, the store's last one clamped to its tokens
    uint32_t kw[4][G::kWpl], vw[8][G::kVW];
    auto load_k = [&](int b) {
        const uint8_t* p = a.kc + ((row0 + (int64_t)b * kBatch) * G::kRowB + tig * (G::kRowB / 4));
        const int cnt = a.tq - b * kBatch - 1;
        if (cnt >= kBatch - 1) {
            p += g * G::kRowB;
#pragma unroll
            for (int j = 0; j < 4; ++j) load_words<G::kWpl>(p + 8 * j * G::kRowB, kw[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) load_words<G::kWpl>(p + min(8 * j + g, cnt) * G::kRowB, kw[j]);
        }
    };
    auto load_v = [&](int b) {
        const uint8_t* p = a.vc + ((row0 + (int64_t)b * kBatch) * G::kRowB + g * G::kVB);
        const int cnt = a.tq - b * kBatch - 1;
        auto one = [&](int k, const uint8_t* at) {
            if constexpr (G::kVB >= 4) load_words<G::kVW>(at, vw[k]);
            else vw[k][0] = __ldcs(reinterpret_cast<const uint16_t*>(at));
        };
        if (cnt >= kBatch - 1) {
            p += 2 * tig * G::kRowB;
#pragma unroll
            for (int k = 0; k < 8; ++k) one(k, p + (8 * (k >> 1) + (k & 1)) * G::kRowB);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) one(k, p + min(8 * (k >> 1) + 2 * tig + (k & 1), cnt) * G::kRowB);
        }
    };
    // (scale, zero point) of token `lane` of a batch, a word per V group; hidden tokens get
    // zeros, since theirs may be NaN
    uint32_t vr[4] = {0u, 0u, 0u, 0u};
    auto load_vm = [&](int b) {
        const int t = b * kBatch + lane;
        const bool live = t >= first && t < a.tq;
        const __nv_bfloat16* ps = a.vs + (row0 + t) * a.ngv;
        const __nv_bfloat16* pz = a.vz + (row0 + t) * a.ngv;
        auto one = [&](int k) {
            vr[k] = 0u;
            if (live) vr[k] = bits_of(ps + k) | (a.vz ? bits_of(pz + k) << 16 : 0u);
        };
        one(0);
        if (a.ngv > 1) one(1);
        if (a.ngv > 2) {
            one(2);
            one(3);
        }
    };
    KRaw kr = {0u, 0u, 0u, 0u};
    int staged = -1, fetched = -1;
    bool kfast = true;
    if (b0 < bs) {
        fetched = b0 * kBatch / a.gk;
        load_k(b0);
        kr = fetch_k_group<BITS, C>(a, o, fetched, lane);
        load_vm(b0);
        load_v(b0);
    }
    __syncthreads();                             // the queries are staged

    int slow = 0;                                // values that may not be finite: 1 in the store, 2 in the buffer
    for (int b = b0; b < bs; ++b) {
        const int t0 = b * kBatch, t1 = min(t0 + kBatch, a.tq);
        if (fetched != staged) {
            kfast = stage_k_group(kr, a.kbias, a.kz != nullptr, kcs[warp], lane, C / 4);
            staged = fetched;
        }
        // the V constants of this batch
        auto fits = [&](int k) { return scale_fits(vr[k]) && zero_exact(bf_hi(vr[k])); };
        bool vfast = fits(0) && fits(1);
        if (a.ngv > 2) vfast = vfast && fits(2) && fits(3);
        vfast = __all_sync(0xFFFFFFFFu, vfast);
        if (!vfast) {                            // far zero points alone give finite values
            auto bad = [&](int k) { return may_be_odd(bf_lo(vr[k]), bf_hi(vr[k])); };
            if (__any_sync(0xFFFFFFFFu, bad(0) || bad(1) || bad(2) || bad(3))) slow |= 1;
        }
        __syncwarp();                            // the batch before has been read
        auto stage = [&](int k) {
            vms[warp][k][lane] = vfast ? (vr[k] & 0xFFFFu) | (biased(vr[k], a.vbias) & 0xFFFF0000u) : vr[k];
        };
        stage(0);
        if (a.ngv > 1) stage(1);
        if (a.ngv > 2) {
            stage(2);
            stage(3);
        }
        __syncwarp();

        float s[MT][4][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[m][j][0] = s[m][j][1] = s[m][j][2] = s[m][j][3] = 0.0f;
        if (kfast) scores_of<BITS, C, MT, true>(s, kw, qf, kcs[warp], kmg, a.kbias, lane);
        else scores_of<BITS, C, MT, false>(s, kw, qf, kcs[warp], kmg, a.kbias, lane);
        if (b + 1 < bs) {
            const int ba = b + kAhead;           // into L2 a few batches ahead: codes, V constants, K group constants
            if (lane < 8 && ba < bs && (ba + 1) * kBatch <= a.tq) {
                if (lane < 2) {
                    bulk_prefetch_l2((lane ? a.vc : a.kc) + (row0 + (int64_t)ba * kBatch) * G::kRowB, kBatch * G::kRowB);
                } else {
                    const bool key = lane >= 4;
                    const __nv_bfloat16* at = (lane & 1) ? (key ? a.kz : a.vz) : (key ? a.ks : a.vs);
                    const int64_t off = key ? (o * a.ngk + ba * kBatch / a.gk) * C + ((lane & 2) ? C / 2 : 0)
                                            : (row0 + (int64_t)ba * kBatch) * a.ngv;
                    if (at) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + off));
                }
            }
            load_k(b + 1);
            const int gk = (b + 1) * kBatch / a.gk;
            if (gk != fetched) {
                fetched = gk;
                kr = fetch_k_group<BITS, C>(a, o, gk, lane);
            }
            load_vm(b + 1);
        }
        uint4 p[2][MT];
        const bool whole = t0 >= first && t1 - t0 == kBatch && t1 - 1 <= last_lo;
        softmax_of<C, ROWS>(a, s, y, st, p, whole, t0, t1, first, last, tig);
        if (vfast) values_of<BITS, C, ROWS, true>(y, p, vw, vm, vmg, a.vbias, tig);
        else values_of<BITS, C, ROWS, false>(y, p, vw, vm, vmg, a.vbias, tig);
        if (b + 1 < bs) load_v(b + 1);
    }

    // ---- the run's buffer batches: bf16 rows
    for (int b = max(b0, sp.nsb); b < b1; ++b) {
        int t0, t1;
        batch_at(a, sp, b, t0, t1);
        const __nv_bfloat16* krow[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            krow[j] = a.kr + ((uint64_t)o * a.rrows + (min(t0 + 8 * j + g, t1 - 1) - a.tq)) * C + tig * (C / 4);
        float s[MT][4][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[m][j][0] = s[m][j][1] = s[m][j][2] = s[m][j][3] = 0.0f;
        scores_of_rows<BITS, C, MT>(s, krow, qf, lane);
        uint4 p[2][MT];
        const bool whole = t0 >= first && t1 - t0 == kBatch && t1 - 1 <= last_lo;
        softmax_of<C, ROWS>(a, s, y, st, p, whole, t0, t1, first, last, tig);
        // this lane's C/8 channels of its tokens, paired by token
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            uint32_t r[4][C / 16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = t0 + 16 * ks + 8 * (e >> 1) + 2 * tig + (e & 1);
#pragma unroll
                for (int i = 0; i < C / 64; ++i) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (t >= first && t < t1)
                        x = reinterpret_cast<const uint4*>(a.vr + ((uint64_t)o * a.rrows + (t - a.tq)) * C + g * (C / 8))[i];
                    r[e][4 * i] = x.x; r[e][4 * i + 1] = x.y; r[e][4 * i + 2] = x.z; r[e][4 * i + 3] = x.w;
                }
            }
            uint32_t bad[2] = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < C / 16; ++i) {
                    bad[e & 1] = add_if_odd(bad[e & 1], r[e][i]);
                    r[e][i] = finite_or_zero(r[e][i]);
                }
            if (__any_sync(0xFFFFFFFFu, (bad[0] | bad[1]) != 0u)) slow |= 2;
#pragma unroll
            for (int nt = 0; nt < C / 8; nt += 2)
                add_values<ROWS, C>(y, nt, p[ks], __byte_perm(r[0][nt / 2], r[1][nt / 2], 0x5410),
                                    __byte_perm(r[2][nt / 2], r[3][nt / 2], 0x5410),
                                    __byte_perm(r[0][nt / 2], r[1][nt / 2], 0x7632),
                                    __byte_perm(r[2][nt / 2], r[3][nt / 2], 0x7632));
        }
    }

    // ---- merge the warps, a row tile at a time; channel of (nt, column e of lane tig) = (2 tig + e) C/8 + nt,
    // transposed: lane (g, tig) has channels g C/8 + i of rows 2 tig and 2 tig + 1
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m > 0) __syncthreads();
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float l = st.l[m][h];
            l = __fadd_rn(l, __shfl_xor_sync(0xFFFFFFFFu, l, 1));
            l = __fadd_rn(l, __shfl_xor_sync(0xFFFFFFFFu, l, 2));
            if (tig == 0) {
                sm[warp][g + 8 * h] = st.m[m][h];
                sl[warp][g + 8 * h] = l;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q4 = 0; q4 < C / 32; ++q4) {
                if constexpr (ROWS == 8) {
                    *reinterpret_cast<float4*>(&sy[warp][2 * tig + h][g * (C / 8) + 4 * q4]) =
                        make_float4(y[0][2 * q4][h], y[0][2 * q4][2 + h], y[0][2 * q4 + 1][h], y[0][2 * q4 + 1][2 + h]);
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float4*>(&sy[warp][g + 8 * h][(2 * tig + e) * (C / 8) + 4 * q4]) =
                            make_float4(y[m][4 * q4][2 * h + e], y[m][4 * q4 + 1][2 * h + e], y[m][4 * q4 + 2][2 * h + e],
                                        y[m][4 * q4 + 3][2 * h + e]);
                }
            }
        if (m == 0 && slow) {
            if (slow & 1) note_rows<BITS, C>(a, o, max(b0 * kBatch, first), min(bs * kBatch, a.tq), odd, lane);
            if (slow & 2) {
                int from, to, skip;
                batch_at(a, sp, max(b0, sp.nsb), from, skip);
                batch_at(a, sp, b1 - 1, skip, to);
                note_rows<BITS, C>(a, o, max(from, first), to, odd, lane);
            }
        }
        __syncthreads();
        for (int k = tid; k < R::kOut * (C / 4); k += kThreads) {
            const int row = k / (C / 4), c4 = (k % (C / 4)) * 4, r = 16 * m + row;
            if (r >= a.rows) break;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w][row]);
            float L = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = part_scale(sm[w][row], M);
                L = __fmaf_rn(sl[w][row], f, L);
                const float4 x = *reinterpret_cast<const float4*>(&sy[w][row][c4]);
                v[0] = __fmaf_rn(x.x, f, v[0]);
                v[1] = __fmaf_rn(x.y, f, v[1]);
                v[2] = __fmaf_rn(x.z, f, v[2]);
                v[3] = __fmaf_rn(x.w, f, v[3]);
            }
            const int4 op = *reinterpret_cast<const int4*>(&odd[c4]), on = *reinterpret_cast<const int4*>(&odd[C + c4]);
            if ((op.x & op.y & op.z & op.w & on.x & on.y & on.z & on.w) != kNever) {
                const int row_last = base + r / a.group;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = __fadd_rn(v[i], odd_value(odd, C, c4 + i, row_last));
            }
            if (A.cluster) {
                *reinterpret_cast<float4*>(&sy[0][row][c4]) = make_float4(v[0], v[1], v[2], v[3]);   // read by this thread only
                if (c4 == 0) {
                    gm[row] = M;
                    gl[row] = L;
                }
            } else if (A.nsplit > 1) {
                float* dst = A.part + ((o * a.rows + r) * A.nsplit + split) * (C + 4);
                *reinterpret_cast<float4*>(dst + c4) = make_float4(v[0], v[1], v[2], v[3]);
                if (c4 == 0) *reinterpret_cast<float2*>(dst + C) = make_float2(M, L);
            } else {
                write_row<C>(A, o, r, c4, M, L, v);
            }
        }
        if (A.cluster) {                         // block rank = split; each takes its share of the rows' pieces
            cluster_sync();
            for (int k = split * kThreads + tid; k < R::kOut * (C / 4); k += A.nsplit * kThreads) {
                const int row = k / (C / 4), c4 = (k % (C / 4)) * 4, r = 16 * m + row;
                if (r >= a.rows) break;
                float M = -INFINITY;
                for (int s = 0; s < A.nsplit; ++s) M = fmaxf(M, remote_f(&gm[row], s));
                float L = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int s = 0; s < A.nsplit; ++s) {
                    const float f = part_scale(remote_f(&gm[row], s), M);
                    const float4 x = remote_f4(&sy[0][row][c4], s);
                    L = __fmaf_rn(remote_f(&gl[row], s), f, L);
                    v[0] = __fmaf_rn(x.x, f, v[0]);
                    v[1] = __fmaf_rn(x.y, f, v[1]);
                    v[2] = __fmaf_rn(x.z, f, v[2]);
                    v[3] = __fmaf_rn(x.w, f, v[3]);
                }
                write_row<C>(A, o, r, c4, M, L, v);
            }
            cluster_sync();                      // nobody leaves, or writes the next tile, before all have read
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

// Up to 8, 16 or 32 rows (four, three, two CTAs a SM); more rows take the
// tensor-core forms of prefill.cu.  Splits of the visible batches: the number that
// gives the shortest run through all waves, counting about three batches for a
// CTA's start and end and three for a second launch.
struct RowsPlan { int64_t nsplit; bool cluster; };

constexpr int64_t kCluster = 8;                  // most splits that a cluster joins
constexpr int64_t kMaxWaves = 2;                 // more CTAs than this are not split further

int64_t slots_of(int64_t rows) { return 152 * (rows <= 8 ? 4 : rows <= 16 ? 3 : 2); }

// Clusters must find their SMs together: on a full GPU (448 CTAs in clusters of 7)
// they cost 73 us where two launches take 56; on 64 CTAs they save the second
// launch (5 us).
bool cluster_ok(int64_t outer, int64_t s, int64_t slots) { return s > 1 && s <= kCluster && 2 * outer * s <= slots; }

// Up to 2048 tokens of few slices the splits stay within a cluster: no workspace.
bool short_cache(int64_t outer, int64_t T, int64_t slots) { return T <= 2048 && cluster_ok(outer, kCluster, slots); }

RowsPlan rows_plan(int64_t outer, int64_t T, int64_t rows)
{
    const int64_t slots = slots_of(rows), nb = (T + kBatch - 1) / kBatch + 1;
    const int64_t most = short_cache(outer, T, slots) ? kCluster : nb;
    RowsPlan p = {1, false};
    int64_t best = INT64_MAX;
    for (int64_t s = 1; s == 1 || (outer * s <= kMaxWaves * slots && s * kWarps <= nb && s <= most); ++s) {
        const bool cluster = cluster_ok(outer, s, slots);
        const int64_t cost = ((outer * s + slots - 1) / slots) * ((nb + s * kWarps - 1) / (s * kWarps) + 3) +
                             (s > 1 && !cluster ? 3 : 0);
        if (cost < best) {
            best = cost;
            p = {s, cluster};
        }
    }
    return p;
}

template <int BITS, int C>
cudaError_t launch_rows(ChunkArgs A, int64_t outer, cudaStream_t st)
{
    const RowsPlan p = rows_plan(outer, A.v.T, A.v.rows);
    A.nsplit = (int32_t)p.nsplit;
    const int64_t grid = outer * p.nsplit;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    A.cluster = p.cluster;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim = {(unsigned)(A.cluster ? p.nsplit : 1), 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = A.v.rows <= 8 ? cudaLaunchKernelEx(&cfg, attend_rows_kernel<BITS, C, 8>, A)
                          : A.v.rows <= 16 ? cudaLaunchKernelEx(&cfg, attend_rows_kernel<BITS, C, 16>, A)
                                           : cudaLaunchKernelEx(&cfg, attend_rows_kernel<BITS, C, 32>, A);
    if (e != cudaSuccess) return e;
    if (p.nsplit > 1 && !p.cluster) {
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
    if (chunk_uses_tc(rows)) return chunk_tc_workspace(outer, C, tmax, rows);
    // every T up to tmax may choose its splits: at most kMaxWaves of CTAs, or one per four batches
    const int64_t slots = slots_of(rows), most = (tmax + kBatch - 1) / kBatch + 1;
    if (short_cache(outer, tmax, slots) || most / kWarps <= 1) return 0;
    return (size_t)(std::min(kMaxWaves * slots, outer * (most / kWarps)) * rows * (C + 4)) * sizeof(float);
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
    v.kbias = 128.0f + (x.k_signed ? (float)(1 << (x.bits - 1)) : 0.0f);
    v.vbias = 128.0f + (x.v_signed ? (float)(1 << (x.bits - 1)) : 0.0f);
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
    if (chunk_uses_tc(A.v.rows)) return launch_attend_tc(A, x.bits, x.C, x.outer, ws, st);
    if (x.bits == 4) return x.C == 128 ? launch_rows<4, 128>(A, x.outer, st) : launch_rows<4, 64>(A, x.outer, st);
    return x.C == 128 ? launch_rows<2, 128>(A, x.outer, st) : launch_rows<2, 64>(A, x.outer, st);
}

}  // namespace kvq
