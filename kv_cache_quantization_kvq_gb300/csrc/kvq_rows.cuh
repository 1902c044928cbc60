// kvq_rows.cuh -- K and V rows of the streaming cache as mma.sync fragments,
// for the kernels of few query rows (chunk.cu, weights.cu).
//
// A batch is 32 consecutive cache tokens, all of the store or all of the
// buffer.  A warp turns a batch's packed codes into the B fragments of
// mma.sync.m16n8k16 (bf16 x bf16 -> float32) in registers: the order of the
// contracted index is free as long as both operands use the same, so each is
// chosen such that a lane reads one contiguous piece of a code row.
//  * scores, contraction over channels: lane (g, tig) = (lane / 4, lane % 4)
//    reads its quarter of token g's row, channels [tig C/4, (tig+1) C/4).  A
//    32-bit code word of F fields holds the channel pairs (i, i + F/2): fields
//    BITS apart in its two halves, so one shift and one mask-and-xor leave both
//    as the bf16 values 128 + field (the xor also turns two's complement into
//    offset binary);
//  * values, contraction over tokens: lane (g, tig) reads channels
//    [g C/8, (g+1) C/8) of the tokens its score fragment covers; a byte permute
//    pairs the words of two tokens, then the same shift and mask.
// One bf16x2 subtraction of 128 + off + zp is exact when |zp| <= 112 and an
// integer (every operand and result is an integer of at most 256), and one
// bf16x2 product with the bf16 scale rounds once: exactly RN_bf16(s (code -
// zp)), what kvq_dequantize stores (its float32 product of an 8-bit and an
// 8-bit significand is exact).  Groups with other zero points take the
// float32 route: subtract, multiply and round as kvq_dequantize does.
// Unpacking is four instructions a pair.  The kernels are bound neither by it nor by
// bytes (half of the issue slots and three quarters of DRAM idle) but by the latency of
// a warp's chain of loads, unpacking and products at the warps that registers allow.
#pragma once

#include "kvq_device.cuh"

namespace kvq {
namespace rows {

constexpr int kBatch = 32;                       // tokens of a batch
constexpr float kLog2e = 1.4426950408889634f;

// The cache as the kernels see it.
struct View {
    const __nv_bfloat16* q;
    const uint8_t *kc, *vc;
    const __nv_bfloat16 *ks, *kz, *kr;           // kz / vz: nullptr for symmetric codes
    const __nv_bfloat16 *vs, *vz, *vr;
    const int32_t* first;
    int64_t cap, rrows;
    int32_t tq, nres, T, n;
    int32_t group, rows;                         // rows = n * group query rows of a slice
    int32_t kv_heads, gk, ngk, gv, ngv;
    uint32_t kflip, vflip;                       // turns two's complement fields into offset binary
    float kbias, vbias;                          // 128 + that offset, 2^(bits-1) or 0
    float scale2;                                // log2(e) / sqrt(C)
};

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float ex2(float x) {  // 2^x, 2 ulp, 0 for -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// ---- the end of a softmax row: maximum m (base 2) and sum l of its weights.
// A NaN among the row's logits never moves m (fmaxf passes over it) and +inf
// makes 2^(inf - inf), so it is l that carries them: NaN, and so are out and lse.
// l = 0 is a row that saw nothing, or logits of -inf only: out 0, lse -inf.
__device__ __forceinline__ float row_scale(float l) { return l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l); }
__device__ __forceinline__ float row_value(float y, float scale) { return scale == 0.0f ? 0.0f : __fmul_rn(y, scale); }
__device__ __forceinline__ float row_lse(float m, float l) {
    return l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(m, log2f(l)), 0.6931471805599453f);
}
// what a part's sums count in the whole: 2^(part's maximum - the whole's), 1 where both are -inf (or +inf), so
// that a part's NaN stays, and never quite 0, so that its infinities do not turn into NaN
__device__ __forceinline__ float part_scale(float m, float M) { return m == M ? 1.0f : fmaxf(ex2(__fsub_rn(m, M)), 0x1p-126f); }
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void mma16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// N 32-bit words (N = 1, 2, 4) from p, aligned to their size; read once.
template <int N>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 x = __ldcs(reinterpret_cast<const uint4*>(p));
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (N == 2) {
        const uint2 x = __ldcs(reinterpret_cast<const uint2*>(p));
        w[0] = x.x; w[1] = x.y;
    } else {
        w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    }
}

__device__ __forceinline__ uint32_t bits_of(const __nv_bfloat16* p) {
    return *reinterpret_cast<const uint16_t*>(p);
}

// whether a zero point may take the bf16 route
__device__ __forceinline__ bool zero_exact(float z) { return fabsf(z) <= 112.0f && z == rintf(z); }
// a pair of zero points as that route wants them: 128 + off + zp
__device__ __forceinline__ uint32_t biased(uint32_t z, float b) {
    return pack_bf16x2(__fadd_rn(b, bf_lo(z)), __fadd_rn(b, bf_hi(z)));
}

template <int BITS, int C>
struct Geo {
    static constexpr int kRowB = C * BITS / 8;   // packed bytes of a token row
    static constexpr int F = 32 / BITS;          // fields of a word
    static constexpr int kWpl = kRowB / 16;      // words of a row per lane, score side
    static constexpr int kSteps = C / 16;        // k-steps of a score product
    static constexpr int kVB = kRowB / 8;        // bytes of a row per lane, value side (2, 4 or 8)
    static constexpr int kVW = kVB >= 4 ? kVB / 4 : 1;
    static constexpr uint32_t kMask = BITS == 4 ? 0x000F000Fu : 0x00030003u;
    // first channel, within its quarter, of pair p; the second is F/2 further
    __host__ __device__ static constexpr int pair_channel(int p) { return p / (F / 2) * F + p % (F / 2); }
};

constexpr uint32_t kOne28 = 0x43004300u;         // bf16 128.0 in both halves

// kOne28 with the sign fields' flip merged in (fields are the low BITS of each half)
template <int BITS>
__device__ __forceinline__ uint32_t magic(uint32_t flip) { return kOne28 | (flip & Geo<BITS, 64>::kMask); }

// One pair of rows' values from two fields of w at bit `sh` of its halves.
template <int BITS, bool FAST>
__device__ __forceinline__ uint32_t value_pair(uint32_t w, int sh, uint32_t mg, uint32_t s, uint32_t z, float bias) {
    const uint32_t x = ((w >> sh) & Geo<BITS, 64>::kMask) ^ mg;
    if constexpr (FAST) return mul_bf16x2(sub_bf16x2(x, z), s);
    // x holds 128 + field: bias = 128 + offset comes off exactly, and nothing is converted from an integer
    const float lo = __fsub_rn(__fsub_rn(bf_lo(x), bias), bf_lo(z));
    const float hi = __fsub_rn(__fsub_rn(bf_hi(x), bias), bf_hi(z));
    return pack_bf16x2(__fmul_rn(lo, bf_lo(s)), __fmul_rn(hi, bf_hi(s)));
}

// ---- values that are not finite
// A token that a row does not see has weight 0 in the row's value product, and 0
// times NaN or infinity would be NaN there.  So the products read such values as 0,
// and a CTA keeps per channel the first of its tokens, padding aside, that holds
// +inf or NaN (odd[c]) and the first that holds -inf or NaN (odd[C + c]); a row
// that sees that token has the infinity added to its sum.  Only slow paths look: the
// fast ones take constants that cannot give such a value.
constexpr int kNever = 0x7FFFFFFF;               // no token: positions are smaller

// whether a scale may take the bf16 route for values: with |code - zp| < 256 its products are finite
// (and so does every one of the scales whose bit patterns, sign aside, are at most this)
constexpr uint32_t kScaleFits = 0x7A00u;         // bf16 1.66e35
__device__ __forceinline__ bool scale_fits(uint32_t sz) { return (sz & 0x7FFFu) <= kScaleFits; }
// whether a scale and zero point can give a value that is not finite
__device__ __forceinline__ bool may_be_odd(float s, float z) { return !(fabsf(s) * (fabsf(z) + 16.0f) < 3.3e38f); }
// 0 as long as every w added is finite (0 times NaN or infinity is NaN): one instruction a pair
__device__ __forceinline__ uint32_t add_if_odd(uint32_t acc, uint32_t w) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(0u), "r"(acc));
    return d;
}
__device__ __forceinline__ bool is_odd(const uint4& x) {
    return add_if_odd(add_if_odd(0u, x.x), x.y) != 0u || add_if_odd(add_if_odd(0u, x.z), x.w) != 0u;
}
// a pair of bf16 with 0 in place of infinities and NaN
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
    uint32_t keep;
    asm("set.le.u32.bf16x2 %0, %1, %2;" : "=r"(keep) : "r"(w & 0x7FFF7FFFu), "r"(0x7F7F7F7Fu));
    return w & keep;
}
// notes bf16 value v of channel c and token t
__device__ __forceinline__ void note_odd(int* odd, int C, int c, uint32_t v, int t) {
    if ((v & 0x7F80u) != 0x7F80u) return;
    const bool nan = v & 0x7Fu, neg = v & 0x8000u;
    if (nan || !neg) atomicMin(&odd[c], t);
    if (nan || neg) atomicMin(&odd[C + c], t);
}
// what a row whose last token is `last` adds to channel c
__device__ __forceinline__ float odd_value(const int* odd, int C, int c, int last) {
    return __fadd_rn(odd[c] <= last ? INFINITY : 0.0f, odd[C + c] <= last ? -INFINITY : 0.0f);
}
// notes a whole row of values, token t of slice o, one element at a time
template <int BITS, int C>
__device__ __forceinline__ void note_row(const View& a, int64_t o, int t, int* odd) {
    const uint8_t* codes = a.vc + ((uint64_t)o * a.cap + t) * (C * BITS / 8);
    const int64_t meta = (o * a.cap + t) * a.ngv;
#pragma unroll 1
    for (int c = 0; c < C; ++c) {
        uint32_t v;
        if (t >= a.tq) {
            v = bits_of(a.vr + ((uint64_t)o * a.rrows + (t - a.tq)) * C + c);
        } else {
            const uint32_t f = ((codes[c * BITS / 8] ^ (a.vflip & 0xFFu)) >> (c * BITS % 8)) & ((1u << BITS) - 1);
            const float z = a.vz ? bf_lo(bits_of(a.vz + meta + c / a.gv)) : 0.0f;
            const float x = __fmul_rn(__fsub_rn(__fsub_rn(__fadd_rn(128.0f, (float)f), a.vbias), z), bf_lo(bits_of(a.vs + meta + c / a.gv)));
            v = pack_bf16x2(x, 0.0f) & 0xFFFFu;
        }
        note_odd(odd, C, c, v, t);
    }
}

// notes the values of tokens [t0, t1) of slice o, by one warp
template <int BITS, int C>
__device__ __noinline__ void note_rows(const View& a, int64_t o, int t0, int t1, int* odd, int lane) {
#pragma unroll 1
    for (int64_t t = (int64_t)t0 + lane; t < t1; t += 32) {
        bool look = t >= a.tq;
        for (int k = 0; !look && k < a.ngv; ++k) {
            const int64_t at = (o * a.cap + t) * a.ngv + k;
            look = may_be_odd(bf_lo(bits_of(a.vs + at)), a.vz ? bf_lo(bits_of(a.vz + at)) : 0.0f);
        }
        if (look) note_row<BITS, C>(a, o, (int)t, odd);
    }
}

// Channel pairs (c, c + F/2) of this lane's quarter of a bf16 row, from the
// quarter's first element: the order of the code words' fields.
template <int BITS, int C>
__device__ __forceinline__ void load_pairs(const __nv_bfloat16* quarter, uint32_t (&pr)[C / 8]) {
    using G = Geo<BITS, C>;
    constexpr int N = C / 8;                     // 32-bit words of the quarter
    uint32_t r[N];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(quarter)[i];
        r[4 * i] = x.x; r[4 * i + 1] = x.y; r[4 * i + 2] = x.z; r[4 * i + 3] = x.w;
    }
#pragma unroll
    for (int p = 0; p < N; ++p) {
        const int c = G::pair_channel(p);
        pr[p] = __byte_perm(r[c / 2], r[(c + G::F / 2) / 2], (c & 1) ? 0x7632 : 0x5410);
    }
}

// ---- K constants of one group, staged in shared memory by the warp that uses
// them: entry (kk, tig) = scale pairs 2 kk, 2 kk + 1 and zero pairs of lane
// quarter tig.  Lane e < C/4 makes entry e.
struct KRaw { uint32_t s0, s1, z0, z1; };

template <int BITS, int C>
__device__ __forceinline__ KRaw fetch_k_group(const View& a, int64_t o, int gk, int lane) {
    using G = Geo<BITS, C>;
    KRaw r = {0u, 0u, 0u, 0u};
    if (lane < C / 4) {
        const int64_t at = (o * a.ngk + gk) * C + (lane & 3) * (C / 4) + G::pair_channel(2 * (lane >> 2));
        r.s0 = *reinterpret_cast<const uint32_t*>(a.ks + at);       // channels c, c + 1
        r.s1 = *reinterpret_cast<const uint32_t*>(a.ks + at + G::F / 2);
        if (a.kz) {
            r.z0 = *reinterpret_cast<const uint32_t*>(a.kz + at);
            r.z1 = *reinterpret_cast<const uint32_t*>(a.kz + at + G::F / 2);
        }
    }
    return r;
}
// Stages them; returns whether the warp may take the bf16 route (the zero
// pairs are then 128 + off + zp, else as stored).
__device__ __forceinline__ bool stage_k_group(const KRaw& r, float bias, bool asym, uint4* kc, int lane, int entries) {
    const uint32_t s0 = __byte_perm(r.s0, r.s1, 0x5410), s1 = __byte_perm(r.s0, r.s1, 0x7632);
    uint32_t z0 = __byte_perm(r.z0, r.z1, 0x5410), z1 = __byte_perm(r.z0, r.z1, 0x7632);
    bool ok = true;
    if (asym)
        ok = __all_sync(0xFFFFFFFFu, zero_exact(bf_lo(z0)) && zero_exact(bf_hi(z0)) && zero_exact(bf_lo(z1)) &&
                                         zero_exact(bf_hi(z1)));
    if (ok) {
        z0 = biased(z0, bias);
        z1 = biased(z1, bias);
    }
    __syncwarp();                                // the group before has been read
    if (lane < entries) kc[lane] = make_uint4(s0, s1, z0, z1);
    __syncwarp();
    return ok;
}

// ---- scores of a batch: s[mt][j] += Q(tile mt) . K(n-tile j, tokens 8 j + g)
// from the lane's code words.  qf: [mt][kk][lane] A fragments.
template <int BITS, int C, int MT, bool FAST>
__device__ __forceinline__ void scores_of(float (&s)[MT][4][4], const uint32_t (&w)[4][Geo<BITS, C>::kWpl],
                                          const uint4* qf, const uint4* kc, uint32_t mg, float bias, int lane) {
    using G = Geo<BITS, C>;
#pragma unroll
    for (int kk = 0; kk < G::kSteps; ++kk) {
        const uint4 k = kc[kk * 4 + (lane & 3)];
        uint4 q[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) q[m] = qf[(m * G::kSteps + kk) * 32 + lane];
        const int wi = 2 * kk / (G::F / 2), sh = BITS * (2 * kk % (G::F / 2));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t b0 = value_pair<BITS, FAST>(w[j][wi], sh, mg, k.x, k.z, bias);
            const uint32_t b1 = value_pair<BITS, FAST>(w[j][wi], sh + BITS, mg, k.y, k.w, bias);
#pragma unroll
            for (int m = 0; m < MT; ++m) mma16816(s[m][j], q[m], b0, b1);
        }
    }
}
// the same from bf16 rows of the buffer (row of token 8 j + g: krow[j], this lane's quarter)
template <int BITS, int C, int MT>
__device__ __forceinline__ void scores_of_rows(float (&s)[MT][4][4], const __nv_bfloat16* (&krow)[4], const uint4* qf,
                                               int lane) {
    using G = Geo<BITS, C>;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t kb[C / 8];
        load_pairs<BITS, C>(krow[j], kb);
#pragma unroll
        for (int kk = 0; kk < G::kSteps; ++kk)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                mma16816(s[m][j], qf[(m * G::kSteps + kk) * 32 + lane], kb[2 * kk], kb[2 * kk + 1]);
    }
}

// the first token of slice o that is not padding, 0 .. T
__device__ __forceinline__ int padding(const View& a, int64_t o) { return a.first ? min(max(a.first[o], 0), a.T) : 0; }

// Which batches of a slice exist: those of the store come first, then the buffer's.
struct Span { int nsb, nb; };                    // store batches, all batches
__device__ __forceinline__ Span span_of(const View& a) {
    Span s;
    s.nsb = (a.tq + kBatch - 1) / kBatch;
    s.nb = s.nsb + (a.nres + kBatch - 1) / kBatch;
    return s;
}
// first token of batch b, and the end of its valid tokens
__device__ __forceinline__ void batch_at(const View& a, const Span& s, int b, int& t0, int& t1) {
    if (b < s.nsb) {
        t0 = b * kBatch;
        t1 = min(t0 + kBatch, a.tq);
    } else {
        t0 = a.tq + (b - s.nsb) * kBatch;
        t1 = min(t0 + kBatch, a.T);
    }
}
// the batch that holds token t (0 <= t < T)
__device__ __forceinline__ int batch_of(const View& a, const Span& s, int t) {
    return t < a.tq ? t / kBatch : s.nsb + (t - a.tq) / kBatch;
}

// query row r of slice o: index of its q row (times C) and of its lse
__device__ __forceinline__ int64_t row_index(const View& a, int64_t o, int r) {
    const int i = r / a.group, j = r - i * a.group;
    const uint32_t b = (uint32_t)o / (uint32_t)a.kv_heads, h = (uint32_t)o - b * (uint32_t)a.kv_heads;
    return ((int64_t)b * a.n + i) * ((int64_t)a.kv_heads * a.group) + (int64_t)h * a.group + j;
}

// A fragments of query rows [r0, r0 + 16 MT) of slice o, made by the whole CTA
// (rows past the last are zeros): entry (mt, kk, lane) = rows g and g + 8 of
// tile mt, channel pairs 2 kk and 2 kk + 1.
template <int BITS, int C, int MT>
__device__ __forceinline__ void stage_queries(const View& a, int64_t o, int r0, uint4* qf, int tid, int threads) {
    using G = Geo<BITS, C>;
    for (int e = tid; e < MT * G::kSteps * 32; e += threads) {
        const int lane = e & 31, kk = (e >> 5) % G::kSteps, mt = (e >> 5) / G::kSteps;
        const int c = (lane & 3) * (C / 4) + G::pair_channel(2 * kk);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = r0 + mt * 16 + (lane >> 2) + 8 * h;
            if (r < a.rows) {
                const __nv_bfloat16* p = a.q + row_index(a, o, r) * C + c;
                const uint32_t x = *reinterpret_cast<const uint32_t*>(p);           // channels c, c + 1
                const uint32_t y = *reinterpret_cast<const uint32_t*>(p + G::F / 2);
                w[h] = __byte_perm(x, y, 0x5410);
                w[2 + h] = __byte_perm(x, y, 0x7632);
            }
        }
        qf[e] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace rows
}  // namespace kvq
