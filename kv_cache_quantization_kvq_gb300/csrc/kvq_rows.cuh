// kvq_rows.cuh -- K and V rows of the streaming cache as mma.sync fragments.
//
// A batch is 32 consecutive cache tokens, all of the store or all of the
// buffer.  A warp turns a batch's packed codes into the B fragments of
// mma.sync.m16n8k16 (bf16 x bf16 -> float32) without shared memory: the order
// of the contracted index is free as long as both operands use the same, so
// each is chosen such that a lane reads one contiguous piece of a code row.
//  * scores, contraction over channels: lane (g, tig) = (lane / 4, lane % 4)
//    reads its quarter of token g's row, channels [tig C/4, (tig+1) C/4).  A
//    32-bit code word of F fields holds the channel pairs (i, i + F/2): fields
//    BITS apart in its two halves, so one shift and one mask-and-or leave both
//    as the bf16 values 128 + field;
//  * values, contraction over tokens: lane (g, tig) reads channels
//    [g C/8, (g+1) C/8) of the four tokens its score fragment covers; a byte
//    permute pairs the words of two tokens, then the same shift and mask.
// One bf16x2 subtraction of 128 + off + zp is exact when |zp| <= 112 and an
// integer (every operand and result is an integer of at most 256), and one
// bf16x2 product with the bf16 scale rounds once: exactly RN_bf16(s (code -
// zp)), what kvq_dequantize stores (its float32 product of an 8-bit and an
// 8-bit significand is exact).  Groups with other zero points take the
// float32 route: subtract, multiply and round as kvq_dequantize does.
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
    float koff, voff;                            // that offset: 2^(bits-1) or 0
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
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// zero point of a pair as the fast route wants it, and whether it may take it
__device__ __forceinline__ bool zero_exact(float z) { return fabsf(z) <= 112.0f && z == rintf(z); }

template <int BITS, int C>
struct Geo {
    static constexpr int kRowB = C * BITS / 8;   // packed bytes of a token row
    static constexpr int F = 32 / BITS;          // fields of a word
    static constexpr int kWpl = kRowB / 16;      // words of a row per lane, score side
    static constexpr int kPairs = C / 8;         // channel pairs per lane, score side
    static constexpr int kSteps = C / 16;        // k-steps of a score product
    static constexpr int kVB = kRowB / 8;        // bytes of a row per lane, value side (2, 4 or 8)
    static constexpr int kVW = kVB >= 4 ? kVB / 4 : 1;
    static constexpr int kTiles = C / 8;         // n-tiles of a value product
    static constexpr uint32_t kMask = BITS == 4 ? 0x000F000Fu : 0x00030003u;
};

constexpr uint32_t kOne28 = 0x43004300u;         // bf16 128.0 in both halves

// Channel pairs (c, c + F/2) of this lane's quarter of a bf16 row, from the
// quarter's first element: the order of the code words' fields.
template <int BITS, int C>
__device__ __forceinline__ void load_pairs(const __nv_bfloat16* quarter, uint32_t (&pr)[Geo<BITS, C>::kPairs]) {
    using G = Geo<BITS, C>;
    constexpr int N = C / 8;                     // 32-bit words of the quarter
    uint32_t r[N];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(quarter)[i];
        r[4 * i] = x.x; r[4 * i + 1] = x.y; r[4 * i + 2] = x.z; r[4 * i + 3] = x.w;
    }
#pragma unroll
    for (int p = 0; p < G::kPairs; ++p) {
        const int c = p / (G::F / 2) * G::F + p % (G::F / 2);
        pr[p] = __byte_perm(r[c / 2], r[(c + G::F / 2) / 2], (c & 1) ? 0x7632 : 0x5410);
    }
}

// K constants of one group for this lane's channels: scales and, in the fast
// form, 128 + off + zp (else the raw zero points).  Returns whether the whole
// warp may take the fast route.
template <int BITS, int C>
__device__ __forceinline__ bool load_k_group(const View& a, int64_t o, int gk, int tig,
                                             uint32_t (&s)[C / 8], uint32_t (&z)[C / 8]) {
    const int64_t at = (o * a.ngk + gk) * C + tig * (C / 4);
    load_pairs<BITS, C>(a.ks + at, s);
    if (!a.kz) {
        const uint32_t v = pack_bf16x2(128.0f + a.koff, 128.0f + a.koff);
#pragma unroll
        for (int p = 0; p < C / 8; ++p) z[p] = v;
        return true;
    }
    load_pairs<BITS, C>(a.kz + at, z);
    bool ok = true;
#pragma unroll
    for (int p = 0; p < C / 8; ++p) ok = ok && zero_exact(bf_lo(z[p])) && zero_exact(bf_hi(z[p]));
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok) {
        const float b = 128.0f + a.koff;
#pragma unroll
        for (int p = 0; p < C / 8; ++p) z[p] = pack_bf16x2(__fadd_rn(b, bf_lo(z[p])), __fadd_rn(b, bf_hi(z[p])));
    }
    return ok;
}

// One pair of rows' values from two fields of w at bit `sh` of its halves.
template <int BITS, bool FAST>
__device__ __forceinline__ uint32_t value_pair(uint32_t w, int sh, uint32_t s, uint32_t z, float off) {
    const uint32_t x = (w >> sh) & Geo<BITS, 64>::kMask;
    if constexpr (FAST) return mul_bf16x2(sub_bf16x2(x | kOne28, z), s);
    const float lo = __fsub_rn(__fsub_rn((float)(x & 0xFFFFu), off), bf_lo(z));
    const float hi = __fsub_rn(__fsub_rn((float)(x >> 16), off), bf_hi(z));
    return pack_bf16x2(__fmul_rn(lo, bf_lo(s)), __fmul_rn(hi, bf_hi(s)));
}

// Scores of one n-tile (8 tokens) from a lane's code words of its token.
template <int BITS, int C, bool FAST>
__device__ __forceinline__ void keys_of(const uint32_t (&w)[Geo<BITS, C>::kWpl], const uint32_t (&s)[C / 8],
                                        const uint32_t (&z)[C / 8], float off, uint32_t (&b)[C / 8]) {
    using G = Geo<BITS, C>;
#pragma unroll
    for (int p = 0; p < G::kPairs; ++p)
        b[p] = value_pair<BITS, FAST>(w[p / (G::F / 2)], BITS * (p % (G::F / 2)), s[p], z[p], off);
}

// Which batches of a slice a set of query rows can see: batches of the store
// come first, then the buffer's.
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

// query row r of slice o: element offset of its q row / index of its lse
__device__ __forceinline__ int64_t row_index(const View& a, int64_t o, int r) {
    const int i = r / a.group, j = r - i * a.group;
    const int64_t b = o / a.kv_heads, h = o - b * a.kv_heads;
    return (b * a.n + i) * ((int64_t)a.kv_heads * a.group) + h * a.group + j;
}

}  // namespace rows
}  // namespace kvq
