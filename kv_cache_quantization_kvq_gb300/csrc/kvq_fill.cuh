// kvq_fill.cuh -- tiles of 128 cache tokens as swizzled bf16 operands of the
// tcgen05 products, unpacked from the codes by 128 threads.
//
// Within every 8 channels a tile holds them in the order 0 4 1 5 2 6 3 7 in which
// a code word gives them up (the other operand is laid out alike).
#pragma once

#include "kvq_fast.cuh"
#include "kvq_rows.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace fill {

using namespace rows;

constexpr int kTile = 128;

// 0 4 1 5 2 6 3 7 from eight bf16 in order
__device__ __forceinline__ uint4 interleave(const uint4& x) {
    return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                      __byte_perm(x.y, x.w, 0x7632));
}

// eight fields of a token's 8-channel piece, (i, i + 4) at bits BITS i of the halves
template <int BITS>
__device__ __forceinline__ uint32_t load_piece(const uint8_t* p) {
    if constexpr (BITS == 4) return __ldcs(reinterpret_cast<const uint32_t*>(p));
    else return __byte_perm((uint32_t)__ldcs(reinterpret_cast<const uint16_t*>(p)), 0u, 0x4140);
}

// one piece: values of fields (i, i + 4), i = 0 .. 3, with their scale and zero pairs
template <int BITS, bool FAST>
__device__ __forceinline__ uint4 unpack_piece(uint32_t w, uint32_t mg, const uint32_t (&s)[4], const uint32_t (&z)[4],
                                              float bias) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = value_pair<BITS, FAST>(w, BITS * i, mg, s[i], z[i], bias);
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Rows [rb, re) of key tile j token by token: at the padding, the store's end, in
// the buffer (hidden and missing tokens are zeros), or with far zero points or
// scales.  Values that are not finite become 0 and are noted in odd[2 C], whose next
// element then says so.  Kept out of line: inlined into the loops below it pushed them out of the instruction
// cache (5.7 warps stalled on fetches per issue).
template <int BITS, int C, bool KEYS>
__device__ __noinline__ void fill_rows(const View& a, int64_t o, int first, int j, int rb, int re, unsigned char* tile,
                                       int tid, int* odd) {
    constexpr int P = C / 8, kStep = 128 / P;
    const int p = tid % P;
    const float bias = KEYS ? a.kbias : a.vbias;
    const uint32_t mg = magic<BITS>(KEYS ? a.kflip : a.vflip);
    const uint8_t* codes = (KEYS ? a.kc : a.vc) + (uint64_t)o * a.cap * (C * BITS / 8) + p * BITS;
    constexpr int kAhead = 4;                    // buffer rows in flight
#pragma unroll 1
    for (int r = rb + tid / P; r < re; r += kAhead * kStep) {
        uint4 x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = j * kTile + r + i * kStep;
            x[i] = make_uint4(0, 0, 0, 0);
            if (r + i * kStep < re && t >= max(first, a.tq) && t < a.T)
                x[i] = *reinterpret_cast<const uint4*>((KEYS ? a.kr : a.vr) + ((uint64_t)o * a.rrows + (t - a.tq)) * C + p * 8);
        }
#pragma unroll 1
        for (int i = 0; i < kAhead; ++i) {
            const int row = r + i * kStep, t = j * kTile + row;
            if (row >= re) break;
            uint4 y = i == 0 ? x[0] : i == 1 ? x[1] : i == 2 ? x[2] : x[3];
            if (t >= a.tq) {
                y = interleave(y);
            } else if (t >= first) {
                uint32_t s[4], z[4];
                if constexpr (KEYS) {
                    const int64_t at = (o * a.ngk + t / a.gk) * C + p * 8;
                    const uint4 s4 = interleave(*reinterpret_cast<const uint4*>(a.ks + at));
                    const uint4 z4 = interleave(a.kz ? *reinterpret_cast<const uint4*>(a.kz + at) : make_uint4(0, 0, 0, 0));
                    s[0] = s4.x; s[1] = s4.y; s[2] = s4.z; s[3] = s4.w;
                    z[0] = z4.x; z[1] = z4.y; z[2] = z4.z; z[3] = z4.w;
                } else {
                    const int64_t at = (o * a.cap + t) * a.ngv + p * 8 / a.gv;
                    s[0] = s[1] = s[2] = s[3] = bits_of(a.vs + at) * 0x10001u;
                    z[0] = z[1] = z[2] = z[3] = a.vz ? bits_of(a.vz + at) * 0x10001u : 0u;
                }
                y = unpack_piece<BITS, false>(load_piece<BITS>(codes + (int64_t)t * (C * BITS / 8)), mg, s, z, bias);
            }
            if constexpr (!KEYS) {
                if (is_odd(y)) {
                    auto note = [&](uint32_t& w, int c) {           // channels c and c + 4 of the piece
                        note_odd(odd, C, p * 8 + c, w & 0xFFFFu, t);
                        note_odd(odd, C, p * 8 + c + 4, w >> 16, t);
                        w = finite_or_zero(w);
                    };
                    note(y.x, 0);
                    note(y.y, 1);
                    note(y.z, 2);
                    note(y.w, 3);
                    odd[2 * C] = 1;
                }
            }
            *reinterpret_cast<uint4*>(tile + p / 8 * (kTile * 128) + tc::swizzled(row, p % 8)) = y;
        }
    }
}

// A run of consecutive tiles of one cache by two groups of 128 threads (four warps),
// a half tile (64 tokens) each, their codes and the keys' constants staged in
// shared memory by another warp's bulk copies, three halves deep.  A thread takes
// 8-channel piece p of every (1024 / C)-th token.  With a warp or two per scheduler,
// what a half takes is the latency of its chains: one group for both halves took
// 702 us where two take 584 (128 rows over 65536 tokens and 64 slices), and
// divisions stay out of it.  Loops over a whole tile stay rolled: unrolled, with
// four quarters' words in registers, they missed the instruction cache (893 us).
template <int BITS, int C, bool KEYS>
struct Staged {
    static constexpr int P = C / 8, kStep = 128 / P, kN = 32 / kStep, kSub = 32 / P;   // rows a pass, passes of 32 tokens, rows of a warp's pass
    static constexpr int kRowB = C * BITS / 8, kHalf = 64, kStages = 3, kAhead = 8;
    static constexpr int kCodesB = kHalf * kRowB, kConstB = 2 * C * 2;                 // up to two key groups' scales
    static constexpr int kStageB = kCodesB + 2 * (C == 128 ? kConstB : 2 * kConstB);   // V: 4 warps x 4 groups x 16 words
    static constexpr int kBytes = kStages * kStageB;
    static constexpr int kOddAt = kBytes + 256;  // values: where those that are not finite are noted, from the stages

    const View& a;
    const int64_t o;
    const int first, me, sub, p, r0;             // sub: which half of every tile
    unsigned char* stage;
    uint64_t *rfull, *rfree;                     // [kStages]
    const uint8_t* codes;                        // of the slice
    const uint32_t mg, place;
    const float bias;
    const int k0;                                // halves staged before this run, in the same stages
    int h0, h1;                                  // the half tiles that are staged: whole, in the store and seen
    int rem;                                     // keys: tokens of the group before the next half
    uint32_t vm[2];                              // values: (scale, zero point) of this lane's row and groups, next half

    // tiles [j0, j0 + n)
    __device__ __forceinline__ Staged(const View& v, int64_t slice, int hidden, int j0, int n, int tid, int part,
                                      unsigned char* st, uint64_t* full, uint64_t* free, int before = 0)
        : a(v), o(slice), first(hidden), me(tid), sub(part), p(tid % P), r0(tid / P), stage(st), rfull(full), rfree(free),
          codes((KEYS ? v.kc : v.vc) + (uint64_t)slice * v.cap * kRowB), mg(magic<BITS>(KEYS ? v.kflip : v.vflip)),
          place(tid % P / 8 * (kTile * 128) + tc::swizzled(tid / P, tid % P % 8)), bias(KEYS ? v.kbias : v.vbias), k0(before) {
        h0 = max(2 * j0, (first + kHalf - 1) / kHalf);
        h1 = max(h0, min(2 * (j0 + n), a.tq / kHalf));
        rem = KEYS ? (int)((int64_t)mine() * kHalf % a.gk) : 0;
    }

    __device__ __forceinline__ int* noted() const { return KEYS ? nullptr : reinterpret_cast<int*>(stage + kOddAt); }
    __device__ __forceinline__ int staged() const { return h1 - h0; }
    __device__ __forceinline__ int mine() const { return h0 + ((h0 ^ sub) & 1); }      // this group's first staged half
    // stages half h (one lane); the stage's last readers are done
    __device__ __forceinline__ void issue(int h) const {
        const int s = (k0 + h - h0) % kStages;
        unsigned char* dst = stage + s * kStageB;
        uint32_t bytes = kCodesB;
        const int64_t t = (int64_t)h * kHalf;
        if constexpr (KEYS) {
            const int g = (int)(t / a.gk), groups = (int)((t + kHalf - 1) / a.gk) - g + 1;
            const uint32_t n = groups * C * 2;
            bytes += a.kz ? 2 * n : n;
            mbar_expect_tx(&rfull[s], bytes);
            bulk_g2s(dst + kCodesB, a.ks + (o * a.ngk + g) * C, n, &rfull[s]);
            if (a.kz) bulk_g2s(dst + kCodesB + kConstB, a.kz + (o * a.ngk + g) * C, n, &rfull[s]);
        } else {
            mbar_expect_tx(&rfull[s], bytes);
        }
        bulk_g2s(dst, codes + t * kRowB, kCodesB, &rfull[s]);
    }
    // values: the constants of half h, to registers: lane = row (l % 16) of the warp's 16, groups l / 16 and + 2
    __device__ __forceinline__ void load_meta(int h) {
        const int row = me & 15, lo = (me >> 4) & 1;
        const int64_t t = (int64_t)h * kHalf + row / kSub * kStep + (me >> 5) * kSub + row % kSub;
        const int64_t at = (o * a.cap + t) * a.ngv + lo;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            vm[k] = 0u;
            if (lo + 2 * k < a.ngv) vm[k] = bits_of(a.vs + at + 2 * k) | (a.vz ? bits_of(a.vz + at + 2 * k) << 16 : 0u);
        }
    }

    // half h of the tile; false: a wait gave up
    template <class Ready>
    __device__ __forceinline__ bool half(int h, unsigned char* tile, const Ready& ready) {
        const int rb = (h & 1) * kHalf;
        if (h < h0 || h >= h1) {
            fill_rows<BITS, C, KEYS>(a, o, first, h >> 1, rb, rb + kHalf, tile, me, noted());
            return true;
        }
        const int k = k0 + h - h0, s = k % kStages;
        unsigned char* st = stage + s * kStageB;
        uint32_t* meta = reinterpret_cast<uint32_t*>(st + kCodesB) + (me >> 5) * 64;   // [4 groups][16 rows] of this warp
        bool fast = true;
        uint32_t mv[2] = {0u, 0u};
        if constexpr (!KEYS) {                   // while the copy is on its way
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mv[i] = (vm[i] & 0xFFFFu) | (biased(vm[i], bias) & 0xFFFF0000u);
                fast = fast && scale_fits(vm[i]) && zero_exact(bf_hi(vm[i]));
            }
            fast = __all_sync(0xFFFFFFFFu, fast);
        }
        // the copy has landed, so the stage's last readers, the other group's among them, are done with it
        if (!ready(&rfull[s], (k / kStages) & 1)) return false;
        if constexpr (!KEYS) {
#pragma unroll
            for (int i = 0; i < 2; ++i) meta[(((me >> 4) & 1) + 2 * i) * 16 + (me & 15)] = mv[i];
            if (h + 2 < h1) load_meta(h + 2);
            __syncwarp();
        }
        const int vg = KEYS ? 0 : p * 8 / a.gv * 16 + r0 % kSub;
        uint32_t sk[4], zk[4];
        bool okq[2] = {fast, fast};
        int held = -1;                           // keys: the group in sk and zk, 0 or 1 of the stage's
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            unsigned char* dst = tile + place + (rb + 32 * q) * 128;
            const unsigned char* src = st + (32 * q + r0) * kRowB + p * BITS;
            if constexpr (KEYS) {
                const int now = q && rem + 32 >= a.gk ? 1 : 0;
                if (now != held) {
                    const unsigned char* c = st + kCodesB + now * (C * 2) + p * 16;
                    const uint4 s4 = interleave(*reinterpret_cast<const uint4*>(c));
                    const uint4 z4 = a.kz ? interleave(*reinterpret_cast<const uint4*>(c + kConstB)) : make_uint4(0, 0, 0, 0);
                    sk[0] = s4.x; sk[1] = s4.y; sk[2] = s4.z; sk[3] = s4.w;
                    zk[0] = z4.x; zk[1] = z4.y; zk[2] = z4.z; zk[3] = z4.w;
                    fast = true;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        fast = fast && zero_exact(bf_lo(zk[i])) && zero_exact(bf_hi(zk[i]));
                        zk[i] = biased(zk[i], bias);
                    }
                    held = now;
                }
                okq[q] = fast;
            }
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                uint32_t w;
                if constexpr (BITS == 4) w = *reinterpret_cast<const uint32_t*>(src + i * kStep * kRowB);
                else w = __byte_perm((uint32_t)*reinterpret_cast<const uint16_t*>(src + i * kStep * kRowB), 0u, 0x4140);
                if constexpr (!KEYS) {
                    const uint32_t x = meta[vg + (32 / kStep * q + i) * kSub];
                    sk[0] = sk[1] = sk[2] = sk[3] = __byte_perm(x, 0u, 0x1010);
                    zk[0] = zk[1] = zk[2] = zk[3] = __byte_perm(x, 0u, 0x3232);
                }
                *reinterpret_cast<uint4*>(dst + i * kStep * 128) = unpack_piece<BITS, true>(w, mg, sk, zk, 0.0f);
            }
        }
        if (!okq[0] || !okq[1]) fill_rows<BITS, C, KEYS>(a, o, first, h >> 1, rb, rb + kHalf, tile, me, noted());
        if constexpr (KEYS) {
            rem += 2 * kHalf;
            while (rem >= a.gk) rem -= a.gk;
        }
        __syncwarp();
        if ((me & 31) == 0) mbar_arrive(&rfree[s]);
        return true;
    }

    // every tile, in order: `enter(j)` waits for tile buffer j's turn and returns it (nullptr: give up), `leave(j)` hands it on
    template <class Ready, class Enter, class Leave>
    __device__ __forceinline__ bool run(int j0, int n, const Ready& ready, const Enter& enter, const Leave& leave) {
        if (!KEYS && mine() < h1) load_meta(mine());
        for (int j = 0; j < n; ++j) {
            unsigned char* tile = enter(j);
            if (!tile || !half(2 * (j0 + j) + sub, tile, ready)) return false;
            leave(j);
        }
        return true;
    }
    // the copies, by one warp: each stage again when its four readers are done; the codes come into L2 before that
    template <class Ready>
    __device__ __forceinline__ bool produce(const Ready& ready) const {
        int h = h0;
        for (; h < h1; ++h) {
            const int k = k0 + h - h0;
            if (k >= kStages && !ready(&rfree[k % kStages], (k / kStages - 1) & 1)) break;
            if (tc::elect()) {
                if (h + kAhead < h1) bulk_prefetch_l2(codes + (int64_t)(h + kAhead) * kHalf * kRowB, kCodesB);
                issue(h);
            }
            __syncwarp();
            if constexpr (!KEYS) {               // and the values' constants: lines of 64 elements of scales, zero points
                const int lane = me & 31, at = (lane >> 1) * 64;
                const __nv_bfloat16* m = (lane & 1) ? a.vz : a.vs;
                if (m && h + kAhead < h1 && at < kHalf * a.ngv)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(m + (o * a.cap + (int64_t)(h + kAhead) * kHalf) * a.ngv + at));
            }
        }
        // before the shared memory goes: every copy issued has landed
        for (int k = k0 + max(0, h - h0 - kStages); k < k0 + h - h0; ++k) tc::drain(&rfull[k % kStages], (k / kStages) & 1);
        return h == h1;
    }
};

}  // namespace fill
}  // namespace kvq
