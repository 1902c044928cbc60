// prefix.cu -- attention of many query rows to a quantized prefix that all of
// them see, on pairs of SMs (kvq_attend_shared, head_dim 128).
//
// Method as in prefill.cu's fused form: codes are unpacked into swizzled bf16 tiles
// by fill warps, and the cache is read once.  Per 128-token tile the unpacking
// takes as long as the products of a few hundred rows, and an SM's tensor memory
// holds 256.  So two SMs share it: their CTAs, a cluster, are a tcgen05 CTA pair, whose products
// take half of the B operand from each SM's shared memory.  Each CTA unpacks the
// keys of half of a tile's tokens and half of the channels of its values, and both
// use all of them for 256 rows each: 512 rows a pair, half of the unpacking and
// half of the shared memory a row.
//
// attend_prefix_kernel: a pair of CTAs per (slice, 512 rows, split of the key
// tiles), two row tiles of 256 rows, of which CTA c has 128 c .. 128 c + 127.  In each CTA
// warps 0-3 and 4-7 are the softmax of its rows of the row tiles, a thread per row;
// in the first CTA warps 8 and 9 issue the pair's products of a row tile each; warps 10 and
// 11 copy the codes by bulk copies; warps 12-15 unpack keys and 16-19 values.  Every row sees every token that
// exists, so only the first and the last tile are masked.  Each split leaves (y, m, l) per row,
// joined in merge_rows_kernel (chunk.cu).
//
// Measured on one GB300: 128 requests x 4 heads, 4 bits, over a prefix of 131072 tokens of 8 KV heads 205 us
// (1.34 PFLOP/s of products; the call, with its own tokens and the joining, 230).  What bounds it is the chain
// scores -> weights -> value product of a row tile, of which an SM has two: tensor pipe 62 %, issue slots 60 %.
#include <algorithm>

#include "kvq_chunk.cuh"
#include "kvq_fill.cuh"

namespace kvq {

namespace {

using namespace rows;
using fill::interleave;
using fill::load_piece;
using fill::unpack_piece;

constexpr int C = 128;
constexpr int kTile = 128;                       // tokens of a key tile, rows of a CTA's part of a row tile
constexpr int kSub = 64;                          // tokens whose scores a row tile holds at a time, twice
constexpr int kSlots = 3;                        // tiles of keys and of values in shared memory
constexpr int kStages = 3;                       // tiles of codes
constexpr int kThreads = 640;                    // 20 warps, 96 registers each at launch (61440 in all):
constexpr int kRegsSoftmax = 144;                // 8 softmax warps take 144, for a row of weights and a quarter of
constexpr int kRegsOther = 64;                   // its scores, and the other twelve keep 64 (61440)
static_assert(256 * kRegsSoftmax + 384 * kRegsOther <= kThreads * 96, "registers of the launch");
constexpr float kSlack = 8.0f;                   // base-2 growth of the maximum that is let pass

// ---------------------------------------------------------------- pairs of CTAs
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
// One arrival on the first CTA's barrier.  What it hands on lies in this SM's shared and tensor memory, which the
// tensor cores of both read, and has been fenced for them before; with a release at cluster scope every arrival waited for
// all of the SM's stores (445 us where 405 are without).
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(at_rank(bar, 0)) : "memory");
}
__device__ __forceinline__ void alloc_pair(uint32_t* slot, uint32_t cols) {      // one warp of each CTA
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void dealloc_pair(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void mma_ss_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_ts_pair(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"((uint32_t)add)
        : "memory");
}
// both CTAs' barriers get one arrival when everything issued before by this thread is done
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_u32(bar)), "h"((uint16_t)3)
                 : "memory");
}

// ---------------------------------------------------------------- shared memory
template <int BITS>
struct Smem {
    static constexpr int kRowB = C * BITS / 8;
    static constexpr int kQB = kTile * C * 2;    // a CTA's rows of a row tile
    static constexpr int kTileB = kQB / 2;       // a CTA's half of a key or value tile
    static constexpr int kRawK = 64 * kRowB + 4 * C * 2;           // codes of 64 tokens, scales and zero points of each 32
    static constexpr int kRawV = kTile * kRowB;  // codes of 128 tokens, all channels
    static constexpr int kQ = 0, kK = 2 * kQB, kV = kK + kSlots * kTileB, kCodesK = kV + kSlots * kTileB;
    static constexpr int kCodesV = kCodesK + kStages * kRawK, kMeta = kCodesV + kStages * kRawV;
    static constexpr int kBars = kMeta + 4 * 64 * 4, kOdd = kBars + 512, kBytes = kOdd + (2 * C + 4) * 4 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    static_assert(kRawK % 128 == 0 && kRawV % 128 == 0, "bulk copies are aligned");
};

struct PrefixArgs {
    ChunkArgs A;
    int32_t ntiles;                              // of 512 rows in a slice
};

// ---------------------------------------------------------------- unpacking
// A CTA's half of the tiles [j0, j0 + n) of keys or values, by 128 threads.  Keys: rows 0 .. 31 are
// tokens 32 c .. of a tile's first 64, rows 32 .. 63 of the others; a thread has 8-channel piece me % 16 of
// rows me / 16 + 8 i.  Values: pieces 8 c + me % 8 of all 128 tokens; a warp has 32 of them.
template <int BITS, bool KEYS>
struct Half {
    using S = Smem<BITS>;
    static constexpr int kRowB = S::kRowB, kRaw = KEYS ? S::kRawK : S::kRawV;

    const View& a;
    const int64_t o;
    const int first, j0, n, c, me;
    int ja, jb;                                  // the tiles whose codes are staged: whole, in the store and not padding
    const int p, r0, step;                       // piece of a row, first row, rows between
    const uint8_t* codes;
    const uint32_t mg;
    const float bias;

    __device__ __forceinline__ Half(const View& v, int64_t slice, int hidden, int j, int count, int rank, int tid)
        : a(v), o(slice), first(hidden), j0(j), n(count), c(rank), me(tid), p(KEYS ? tid % 16 : rank * 8 + tid % 8),
          r0(KEYS ? tid / 16 : tid / 32 * 32 + tid % 32 / 8), step(KEYS ? 8 : 4),
          codes((KEYS ? v.kc : v.vc) + (uint64_t)slice * v.cap * kRowB), mg(magic<BITS>(KEYS ? v.kflip : v.vflip)),
          bias(KEYS ? v.kbias : v.vbias) {
        ja = max(j0, (first + kTile - 1) / kTile);
        jb = max(ja, min(j0 + n, a.tq / kTile));
    }
    __device__ __forceinline__ int token(int j, int row) const {
        return j * kTile + (KEYS ? row / 32 * kSub + 32 * c + row % 32 : row);
    }
    __device__ __forceinline__ uint32_t place(int row) const {
        return KEYS ? p / 8 * (64 * 128) + tc::swizzled(row, p % 8) : tc::swizzled(row, p % 8);
    }

    // the copies, by one warp: tile j's into its stage
    __device__ __forceinline__ void issue(int j, unsigned char* raw, uint64_t* full) const {
        const int s = (j - ja) % kStages;
        unsigned char* dst = raw + s * kRaw;
        if constexpr (KEYS) {                    // 32 tokens are of one group
            mbar_expect_tx(&full[s], 64 * kRowB + (a.kz ? 4 : 2) * C * 2);
            for (int q = 0; q < 2; ++q) {
                const int64_t t = token(j, 32 * q), g = (o * a.ngk + t / a.gk) * C;
                bulk_g2s(dst + 32 * q * kRowB, codes + t * kRowB, 32 * kRowB, &full[s]);
                bulk_g2s(dst + 64 * kRowB + q * C * 2, a.ks + g, C * 2, &full[s]);
                if (a.kz) bulk_g2s(dst + 64 * kRowB + (2 + q) * C * 2, a.kz + g, C * 2, &full[s]);
            }
        } else {
            mbar_expect_tx(&full[s], kTile * kRowB);
            bulk_g2s(dst, codes + (int64_t)j * kTile * kRowB, kTile * kRowB, &full[s]);
        }
        // into L2 some tiles ahead: the first CTA fetches keys, the second values
        if (j + 8 < jb && c == (KEYS ? 0 : 1)) bulk_prefetch_l2(codes + (int64_t)(j + 8) * kTile * kRowB, kTile * kRowB);
    }
    template <class Ready>
    __device__ __forceinline__ void copy(unsigned char* raw, uint64_t* full, uint64_t* free, const Ready& ready) const {
        int j = ja;
        for (; j < jb; ++j) {
            const int k = j - ja;
            if (k >= kStages && !ready(&free[k % kStages], (k / kStages - 1) & 1)) break;
            if (tc::elect()) issue(j, raw, full);
            __syncwarp();
        }
        // before the shared memory goes: every copy issued has landed
        for (int k = max(0, j - ja - kStages); k < j - ja; ++k) tc::drain(&full[k % kStages], (k / kStages) & 1);
    }

    // tile j row by row: at the padding, the store's end, in the buffer (what does not exist is zeros), or with
    // far zero points or scales; values that are not finite become 0 and are noted
    __device__ __noinline__ void slow(int j, unsigned char* tile, int* odd) const {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const int row = r0 + i * step, t = token(j, row);
            uint4 y = make_uint4(0, 0, 0, 0);
            if (t >= first && t < a.T) {
                if (t >= a.tq) {
                    y = interleave(*reinterpret_cast<const uint4*>((KEYS ? a.kr : a.vr) + ((uint64_t)o * a.rrows + (t - a.tq)) * C + p * 8));
                } else {
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
                    y = unpack_piece<BITS, false>(load_piece<BITS>(codes + (int64_t)t * kRowB + p * BITS), mg, s, z, bias);
                }
            }
            if constexpr (!KEYS) {
                if (is_odd(y)) {
                    auto note = [&](uint32_t& w, int ch) {          // channels ch and ch + 4 of the piece
                        note_odd(odd, C, p * 8 + ch, w & 0xFFFFu, t);
                        note_odd(odd, C, p * 8 + ch + 4, w >> 16, t);
                        w = finite_or_zero(w);
                    };
                    note(y.x, 0);
                    note(y.y, 1);
                    note(y.z, 2);
                    note(y.w, 3);
                    odd[2 * C] = 1;
                }
            }
            *reinterpret_cast<uint4*>(tile + place(row)) = y;
        }
    }

    // values: (scale, zero point) of token `lane` of the warp's 32 of tile j, a word for each of the half's groups
    __device__ __forceinline__ void load_meta(int j, uint32_t (&vm)[2]) const {
        const int64_t t = (int64_t)j * kTile + (me & ~31) + (me & 31);
        const int64_t at = (o * a.cap + t) * a.ngv + c * 64 / a.gv;
        vm[0] = bits_of(a.vs + at) | (a.vz ? bits_of(a.vz + at) << 16 : 0u);
        vm[1] = a.gv == 32 ? bits_of(a.vs + at + 1) | (a.vz ? bits_of(a.vz + at + 1) << 16 : 0u) : vm[0];
    }

    // every tile, in order: enter(i) waits for the turn of tile j0 + i and returns its buffer (nullptr: give up),
    // leave(i) hands it on
    template <class Ready, class Enter, class Leave>
    __device__ __forceinline__ void run(unsigned char* raw, uint32_t* meta, uint64_t* full, uint64_t* free, int* odd,
                                        const Ready& ready, const Enter& enter, const Leave& leave) const {
        const int lane = me & 31;
        uint32_t vm[2] = {0u, 0u};
        auto staged = [&](int j) { return j >= ja && j < jb; };
        if (!KEYS && staged(j0)) load_meta(j0, vm);
        for (int i = 0; i < n; ++i) {
            const int j = j0 + i;
            unsigned char* tile = enter(i);
            if (!tile) return;
            if (!staged(j)) {
                slow(j, tile, odd);
                if (!KEYS && staged(j + 1)) load_meta(j + 1, vm);
            } else {
                const int k = j - ja, s = k % kStages;
                const unsigned char* st = raw + s * kRaw;
                bool fast = true;
                if constexpr (!KEYS) {           // while the copy is on its way
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        meta[g * 32 + lane] = (vm[g] & 0xFFFFu) | (biased(vm[g], bias) & 0xFFFF0000u);
                        fast = fast && scale_fits(vm[g]) && zero_exact(bf_hi(vm[g]));
                    }
                    fast = __all_sync(0xFFFFFFFFu, fast);
                    if (staged(j + 1)) load_meta(j + 1, vm);
                }
                if (!ready(&full[s], (k / kStages) & 1)) return;
                if constexpr (KEYS) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t sk[4], zk[4];
                        const unsigned char* cst = st + 64 * kRowB + q * C * 2 + p * 16;
                        const uint4 s4 = interleave(*reinterpret_cast<const uint4*>(cst));
                        const uint4 z4 = a.kz ? interleave(*reinterpret_cast<const uint4*>(cst + 2 * C * 2)) : make_uint4(0, 0, 0, 0);
                        sk[0] = s4.x; sk[1] = s4.y; sk[2] = s4.z; sk[3] = s4.w;
                        zk[0] = z4.x; zk[1] = z4.y; zk[2] = z4.z; zk[3] = z4.w;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            fast = fast && zero_exact(bf_lo(zk[e])) && zero_exact(bf_hi(zk[e]));
                            zk[e] = biased(zk[e], bias);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int row = r0 + (4 * q + e) * 8;
                            const unsigned char* src = st + row * kRowB + p * BITS;
                            uint32_t w;
                            if constexpr (BITS == 4) w = *reinterpret_cast<const uint32_t*>(src);
                            else w = __byte_perm((uint32_t)*reinterpret_cast<const uint16_t*>(src), 0u, 0x4140);
                            *reinterpret_cast<uint4*>(tile + place(row)) = unpack_piece<BITS, true>(w, mg, sk, zk, 0.0f);
                        }
                    }
                } else {
                    __syncwarp();
                    const uint32_t* m = meta + (p * 8 % 64 >= 32 && a.gv == 32 ? 32 : 0);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int row = r0 + e * 4;
                        const unsigned char* src = st + row * kRowB + p * BITS;
                        uint32_t w;
                        if constexpr (BITS == 4) w = *reinterpret_cast<const uint32_t*>(src);
                        else w = __byte_perm((uint32_t)*reinterpret_cast<const uint16_t*>(src), 0u, 0x4140);
                        const uint32_t x = m[row & 31], sv = __byte_perm(x, 0u, 0x1010), zv = __byte_perm(x, 0u, 0x3232);
                        const uint32_t s4[4] = {sv, sv, sv, sv}, z4[4] = {zv, zv, zv, zv};
                        *reinterpret_cast<uint4*>(tile + place(row)) = unpack_piece<BITS, true>(w, mg, s4, z4, 0.0f);
                    }
                }
                // a thread writes the same pieces either way
                if (!fast) slow(j, tile, odd);
                __syncwarp();
                if (lane == 0) mbar_arrive(&free[s]);
            }
            leave(i);
        }
    }
};

template <int BITS>
__global__ void __launch_bounds__(kThreads, 1)
attend_prefix_kernel(const __grid_constant__ PrefixArgs X)
{
    using S = Smem<BITS>;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);          // alike in both CTAs
    // of the first CTA's, both arrive on these:
    uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + S::kBars);  // [kSlots] both halves of a key tile are unpacked
    uint64_t* vfull = kfull + kSlots;
    uint64_t* pfull = vfull + kSlots;            // [2 x 2] weights of a row tile's half are in tensor memory
    // and these are each CTA's own:
    uint64_t* kfree = pfull + 4;                 // [kSlots] every row tile is done with it
    uint64_t* vfree = kfree + kSlots;
    uint64_t* sfull = vfree + kSlots;            // [2 x 2] its scores are
    uint64_t* odone = sfull + 4;                 // [2 x 2] its value product is done
    uint64_t* rk = odone + 4;                    // [2][kStages] codes of keys: full, free
    uint64_t* rv = rk + 2 * kStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rv + 2 * kStages);
    volatile int* gone = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* odd = reinterpret_cast<int*>(sm + S::kOdd);               // [2 C], and whether any is noted

    const ChunkArgs& A = X.A;
    const View& a = A.v;
    // the shuffle tells the compiler that a warp's number is uniform: the products' operands then are, too
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int rank = (int)cta_rank();
    const int pair = blockIdx.x >> 1, split = pair % A.nsplit, tile = pair / A.nsplit % X.ntiles;
    const int64_t o = pair / A.nsplit / X.ntiles;
    const int r0 = tile * 512, nrows = min(512, a.rows - r0), nt = nrows > 256 ? 2 : 1;
    const int first = padding(a, o);
    int j0 = 0, n = 0;
    if (first < a.T) {                           // this split's tiles of the ones with tokens
        const int lo = first / kTile;
        const int64_t len = (a.T + kTile - 1) / kTile - lo;
        j0 = lo + (int)(len * split / A.nsplit);
        n = lo + (int)(len * (split + 1) / A.nsplit) - j0;
    }

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&kfull[i], 8);             // four warps of each CTA
            mbar_init(&vfull[i], 8);
            mbar_init(&kfree[i], nt);
            mbar_init(&vfree[i], nt);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&pfull[i], 8);
            mbar_init(&sfull[i], 1);
            mbar_init(&odone[i], 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&rk[i], 1);
            mbar_init(&rk[kStages + i], 4);
            mbar_init(&rv[i], 1);
            mbar_init(&rv[kStages + i], 4);
        }
        *gone = 0;
        mbar_init_fence();
    }
    for (int i = tid; i <= 2 * C; i += kThreads) odd[i] = i < 2 * C ? kNever : 0;
    if (warp == 8) alloc_pair(tmem_slot, 512);
    if (tid == 352 && n > 0 && j0 * kTile < a.tq)                  // the first codes into L2, while the CTAs meet
        bulk_prefetch_l2((rank ? a.vc : a.kc) + ((uint64_t)o * a.cap + j0 * kTile) * S::kRowB, min(8 * kTile, (a.tq - j0 * kTile)) * S::kRowB);
    {
        // the queries, four of a thread's pieces in flight at once
        constexpr int kEach = 4;
#pragma unroll 1
        for (int k0 = tid; k0 < nt * kTile * (C / 8); k0 += kEach * kThreads) {
            uint4 x[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int k = k0 + i * kThreads, t = k / (kTile * (C / 8)), row = k / (C / 8) % kTile, p = k % (C / 8);
                const int r = r0 + t * 256 + rank * kTile + row;
                x[i] = make_uint4(0, 0, 0, 0);
                if (t < nt && r < a.rows) x[i] = *reinterpret_cast<const uint4*>(a.q + row_index<true>(a, o, r) * C + p * 8);
            }
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int k = k0 + i * kThreads, t = k / (kTile * (C / 8)), row = k / (C / 8) % kTile, p = k % (C / 8);
                if (t < nt)
                    *reinterpret_cast<uint4*>(sm + S::kQ + t * S::kQB + (p / 8) * (kTile * 128) + tc::swizzled(row, p % 8)) = interleave(x[i]);
            }
        }
    }
    tc::async_fence();
    tc::before_sync();
    __syncthreads();
    cluster_sync();                              // both CTAs' barriers, queries and tensor memory are there
    tc::after_sync();
    const uint32_t tmem = *tmem_slot;
    auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, tc::wait(bar, parity & 1, gone)) != 0; };

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    if (warp >= 12) {
        // ---- unpacking
        auto role = [&](const auto& f, unsigned char* codes, uint64_t* bars, uint64_t* full, uint64_t* free, unsigned char* tiles) {
            f.run(codes, reinterpret_cast<uint32_t*>(sm + S::kMeta) + (warp & 3) * 64, bars, bars + kStages, odd, ready,
                  [&](int i) -> unsigned char* {
                      return i >= kSlots && !ready(&free[i % kSlots], i / kSlots - 1) ? nullptr : tiles + i % kSlots * S::kTileB;
                  },
                  [&](int i) {
                      tc::async_fence();
                      __syncwarp();
                      if (lane == 0) arrive_first(&full[i % kSlots]);
                  });
        };
        if (warp < 16) role(Half<BITS, true>(a, o, first, j0, n, rank, tid & 127), sm + S::kCodesK, rk, kfull, kfree, sm + S::kK);
        else role(Half<BITS, false>(a, o, first, j0, n, rank, tid & 127), sm + S::kCodesV, rv, vfull, vfree, sm + S::kV);
    } else if (warp >= 10) {
        if (warp == 10) Half<BITS, true>(a, o, first, j0, n, rank, lane).copy(sm + S::kCodesK, rk, rk + kStages, ready);
        else Half<BITS, false>(a, o, first, j0, n, rank, lane).copy(sm + S::kCodesV, rv, rv + kStages, ready);
    } else if (warp >= 8) {
        // ---- products of row tile t, of both CTAs
        const int t = warp - 8;
        if (rank == 0 && t < nt && n > 0) {
            constexpr uint32_t kScores = tc::instr_desc(256, kSub, false), kValues = tc::instr_desc(256, C, true);
            const uint32_t q_at = smem_u32(sm + S::kQ) + t * S::kQB, k_at = smem_u32(sm + S::kK), v_at = smem_u32(sm + S::kV);
            const uint32_t s_at = tmem + t * kTile, o_at = tmem + 256 + t * C;
            auto scores = [&](int u) {           // of half tile u
                const uint32_t at = k_at + (u >> 1) % kSlots * S::kTileB + (u & 1) * (32 * 128);
#pragma unroll
                for (int k = 0; k < C / 16; ++k)
                    mma_ss_pair(s_at + (u & 1) * kSub, tc::smem_desc(q_at + (k / 4) * (kTile * 128) + (k % 4) * 32, 16),
                                tc::smem_desc(at + (k / 4) * (64 * 128) + (k % 4) * 32, 16), kScores, k > 0);
                commit_pair(&sfull[2 * t + (u & 1)]);
                if (u & 1) commit_pair(&kfree[(u >> 1) % kSlots]);
            };
            bool ok = ready(&kfull[0], 0);
            tc::after_sync();
            if (ok && tc::elect()) {
                scores(0);
                scores(1);
            }
            __syncwarp();
            for (int u = 0; ok && u < 2 * n; ++u) {
                const int j = u >> 1, s = j % kSlots;
                if (!(u & 1)) {
                    ok = ready(&vfull[s], j / kSlots);
                    if (j + 1 < n) ok = ok && ready(&kfull[(j + 1) % kSlots], (j + 1) / kSlots);
                }
                ok = ok && ready(&pfull[2 * t + (u & 1)], j);
                if (!ok) break;
                tc::after_sync();
                if (tc::elect()) {
                    const uint32_t at = v_at + s * S::kTileB + (u & 1) * (kSub * 128);
#pragma unroll
                    for (int k = 0; k < kSub / 16; ++k)
                        mma_ts_pair(o_at, s_at + (u & 1) * kSub + k * 8, tc::smem_desc(at + k * 2048, kTile * 128), kValues,
                                    u > 0 || k > 0);
                    commit_pair(&odone[2 * t + (u & 1)]);
                    if (u & 1) commit_pair(&vfree[s]);
                    if (j + 1 < n) scores(u + 2);
                }
                __syncwarp();
            }
        }
    } else if (warp < 4 * nt) {
        // ---- softmax of this CTA's rows of row tile t, a thread per row
        const int t = warp / 4;
        const int r = r0 + t * 256 + rank * kTile + (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + t * kTile, o_at = tmem + lanes + 256 + t * C;
        float m = -INFINITY;
        u64 sum = 0;
        bool ok = true;
        for (int u = 0; ok && u < 2 * n; ++u) {  // half tiles of 64 tokens
            const uint32_t su = s_at + (u & 1) * kSub;
            ok = ready(&sfull[2 * t + (u & 1)], u >> 1);
            if (!ok) break;
            tc::after_sync();
            uint32_t s[kSub];
            tc::ld32(su, s);
            tc::ld32(su + 32, s + 32);
            tc::wait_ld();
            // tokens [lo, hi) of the half tile exist and are not padding
            const int c0 = j0 * kTile + u * kSub, lo = first - c0, hi = a.T - c0;
            if (lo > 0 || hi < kSub) {
#pragma unroll
                for (int i = 0; i < kSub; ++i)
                    if (i < lo || i >= hi) s[i] = 0xFF800000u;     // -inf
            }
            float x0 = -INFINITY, x1 = -INFINITY, x2 = -INFINITY, x3 = -INFINITY;
#pragma unroll
            for (int i = 0; i < kSub; i += 4) {
                x0 = fmaxf(x0, __uint_as_float(s[i]));
                x1 = fmaxf(x1, __uint_as_float(s[i + 1]));
                x2 = fmaxf(x2, __uint_as_float(s[i + 2]));
                x3 = fmaxf(x3, __uint_as_float(s[i + 3]));
            }
            const float top = __fmul_rn(fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)), a.scale2);
            const bool grow = top > __fadd_rn(m, kSlack);           // m = -inf: whenever anything is seen
            if (__any_sync(0xFFFFFFFFu, grow)) {
                const float f = grow ? ex2(__fsub_rn(m, top)) : 1.0f;
                if (grow) m = top;
                sum = mul2(sum, pk(f, f));
                if (u > 0) {
                    // the products before this half tile's are done (the scores' arrival says so of those before them)
                    ok = ready(&odone[2 * t + ((u - 1) & 1)], (u - 1) >> 1);
                    if (!ok) break;
                    tc::after_sync();
#pragma unroll 1
                    for (int i = 0; i < C / 32; ++i) {
                        uint32_t y[32];
                        tc::ld32(o_at + 32 * i, y);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__fmul_rn(__uint_as_float(y[e]), f));
                        tc::st32(o_at + 32 * i, y);
                    }
                }
            }
            const float neg = m == -INFINITY ? 0.0f : -m;
            const u64 sc2 = pk(a.scale2, a.scale2), ng2 = pk(neg, neg);
            uint32_t p[kSub / 2];
            u64 s0 = 0, s1 = 0;
#pragma unroll
            for (int i = 0; i < kSub / 2; ++i) {
                const u64 e = fma2(pk(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sc2, ng2);
                const float e0 = ex2(lo_of(e)), e1 = ex2(hi_of(e));
                if (i & 1) s1 = add2(s1, pk(e0, e1));
                else s0 = add2(s0, pk(e0, e1));
                p[i] = pack_bf16x2(e0, e1);
            }
            sum = add2(sum, add2(s0, s1));
            tc::st32(su, p);
            tc::wait_st();
            tc::before_sync();
            __syncwarp();
            if (lane == 0) arrive_first(&pfull[2 * t + (u & 1)]);
        }
        // ---- the row's sums
        asm volatile("griddepcontrol.launch_dependents;");
        float l = 0.0f;
        if (ok && n > 0) {
            ok = ready(&odone[2 * t + 1], n - 1);
            tc::after_sync();
            l = __fadd_rn(lo_of(sum), hi_of(sum));
        }
        // By way of shared memory, 32 channels at a time, so that a warp writes 128 bytes of a row side by side (a row
        // per lane took 9 us): the row tile's queries are not needed any more.  Pieces of 16 bytes, in places that a
        // row's number permutes.
        unsigned char* stage = sm + S::kQ + t * S::kQB + (warp & 3) * (32 * 128);
        float* part = A.part + ((o * a.rows + (r - lane)) * A.nsplit + split) * (C + 4);     // of the warp's first row
        const int64_t pitch = (int64_t)A.nsplit * (C + 4);
        const int rows = ok ? min(32, a.rows - (r - lane)) : 0;              // that exist
#pragma unroll 1
        for (int i = 0; i < C / 32; ++i) {
            uint32_t y[32];
            if (ok && n > 0) {
                tc::ld32(o_at + 32 * i, y);
                tc::wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = 0u;
            }
            __syncwarp();                        // the piece before has been read
#pragma unroll
            for (int e = 0; e < 4; ++e) {        // channels 0 .. 7 sit in columns 0 2 4 6 1 3 5 7
                const uint32_t* z = y + 8 * e;
                *reinterpret_cast<uint4*>(stage + lane * 128 + ((2 * e) ^ (lane & 7)) * 16) = make_uint4(z[0], z[2], z[4], z[6]);
                *reinterpret_cast<uint4*>(stage + lane * 128 + ((2 * e + 1) ^ (lane & 7)) * 16) = make_uint4(z[1], z[3], z[5], z[7]);
            }
            __syncwarp();
#pragma unroll 4
            for (int e = 0; e < 8; ++e) {        // four rows at a time
                const int row = 4 * e + lane / 8, p = lane & 7;
                if (row < rows)
                    *reinterpret_cast<uint4*>(part + row * pitch + 32 * i + 4 * p) =
                        *reinterpret_cast<const uint4*>(stage + row * 128 + (p ^ (row & 7)) * 16);
            }
        }
        if (lane < rows) *reinterpret_cast<float2*>(part + lane * pitch + C) = make_float2(m, l);
    }
    __syncwarp();
    tc::before_sync();
    __syncthreads();
    cluster_sync();                              // nobody leaves, or reads what the other noted, before both are done
    tc::after_sync();
    if (warp == 8) dealloc_pair(tmem, 512);
    // values that are not finite, noted by the CTA that has their channels: every row sees them
    uint32_t noted[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(noted[h]) : "r"(at_rank(&odd[2 * C], h)) : "memory");
    if ((noted[0] | noted[1]) != 0u && !*gone) {
        for (int i = tid; i < nt * kTile; i += kThreads) {
            const int r = r0 + (i / kTile) * 256 + rank * kTile + i % kTile;
            if (r >= a.rows) continue;
            float* part = A.part + ((o * a.rows + r) * A.nsplit + split) * (C + 4);
#pragma unroll 1
            for (int ch = 0; ch < C; ++ch) {
                uint32_t up, dn;
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(up) : "r"(at_rank(&odd[ch], ch / 64)) : "memory");
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(dn) : "r"(at_rank(&odd[C + ch], ch / 64)) : "memory");
                const float x = __fadd_rn(up != (uint32_t)kNever ? INFINITY : 0.0f, dn != (uint32_t)kNever ? -INFINITY : 0.0f);
                if (x != 0.0f) part[ch] = __fadd_rn(part[ch], x);
            }
        }
    }
    cluster_sync();                              // the other has read what this one noted
    asm volatile("griddepcontrol.wait;" ::: "memory");              // so that what follows this launch follows the one before, too
}

constexpr int64_t kPairs = 76;                   // of SMs
constexpr int64_t kMaxPairs = 4 * kPairs;        // of CTAs with splits: bounds the partial results

// Splits of the key tiles: the shortest way through all waves, in key tiles, with about six for a pair's start and end.
int64_t splits_of(int64_t tiles, int64_t keys)
{
    int64_t best = INT64_MAX, s = 1;
    for (int64_t k = 1; k == 1 || (k * 2 <= keys && tiles * k <= kMaxPairs); ++k) {
        const int64_t cost = (tiles * k + kPairs - 1) / kPairs * ((keys + k - 1) / k + 6) + k / 4;
        if (cost < best) {
            best = cost;
            s = k;
        }
    }
    return s;
}

template <int BITS>
cudaError_t launch(PrefixArgs X, int64_t outer, cudaStream_t st)
{
    const cudaError_t e = ensure_kernel_attrs(reinterpret_cast<const void*>(attend_prefix_kernel<BITS>), Smem<BITS>::kBytes);
    if (e != cudaSuccess) return e;
    const int64_t grid = 2 * outer * X.ntiles * X.A.nsplit;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {2, 1, 1};
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Smem<BITS>::kBytes;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = X.A.own_part ? 2 : 1;         // the launch before is the rows kernel of this call
    const cudaError_t l = cudaLaunchKernelEx(&cfg, attend_prefix_kernel<BITS>, X);
    return l != cudaSuccess ? l : cudaGetLastError();
}

}  // namespace

// Below, an SM's tensor memory holds the rows of a tile by itself; far above, one expansion costs less than unpacking for
// every 512 rows.  In us, pairs against the other forms (chunk.cu, prefill.cu), at 4 bits (2 bits alike):
//   rows                            64        128        160        256       2048       2560       3000       4096
//   8 slices of  1000 tokens   22 :  21   23 :  24   23 :  27   23 :  31   37 :  33   43 :  33   45 :  33   50 :  33
//   8 slices of  8192 tokens   25 :  24   27 :  27   27 :  31   28 :  35   76 :  87  107 : 128  114 : 130  133 : 112
//   8 slices of 32768 tokens   52 :  49   53 :  52   53 :  62   53 :  65  228 : 264  301 : 332  312 : 325  435 : 395
//   2 slices of 65536 tokens   36 :  36   36 :  39   37 :  44   37 :  48  110 : 129  136 : 151  158 : 167  214 : 226
// So the upper end is too low for long prefixes and too high for one of 1000 tokens, where pairs pay up to 1024 rows (30 : 33);
// the rule does not look at the prefix's length.
bool prefix_uses_pairs(int64_t dim, int64_t rows) { return dim == C && rows > 128 && rows <= 2048; }

size_t prefix_workspace(int64_t outer, int64_t tmax, int64_t rows)
{
    const int64_t tiles = outer * ((rows + 511) / 512), keys = std::max<int64_t>((tmax + kTile - 1) / kTile, 1);
    const int64_t pairs = std::max(tiles, std::min(kMaxPairs, tiles * std::max<int64_t>(keys / 2, 1)));
    return (size_t)(pairs * std::min<int64_t>(rows, 512) * (C + 4)) * sizeof(float);
}

cudaError_t launch_attend_prefix(ChunkArgs A, int bits, int64_t outer, void* ws, cudaStream_t st)
{
    PrefixArgs X;
    X.ntiles = (A.v.rows + 511) / 512;
    A.part = static_cast<float*>(ws);
    A.nsplit = (int32_t)splits_of(outer * X.ntiles, (A.v.T + kTile - 1) / kTile);
    X.A = A;
    const cudaError_t e = bits == 4 ? launch<4>(X, outer, st) : launch<2>(X, outer, st);
    return e != cudaSuccess ? e : launch_merge_rows(A, C, outer, st);
}

}  // namespace kvq
