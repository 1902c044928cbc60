// prefill.cu -- causal attention of many query rows over the streaming
// quantized cache, on tcgen05 tensor cores (kvq_attend_chunk with enough rows).
//
// Method as in chunk.cu.  With R query rows per slice the products cost 4 R C
// operations a token while its codes are C bytes, so for hundreds of rows the
// tensor cores bound it, and unpacking each key and value once per 256 rows
// would compete with the softmax for issue slots.  So:
//  1. expand_kernel writes the cache's bf16 rows, K^ and V^ [slice][Tp][C] (Tp =
//     T rounded up to 128), once; hidden and missing tokens become zeros, so
//     whatever lies there (NaN) never reaches a product;
//  2. attend_tc_kernel, a CTA per (slice, 256 rows, split of the key tiles):
//     two M = 128 tiles of query rows share every 128-token key and value tile.
//     Warp 8 loads tiles by TMA into a ring; warps 9 and 10 issue the products of
//     a row tile each (one warp for both left the tensor cores idle at every
//     wait: 1.85 ms for the chunk below); warps 0-3 and 4-7 are the softmax of the two row tiles, a
//     thread per row: S (128 float32 columns of tensor memory) -> registers ->
//     P in bf16 over the same columns, which the value product reads as its A
//     operand from tensor memory.  While one tile is in its softmax the tensor
//     cores work on the other.
//     The running maximum is moved (and the output in tensor memory rescaled)
//     only when it grows by more than 2^8: until then the weights are at most
//     256, which costs float32 sums and bf16 weights no relative precision.
//
// Measured on one GB300: 4096 queries x 4 heads over 32768 tokens and 8 slices 1.32
// ms (1.56 PFLOP/s); the expansion takes 40 us of it.  attend_tc_kernel has the tensor
// cores busy 72 % of its cycles, the issue slots 38 %.
// The weights enter the value product as one bf16 (its operands are of one type): hi +
// lo would be half as many products again where they are most of the time, for an
// error of 2^-8 of each weight at most, the size of out's own rounding.
#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kvq_chunk.cuh"
#include "kvq_fill.cuh"

namespace kvq {

namespace {

using namespace rows;
using fill::kTile;                               // 128 tokens of a key tile, 128 rows of a query tile
using fill::Staged;
using fill::interleave;

constexpr int kSlots = 4;                        // ring slots of one K or V tile
constexpr int kThreadsTc = 384;                 // 12 warps, 168 registers each at launch (64512 in all):
constexpr int kRegsSoftmax = 216;                // 8 softmax warps take 216 and the other four keep 56
constexpr int kRegsOther = 56;                   // (62464), so a row of 128 scores stays in registers
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreadsTc * 168, "registers of the launch");
constexpr float kSlack = 8.0f;                   // base-2 growth of the maximum that is let pass

// ---------------------------------------------------------------- expansion
// A thread takes one piece of 8 channels of 8 consecutive tokens: of K (its
// group's scales and zero points read once) or of V.  odd[slice][Tp / 8] says which
// 8 tokens hold values that are not finite; those become 0.
template <int BITS, int C>
__global__ void __launch_bounds__(256)
expand_kernel(const View a, int64_t o0, int64_t slices, int64_t Tp, __nv_bfloat16* kx, __nv_bfloat16* vx, uint8_t* odd)
{
    using W = typename CodeWord<BITS>::T;
    constexpr int P = C / 8;
    const int64_t oct = Tp / 8, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= slices * oct * P) return;
    const bool keys = blockIdx.y == 0;
    const int p = (int)(id % P);
    const int64_t so = id / P / oct;
    const int t0 = (int)(id / P - so * oct) * 8;
    const int64_t o = o0 + so;
    const int first = a.first ? a.first[o] : 0;
    const uint8_t* codes = keys ? a.kc : a.vc;
    const __nv_bfloat16* sc = keys ? a.ks : a.vs;
    const __nv_bfloat16* ze = keys ? a.kz : a.vz;
    const float off = (keys ? a.kbias : a.vbias) - 128.0f;
    const uint32_t flip = keys ? a.kflip : a.vflip;
    __nv_bfloat16* dst = (keys ? kx : vx) + (so * Tp + t0) * C + p * 8;
    float s[8], z[8];
    bool bad = false;
    if (keys && t0 < a.tq) {
        const int64_t at = (o * a.ngk + t0 / a.gk) * C + p * 8;     // 8 tokens lie in one group
        Raw8<__nv_bfloat16> r;
        load_raw8(sc + at, r);
        widen8(r, s);
        if (ze) {
            load_raw8(ze + at, r);
            widen8(r, z);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int t = t0 + i;
        uint4 x = make_uint4(0, 0, 0, 0);
        bool look = false;                       // values that may not be finite
        if (t >= first && t < a.T) {
            if (t >= a.tq) {
                look = !keys;
                x = *reinterpret_cast<const uint4*>((keys ? a.kr : a.vr) + ((uint64_t)o * a.rrows + (t - a.tq)) * C + p * 8);
            } else {
                if (!keys) {
                    const int64_t at = (o * a.cap + t) * a.ngv + p * 8 / a.gv;
                    const float sv = __bfloat162float(sc[at]), zv = ze ? __bfloat162float(ze[at]) : 0.0f;
                    look = may_be_odd(sv, zv);
#pragma unroll
                    for (int k = 0; k < 8; ++k) { s[k] = sv; z[k] = zv; }
                }
                W w = *reinterpret_cast<const W*>(codes + ((uint64_t)o * a.cap + t) * (C * BITS / 8) + p * BITS);
                w ^= (W)flip;
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float c = __fsub_rn((float)((w >> (BITS * k)) & ((1 << BITS) - 1)), off);
                    v[k] = __fmul_rn(ze ? __fsub_rn(c, z[k]) : c, s[k]);
                }
                store8(reinterpret_cast<__nv_bfloat16*>(&x), v);
            }
        }
        if (look && is_odd(x)) {
            bad = true;
            x = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
        }
        *reinterpret_cast<uint4*>(dst + (int64_t)i * C) = x;
    }
    if (!keys) {                                 // whole warps are here: Tp / 8 P is a multiple of 128
        const uint32_t any = __ballot_sync(0xFFFFFFFFu, bad) >> (threadIdx.x & 31 & ~(P - 1)) & ((1u << P) - 1);
        if (p == 0) odd[id / P] = any ? 1 : 0;
    }
}

// ---------------------------------------------------------------- attention
template <int C>
struct Smem {
    static constexpr int kTileB = kTile * C * 2; // one Q, K or V tile
    static constexpr int kQ = 0, kRing = 2 * kTileB, kBars = kRing + kSlots * kTileB, kOdd = kBars + 256;
    static constexpr int kSums = kOdd + (2 * C + 4) * 4, kBytes = kSums + 2 * kTile * 4 + 1024;    // and room to align to 1024
};

struct TcArgs {
    ChunkArgs A;                                 // nsplit: of the split tiles
    int64_t o0, slices, Tp;
    int32_t nwhole;                              // query tiles taken whole; the others are split
    int32_t trows;                               // rows of a tile that partial results are kept for
    int32_t bits;
    const uint8_t* odd;                          // [slices][Tp / 8], as expand_kernel writes it
};

// The query tile and split of a CTA.
struct TileOf {
    int tile, split, nsplit, r0, nrows, nt;      // tile of up to 256 rows from r0; nt row tiles of 128 in use
    int64_t so, o;                               // slice of this launch, slice
    __device__ __forceinline__ explicit TileOf(const TcArgs& X) {
        tile = blockIdx.x;                       // the longest of a slice first
        split = 0;
        nsplit = 1;
        if (tile >= X.nwhole) {
            nsplit = X.A.nsplit;
            split = (tile - X.nwhole) % nsplit;
            tile = X.nwhole + (tile - X.nwhole) / nsplit;
        }
        so = tile / X.A.ntiles;
        o = X.o0 + so;
        r0 = (X.A.ntiles - 1 - tile % X.A.ntiles) * 2 * kTile;
        nrows = min(2 * kTile, X.A.v.rows - r0);
        nt = nrows > kTile ? 2 : 1;
    }
    // the key tiles [j0, j0 + n) it sees; returns the first token that is not padding
    __device__ __forceinline__ int keys(const TcArgs& X, int& j0, int& n) const {
        const View& a = X.A.v;
        const int first = padding(a, o);
        const int last_hi = a.T - a.n + (r0 + nrows - 1) / a.group;
        int j1 = 0;
        j0 = 0;
        if (first <= last_hi) {
            j0 = first / kTile;
            j1 = last_hi / kTile + 1;
        }
        const int64_t len = j1 - j0;
        n = (int)(len * (split + 1) / nsplit) - (int)(len * split / nsplit);
        j0 += (int)(len * split / nsplit);
        return first;
    }
    // where row r's sums go, nullptr: out and lse are written; at: its row_index
    template <bool JOIN>
    __device__ __forceinline__ float* sums_of(const TcArgs& X, int r, int64_t at, int C) const {
        if (JOIN ? tile >= X.nwhole : nsplit > 1) return X.A.part + (((int64_t)(tile - X.nwhole) * X.trows + (r - r0)) * nsplit + split) * (C + 4);
        return JOIN && X.A.sums ? X.A.sums + at * (C + 4) : nullptr;
    }
};

// Adds the values that are not finite to the rows that the CTA has written: a thread
// per row, after everything else (in the softmax warps' epilogue it cost the fused
// form 6 us of 93).  sums: the rows' sums of weights.
template <int C, bool JOIN>
__device__ __noinline__ void add_odd(const TcArgs& X, const TileOf& w, const int* odd, const float* sums, int tid, int threads) {
    const View& a = X.A.v;
    for (int i = tid; i < w.nrows; i += threads) {
        const int r = w.r0 + i, last = a.T - a.n + r / a.group;
        const int64_t at = row_index<JOIN>(a, w.o, r);
        float* part = w.sums_of<JOIN>(X, r, at, C);
        __nv_bfloat16* out = X.A.out + at * C;
#pragma unroll 1
        for (int c = 0; c < C; ++c) {
            const float x = odd_value(odd, C, c, last);
            if (x == 0.0f) continue;
            if (part) part[c] = __fadd_rn(part[c], x);
            else if (sums[i] != 0.0f) out[c] = __float2bfloat16(__fadd_rn(__bfloat162float(out[c]), x));
        }
    }
}

template <int C, bool JOIN>
__global__ void __launch_bounds__(kThreadsTc, 1)
attend_tc_kernel(const TcArgs X, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using S = Smem<C>;
    constexpr int kHalves = C / 64;              // 64-channel halves of a tile, 16 KB each
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::kBars);
    uint64_t* empty = full + kSlots;
    uint64_t* sfull = empty + kSlots;            // [2] scores of a row tile are in tensor memory
    uint64_t* pfull = sfull + 2;                 // [2] its weights are
    uint64_t* odone = pfull + 2;                 // [2] its output is complete
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(odone + 2);
    volatile int* gone = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* odd = reinterpret_cast<int*>(sm + S::kOdd);               // [2 C], and whether any is noted
    float* sums = reinterpret_cast<float*>(sm + S::kSums);         // [256] the rows' sums of weights

    const ChunkArgs& A = X.A;
    const View& a = A.v;
    // the shuffle tells the compiler that a warp's number is uniform: the products' operands then are, too (the chunk
    // above 1.40 -> 1.32 ms)
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const TileOf w(X);
    const int64_t so = w.so, o = w.o;
    const int r0 = w.r0, nrows = w.nrows, nt = w.nt, base = a.T - a.n;
    int j0, n;
    const int first = w.keys(X, j0, n), j1 = j0 + n;

    // ---- setup: barriers, tensor memory, the query rows
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], nt);            // every row tile is done with it
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);
            mbar_init(&odone[i], 1);
        }
        *gone = 0;
        mbar_init_fence();
    }
    if (warp == 9) tc::alloc(tmem_slot, 512);
    for (int k = tid; k < nt * kTile * (C / 8); k += kThreadsTc) {
        const int r = k / (C / 8), c = k % (C / 8);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < nrows) x = *reinterpret_cast<const uint4*>(a.q + row_index<JOIN>(a, o, r0 + r) * C + c * 8);
        *reinterpret_cast<uint4*>(sm + S::kQ + (r / kTile) * S::kTileB + (c / 8) * (kTile * 128) +
                                  tc::swizzled(r % kTile, c % 8)) = x;
    }
    // a key tile's flags are 16 bytes; what they point to is looked up in the cache itself
    const uint4* flags = reinterpret_cast<const uint4*>(X.odd + so * (X.Tp / 8)) + j0;
    uint32_t mine = 0;
    for (int j = tid; j < n; j += kThreadsTc) {
        const uint4 f = flags[j];
        mine |= f.x | f.y | f.z | f.w;
    }
    for (int c = tid; c < 2 * C; c += kThreadsTc) odd[c] = kNever;
    tc::async_fence();
    tc::before_sync();
    const bool any_odd = __syncthreads_or(mine != 0);
    tc::after_sync();
    const uint32_t tmem = *tmem_slot;
    if (tid == 0) odd[2 * C] = any_odd;
    if (any_odd) {
        for (int t = tid; t < n * kTile; t += kThreadsTc) {
            const int tok = j0 * kTile + t;
            if (reinterpret_cast<const uint8_t*>(flags)[t / 8] == 0 || tok < first || tok >= a.T) continue;
            if (X.bits == 4) note_row<4, C>(a, o, tok, odd);
            else note_row<2, C>(a, o, tok, odd);
        }
        __syncthreads();
    }

    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) {
        // ---- tiles by TMA, in the order the products take them: K0, K1, V0, K2, V1, ...
        int it = 0;
        auto load = [&](const CUtensorMap* map, int j) {
            const int s = it % kSlots;
            if (it >= kSlots && !__all_sync(0xFFFFFFFFu, tc::wait(&empty[s], ((it / kSlots) - 1) & 1, gone))) return false;
            if (tc::elect()) {
                mbar_expect_tx(&full[s], S::kTileB);
                for (int h = 0; h < kHalves; ++h)
                    tma_load_2d(sm + S::kRing + s * S::kTileB + h * (kTile * 128), map, h * 64,
                                (int)(so * X.Tp) + j * kTile, &full[s]);
            }
            __syncwarp();
            ++it;
            return true;
        };
        if (n > 0) {
            bool ok = load(&kmap, j0);
            for (int j = j0; ok && j < j1; ++j) {
                if (j + 1 < j1) ok = load(&kmap, j + 1);
                ok = ok && load(&vmap, j);
            }
        }
        // every copy issued lands before the CTA's shared memory goes
        for (int i = max(0, it - kSlots); i < it; ++i) tc::drain(&full[i % kSlots], (i / kSlots) & 1);
    } else if (warp <= 8 + nt && n > 0) {
        // ---- products of row tile t
        const int t = warp - 9;
        constexpr uint32_t kScores = tc::instr_desc(kTile, kTile, false), kValues = tc::instr_desc(kTile, C, true);
        const uint32_t q_at = smem_u32(sm + S::kQ) + t * S::kTileB, ring = smem_u32(sm + S::kRing);
        const uint32_t s_at = tmem + t * kTile, o_at = tmem + 256 + t * C;
        auto scores = [&](int s) {
#pragma unroll
            for (int k = 0; k < C / 16; ++k) {
                const uint32_t at = (k / 4) * (kTile * 128) + (k % 4) * 32;
                tc::mma_ss(s_at, tc::smem_desc(q_at + at, 16), tc::smem_desc(ring + s * S::kTileB + at, 16), kScores, k > 0);
            }
            tc::commit(&sfull[t]);
        };
        auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, tc::wait(bar, parity, gone)) != 0; };
        int it = 0;
        bool ok = ready(&full[0], 0);
        if (ok && tc::elect()) {
            scores(0);
            tc::commit(&empty[0]);
        }
        __syncwarp();
        ++it;
        for (int j = 0; ok && j < n; ++j) {
            int ks = -1;
            if (j + 1 < n) {
                ks = it % kSlots;
                ok = ready(&full[ks], (it / kSlots) & 1);
                ++it;
            }
            const int vs = it % kSlots;
            ok = ok && ready(&full[vs], (it / kSlots) & 1) && ready(&pfull[t], j & 1);
            ++it;
            if (!ok) break;
            tc::after_sync();
            if (tc::elect()) {
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    tc::mma_ts(o_at, s_at + k * 8, tc::smem_desc(ring + vs * S::kTileB + k * 2048, kTile * 128), kValues,
                               j > 0 || k > 0);
                if (ks >= 0) {
                    scores(ks);
                    tc::commit(&empty[vs]);
                    tc::commit(&empty[ks]);
                } else {
                    tc::commit(&empty[vs]);
                    tc::commit(&odone[t]);
                }
            }
            __syncwarp();
        }
    }
    } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    if (warp < 4 * nt) {
        // ---- softmax of row tile t, a thread per row
        const int t = warp / 4;
        const int r = r0 + t * kTile + (warp & 3) * 32 + lane;
        const int last = r < a.rows ? base + r / a.group : a.T;     // rows past the last are not written
        const int tile_lo = base + (r0 + t * kTile) / a.group;      // the fewest tokens a row of the tile sees
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + t * kTile, o_at = tmem + lanes + 256 + t * C;
        float m = -INFINITY;
        u64 sum = 0;
        bool ok = true;
        for (int j = 0; ok && j < n; ++j) {
            ok = tc::wait(&sfull[t], j & 1, gone);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc::after_sync();
            uint32_t s[kTile];
#pragma unroll
            for (int c = 0; c < 4; ++c) tc::ld32(s_at + 32 * c, s + 32 * c);
            tc::wait_ld();
            const int c0 = (j0 + j) * kTile;
            if (c0 < first || c0 + kTile - 1 > tile_lo) {
#pragma unroll
                for (int c = 0; c < kTile; ++c)
                    if (c0 + c < first || c0 + c > last) s[c] = 0xFF800000u;         // -inf
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
            const bool grow = top > __fadd_rn(m, kSlack);           // m = -inf: whenever anything is seen
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
            for (int h = 0; h < 2; ++h) {        // 64 scores -> 32 columns of weight pairs
                uint32_t p[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int c = 64 * h + 2 * i;
                    const u64 e = fma2(pk(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, ng2);
                    const float e0 = ex2(lo_of(e)), e1 = ex2(hi_of(e));
                    sum = add2(sum, pk(e0, e1));
                    p[i] = pack_bf16x2(e0, e1);
                }
                tc::st32(s_at + 32 * h, p);
            }
            tc::wait_st();
            tc::before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[t]);
        }
        // ---- output
        float l = 0.0f;
        if (ok && n > 0) {
            ok = __all_sync(0xFFFFFFFFu, tc::wait(&odone[t], 0, gone));
            tc::after_sync();
            l = __fadd_rn(lo_of(sum), hi_of(sum));
        }
        const bool write = ok && r < a.rows;
        const int64_t at = write ? row_index<JOIN>(a, o, r) : 0;
        float* part = w.sums_of<JOIN>(X, r, at, C);
        // a whole tile of a launch to be joined: what the row has seen elsewhere is added here
        float fm = 1.0f, fo = 0.0f;
        const float* own_sums = nullptr;
        const __nv_bfloat16* own_out = nullptr;
        if constexpr (JOIN) {
            if (write && !part && A.shared) {
                float mo = -INFINITY, lo = 0.0f;
                if (A.own_sums) {
                    own_sums = A.own_sums + at * (C + 4);
                    mo = own_sums[C];
                    lo = own_sums[C + 1];
                } else if (A.own_lse) {
                    const float z = A.own_lse[at];
                    if (z != -INFINITY) {
                        own_out = A.own_out + at * C;
                        mo = __fmul_rn(z, kLog2e);
                        lo = z != z ? z : 1.0f;
                    }
                }
                const float M = fmaxf(m, mo);
                fm = part_scale(m, M);
                fo = part_scale(mo, M);
                l = __fmaf_rn(l, fm, __fmul_rn(lo, fo));
                m = M;
            }
        }
        const float inv = row_scale(l);
#pragma unroll
        for (int c = 0; c < C / 32; ++c) {
            uint32_t y[32];
            if (ok && n > 0) {
                tc::ld32(o_at + 32 * c, y);
                tc::wait_ld();
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = 0u;
            }
            if constexpr (JOIN) {
                if (own_sums) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 x = *reinterpret_cast<const float4*>(own_sums + 32 * c + 4 * i);
                        const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            y[4 * i + k] = __float_as_uint(__fmaf_rn(__uint_as_float(y[4 * i + k]), fm, __fmul_rn(v[k], fo)));
                    }
                } else if (own_out) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4*>(own_out + 32 * c + 8 * i);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t* z = y + 8 * i + 2 * k;
                            z[0] = __float_as_uint(__fmaf_rn(__uint_as_float(z[0]), fm, __fmul_rn(bf_lo(w[k]), fo)));
                            z[1] = __float_as_uint(__fmaf_rn(__uint_as_float(z[1]), fm, __fmul_rn(bf_hi(w[k]), fo)));
                        }
                    }
                }
            }
            if (write && part) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(part + 32 * c + 4 * i) = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            } else if (write) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = pack_bf16x2(row_value(__uint_as_float(y[8 * i + 2 * k]), inv),
                                           row_value(__uint_as_float(y[8 * i + 2 * k + 1]), inv));
                    *reinterpret_cast<uint4*>(A.out + at * C + 32 * c + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            __syncwarp();                        // the next load wants the whole warp
        }
        if (write) sums[r - r0] = l;
        if (write && part) *reinterpret_cast<float2*>(part + C) = make_float2(m, l);
        if (write && !part && A.lse)
            A.lse[at] = row_lse(m, l);
    }
    }
    __syncwarp();
    tc::before_sync();
    __syncthreads();
    tc::after_sync();
    if (warp == 9) tc::dealloc(tmem, 512);
    if (odd[2 * C] && !*gone) add_odd<C, JOIN>(X, w, odd, sums, tid, kThreadsTc);
}

// ---------------------------------------------------------------- fused form
// The same without the expansion, for fewer query rows: sixteen fill warps turn
// the packed codes into the swizzled bf16 tiles themselves (warps 12-19 the
// keys, 20-27 the values), so the cache is read once, as codes.  Per 128-token
// tile that is 32768 values, four instructions a pair: about as long as the
// products of 256 rows take, so more rows are better served by expanding once.
// Within every 8 channels the tiles hold them in the order 0 4 1 5 2 6 3 7 in
// which a code word gives them up; the query rows are staged, and the output is
// written, accordingly.  With 896 threads a softmax thread has 72 registers and
// reads its 128 scores twice, 32 at a time.
constexpr int kFusedWarps = 28;
constexpr int kFusedThreads = kFusedWarps * 32;

template <int BITS, int C>
struct SmemF {
    static constexpr int kTileB = kTile * C * 2;
    static constexpr int kQ = 0, kK = 2 * kTileB, kV = kK + 2 * kTileB, kRawK = kV + 2 * kTileB;    // two K, two V tiles,
    static constexpr int kRawV = kRawK + Staged<BITS, C, true>::kBytes;                 // and their staged codes
    static constexpr int kBars = kRawV + Staged<BITS, C, false>::kBytes, kOdd = kRawV + Staged<BITS, C, false>::kOddAt;
    static_assert(kOdd == kBars + 256, "behind the barriers");
    static constexpr int kSums = kOdd + (2 * C + 4) * 4, kBytes = kSums + 2 * kTile * 4 + 1024;
};

template <int BITS, int C, bool JOIN>
__global__ void __launch_bounds__(kFusedThreads, 1)
attend_fused_kernel(const __grid_constant__ TcArgs X)
{
    using S = SmemF<BITS, C>;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + S::kBars);  // [2] a key tile is in shared memory (8 warps)
    uint64_t* kfree = kfull + 2;                 // [2] every row tile is done with it
    uint64_t* vfull = kfree + 2;
    uint64_t* vfree = vfull + 2;
    uint64_t* sfull = vfree + 2;                 // [2] per row tile, as in attend_tc_kernel
    uint64_t* pfull = sfull + 2;
    uint64_t* odone = pfull + 2;
    uint64_t* raw_bars = odone + 2;              // [K full, K free, V full, V free][3]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(raw_bars + 12);
    volatile int* gone = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* odd = reinterpret_cast<int*>(sm + S::kOdd);               // [2 C], and whether any is noted
    float* sums = reinterpret_cast<float*>(sm + S::kSums);         // [256] the rows' sums of weights

    const ChunkArgs& A = X.A;
    const View& a = A.v;
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const TileOf w(X);
    const int64_t o = w.o;
    const int r0 = w.r0, nrows = w.nrows, nt = w.nt, base = a.T - a.n;
    int j0, n;
    const int first = w.keys(X, j0, n);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&kfull[i], 8);
            mbar_init(&kfree[i], nt);
            mbar_init(&vfull[i], 8);
            mbar_init(&vfree[i], nt);
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);
            mbar_init(&odone[i], 1);
        }
        for (int i = 0; i < 12; ++i) mbar_init(&raw_bars[i], i / 3 % 2 ? 4 : 1);
        *gone = 0;
        mbar_init_fence();
    }
    if (warp == 8) tc::alloc(tmem_slot, 512);
    for (int c = tid; c <= 2 * C; c += kFusedThreads) odd[c] = c < 2 * C ? kNever : 0;
    if (warp < 12)
        for (int k = tid; k < nt * kTile * (C / 8); k += 384) {
            const int r = k / (C / 8), c = k % (C / 8);
            uint4 x = make_uint4(0, 0, 0, 0);
            if (r < nrows) x = interleave(*reinterpret_cast<const uint4*>(a.q + row_index<JOIN>(a, o, r0 + r) * C + c * 8));
            *reinterpret_cast<uint4*>(sm + S::kQ + (r / kTile) * S::kTileB + (c / 8) * (kTile * 128) +
                                      tc::swizzled(r % kTile, c % 8)) = x;
        }
    tc::async_fence();
    tc::before_sync();
    __syncthreads();
    tc::after_sync();
    const uint32_t tmem = *tmem_slot;
    auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, tc::wait(bar, parity, gone)) != 0; };

    if (warp >= 10) {
        // ---- fill: warps 12-19 the keys, 20-27 the values; warps 10 and 11 copy their codes
        const int me = tid & 127, sub = ((warp - 12) >> 2) & 1;      // two groups of four warps each
        const bool keys = warp < 12 ? warp == 10 : warp < 20;
        auto role = [&](auto f, uint64_t* full, uint64_t* free, unsigned char* tiles) {
            if (warp < 12) {
                f.produce(ready);
                return;
            }
            f.run(j0, n, ready,
                  [&](int j) -> unsigned char* {
                      return j >= 2 && !ready(&free[j & 1], ((j >> 1) - 1) & 1) ? nullptr : tiles + (j & 1) * S::kTileB;
                  },
                  [&](int j) {
                      tc::async_fence();
                      __syncwarp();
                      if (lane == 0) mbar_arrive(&full[j & 1]);
                  });
        };
        if (keys) role(Staged<BITS, C, true>(a, o, first, j0, n, me, sub, sm + S::kRawK, raw_bars, raw_bars + 3), kfull, kfree, sm + S::kK);
        else role(Staged<BITS, C, false>(a, o, first, j0, n, me, sub, sm + S::kRawV, raw_bars + 6, raw_bars + 9), vfull, vfree, sm + S::kV);
    } else if (warp >= 8) {
        // ---- products of row tile t (warps 8 and 9)
        const int t = warp - 8;
        if (t < nt && n > 0) {
            constexpr uint32_t kScores = tc::instr_desc(kTile, kTile, false), kValues = tc::instr_desc(kTile, C, true);
            const uint32_t q_at = smem_u32(sm + S::kQ) + t * S::kTileB, k_at = smem_u32(sm + S::kK), v_at = smem_u32(sm + S::kV);
            const uint32_t s_at = tmem + t * kTile, o_at = tmem + 256 + t * C;
            auto scores = [&](int s) {
#pragma unroll
                for (int k = 0; k < C / 16; ++k) {
                    const uint32_t at = (k / 4) * (kTile * 128) + (k % 4) * 32;
                    tc::mma_ss(s_at, tc::smem_desc(q_at + at, 16), tc::smem_desc(k_at + s * S::kTileB + at, 16), kScores, k > 0);
                }
                tc::commit(&sfull[t]);
                tc::commit(&kfree[s]);
            };
            bool ok = ready(&kfull[0], 0);
            tc::after_sync();
            if (ok && tc::elect()) scores(0);
            __syncwarp();
            for (int j = 0; ok && j < n; ++j) {
                const int s = j & 1;
                if (j + 1 < n) ok = ready(&kfull[s ^ 1], ((j + 1) >> 1) & 1);
                ok = ok && ready(&vfull[s], (j >> 1) & 1) && ready(&pfull[t], j & 1);
                if (!ok) break;
                tc::after_sync();
                if (tc::elect()) {
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        tc::mma_ts(o_at, s_at + k * 8, tc::smem_desc(v_at + s * S::kTileB + k * 2048, kTile * 128), kValues,
                                   j > 0 || k > 0);
                    tc::commit(&vfree[s]);
                    if (j + 1 < n) scores(s ^ 1);
                    else tc::commit(&odone[t]);
                }
                __syncwarp();
            }
        }
    } else if (warp < 4 * nt) {
        // ---- softmax of row tile t, a thread per row
        const int t = warp / 4;
        const int r = r0 + t * kTile + (warp & 3) * 32 + lane;
        const int last = r < a.rows ? base + r / a.group : a.T;
        const int tile_lo = base + (r0 + t * kTile) / a.group;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + t * kTile, o_at = tmem + lanes + 256 + t * C;
        float m = -INFINITY;
        u64 sum = 0;
        bool ok = true;
        for (int j = 0; ok && j < n; ++j) {
            ok = ready(&sfull[t], j & 1);
            if (!ok) break;
            tc::after_sync();
            const int c0 = (j0 + j) * kTile;
            const bool cut = c0 < first || c0 + kTile - 1 > tile_lo;
            // tokens [lo, hi] of the tile are seen
            const int lo = first - c0, hi = last - c0;
            float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
                uint32_t s[32];
                tc::ld32(s_at + 32 * h, s);
                tc::wait_ld();
                if (cut) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (32 * h + c < lo || 32 * h + c > hi) s[c] = 0xFF800000u;  // -inf
                }
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    x0 = fmaxf(x0, __uint_as_float(s[c]));
                    x1 = fmaxf(x1, __uint_as_float(s[c + 1]));
                }
            }
            const float top = __fmul_rn(fmaxf(x0, x1), a.scale2);
            const bool grow = top > __fadd_rn(m, kSlack);
            if (__any_sync(0xFFFFFFFFu, grow)) {
                const float f = grow ? ex2(__fsub_rn(m, top)) : 1.0f;
                if (grow) m = top;
                sum = mul2(sum, pk(f, f));
                if (j > 0) {
#pragma unroll 1
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
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {        // 32 scores -> 16 columns of weight pairs, over scores read already
                uint32_t s[32], p[16];
                tc::ld32(s_at + 32 * h, s);
                tc::wait_ld();
                if (cut) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (32 * h + c < lo || 32 * h + c > hi) s[c] = 0xFF800000u;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const u64 e = fma2(pk(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sc2, ng2);
                    const float e0 = ex2(lo_of(e)), e1 = ex2(hi_of(e));
                    sum = add2(sum, pk(e0, e1));
                    p[i] = pack_bf16x2(e0, e1);
                }
                tc::st16(s_at + 16 * h, p);
            }
            tc::wait_st();
            tc::before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[t]);
        }
        // ---- output
        float l = 0.0f;
        if (ok && n > 0) {
            ok = ready(&odone[t], 0);
            tc::after_sync();
            l = __fadd_rn(lo_of(sum), hi_of(sum));
        }
        const bool write = ok && r < a.rows;
        const int64_t at = write ? row_index<JOIN>(a, o, r) : 0;
        float* part = w.sums_of<JOIN>(X, r, at, C);
        const float inv = row_scale(l);
#pragma unroll
        for (int c = 0; c < C / 32; ++c) {
            uint32_t y[32];
            if (ok && n > 0) {
                tc::ld32(o_at + 32 * c, y);
                tc::wait_ld();
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = 0u;
            }
            if (write) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {    // channels 0 .. 7 sit in columns 0 2 4 6 1 3 5 7
                    const uint32_t* z = y + 8 * i;
                    if (part) {
                        *reinterpret_cast<uint4*>(part + 32 * c + 8 * i) = make_uint4(z[0], z[2], z[4], z[6]);
                        *reinterpret_cast<uint4*>(part + 32 * c + 8 * i + 4) = make_uint4(z[1], z[3], z[5], z[7]);
                    } else {
                        float v[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            v[k] = row_value(__uint_as_float(z[2 * k]), inv);
                            v[4 + k] = row_value(__uint_as_float(z[2 * k + 1]), inv);
                        }
                        store8(A.out + at * C + 32 * c + 8 * i, v);
                    }
                }
            }
            __syncwarp();
        }
        if (write) sums[r - r0] = l;
        if (write && part) *reinterpret_cast<float2*>(part + C) = make_float2(m, l);
        if (write && !part && A.lse)
            A.lse[at] = row_lse(m, l);
    }
    __syncwarp();
    tc::before_sync();
    __syncthreads();
    tc::after_sync();
    if (warp == 8) tc::dealloc(tmem, 512);
    if (odd[2 * C] && !*gone) add_odd<C, JOIN>(X, w, odd, sums, tid, kFusedThreads);
}

// One warp per row of the split query tiles joins their partial results.
template <int C, bool JOIN>
__global__ void __launch_bounds__(256)
merge_tiles_kernel(const TcArgs X, int64_t total)
{
    const ChunkArgs& A = X.A;
    const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (at >= total) return;
    const int tile = X.nwhole + (int)(at / X.trows);
    const int r = (A.ntiles - 1 - tile % A.ntiles) * 2 * kTile + (int)(at % X.trows);
    if (r < A.v.rows)
        merge_row<C, JOIN>(A, X.o0 + tile / A.ntiles, r, A.part + at * A.nsplit * (C + 4), threadIdx.x & 31);
}

constexpr int64_t kExpandBytes = int64_t(1) << 30;                  // expanded K and V held at once

// One query tile of up to 256 rows reads the codes itself; more rows share one
// expansion (64 slices of 32768 tokens: 256 rows 421 us fused, 630 expanded; 512
// rows 815 and 766).
bool fused_form(int64_t rows) { return rows <= 2 * kTile; }

struct TcPlan { int64_t Tp, slices, ntiles; };

TcPlan tc_plan(int64_t outer, int64_t C, int64_t T, int64_t rows)
{
    TcPlan p;
    p.Tp = (T + kTile - 1) / kTile * kTile;
    p.slices = std::max<int64_t>(1, std::min<int64_t>(outer, kExpandBytes / std::max<int64_t>(p.Tp * C * 4, 1)));
    p.ntiles = (rows + 2 * kTile - 1) / (2 * kTile);
    return p;
}

// One CTA fits on an SM.  Either every query tile is split into the same number
// of key ranges, or full waves of 152 tiles are taken whole and the rest is split
// over the 152 SMs (512 tiles: 3.37 waves end after 3.5 instead of 4, 1.58 -> 1.40
// ms); the cheaper one, in key tiles through all waves with about six for a
// CTA's start and end and eight for joining.
constexpr int64_t kSms = 152;
constexpr int64_t kMaxSplitCtas = 4 * kSms;      // CTAs of split tiles: bounds the partial results

struct Waves { int64_t whole, tail, nsplit; };

Waves waves_of(int64_t tiles, int64_t Tp, bool parts)
{
    const int64_t keys = Tp / kTile;
    Waves w = {parts ? 0 : tiles, parts ? tiles : 0, 1};            // parts: every tile's results are joined later
    int64_t best = (tiles + kSms - 1) / kSms * (keys + 6) + (parts ? 8 : 0);
    for (int64_t s = 2; s * 2 <= keys && tiles * s <= kMaxSplitCtas; ++s) {
        const int64_t cost = (tiles * s + kSms - 1) / kSms * ((keys + s - 1) / s + 6) + 8;
        if (cost < best) {
            best = cost;
            w = {0, tiles, s};
        }
    }
    const int64_t tail = tiles % kSms, s = tail ? std::min<int64_t>(kSms / tail, keys / 2) : 1;
    if (!parts && tiles > kSms && s > 1 && tiles / kSms * (keys + 6) + (keys + s - 1) / s + 14 < best) w = {tiles - tail, tail, s};
    return w;
}

template <int BITS, int C, bool JOIN>
cudaError_t launch_tc(const ChunkArgs& A0, int64_t outer, void* ws, cudaStream_t st)
{
    const bool fused = fused_form(A0.v.rows) || A0.v.T == 0;        // an empty cache has nothing to expand
    TcPlan p = tc_plan(outer, C, A0.v.T, A0.v.rows);
    if (fused) p.slices = outer;
    TcArgs X;
    X.A = A0;
    X.A.ntiles = (int32_t)p.ntiles;
    X.Tp = p.Tp;
    X.trows = (int32_t)std::min<int64_t>(A0.v.rows, 2 * kTile);
    __nv_bfloat16* kx = static_cast<__nv_bfloat16*>(ws);
    __nv_bfloat16* vx = kx + p.slices * p.Tp * C;
    X.bits = BITS;
    uint8_t* odd = reinterpret_cast<uint8_t*>(vx + p.slices * p.Tp * C);
    X.odd = odd;
    X.A.part = fused ? static_cast<float*>(ws) : reinterpret_cast<float*>(odd + p.slices * (p.Tp / 8));
    if ((!fused && p.slices * p.Tp > 0x7FFFFFFF) || p.slices * p.ntiles > 0x7FFFFFFF - kMaxSplitCtas)
        return cudaErrorInvalidConfiguration;
    CUtensorMap km, vm;
    if (!fused && (!encode_rows_tile_map(kx, p.slices * p.Tp, C, &km) || !encode_rows_tile_map(vx, p.slices * p.Tp, C, &vm)))
        return cudaErrorNotSupported;
    const cudaError_t e = fused
        ? ensure_kernel_attrs(reinterpret_cast<const void*>(attend_fused_kernel<BITS, C, JOIN>), (SmemF<BITS, C>::kBytes))
        : ensure_kernel_attrs(reinterpret_cast<const void*>(attend_tc_kernel<C, JOIN>), Smem<C>::kBytes);
    if (e != cudaSuccess) return e;
    for (int64_t o0 = 0; o0 < outer; o0 += p.slices) {
        X.o0 = o0;
        X.slices = std::min(p.slices, outer - o0);
        const Waves w = waves_of(X.slices * p.ntiles, p.Tp, X.A.shared && (fused || X.A.own_part));
        X.nwhole = (int32_t)w.whole;
        X.A.nsplit = (int32_t)w.nsplit;
        const unsigned grid = (unsigned)(w.whole + w.tail * w.nsplit);
        if (fused) {
            attend_fused_kernel<BITS, C, JOIN><<<grid, kFusedThreads, (SmemF<BITS, C>::kBytes), st>>>(X);
        } else {
            const int64_t items = X.slices * (p.Tp / 8) * (C / 8);
            expand_kernel<BITS, C><<<dim3((unsigned)((items + 255) / 256), 2), 256, 0, st>>>(X.A.v, o0, X.slices, p.Tp, kx, vx, odd);
            attend_tc_kernel<C, JOIN><<<grid, kThreadsTc, Smem<C>::kBytes, st>>>(X, km, vm);
        }
        if (w.tail) {
            const int64_t total = w.tail * X.trows;
            merge_tiles_kernel<C, JOIN><<<(unsigned)((total + 7) / 8), 256, 0, st>>>(X, total);
        }
    }
    return cudaGetLastError();
}

}  // namespace

// [rows, C] bf16 as boxes of 64 channels x 128 rows, 128-byte swizzle
bool encode_rows_tile_map(const void* x, int64_t rows, int64_t C, CUtensorMap* map)
{
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_fn());
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)C, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)C * 2};
    const cuuint32_t box[2] = {64, kTile};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(x), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows from which the tensor-core forms are taken (64 slices of 32768 tokens: 32
// rows 249 us on mma.sync and 311 here, 64 rows 506 and 313).
bool chunk_uses_tc(int64_t rows) { return rows > 32; }

// Enough for every T up to tmax: a shorter cache may take more slices at once,
// but never more than the bound on expanded bytes.
size_t chunk_tc_workspace(int64_t outer, int64_t C, int64_t tmax, int64_t rows, bool shared)
{
    const TcPlan p = tc_plan(outer, C, tmax, rows);
    size_t b = fused_form(rows) ? 0 : (size_t)std::min(outer * p.Tp * C * 4, std::max(kExpandBytes, p.Tp * C * 4));
    b += b / (32 * C);                           // a flag for 8 tokens
    const int64_t trows = std::min<int64_t>(rows, 2 * kTile), tiles = outer * p.ntiles;
    int64_t ctas = std::min(kMaxSplitCtas, tiles * std::max<int64_t>(p.Tp / kTile / 2, 1));
    if (shared) ctas = std::max(ctas, tiles);    // whole tiles leave their sums too
    b += (size_t)(ctas * trows * (C + 4)) * 4;
    return b;
}

template <bool JOIN>
static cudaError_t launch_any(const ChunkArgs& A, int bits, int64_t C, int64_t outer, void* ws, cudaStream_t st)
{
    if (bits == 4) return C == 128 ? launch_tc<4, 128, JOIN>(A, outer, ws, st) : launch_tc<4, 64, JOIN>(A, outer, ws, st);
    return C == 128 ? launch_tc<2, 128, JOIN>(A, outer, ws, st) : launch_tc<2, 64, JOIN>(A, outer, ws, st);
}

cudaError_t launch_attend_tc(const ChunkArgs& A, int bits, int64_t C, int64_t outer, void* ws, cudaStream_t st)
{
    return A.sums || A.shared ? launch_any<true>(A, bits, C, outer, ws, st) : launch_any<false>(A, bits, C, outer, ws, st);
}

}  // namespace kvq
