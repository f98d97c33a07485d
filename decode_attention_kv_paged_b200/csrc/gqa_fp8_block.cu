// gqa_fp8_block.cu -- decode attention over the block-scaled fp8 cache, the
// E4M3 codes fed to the tcgen05 tensor cores as they are.
//
//   o_r = sum_j w_rj V_j / sum_j w_rj,   w_rj = exp(scale q_r . K_j)
//
// With one scale per (block, head), K_j = ks c_j and V_j = vs e_j with the same
// ks, vs for 64 keys, so both products run on codes and the scales meet the
// scores and the weights in fp32, once per (key, row).
//
// Shapes.  A unit is one K/V head with up to NQ of the query rows that share
// it (group heads x q_len positions).  The keys are the wide side, so they
// take the M side of both products:
//     S^T [128 keys][rows]  = K [128][d] . Q^T        K as loaded (K-major)
//     O^T [d][rows]         = V^T [d][128] . P        V as loaded (MN-major)
// and the few query rows the N side, which costs least (an MMA of M = 128,
// K = 32 takes 47 cycles for any N <= 64, measured).  An operand of more bits
// against 8-bit codes is split into E4M3 columns, each the rounded remainder of
// those before it: x = a + b / 32 + c / 1024, a = RNE(x), b = RNE(32 (x - a)),
// c = RNE(1024 (x - a - b / 32)); each holds 4 significant bits.  For Q (8 bits,
// scaled by a power of two per row) two are exact down to 2^-22 of the row's
// largest value.  The weights are rounded to f16 (2^-11 of a weight), which
// three hold exactly down to 2^-14, and within 2^-28, of the tile's largest.
// (Two left 2^-8 of a weight, the one rounding that showed beside the output's:
// relative L2 1.8e-3 against 1.65e-3.)
//
// Softmax.  One thread per key; the largest score of each row comes from a
// warp reduction and an exchange between the four warps.  Two references, as
// the sum of the weights knows nothing of V scales: exponentials are taken
// relative to the block's own largest score.  With one factor a row they join
// the sum of weights, relative to the running largest score; with another they
// become the operand P, relative to the tile's largest (weight x V scale), not
// a running one: the E4M3 pieces then lose nothing to a key far ahead in
// another tile.  Both factors are at most 1 for any V scales, so that blocks
// 2^240 apart stand beside one another.  The tile's O^T is read from tensor
// memory and added to fp32 registers with the factor that brings it to its
// running reference; sums of weights stay in fp32 registers, per key lane,
// until the unit's end, where the two references meet.
//
// Roles (one CTA per SM, 16 warps): warp 0 loads tiles of two blocks by TMA
// (swizzled as the MMA reads them) into two rings, and writes a record of each
// tile (positions, flags, scales) that the others go by; warps 1 and 2 issue
// the two products; warp 3 prepares the next unit's queries; warps 4-7 and 8-11
// are the softmax, on even and odd tiles (a tile is one long chain of latencies
// for its four warps, so two are kept going) or, with 32 rows, on 16 rows each;
// warps 12-15 keep the output.  S is double-buffered, P and O^T four deep.
// Every wait is bounded, and tensor memory always freed.
//
// The work is split over all SMs by visible blocks (plan.cuh); a unit cut by a
// CTA boundary leaves fp32 partials, which a second kernel, waiting on the
// first by programmatic launch, joins: one CTA per cut, splits in order.
//
// What bounds it (device time; floor: codes once at the copy rate).  32 heads
// of their own, 8 x 32768 tokens, d = 128: 336 us, 0.98 of the copy rate, for
// the first 50 ms; a loop that goes on reaches the 1000 W cap, the SM clock
// falls from 1965 to 1690 MHz, and it takes 346 to 386 us on different devices.
// Up to 8 columns a tile of 128 keys costs its bytes (0.74 us at d = 128).
// With 32 columns it is the softmax, 1.44 us a tile whether 20 or 32 rows are
// used: both groups work on one tile, some 2900 cycles from one to the next.
// Beside the tiles a call takes 14 us with up to 8 columns, 18 with d = 256, 24
// with 32 (fits over lengths): the first K tile is there after 4.0 us (lengths,
// table and codes are loads that wait for one another), its weights after 6.0,
// then come the uneven ends of the CTAs and the second kernel (16 x 4096 tokens,
// 8 K/V heads: 34.7 us, floor 20.5).  The instruction cache mattered as much as
// anything: no warp's loop may be long, so records replace walks over the work
// list, and slow paths are out of line.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fp8_block.cuh"
#include "host_state.cuh"
#include "tc_common.cuh"

namespace attn {

constexpr int kFbThreads = 512;
constexpr int kFbMaxStages = 8;
constexpr int kFbWholeBlocks = 32;                    // see launch_gqa_fp8_block
constexpr int kFbTile = 2 * kBlockSize;               // keys of a tile

template <int D, int NQ>
struct FbCfg {
    static constexpr int kRowBytes = D == 64 ? 64 : 128;      // swizzle span
    static constexpr int kBoxes = D / kRowBytes;
    static constexpr int kHalves = D == 256 ? 2 : 1;          // M = 128 pieces of O^T
    static constexpr int kM = D == 64 ? 64 : 128;             // M of O^T
    static constexpr int kN = 2 * NQ;                         // columns of S: two pieces of Q
    // columns of P and O^T: three pieces, 16 at a time (M = 128 takes N so)
    static constexpr int kNP = NQ == 8 ? 32 : 3 * NQ;
    static constexpr int kBoxBytes = kFbTile * kRowBytes;     // one box of a tile
    static constexpr int kSlot = kFbTile * D;
    static constexpr int kQBytes = kN * D;
    static constexpr int kPBytes = kNP * kFbTile;
    // P and O^T buffers: four, so that the softmax seldom waits for the products
    // and the output of its earlier tiles, where tensor memory has the room.
    static constexpr int kOut = D == 256 && NQ == 32 ? 2 : 4;
    static constexpr int kFixed = 3 * kQBytes + kOut * kPBytes + 16 * 1024 + 1024 /*align*/;
    static constexpr int kSlots = (227 * 1024 - kFixed) / kSlot;
    static constexpr int kKStages = kSlots / 2 > kFbMaxStages ? kFbMaxStages : kSlots / 2;
    static constexpr int kVStages =
        kSlots - kKStages > kFbMaxStages ? kFbMaxStages : kSlots - kKStages;
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + kKStages * kSlot;
    static constexpr int kOffQ = kOffV + kVStages * kSlot;
    // the next unit's queries as they are in memory: [NQ][D] bf16
    static constexpr int kOffRaw = kOffQ + 2 * kQBytes;
    static constexpr int kOffP = kOffRaw + kQBytes;
    static constexpr int kOffBar = kOffP + kOut * kPBytes;
    static constexpr int kSmem = kOffBar + 16 * 1024 + 1024;
    static constexpr uint32_t kTmemS = 0, kTmemO = 2 * kN;
    static constexpr uint32_t kTmemUsed = 2 * kN + kOut * kHalves * kNP;
    static constexpr uint32_t kTmemCols =
        kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
    static_assert(kKStages >= 2 && kVStages >= 2, "at least two stages per ring");
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kTmemUsed <= 512, "tensor memory");
};

// A tile, as the load warp tells the others: first positions of its blocks,
// flags and the unit's running number, blocks of the CTA's range behind it.
struct __align__(16) FbTile {
    int pos[2], flags, left;
};
constexpr int kFbFirst = 1, kFbLast = 2, kFbLastPair = 4, kFbTwo = 8, kFbSegShift = 4;
// A unit's part: sequence, its length, the window its queries have (0: none),
// K/V head, query rows; whether the part is all of the unit.
struct __align__(16) FbPart {
    int b, T, window, kvh, row0, rows, whole, pad;
};
// Both rings hold whatever any role may still look at: the loads are at most a
// ring ahead of the products, and those four tiles ahead of the output.
constexpr int kFbRing = 16;
static_assert(kFbMaxStages + 7 <= kFbRing, "records outlive their readers");

template <int NQ>
struct FbShared {
    // With 32 columns the two softmax groups take half of the rows of every
    // tile each, else all rows of every other tile: the code of a group stays
    // small (32 rows in one thread took 30% misses in the instruction cache and
    // twice the time).
    static constexpr bool kRowSplit = NQ == 32;
    static constexpr int kRows = kRowSplit ? 16 : NQ;        // of a softmax thread
    // In the order of the arrivals that complete them (see their set-up).
    uint64_t k_full[kFbMaxStages], k_empty[kFbMaxStages];
    uint64_t v_full[kFbMaxStages], v_empty[kFbMaxStages];
    uint64_t q_full[2], o_full[4], q_empty[2], s_full[2], mma_final;
    uint64_t o_free[4], g_sync[2], s_free[2], p_full[4], unsignalled;
    static constexpr int kBars = 4 * kFbMaxStages + 24;
    alignas(16) FbTile tile[kFbRing];
    alignas(16) FbPart part[kFbRing];
    // Per tile and block: K scale x softmax scale (log2 units), log2 of the V
    // scale (of 0: -inf), 0 where there is no block.
    alignas(16) float4 info[kFbRing][2];
    alignas(16) float qsc[kFbRing][NQ];    // power-of-two scale of each query row
    alignas(16) int row_at[kFbRing][NQ];   // its position
    // per softmax group, on even and odd turns: largest scores per warp
    alignas(16) float wmax[2][2][4][kRows];
    // Per softmax warp: what the exponentials are relative to (negative), their
    // factors in the sum and in P, the factor of the sum so far.
    alignas(16) float ref[8][kRows], fac[8][kRows], pfac[8][kRows], grow[8][kRows];
    alignas(16) float top[4][NQ];  // a tile's largest score with its V scale
    alignas(16) float join[4][2][NQ];   // per output warp: factor of the tile, of the rest
    // at a part's end, per softmax group that had a tile: sums of weights, the
    // scores they are relative to (row split: the first group's place holds all rows)
    float lsum[4][2][4][NQ];
    float ltop[4][2][NQ];
    uint32_t tmem_base;
    int abort, never;             // set when a wait gave up; stays 0
    PlanScratch plan;
};
static_assert(sizeof(FbShared<32>) <= 16 * 1024, "shared block");

// Largest of x over the warp (NaN only where every lane is NaN).
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Two f16 numbers as E4M3 codes (nearest even, saturated, NaN kept), and back.
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
    return r;
}

// The first E4M3 piece of two f16 numbers of at most 256 in size; x becomes 32
// times what is left (at most 256 again; few bits: exact in f16).
__device__ __forceinline__ uint32_t e4m3_piece(uint32_t &x) {
    const uint32_t c = f16x2_to_e4m3x2(x), back = e4m3x2_to_f16x2(c);
    const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&x),
                                      *reinterpret_cast<const __half2 *>(&back)),
                              __floats2half2_rn(32.f, 32.f));
    x = *reinterpret_cast<const uint32_t *>(&r);
    return c;
}

// UMMA shared-memory descriptor; layout 0: no swizzle, 2: 128-byte, 4: 64-byte.
__device__ __forceinline__ uint64_t fb_desc(uint32_t start, uint32_t lbo, uint32_t sbo,
                                            int layout) {
    return (uint64_t)((start & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)layout << 61);
}

// kind::f8f6f4, E4M3 operands, fp32 accumulator.
__host__ __device__ constexpr uint32_t fb_idesc(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Issued by the lane whose `lead` is set; the whole warp comes here, so that the
// descriptors stay in uniform registers (in a branch of one lane each of them is
// moved there first: some 110 cycles an MMA, now 85).
__device__ __forceinline__ void umma_f8(uint32_t lead, uint32_t d_tmem, uint64_t a, uint64_t b,
                                        uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void umma_commit_by(uint32_t lead, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(lead)
        : "memory");
}

template <int N>
__device__ __forceinline__ void fb_tmem_ld(uint32_t addr, float *v) {
    static_assert(N == 16 || N == 32, "columns of a load");
    if constexpr (N == 32) tmem_ld32(addr, v);
    else tmem_ld16(addr, v);
}

// mbar_wait out of line: the slow half of every wait, kept out of the loops
// (their code has to stay in the instruction cache).
__device__ __noinline__ bool fb_wait_slow(uint64_t *bar, uint32_t parity,
                                          unsigned long long timeout_ns, unsigned *err,
                                          volatile int *abort) {
    return mbar_wait(bar, parity, timeout_ns, err, abort);
}

// A warp's wait: it tests for a while (a suspended wait wakes up some 200
// cycles late), then sleeps.  The lanes leave together.
__device__ __forceinline__ bool fb_wait(uint64_t *bar, uint32_t parity,
                                        const GqaFp8BlockParams &p, volatile int *abort) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
        if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
    return __all_sync(0xffffffffu, fb_wait_slow(bar, parity, p.timeout_ns, p.err, abort));
}

// The same for the warps that issue the products, which everything else waits
// on: they never sleep.
__device__ __noinline__ bool fb_poll_slow(uint64_t *bar, uint32_t parity,
                                          unsigned long long timeout_ns, unsigned *err,
                                          volatile int *abort) {
    unsigned long long t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
        if ((it & 15u) == 15u && __any_sync(0xffffffffu, *abort)) return false;
        if ((it & 1023u) == 1023u) {
            const unsigned long long now = __shfl_sync(0xffffffffu, global_timer_ns(), 0);
            if (t0 == 0) {
                t0 = now;
            } else if (now - t0 > timeout_ns) {
                raise_error(err, kErrTimeout);
                *abort = 1;
                return false;
            }
        }
    }
}

// The part of the work list that a CTA takes, walked unit by unit: `len`
// visible blocks of unit `unit` of sequence b, from its block blk_off on.
template <bool G>
struct FbWalk {
    SegmentWalkerT<G> w;      // its block mapping; pos and end are not used
    int rest, len;            // blocks of the range left, of this unit's part

    __device__ void part() { len = min(rest, w.nb - w.blk_off); }
    __device__ void init(const PlanArgs &pa, int blocks, int b, long long off) {
        w.seq_lens = pa.seq_lens;
        w.B = pa.B;
        w.units = pa.units_per_seq;
        w.vis = pa.vis;
        w.max_blocks = pa.max_blocks;
        rest = blocks;
        len = 0;
        if (rest <= 0) return;
        w.b = b;
        w.load_seq();
        w.unit = off >> 32 ? (int)(off / w.nb) : (int)((unsigned)off / (unsigned)w.nb);
        w.blk_off = (int)(off - (long long)w.unit * w.nb);
        part();
    }
    __device__ bool done() const { return rest <= 0; }
    __device__ bool whole() const { return len == w.nb; }
    __device__ void next() {
        rest -= len;
        w.blk_off += len;
        if (rest <= 0) return;
        if (w.blk_off == w.nb) {
            w.blk_off = 0;
            if (++w.unit == w.units) {
                w.unit = 0;
                do { ++w.b; w.load_seq(); } while (w.nb == 0 && w.b + 1 < w.B);
            }
        }
        part();
    }
};

// Where a CTA's range begins: blocks in it, sequence, blocks of that sequence
// before it, and the length of the whole list.
struct FbPlace {
    int blocks, b;
    long long off, W;
};

// plan_locate for at most 32 sequences and a list that 32 bits count, by each
// warp for itself: one load, one scan, no barrier.
template <bool G>
__device__ __forceinline__ FbPlace fb_place(const PlanArgs &a, int cta, int lane,
                                            unsigned *err) {
    unsigned work = 0;
    bool bad = false;
    if (lane < a.B) {
        int fb, sb;
        work = (unsigned)visible_blocks<G>(a.seq_lens[lane], a.vis, a.max_blocks, &fb, &sb, &bad,
                                           lane) *
               a.units_per_seq;
    }
    unsigned x = work;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    const unsigned W = __shfl_sync(0xffffffffu, x, 31);
    const unsigned P = min(W, (unsigned)a.num_ctas);
    if (err && __any_sync(0xffffffffu, bad) && lane == 0) raise_error(err, kErrBadSeqLen);
    FbPlace at{0, 0, 0, (long long)W};
    if ((unsigned)cta >= P) return at;
    const unsigned lo = (unsigned)cta * W / P, hi = ((unsigned)cta + 1u) * W / P;
    const unsigned hit = __ballot_sync(0xffffffffu, x - work <= lo && lo < x);
    at.b = __ffs(hit) - 1;
    at.blocks = (int)(hi - lo);
    at.off = lo - __shfl_sync(0xffffffffu, x - work, at.b);
    return at;
}

struct FbUnit {      // what a unit's index stands for
    int kvh, row0, rows;
};
__device__ __forceinline__ FbUnit fb_unit(const GqaFp8BlockParams &p, int unit) {
    FbUnit u;
    u.kvh = unit / p.chunks;
    u.row0 = (unit % p.chunks) * p.chunk_rows;
    u.rows = min(p.chunk_rows, p.group * p.q_len - u.row0);
    return u;
}

// 16 bytes from global to shared memory, for fb_copies_done to wait for.
__device__ __forceinline__ void fb_copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void fb_copies_done() {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
}

// Starts copying a unit's query rows first, first + step, ...; one warp.
template <int D>
__device__ __forceinline__ void fb_fetch_q(const GqaFp8BlockParams &p, int b, const FbUnit &u,
                                           unsigned char *raw, int first, int step) {
    constexpr int kChunks = D / 8;             // of a row, a power of two
    constexpr int kAtOnce = kChunks < 32 ? 32 / kChunks : 1;
    const int lane = threadIdx.x & 31;
    for (int r = first + (lane / kChunks) * step; r < u.rows; r += kAtOnce * step) {
        const int row = u.row0 + r, i = row / p.group, g = row - i * p.group, c = lane % kChunks;
        fb_copy16(raw + (r * kChunks + c) * 16,
                  p.q + ((int64_t)b * p.q_len + i) * p.q_stride +
                      (size_t)(u.kvh * p.group + g) * D + c * 8);
    }
}

// The rows that this warp copied to `raw` into a Q buffer: row r in columns r
// (hi) and NQ + r (lo) of the N side, scaled so that its largest value is in
// [128, 256).  A row with an infinity or a NaN becomes NaN.  (Not inlined: two
// callers, and the code that an SM has to fetch before its first tile counts.)
template <int D, int NQ>
__device__ __noinline__ void fb_prepare_q(const unsigned char *raw, unsigned char *q_buf,
                                          float *qsc, int *row_at, int at0, int row0, int rows,
                                          int group, int first, int step) {
    using C = FbCfg<D, NQ>;
    constexpr int kE = D / 32;                 // values of a lane
    const int lane = threadIdx.x & 31;
#pragma unroll 2
    for (int r = first; r < rows; r += step) {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(raw + r * 2 * D + lane * 2 * kE);
        uint32_t w[kE / 2], top = 0;
        if constexpr (kE == 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(src);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (kE == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(src);
            w[0] = v.x; w[1] = v.y;
        } else {
            w[0] = *src;
        }
#pragma unroll
        for (int j = 0; j < kE / 2; ++j)
            top = max(top, max((w[j] << 16) & 0x7FFFFFFFu, w[j] & 0x7FFF0000u));
        top = __reduce_max_sync(0xffffffffu, top);
        // 2^(exponent - 7), at least the smallest normal number
        const uint32_t e = (uint32_t)max((int)(top >> 23) - 7, 1);
        const float s = __uint_as_float(e << 23), by = __uint_as_float((254u - e) << 23);
        uint32_t hi[kE / 2], lo[kE / 2];
#pragma unroll
        for (int j = 0; j < kE / 2; ++j) {
            uint32_t x = pack_f16x2(bf16lo(w[j]) * by, bf16hi(w[j]) * by);
            hi[j] = e4m3_piece(x);
            lo[j] = f16x2_to_e4m3x2(x);
            if (top >= 0x7F800000u) hi[j] = 0x7F7Fu;
        }
#pragma unroll
        for (int piece = 0; piece < 2; ++piece) {
            const uint32_t *c = piece ? lo : hi;
            const int n = r + piece * NQ, byte = lane * kE;
            int off = n * C::kRowBytes + byte % C::kRowBytes;
            off ^= C::kRowBytes == 128 ? ((off >> 7) & 7) << 4 : ((off >> 7) & 3) << 4;
            unsigned char *dst = q_buf + (byte / C::kRowBytes) * (C::kN * C::kRowBytes) + off;
            if constexpr (kE == 8)
                *reinterpret_cast<uint2 *>(dst) =
                    make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
            else if constexpr (kE == 4)
                *reinterpret_cast<uint32_t *>(dst) = c[0] | (c[1] << 16);
            else
                *reinterpret_cast<uint16_t *>(dst) = (uint16_t)c[0];
        }
        if (lane == 0) {
            qsc[r] = s;
            row_at[r] = at0 + (row0 + r) / group;
        }
    }
}

// Sums v[q] over the warp; lane l gets the sum of q = l % NQ.
template <int NQ>
__device__ __forceinline__ float warp_sums(float *v, int lane) {
#pragma unroll
    for (int o = NQ / 2; o >= 1; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float keep = up ? v[j + o] : v[j], give = up ? v[j] : v[j + o];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    float x = v[0];
#pragma unroll
    for (int o = NQ; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int D, int NQ, bool G>
__global__ void __launch_bounds__(kFbThreads, 1)
gqa_fp8_block_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const GqaFp8BlockParams p) {
    using C = FbCfg<D, NQ>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *sK = smem + C::kOffK, *sV = smem + C::kOffV, *sQ = smem + C::kOffQ,
                  *sP = smem + C::kOffP;
    FbShared<NQ> *sh = reinterpret_cast<FbShared<NQ> *>(smem + C::kOffBar);
    volatile int *abort_flag = &sh->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 0) {
        // the barriers, one lane each: arrivals that complete a phase
        for (int i = lane; i < FbShared<NQ>::kBars; i += 32) {
            uint64_t *bar = sh->k_full + i;
            constexpr uint32_t kWarps = FbShared<NQ>::kRowSplit ? 8 : 4;
            const uint32_t count = bar >= sh->s_free ? kWarps        // a tile's softmax warps
                                   : bar >= sh->o_free ? 4           // warps of a group
                                   : bar >= sh->s_full ? 2   // the products and their issuer
                                                       : 1;
            mbar_init(bar, count);
        }
        if (lane == 0) {
            sh->abort = 0;
            sh->never = 0;
            tma_prefetch_map(&tm_k);
            tma_prefetch_map(&tm_v);
        }
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(&sh->tmem_base, C::kTmemCols);
    // Rows of Q behind a unit's stay what they are: zeros from here on, or an
    // earlier unit's rows (their columns are never written out).
    for (int i = tid; i < 2 * C::kQBytes / 16; i += kFbThreads)
        reinterpret_cast<uint4 *>(sQ)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < kFbRing * NQ; i += kFbThreads) {
        (&sh->qsc[0][0])[i] = 0.f;
        (&sh->row_at[0][0])[i] = 0;
    }

    // What came before on the stream wrote the inputs.
    pdl_wait_primary();
    pdl_launch_dependents();

    // The visible blocks of any of a sequence's queries.
    Visibility vis = p.vis;
    if (vis.window > 0) vis.window += p.q_len - 1;
    const int units = p.H_kv * p.chunks;
    const PlanArgs pa{p.seq_lens, p.B, units, vis, p.max_blocks, p.num_ctas};
    FbWalk<G> walk;
    long long W = 0;
    if (p.whole_units) {
        // one CTA per unit
        const int b = blockIdx.x / units;
        int fb, sb;
        bool bad;
        const int nb = visible_blocks<G>(p.seq_lens[b], vis, p.max_blocks, &fb, &sb, &bad, b);
        if (bad && tid == 0) raise_error(p.err, kErrBadSeqLen);
        walk.init(pa, nb, b, (long long)(blockIdx.x % units) * nb);
    } else if (p.small_plan) {
        const FbPlace at = fb_place<G>(pa, blockIdx.x, lane,
                                       blockIdx.x == 0 && warp == 0 ? p.err : nullptr);
        W = at.W;
        walk.init(pa, at.blocks, at.b, at.off);
    } else {
        plan_locate(pa, blockIdx.x, &sh->plan, nullptr, p.err);
        W = sh->plan.total;
        const int P = working_ctas(W, p.num_ctas);
        const bool works = (int)blockIdx.x < P;
        const long long lo = works ? cta_bound(blockIdx.x, W, P) : 0;
        const long long hi = works ? cta_bound(blockIdx.x + 1, W, P) : 0;
        walk.init(pa, (int)(hi - lo), sh->plan.seq, lo - sh->plan.base);
    }
    // Table entries of up to 32 blocks of the unit's part, one per lane of warp
    // 0 (-1: none); the first ones while the CTA is still setting up.
    auto entries = [&](int base) {
        return base + lane < walk.len
                   ? p.block_table[(size_t)walk.w.b * p.max_blocks +
                                   walk.w.slot(walk.w.blk_off + base + lane)]
                   : -1;
    };
    int entry = -1;
    if (warp == 0 && !walk.done()) entry = entries(0);
    // The first unit's queries, by all warps that have nothing else to do yet.
    constexpr int kHelpers = kFbThreads / 32 - 3;
    if (warp >= 3 && !walk.done())
        fb_fetch_q<D>(p, walk.w.b, fb_unit(p, walk.w.unit), smem + C::kOffRaw, warp - 3, kHelpers);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem_base;

    if (warp >= 3) {
        if (!walk.done()) {
            const FbUnit u = fb_unit(p, walk.w.unit);
            fb_copies_done();
            fb_prepare_q<D, NQ>(smem + C::kOffRaw, sQ, sh->qsc[0], sh->row_at[0],
                                walk.w.T - p.q_len, u.row0, u.rows, p.group, warp - 3, kHelpers);
            fence_proxy_async_smem();
        }
        named_barrier(1, kHelpers * 32);
    }
    if (walk.done()) {
        // no work: nothing waits for this CTA
        if (warp == 3 && lane == 0 && !p.whole_units && (int)blockIdx.x + 1 < p.num_ctas)
            p.ws_cut[blockIdx.x] = FbCut{0, -1, 0, 0, 0};
    } else if (warp == 0) {
        // ============================================================ loads
        const uint64_t pol = l2_policy_evict_first();
        int n_k = 0, n_v = 0;                   // copies of K and V issued (lane 0)
        int tile = 0, ks = 0, vs = 0, seg = -1;
        uint32_t k_par = 1, v_par = 1;          // of the rings' last round
        bool ok = true;
        int base = 0, kvh = walk.w.unit / p.chunks, left = walk.rest;
        // This lane's block of a batch: its row among the codes, its scales.
        int row = 0;
        float k_scale = 0.f, v_scale = 0.f;
        bool there = false;
        auto look_up = [&](bool wanted) {
            row = p.num_blocks * p.H_kv * kBlockSize;           // behind the pool: zeros
            there = wanted && entry >= 0 && entry < p.num_blocks;
            if (there) {
                const size_t at = (size_t)entry * p.H_kv + kvh;
                row = (int)at * kBlockSize;
                k_scale = p.k_scale[at];
                v_scale = p.v_scale[at];
            } else if (wanted) {
                raise_error(p.err, kErrBadBlock);
            }
        };
        look_up(lane < walk.len);
        while (ok && !walk.done()) {
            // One batch: `count` blocks, looked up.  The next one's entries are
            // read after its first tile is under way, its scales behind its
            // last, so that neither is waited for.
            const int base0 = base, len = walk.len, count = min(32, len - base);
            const int my_row = row;
            const int my_pos = lane < count
                                   ? walk.w.logical(walk.w.blk_off + base + lane) * kBlockSize
                                   : 0;
            const float my_ks = k_scale, my_vs = v_scale;
            const bool my_block = there;
            if (base == 0) {
                ++seg;
                const FbUnit u = fb_unit(p, walk.w.unit);
                const bool global = G && global_query(p.vis, walk.w.b, walk.w.T);
                if (lane == 0)
                    sh->part[seg % kFbRing] =
                        FbPart{walk.w.b, walk.w.T, global ? 0 : p.vis.window, u.kvh, u.row0,
                               u.rows, walk.whole() ? 1 : 0, 0};
            }
#pragma unroll 1
            for (int j = 0; j < count; j += 2, ++tile) {
                const int row0 = __shfl_sync(0xffffffffu, my_row, j);
                const int row1 = __shfl_sync(0xffffffffu, my_row, (j + 1) & 31);
                const int pos0 = __shfl_sync(0xffffffffu, my_pos, j);
                const int pos1 = __shfl_sync(0xffffffffu, my_pos, (j + 1) & 31);
                const bool two = j + 1 < count;
                const uint32_t bytes = (two ? 2 : 1) * kBlockSize * D;
                left -= two ? 2 : 1;
                if (lane == 0) {
                    ok = tile < C::kKStages || mbar_test(&sh->k_empty[ks], k_par) ||
                         fb_wait_slow(&sh->k_empty[ks], k_par, p.timeout_ns, p.err, abort_flag);
                    if (ok) {
#pragma unroll
                        for (int x = 0; x < C::kBoxes; ++x) {
                            unsigned char *dst = sK + ks * C::kSlot + x * C::kBoxBytes;
                            tma_load_2d(dst, &tm_k, x * C::kRowBytes, row0, &sh->k_full[ks], pol);
                            if (two)
                                tma_load_2d(dst + kBlockSize * C::kRowBytes, &tm_k,
                                            x * C::kRowBytes, row1, &sh->k_full[ks], pol);
                        }
                        const int at = base0 + j;
                        sh->tile[tile % kFbRing] =
                            FbTile{{pos0, pos1},
                                   (two ? kFbTwo : 0) | (at == 0 ? kFbFirst : 0) |
                                       (at + 2 >= len ? kFbLast : 0) |
                                       (at + 4 >= len ? kFbLastPair : 0) | seg << kFbSegShift,
                                   left};
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                // The scales may arrive after the copies set out: the arrival
                // that lets others see the tile comes behind them.
                if (lane == j || lane == j + 1) {
                    sh->info[tile % kFbRing][lane - j] =
                        my_block && lane < count
                            ? make_float4(my_ks * p.scale_log2,
                                          my_vs == 0.f ? -INFINITY : log2f(my_vs), 1.f, 0.f)
                            : make_float4(0.f, -INFINITY, 0.f, 0.f);
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh->k_full[ks], bytes);
                    n_k = tile + 1;
                    ok = tile < C::kVStages || mbar_test(&sh->v_empty[vs], v_par) ||
                         fb_wait_slow(&sh->v_empty[vs], v_par, p.timeout_ns, p.err, abort_flag);
                    if (ok) {
                        mbar_arrive_expect_tx(&sh->v_full[vs], bytes);
#pragma unroll
                        for (int x = 0; x < C::kBoxes; ++x) {
                            unsigned char *dst = sV + vs * C::kSlot + x * C::kBoxBytes;
                            tma_load_2d(dst, &tm_v, x * C::kRowBytes, row0, &sh->v_full[vs], pol);
                            if (two)
                                tma_load_2d(dst + kBlockSize * C::kRowBytes, &tm_v,
                                            x * C::kRowBytes, row1, &sh->v_full[vs], pol);
                        }
                        n_v = tile + 1;
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                if (++ks == C::kKStages) {
                    ks = 0;
                    k_par ^= 1u;
                }
                if (++vs == C::kVStages) {
                    vs = 0;
                    v_par ^= 1u;
                }
                if (j == 0) {
                    base += 32;
                    if (base >= walk.len) {
                        walk.next();
                        base = 0;
                        if (!walk.done()) kvh = walk.w.unit / p.chunks;
                    }
                    entry = walk.done() ? -1 : entries(base);
                }
            }
            if (ok && !walk.done()) look_up(base + lane < walk.len);
        }
        // Copies still under way must land before the CTA ends.
        if (lane == 0) {
            for (int t = max(n_k - C::kKStages, 0); t < n_k; ++t)
                fb_wait_slow(&sh->k_full[t % C::kKStages], (uint32_t)((t / C::kKStages) & 1),
                             p.timeout_ns, p.err, abort_flag + 1);
            for (int t = max(n_v - C::kVStages, 0); t < n_v; ++t)
                fb_wait_slow(&sh->v_full[t % C::kVStages], (uint32_t)((t / C::kVStages) & 1),
                             p.timeout_ns, p.err, abort_flag + 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ===================================================== S^T = K Q^T
        constexpr uint32_t idesc = fb_idesc(128, C::kN, 0, 0);
        constexpr int kLayout = C::kRowBytes == 128 ? 2 : 4;
        constexpr int kSteps = C::kRowBytes / 32;
        const uint64_t dk = fb_desc(smem_u32(sK), 16, C::kRowBytes * 8, kLayout);
        const uint64_t dq = fb_desc(smem_u32(sQ), 16, C::kRowBytes * 8, kLayout);
        const uint32_t lead = lane == 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_test(bar, parity)) ||
                   fb_poll_slow(bar, parity, p.timeout_ns, p.err, abort_flag);
        };
        int ks = 0, seg = -1;
        uint32_t k_par = 0;
        const bool go = !p.force_timeout || wait(&sh->unsignalled, 0);
        for (int n = 0; go; ++n) {
            if (n >= 2 && !wait(&sh->s_free[n & 1], (uint32_t)((n / 2 - 1) & 1))) break;
            if (!wait(&sh->k_full[ks], k_par)) break;
            const FbTile at = sh->tile[n % kFbRing];
            if (__any_sync(0xffffffffu, at.flags & kFbFirst)) {
                ++seg;
                if (!wait(&sh->q_full[seg & 1], (uint32_t)((seg >> 1) & 1))) break;
            }
            tc_fence_after();
            const uint32_t d = tmem + C::kTmemS + (n & 1) * C::kN;
            const uint64_t a0 = dk + ((ks * C::kSlot) >> 4);   // addresses count in 16 bytes
            const uint64_t b0 = dq + (((seg & 1) * C::kQBytes) >> 4);
#pragma unroll
            for (int s = 0; s < C::kBoxes * kSteps; ++s) {
                const int x = s / kSteps, o = (s % kSteps) * 32;
                umma_f8(lead, d, a0 + ((x * C::kBoxBytes + o) >> 4),
                        b0 + ((x * C::kN * C::kRowBytes + o) >> 4), idesc, s != 0);
            }
            umma_commit_by(lead, &sh->s_full[n & 1]);
            // what this thread has seen (tile, scales), the softmax may too
            if (lead) mbar_arrive(&sh->s_full[n & 1]);
            umma_commit_by(lead, &sh->k_empty[ks]);
            if (__any_sync(0xffffffffu, at.flags & kFbLast))
                umma_commit_by(lead, &sh->q_empty[seg & 1]);
            if (__any_sync(0xffffffffu, at.left == 0)) break;
            if (++ks == C::kKStages) {
                ks = 0;
                k_par ^= 1u;
            }
        }
        umma_commit_by(lead, &sh->mma_final);
        __syncwarp();
    } else if (warp == 2) {
        // ====================================================== O^T = V^T P
        constexpr uint32_t idesc = fb_idesc(C::kM, C::kNP, 1, 1);
        constexpr int kLayout = C::kRowBytes == 128 ? 2 : 4;
        const uint64_t dv = fb_desc(smem_u32(sV), 16, C::kRowBytes * 8, kLayout);
        const uint64_t dp = fb_desc(smem_u32(sP), 128, 2048, 0);
        const uint32_t lead = lane == 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_test(bar, parity)) ||
                   fb_poll_slow(bar, parity, p.timeout_ns, p.err, abort_flag);
        };
        int vs = 0;
        uint32_t v_par = 0;
        for (int n = 0;; ++n) {
            const int buf = n % C::kOut;
            const uint32_t par = (uint32_t)((n / C::kOut) & 1);
            if (!wait(&sh->v_full[vs], v_par)) break;
            if (n >= C::kOut && !wait(&sh->o_free[buf], par ^ 1u)) break;
            if (!wait(&sh->p_full[buf], par)) break;
            tc_fence_after();
            const uint32_t d = tmem + C::kTmemO + buf * (C::kHalves * C::kNP);
            const uint64_t a0 = dv + ((vs * C::kSlot) >> 4);
            const uint64_t b0 = dp + ((buf * C::kPBytes) >> 4);
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                for (int s = 0; s < kFbTile / 32; ++s)
                    umma_f8(lead, d + h * C::kNP,
                            a0 + ((h * C::kBoxBytes + s * 32 * C::kRowBytes) >> 4),
                            b0 + ((s * 512) >> 4), idesc, s != 0);
            umma_commit_by(lead, &sh->o_full[buf]);
            umma_commit_by(lead, &sh->v_empty[vs]);
            if (__any_sync(0xffffffffu, sh->tile[n % kFbRing].left == 0)) break;
            if (++vs == C::kVStages) {
                vs = 0;
                v_par ^= 1u;
            }
        }
        umma_commit_by(lead, &sh->mma_final);
        // Both issuers' products are done before tensor memory is freed.
        fb_wait_slow(&sh->mma_final, 0, p.timeout_ns, p.err, abort_flag + 1);
        __syncwarp();
    } else if (warp == 3) {
        // ====================================================== next queries
        bool ok = true;
        FbCut end{0, -1, 0, 0, 0};             // the unit cut at the range's end
        for (int seg = 0; !walk.done(); ++seg) {
            const int buf = seg & 1;
            // Where a wait gives up, the walk still goes on to the range's end:
            // the second kernel reads what is cut there.
            if (seg >= 2 && ok)
                ok = __all_sync(0xffffffffu,
                                fb_wait_slow(&sh->q_empty[buf], (uint32_t)((seg / 2 - 1) & 1),
                                             p.timeout_ns, p.err, abort_flag));
            if (seg > 0) {
                const FbUnit u = fb_unit(p, walk.w.unit);
                fb_copies_done();
                fb_prepare_q<D, NQ>(smem + C::kOffRaw, sQ + buf * C::kQBytes,
                                    sh->qsc[seg % kFbRing], sh->row_at[seg % kFbRing],
                                    walk.w.T - p.q_len, u.row0, u.rows, p.group, 0, 1);
                fence_proxy_async_smem();
            }
            mbar_arrive_warp(&sh->q_full[buf]);
            // A unit that goes on in the next CTA: the CTAs that hold it, and the
            // first one's partial.
            if (lane == 0 && !p.whole_units && walk.w.blk_off + walk.len < walk.w.nb) {
                const int P = working_ctas(W, p.num_ctas);
                // the unit's first block in the list; this part starts `rest`
                // before the range's end
                const long long su =
                    cta_bound(blockIdx.x + 1, W, P) - walk.rest - walk.w.blk_off;
                const int c0 = cta_of(su, W, P);
                end = FbCut{c0, cta_of(su + walk.w.nb - 1, W, P),
                            2 * c0 + (cta_bound(c0, W, P) == su ? 0 : 1), walk.w.b, walk.w.unit};
            }
            walk.next();
            __syncwarp();
            if (!walk.done())
                fb_fetch_q<D>(p, walk.w.b, fb_unit(p, walk.w.unit), smem + C::kOffRaw, 0, 1);
        }
        if (!p.whole_units && lane == 0 && (int)blockIdx.x + 1 < p.num_ctas)
            p.ws_cut[blockIdx.x] = end;
    } else if (warp < 12) {
        // ========================================================== softmax
        constexpr bool kSplit = FbShared<NQ>::kRowSplit;
        constexpr int R = FbShared<NQ>::kRows;                 // rows of a thread
        constexpr int kStep = kSplit ? 1 : 2;                  // tiles from one to the next
        const int grp = (warp - 4) >> 2, w = warp & 3, half = w >> 1;
        const int q0 = kSplit ? R * grp : 0;                   // first row
        const int key = 32 * w + lane;                         // of the tile
        const uint32_t tlane = (uint32_t)(32 * w) << 16;
        const int L = p.q_len, sink = p.vis.sink;
        float *ref = sh->ref[warp - 4], *fac = sh->fac[warp - 4], *pfac = sh->pfac[warp - 4],
              *grow = sh->grow[warp - 4];
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return fb_wait(bar, parity, p, abort_flag);
        };
        float2 l[R / 2];
        float top = -INFINITY;                                 // largest score of row q0 + lane
        int seg = -1, turns = 0;                               // tiles of this group so far
        for (int n = kSplit ? 0 : grp, left = walk.rest;; n += kStep, ++turns) {
            if (!kSplit && n > 0) {
                // Whether there is a tile n: one block behind tile n - 2 is
                // tile n - 1; two may be one tile or two.
                if (left <= 1) break;
                if (left == 2) {
                    const int o = n - 1;
                    if (!wait(&sh->s_full[o & 1], (uint32_t)((o >> 1) & 1))) break;
                    if (sh->tile[o % kFbRing].left == 0) break;
                }
            }
            const int buf = n & 1, ob = n % C::kOut;
            if (!wait(&sh->s_full[buf], (uint32_t)((n >> 1) & 1))) break;
            const FbTile tile = sh->tile[n % kFbRing];
            const float4 info = sh->info[n % kFbRing][half];
            left = tile.left;
            if ((tile.flags >> kFbSegShift) != seg) {
                seg = tile.flags >> kFbSegShift;
                top = -INFINITY;
#pragma unroll
                for (int q = 0; q < R / 2; ++q) l[q] = make_float2(0.f, 0.f);
            }
            const FbPart &part = sh->part[seg % kFbRing];
            const int T = part.T, window = part.window;
            const int first = (half ? tile.pos[1] : tile.pos[0]) + 32 * (w & 1);
            const int pos = first + lane;
            // this warp's block, and whether its values are 0
            const bool there = (half == 0 || (tile.flags & kFbTwo)) && info.z != 0.f;
            const bool zero = info.y == -INFINITY;
            // every key of the warp seen by every query
            const bool all = there && first + 31 <= T - L &&
                             (window <= 0 || first > T - 1 - window || first + 31 < sink);
            bool early = window <= 0 || pos < sink;             // whatever the window
            if (!all || zero) {
                if (G && there && window > 0 && first <= T - 1 - window)
                    early |= (global_mask(p.vis, part.b, first / kBlockSize, lane) >> (pos & 63)) &
                             1ull;
                // Rows that no query sees may hold NaN codes: they are zeroed,
                // since 0 x NaN would reach every row's sum.  So are those whose
                // scale is 0.  (Row split: either group zeroes half of a row.)
                const int vs = n % C::kVStages;
                if (!wait(&sh->v_full[vs], (uint32_t)((n / C::kVStages) & 1))) break;
                if (!(there && pos < T && !zero && (early || pos > T - L - window))) {
                    constexpr int kZero = C::kRowBytes / 16 / (kSplit ? 2 : 1);
                    uint4 *v = reinterpret_cast<uint4 *>(sV + vs * C::kSlot +
                                                         key * C::kRowBytes) +
                               (kSplit ? grp * kZero : 0);
#pragma unroll
                    for (int x = 0; x < C::kBoxes; ++x)
#pragma unroll
                        for (int c = 0; c < kZero; ++c)
                            v[x * (C::kBoxBytes / 16) + c] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            tc_fence_after();
            float2 s[R / 2];
            {
                float x[2 * R];
                const uint32_t at = tmem + C::kTmemS + buf * C::kN + q0 + tlane;
                if constexpr (!kSplit) {
                    fb_tmem_ld<2 * R>(at, x);
                } else {
                    fb_tmem_ld<R>(at, x);
                    fb_tmem_ld<R>(at + NQ, x + R);
                }
                tc_fence_before();
                mbar_arrive_warp(&sh->s_free[buf]);
                // scores in log2 units
                const float2 k2 = make_float2(info.x, info.x);
                const float2 piece = make_float2(0.03125f, 0.03125f);
                const float *qsc = &sh->qsc[seg % kFbRing][q0], *y = x + R;
#pragma unroll
                for (int q = 0; q < R; q += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(qsc + q);
                    s[q / 2] = __fmul2_rn(__ffma2_rn(make_float2(y[q], y[q + 1]), piece,
                                                     make_float2(x[q], x[q + 1])),
                                          __fmul2_rn(make_float2(f.x, f.y), k2));
                    s[q / 2 + 1] = __fmul2_rn(__ffma2_rn(make_float2(y[q + 2], y[q + 3]), piece,
                                                         make_float2(x[q + 2], x[q + 3])),
                                              __fmul2_rn(make_float2(f.z, f.w), k2));
                }
            }
            if (!all) {
                // a row at position `at` sees the `span` positions up to it
                const unsigned span = !there ? 0u : early ? 1u << 31 : (unsigned)window;
                const int *row_at = &sh->row_at[seg % kFbRing][q0];
#pragma unroll
                for (int q = 0; q < R; q += 4) {
                    const int4 at = *reinterpret_cast<const int4 *>(row_at + q);
                    if ((unsigned)(at.x - pos) >= span) s[q / 2].x = -INFINITY;
                    if ((unsigned)(at.y - pos) >= span) s[q / 2].y = -INFINITY;
                    if ((unsigned)(at.z - pos) >= span) s[q / 2 + 1].x = -INFINITY;
                    if ((unsigned)(at.w - pos) >= span) s[q / 2 + 1].y = -INFINITY;
                }
            }
            // The P buffer, and what goes with it, is free again (long ago, as a
            // rule: tested here, where the scores' arithmetic hides it).
            if (n >= C::kOut && !wait(&sh->o_free[ob], (uint32_t)((n / C::kOut - 1) & 1))) break;
            // largest of the warp's keys, per row (every lane has it: one writes)
            {
                float m[R];
#pragma unroll
                for (int q = 0; q < R; q += 2) {
                    m[q] = warp_max(s[q / 2].x);
                    m[q + 1] = warp_max(s[q / 2].y);
                }
                if (lane == 0) {
#pragma unroll
                    for (int q = 0; q < R; q += 4)
                        *reinterpret_cast<float4 *>(&sh->wmax[grp][turns & 1][w][q]) =
                            make_float4(m[q], m[q + 1], m[q + 2], m[q + 3]);
                }
            }
            mbar_arrive_warp(&sh->g_sync[grp]);
            if (!wait(&sh->g_sync[grp], (uint32_t)(turns & 1))) break;
            bool grew = false;
            if (lane < R) {
                const float(*wm)[R] = sh->wmax[grp][turns & 1];
                const float m0 = fmaxf(wm[0][lane], wm[1][lane]);    // of either block
                const float m1 = fmaxf(wm[2][lane], wm[3][lane]);
                const float m = half ? m1 : m0, both = fmaxf(m0, m1);
                const float now = both != both ? both : fmaxf(top, both);
                const float v0 = m0 + sh->info[n % kFbRing][0].y;    // with their V scales
                const float v1 = m1 + sh->info[n % kFbRing][1].y;
                const float v = half ? v1 : v0, most = fmaxf(v0, v1);
                const float a = top == now ? 1.f : exp2_approx(top - now);
                // 2^8 is in the exponentials; P keeps it
                ref[lane] = m == -INFINITY ? 0.f : 8.f - m;
                fac[lane] = m == -INFINITY ? 0.f : exp2_approx(m - now - 8.f);
                pfac[lane] = v == -INFINITY ? 0.f : v == most ? 1.f : exp2_approx(v - most);
                grow[lane] = a;
                grew = a != 1.f;
                top = now;
                if (w == 0) sh->top[ob][q0 + lane] = most;
            }
            grew = __any_sync(0xffffffffu, grew);
            __syncwarp();
            if (grew) {
#pragma unroll
                for (int q = 0; q < R; q += 2)
                    l[q / 2] = __fmul2_rn(l[q / 2], *reinterpret_cast<const float2 *>(grow + q));
            }
            uint32_t pa[R / 4], pb[R / 4], pc[R / 4];              // the pieces
#pragma unroll
            for (int q = 0; q < R; q += 4) {
                const float4 r = *reinterpret_cast<const float4 *>(ref + q);
                const float4 f = *reinterpret_cast<const float4 *>(fac + q);
                const float4 g = *reinterpret_cast<const float4 *>(pfac + q);
                float2 x = __fadd2_rn(s[q / 2], make_float2(r.x, r.y));
                float2 y = __fadd2_rn(s[q / 2 + 1], make_float2(r.z, r.w));
                x.x = exp2_approx(x.x);
                x.y = exp2_approx(x.y);
                y.x = exp2_approx(y.x);
                y.y = exp2_approx(y.y);
                l[q / 2] = __ffma2_rn(x, make_float2(f.x, f.y), l[q / 2]);
                l[q / 2 + 1] = __ffma2_rn(y, make_float2(f.z, f.w), l[q / 2 + 1]);
                x = __fmul2_rn(x, make_float2(g.x, g.y));
                y = __fmul2_rn(y, make_float2(g.z, g.w));
                uint32_t u = pack_f16x2(x.x, x.y), v = pack_f16x2(y.x, y.y);
                pa[q / 4] = __byte_perm(e4m3_piece(u), e4m3_piece(v), 0x5410);
                pb[q / 4] = __byte_perm(e4m3_piece(u), e4m3_piece(v), 0x5410);
                pc[q / 4] = __byte_perm(f16x2_to_e4m3x2(u), f16x2_to_e4m3x2(v), 0x5410);
            }
            // 16 columns of a key are 16 bytes, keys one after another
            unsigned char *pk = sP + ob * C::kPBytes + key * 16;
            if constexpr (NQ == 8) {
                *reinterpret_cast<uint4 *>(pk) = make_uint4(pa[0], pa[1], pb[0], pb[1]);
                *reinterpret_cast<uint4 *>(pk + 2048) = make_uint4(pc[0], pc[1], 0u, 0u);
            } else {
                constexpr int kPiece = (NQ / 16) * 2048;
                pk += kSplit ? grp * 2048 : 0;
                *reinterpret_cast<uint4 *>(pk) = make_uint4(pa[0], pa[1], pa[2], pa[3]);
                *reinterpret_cast<uint4 *>(pk + kPiece) = make_uint4(pb[0], pb[1], pb[2], pb[3]);
                *reinterpret_cast<uint4 *>(pk + 2 * kPiece) =
                    make_uint4(pc[0], pc[1], pc[2], pc[3]);
            }
            if (tile.flags & (kSplit ? kFbLast : kFbLastPair)) {    // the group's last of the part
                float v[R];
#pragma unroll
                for (int q = 0; q < R; ++q) v[q] = q & 1 ? l[q / 2].y : l[q / 2].x;
                const float sum = warp_sums<R>(v, lane);
                if (lane < R) {
                    sh->lsum[seg & 3][kSplit ? 0 : grp][w][q0 + lane] = sum;
                    if (w == 0) sh->ltop[seg & 3][kSplit ? 0 : grp][q0 + lane] = top;
                }
            }
            fence_proxy_async_smem();
            mbar_arrive_warp(&sh->p_full[ob]);
            if (kSplit && left == 0) break;
        }
    } else {
        // =========================================================== output
        const int w = warp & 3;
        const uint32_t tlane = (uint32_t)(32 * w) << 16;
        const int col = C::kM == 64 ? 16 * w + lane : 32 * w + lane;
        const bool mine = C::kM == 128 || lane < 16;
        float *join = sh->join[w][0], *keep = sh->join[w][1];
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return fb_wait(bar, parity, p, abort_flag);
        };
        float2 o[C::kHalves][NQ / 2];
        float top = -INFINITY;
        int n0 = 0;                                            // the part's first tile
        for (int n = 0;; ++n) {
            const int buf = n % C::kOut;
            const uint32_t par = (uint32_t)((n / C::kOut) & 1);
            if (!wait(&sh->p_full[buf], par)) break;
            const FbTile tile = sh->tile[n % kFbRing];
            if (tile.flags & kFbFirst) {
                n0 = n;
                top = -INFINITY;
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                    for (int q = 0; q < NQ / 2; ++q) o[h][q] = make_float2(0.f, 0.f);
            }
            if (lane < NQ) {
                const float m = sh->top[buf][lane];
                const float now = m != m ? m : fmaxf(top, m);
                // a tile that the row does not see, or whose values are 0, adds nothing
                join[lane] = m == -INFINITY ? 0.f : exp2_approx(m - now - 8.f);
                keep[lane] = top == now ? 1.f : exp2_approx(top - now);
                top = now;
            }
            __syncwarp();
            if (!wait(&sh->o_full[buf], par)) break;
            tc_fence_after();
            constexpr int kCols = NQ < 16 ? NQ : 16;
            const float2 piece = make_float2(0.03125f, 0.03125f);
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                for (int c0 = 0; c0 < NQ; c0 += kCols) {
                    // the pieces of kCols columns, the last first (of 16, two at a
                    // time: registers are short)
                    float2 x[kCols / 2];
                    const uint32_t at =
                        tmem + C::kTmemO + (buf * C::kHalves + h) * C::kNP + c0 + tlane;
                    if constexpr (NQ == 8) {
                        float t[32];
                        tmem_ld32(at, t);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float2 yz = __ffma2_rn(make_float2(t[16 + 2 * q], t[17 + 2 * q]),
                                                         piece,
                                                         make_float2(t[8 + 2 * q], t[9 + 2 * q]));
                            x[q] = __ffma2_rn(yz, piece, make_float2(t[2 * q], t[2 * q + 1]));
                        }
                    } else {
                        float t[16];
                        tmem_ld16(at + 2 * NQ, t);
#pragma unroll
                        for (int q = 0; q < 8; ++q) x[q] = make_float2(t[2 * q], t[2 * q + 1]);
#pragma unroll
                        for (int part = 1; part >= 0; --part) {
                            tmem_ld16(at + part * NQ, t);
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                x[q] = __ffma2_rn(x[q], piece, make_float2(t[2 * q], t[2 * q + 1]));
                        }
                    }
#pragma unroll
                    for (int q = 0; q < kCols; q += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(join + c0 + q);
                        const float4 k = *reinterpret_cast<const float4 *>(keep + c0 + q);
                        float2 *d = &o[h][(c0 + q) / 2];
                        d[0] = __ffma2_rn(x[q / 2], make_float2(f.x, f.y),
                                          __fmul2_rn(d[0], make_float2(k.x, k.y)));
                        d[1] = __ffma2_rn(x[q / 2 + 1], make_float2(f.z, f.w),
                                          __fmul2_rn(d[1], make_float2(k.z, k.w)));
                    }
                }
            if (tile.flags & kFbLast) {
                const int seg = tile.flags >> kFbSegShift;
                const FbPart part = sh->part[seg % kFbRing];
                float sum = 0.f, high = -INFINITY;             // of row `lane`
                int out_row = 0;
                if (lane < part.rows) {
                    // the sum, relative to the row's largest score, of the groups
                    // that have a tile of this part
                    constexpr int kGroups = FbShared<NQ>::kRowSplit ? 1 : 2;
                    float lt[kGroups];
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        lt[g] = kGroups == 2 && n == n0 && (n & 1) != g
                                    ? -INFINITY
                                    : sh->ltop[seg & 3][g][lane];
                        high = fmaxf(high, lt[g]);
                    }
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const float *ls = &sh->lsum[seg & 3][g][0][lane];
                        const float s = (ls[0] + ls[NQ]) + (ls[2 * NQ] + ls[3 * NQ]);
                        if (lt[g] != -INFINITY) sum = fmaf(s, exp2_approx(lt[g] - high), sum);
                    }
                    const int row = part.row0 + lane, i = row / p.group;
                    out_row = (part.b * p.q_len + i) * p.H_q + part.kvh * p.group +
                              (row - i * p.group);
                }
                if (part.whole) {
                    // two factors: their product may be too small for fp32
                    const float by = sum != 0.f ? 1.f / sum : 0.f;
                    const float over = sum != 0.f ? exp2f(top - high) : 0.f;
                    __nv_bfloat16 *dst = p.out + col;
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        const float f = __shfl_sync(0xffffffffu, by, q);
                        const float e = __shfl_sync(0xffffffffu, over, q);
                        const int r = __shfl_sync(0xffffffffu, out_row, q);
                        if (q < part.rows && mine) {
#pragma unroll
                            for (int h = 0; h < C::kHalves; ++h)
                                dst[(size_t)r * D + h * 128] = __float2bfloat16_rn(
                                    (q & 1 ? o[h][q / 2].y : o[h][q / 2].x) * f * e);
                        }
                    }
                } else {
                    const int slot = 2 * blockIdx.x + (seg == 0 ? 0 : 1);
                    float *dst = p.ws_o + (size_t)slot * NQ * D + col;
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
                        if (q < part.rows && mine) {
#pragma unroll
                            for (int h = 0; h < C::kHalves; ++h)
                                dst[q * D + h * 128] = q & 1 ? o[h][q / 2].y : o[h][q / 2].x;
                        }
                    if (w == 0 && lane < part.rows)
                        p.ws_ml[slot * NQ + lane] = make_float4(top, high, sum, 0.f);
                }
            }
            tc_fence_before();
            mbar_arrive_warp(&sh->o_free[buf]);
            if (tile.left == 0) break;
        }
    }

    // Sequences without a visible key: rows of zeros.
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        int fb, sb;
        bool bad;
        if (visible_blocks<G>(p.seq_lens[b], vis, p.max_blocks, &fb, &sb, &bad, b) == 0) {
            const size_t n = (size_t)p.q_len * p.H_q * D / 8;
            uint4 *dst = reinterpret_cast<uint4 *>(p.out + (size_t)b * p.q_len * p.H_q * D);
            for (size_t i = tid; i < n; i += kFbThreads) dst[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// Joins the partials of the unit cut between main CTAs i and i + 1 (i =
// blockIdx.x), if one is; the CTAs of a unit's cuts share its columns.  First a
// warp per row turns the splits' sums and references into weights, then each
// thread adds up four columns of a row (several threads a share of the splits
// each, where there are few columns).
constexpr int kFbJoinThreads = 512;
template <int D, int NQ>
__global__ void __launch_bounds__(kFbJoinThreads)
gqa_fp8_block_join_kernel(const GqaFp8BlockParams p) {
    constexpr int kC = D / 4, kAhead = 8;
    extern __shared__ __align__(16) unsigned char join_smem[];
    __shared__ float2 s_by[NQ];
    pdl_wait_primary();
    pdl_launch_dependents();
    const FbCut cut = p.ws_cut[blockIdx.x];
    if (cut.last < cut.first) return;
    const int part = (int)blockIdx.x - cut.first, parts = cut.last - cut.first;
    const FbUnit u = fb_unit(p, cut.unit);
    const int n = cut.last - cut.first + 1, items = u.rows * kC;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float4 *s_o = reinterpret_cast<float4 *>(join_smem);
    float *s_w = reinterpret_cast<float *>(s_o + kFbJoinThreads);         // [rows][n]
    auto slot = [&](int k) { return (size_t)(k == 0 ? cut.slot : 2 * (cut.first + k)) * NQ; };
    for (int q = warp; q < u.rows; q += kFbJoinThreads / 32) {
        float top = -INFINITY, high = -INFINITY, sum = 0.f;
        bool nan = false;
        for (int k = lane; k < n; k += 32) {
            const float4 ml = __ldcg(p.ws_ml + slot(k) + q);
            nan |= ml.x != ml.x || ml.y != ml.y;
            top = fmaxf(top, ml.x);
            high = fmaxf(high, ml.y);
        }
        nan = __any_sync(0xffffffffu, nan);
        top = nan ? NAN : warp_max(top);
        high = nan ? NAN : warp_max(high);
        for (int k = lane; k < n; k += 32) {
            const float4 ml = __ldcg(p.ws_ml + slot(k) + q);
            // a split whose keys the row does not see adds nothing, one whose
            // values are 0 its weights
            s_w[q * n + k] = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
            if (ml.y != -INFINITY) sum = fmaf(exp2f(ml.y - high), ml.z, sum);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0)
            s_by[q] = sum != 0.f ? make_float2(1.f / sum, exp2f(top - high)) : make_float2(0.f, 0.f);
    }
    __syncthreads();
    // Threads of an item: a power of two, while each still has splits to add.
    int par = 1;
    while (2 * par * items <= kFbJoinThreads * parts && 2 * par < n) par *= 2;
    const int sub = tid & (par - 1);
    for (int it0 = part * (kFbJoinThreads / par); it0 < items; it0 += parts * (kFbJoinThreads / par)) {
        const int it = it0 + tid / par;
        const int q = it / kC, c = (it % kC) * 4;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (it < items)
            for (int k0 = sub; k0 < n; k0 += kAhead * par) {
                float4 v[kAhead];
                float f[kAhead];
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {     // all loads before any use
                    const int k = min(k0 + a * par, n - 1);
                    v[a] = __ldcg(
                        reinterpret_cast<const float4 *>(p.ws_o + (slot(k) + q) * D + c));
                    f[a] = k0 + a * par < n ? s_w[q * n + k] : 0.f;
                }
#pragma unroll
                for (int a = 0; a < kAhead; ++a)
                    if (k0 + a * par < n)
                        o = make_float4(fmaf(f[a], v[a].x, o.x), fmaf(f[a], v[a].y, o.y),
                                        fmaf(f[a], v[a].z, o.z), fmaf(f[a], v[a].w, o.w));
            }
        if (par > 1) {
            __syncthreads();                   // the last round's are read
            s_o[tid] = o;
            __syncthreads();
            if (sub == 0 && it < items)
                for (int k = 1; k < par; ++k) {
                    const float4 x = s_o[tid + k];
                    o = make_float4(o.x + x.x, o.y + x.y, o.z + x.z, o.w + x.w);
                }
        }
        if (sub == 0 && it < items) {
            const int row = u.row0 + q, i = row / p.group, g = row % p.group;
            const float2 by = s_by[q];
            __nv_bfloat162 w[2] = {__floats2bfloat162_rn(o.x * by.x * by.y, o.y * by.x * by.y),
                                   __floats2bfloat162_rn(o.z * by.x * by.y, o.w * by.x * by.y)};
            *reinterpret_cast<uint2 *>(p.out + ((size_t)(cut.b * p.q_len + i) * p.H_q +
                                                u.kvh * p.group + g) * D + c) =
                *reinterpret_cast<const uint2 *>(w);
        }
    }
}

// -------------------------------------------------------------- host side

int fp8_block_rows(int rows) {
    const int chunks = (rows + 31) / 32, each = (rows + chunks - 1) / chunks;
    return each;
}

static int fb_columns(int chunk_rows) { return chunk_rows <= 8 ? 8 : chunk_rows <= 16 ? 16 : 32; }

// The workspace: cuts, partials, their two references and sums.
int64_t fp8_block_workspace_bytes(int num_ctas, int rows, int d) {
    const int64_t nq = fb_columns(fp8_block_rows(rows));
    return (int64_t)sizeof(FbCut) * kFp8BlockMaxCtas + 2ll * num_ctas * nq * (d * 4 + 16);
}

namespace {

// Codes as a matrix of [rows][D] bytes, boxes of 64 rows and at most 128 bytes.
bool fb_make_map(CUtensorMap *m, const void *base, int D, uint64_t rows) {
    const auto fn = tc_encode_fn();
    if (!fn) return false;
    const int width = D == 64 ? 64 : 128;
    cuuint64_t dims[2] = {(cuuint64_t)D, rows};
    cuuint64_t strides[1] = {(cuuint64_t)D};
    cuuint32_t box[2] = {(cuuint32_t)width, (cuuint32_t)kBlockSize};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NQ, bool G>
cudaError_t fb_launch(const GqaFp8BlockParams &p, const FbEvents &events, cudaStream_t stream) {
    using C = FbCfg<D, NQ>;
    static PerDeviceFlag configured;
    cudaError_t e = configure_once_per_device(configured, [] {
        const cudaError_t r = cudaFuncSetAttribute(
            gqa_fp8_block_join_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
            kFbJoinThreads * 16 + NQ * kFp8BlockMaxCtas * 4);
        if (r != cudaSuccess) return r;
        return cudaFuncSetAttribute(gqa_fp8_block_kernel<D, NQ, G>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap tk, tv;
    const uint64_t rows = (uint64_t)p.num_blocks * p.H_kv * kBlockSize;
    if (!fb_make_map(&tk, p.k_cache, D, rows) || !fb_make_map(&tv, p.v_cache, D, rows))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.whole_units ? p.B * p.H_kv * p.chunks : p.num_ctas));
    cfg.blockDim = dim3(kFbThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (events.start && (e = cudaEventRecord(events.start, stream)) != cudaSuccess) return e;
    e = cudaLaunchKernelEx(&cfg, gqa_fp8_block_kernel<D, NQ, G>, tk, tv, p);
    if (e == cudaSuccess && events.stop) e = cudaEventRecord(events.stop, stream);
    if (e != cudaSuccess || p.whole_units || p.num_ctas == 1) return e;
    cfg.gridDim = dim3((unsigned)p.num_ctas - 1);
    cfg.blockDim = dim3(kFbJoinThreads);
    cfg.dynamicSmemBytes = kFbJoinThreads * 16 + NQ * p.num_ctas * 4;
    return cudaLaunchKernelEx(&cfg, gqa_fp8_block_join_kernel<D, NQ>, p);
}

template <int D>
cudaError_t fb_launch_d(const GqaFp8BlockParams &p, const FbEvents &e, cudaStream_t s) {
    const bool g = p.vis.n_g > 0;
    switch (fb_columns(p.chunk_rows)) {
        case 8: return g ? fb_launch<D, 8, true>(p, e, s) : fb_launch<D, 8, false>(p, e, s);
        case 16: return g ? fb_launch<D, 16, true>(p, e, s) : fb_launch<D, 16, false>(p, e, s);
        default: return g ? fb_launch<D, 32, true>(p, e, s) : fb_launch<D, 32, false>(p, e, s);
    }
}

}  // namespace

cudaError_t launch_gqa_fp8_block(const GqaFp8BlockParams &given, int d, void *workspace,
                                 const FbEvents &events, cudaStream_t stream) {
    GqaFp8BlockParams p = given;
    const int rows = p.group * p.q_len;
    p.chunk_rows = fp8_block_rows(rows);
    p.chunks = (rows + p.chunk_rows - 1) / p.chunk_rows;
    const size_t slots = 2 * (size_t)p.num_ctas * fb_columns(p.chunk_rows);
    p.ws_cut = static_cast<FbCut *>(workspace);
    p.ws_o = reinterpret_cast<float *>(p.ws_cut + kFp8BlockMaxCtas);
    p.ws_ml = reinterpret_cast<float4 *>(p.ws_o + slots * d);
    // Where no sequence can be long and there is an SM for every unit, a unit
    // is not split: that saves the plan and the second kernel.  The lengths are
    // on the device, so the table's width decides: a wider table takes the split
    // whatever its sequences hold.  Measured, whole against split, d = 128: 32
    // units of 4 rows 8.8 us against 16.3 at 512 tokens, 11.8 against 17.0 at
    // 1024, 17.3 against 17.6 at 2048; 128 units 10.3 against 17.9 and 18.4
    // against 24.5 at 512 and 2048; one unit of 32 rows 12.8 against 15.7 at 512,
    // but 30.2 against 21.3 at 2048.
    p.whole_units = p.max_blocks <= kFbWholeBlocks &&
                    (long long)p.B * p.H_kv * p.chunks <= p.num_ctas;
    p.small_plan = p.B <= 32 &&
                   (double)p.B * p.H_kv * p.chunks * p.max_blocks * (p.num_ctas + 1.0) < 4e9;
    switch (d) {
        case 64: return fb_launch_d<64>(p, events, stream);
        case 128: return fb_launch_d<128>(p, events, stream);
        default: return fb_launch_d<256>(p, events, stream);
    }
}

}  // namespace attn
