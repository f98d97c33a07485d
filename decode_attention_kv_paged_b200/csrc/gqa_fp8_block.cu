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
// K = 32 takes 47 cycles for any N <= 64, measured).  A bf16 or fp32 operand
// against 8-bit codes is split into two E4M3 columns: x = hi + lo / 32, hi =
// RNE(x), lo = RNE(32 (x - hi)).  For Q (8 significant bits, scaled by a power
// of two per row) that is exact down to 2^-22 of the row's largest value.  For
// the weights it leaves 2^-8 of a weight at most (each step rounds by 2^-4),
// half of what a bf16 output rounds by, and 2^-22 of the largest weight of the
// tile where the pieces are subnormal.
//
// Softmax.  One thread per key; the largest score of each row comes from a
// warp reduction and an exchange between the four warps.  A tile's weights are
// taken relative to its own largest (weight x V scale), not to a running one:
// the two E4M3 pieces then lose nothing to a key far ahead in another tile.
// The tile's O^T is read from tensor memory and added to fp32 registers with
// the factor that brings it to the running reference.  Sums of weights stay in
// fp32 registers, per key lane, until the unit's end.
//
// Roles (one CTA per SM, 16 warps): warp 0 loads tiles of two blocks by TMA
// (swizzled as the MMA reads them) into two rings, with the block scales;
// warps 1 and 2 issue the two products; warp 3 prepares the next unit's
// queries; warps 4-7 and 8-11 are the softmax, on even and odd tiles (a tile
// is one long chain of latencies for its four warps, so two are kept going);
// warps 12-15 keep the output.  S, P and O are double-buffered.  Every wait is
// bounded, and tensor memory always freed.
//
// The work is split over all SMs by visible blocks (plan.cuh); a unit cut by a
// CTA boundary leaves fp32 partials, which a second kernel, waiting on the
// first by programmatic launch, joins: one CTA per boundary.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fp8_block.cuh"
#include "gqa_tc.cuh"
#include "host_state.cuh"
#include "tc_common.cuh"

namespace attn {

constexpr int kFbThreads = 512;
constexpr int kFbMaxStages = 8;
constexpr int kFbWholeBlocks = 8;                     // see launch_gqa_fp8_block
constexpr int kFbTile = 2 * kBlockSize;               // keys of a tile

template <int D, int NQ>
struct FbCfg {
    static constexpr int kRowBytes = D == 64 ? 64 : 128;      // swizzle span
    static constexpr int kBoxes = D / kRowBytes;
    static constexpr int kHalves = D == 256 ? 2 : 1;          // M = 128 pieces of O^T
    static constexpr int kM = D == 64 ? 64 : 128;             // M of O^T
    static constexpr int kN = 2 * NQ;                         // hi and lo columns
    static constexpr int kBoxBytes = kFbTile * kRowBytes;     // one box of a tile
    static constexpr int kSlot = kFbTile * D;
    static constexpr int kQBytes = kN * D;
    static constexpr int kPBytes = kN * kFbTile;
    static constexpr int kFixed = 2 * kQBytes + 2 * kPBytes + 10 * 1024 + 1024 /*align*/;
    static constexpr int kSlots = (227 * 1024 - kFixed) / kSlot;
    static constexpr int kKStages = kSlots / 2 > kFbMaxStages ? kFbMaxStages : kSlots / 2;
    static constexpr int kVStages =
        kSlots - kKStages > kFbMaxStages ? kFbMaxStages : kSlots - kKStages;
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + kKStages * kSlot;
    static constexpr int kOffQ = kOffV + kVStages * kSlot;
    static constexpr int kOffP = kOffQ + 2 * kQBytes;
    static constexpr int kOffBar = kOffP + 2 * kPBytes;
    static constexpr int kSmem = kOffBar + 10 * 1024 + 1024;
    static constexpr uint32_t kTmemS = 0, kTmemO = 2 * kN;
    static constexpr uint32_t kTmemUsed = 2 * kN + 2 * kHalves * kN;
    static constexpr uint32_t kTmemCols =
        kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
    // With 32 columns the softmax needs more than its even share of registers.
    static constexpr bool kSplitRegs = NQ == 32;
    static constexpr int kRegsLoad = 72, kRegsSoftmax = 152, kRegsOutput = 136;
    static_assert(kRegsLoad + 2 * kRegsSoftmax + kRegsOutput <= 4 * 128, "register split");
    static_assert(kKStages >= 2 && kVStages >= 2, "at least two stages per ring");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

template <int NQ>
struct FbShared {
    // In the order of the arrivals that complete them (see their set-up).
    uint64_t k_full[kFbMaxStages], k_empty[kFbMaxStages];
    uint64_t v_full[kFbMaxStages], v_empty[kFbMaxStages];
    uint64_t q_full[2], s_full[2], o_full[2], q_empty[2], s_free[2], p_full[2], o_free[2];
    uint64_t mma_final;
    static constexpr int kBars = 4 * kFbMaxStages + 15;
    // Per V slot and block of the tile: K scale x softmax scale (log2 units),
    // log2 of the V scale, its reciprocal, 0 where the V scale is 0.
    alignas(16) float4 info[kFbMaxStages][2];
    alignas(16) float qsc[2][NQ];  // power-of-two scale of each query row
    alignas(16) int row_i[2][NQ];  // query position of each row
    alignas(16) float wmax[2][4][NQ];   // per softmax group: largest scores per warp
    alignas(16) float2 ref[8][NQ]; // per softmax warp: reference of the weights, factor in the sum
    alignas(16) float grow[8][NQ]; // per softmax warp: factor of the sum so far
    alignas(16) float top[2][NQ];  // a tile's largest score (with its V scale)
    alignas(16) float2 join[4][NQ];     // per output warp: factor of the tile, of the rest
    // at a unit's end, per softmax group: sums of weights, what they are relative to
    float lsum[2][2][4][NQ];
    float ltop[2][2][NQ];
    uint32_t tmem_base;
    int abort;
    PlanScratch plan;
};
static_assert(sizeof(FbShared<32>) <= 10 * 1024, "shared block");

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

// x = hi + lo / 32 for two numbers of at most 256 in size.
__device__ __forceinline__ void e4m3_split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    const uint32_t x = pack_f16x2(a, b);
    hi = f16x2_to_e4m3x2(x);
    const uint32_t back = e4m3x2_to_f16x2(hi);
    const __half2 k = __floats2half2_rn(32.f, 32.f);
    // the difference has few bits: exact in f16
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&x),
                              *reinterpret_cast<const __half2 *>(&back));
    const __half2 r = __hmul2(d, k);
    lo = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t *>(&r));
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

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int N>
__device__ __forceinline__ void fb_tmem_ld(uint32_t addr, float *v) {
    if constexpr (N == 64) tmem_ld64(addr, v);
    else if constexpr (N == 32) tmem_ld32(addr, v);
    else tmem_ld16(addr, v);
}

// Waits by testing the barrier over and over: for the threads that issue the
// products, which everything else waits on (a suspended wait wakes up some 200
// cycles late).  Bounds and results as mbar_wait.
__device__ __forceinline__ bool mbar_poll(uint64_t *bar, uint32_t parity,
                                          unsigned long long timeout_ns, unsigned *err,
                                          volatile int *abort) {
    unsigned long long t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (mbar_test(bar, parity)) return true;
        if ((it & 15u) == 15u && *abort) return false;
        if ((it & 1023u) == 1023u) {
            const unsigned long long now = global_timer_ns();
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
    __device__ int tiles() const { return (len + 1) / 2; }
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

// Query rows [first, rows) in steps of `step`, one warp each, into a Q buffer:
// row r in columns r (hi) and NQ + r (lo) of the N side, scaled so that its
// largest value is in [128, 256).  A row with an infinity or a NaN becomes NaN.
template <int D, int NQ>
__device__ __forceinline__ void fb_prepare_q(const GqaFp8BlockParams &p, int b, const FbUnit &u,
                                             unsigned char *q_buf, float *qsc, int *row_i,
                                             int first, int step) {
    using C = FbCfg<D, NQ>;
    constexpr int kE = D / 32;                 // values of a lane
    constexpr int kAhead = 4;                  // rows whose loads are in flight
    const int lane = threadIdx.x & 31;
    for (int r0 = first; r0 < u.rows; r0 += kAhead * step) {
        __nv_bfloat162 x[kAhead][kE / 2];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int r = r0 + k * step, row = u.row0 + r;
            if (r >= u.rows) break;
            const int i = row / p.group, g = row % p.group;
            const __nv_bfloat162 *src = reinterpret_cast<const __nv_bfloat162 *>(
                p.q + ((int64_t)b * p.q_len + i) * p.q_stride +
                (size_t)(u.kvh * p.group + g) * D + lane * kE);
            if constexpr (kE == 8) {
                const uint4 v = *reinterpret_cast<const uint4 *>(src);
                x[k][0] = *reinterpret_cast<const __nv_bfloat162 *>(&v.x);
                x[k][1] = *reinterpret_cast<const __nv_bfloat162 *>(&v.y);
                x[k][2] = *reinterpret_cast<const __nv_bfloat162 *>(&v.z);
                x[k][3] = *reinterpret_cast<const __nv_bfloat162 *>(&v.w);
            } else if constexpr (kE == 4) {
                const uint2 v = *reinterpret_cast<const uint2 *>(src);
                x[k][0] = *reinterpret_cast<const __nv_bfloat162 *>(&v.x);
                x[k][1] = *reinterpret_cast<const __nv_bfloat162 *>(&v.y);
            } else {
                x[k][0] = *src;
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int r = r0 + k * step, row = u.row0 + r;
            if (r >= u.rows) break;
            float f[kE];
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < kE / 2; ++e) {
                f[2 * e] = __low2float(x[k][e]);
                f[2 * e + 1] = __high2float(x[k][e]);
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) top = max(top, __float_as_uint(f[e]) & 0x7FFFFFFFu);
            top = __reduce_max_sync(0xffffffffu, top);
            const bool finite = top < 0x7F800000u;
            // 2^(exponent - 7), at least the smallest normal number
            const float s = __uint_as_float((uint32_t)max((int)(top >> 23) - 7, 1) << 23);
            const float by = 1.f / s;
            uint32_t hi[kE / 2], lo[kE / 2];
#pragma unroll
            for (int e = 0; e < kE / 2; ++e) {
                e4m3_split2(f[2 * e] * by, f[2 * e + 1] * by, hi[e], lo[e]);
                if (!finite) hi[e] = 0x7F7Fu;
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
                row_i[r] = row / p.group;
            }
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
            const uint32_t count = bar == &sh->mma_final ? 2             // both issuers
                                   : bar >= sh->s_free ? 4               // warps
                                   : bar >= sh->q_empty ? 9    // the issuer, the softmax warps
                                                        : 1;
            mbar_init(bar, count);
        }
        if (lane == 0) {
            sh->abort = 0;
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
    if (tid < 2 * NQ) {
        sh->qsc[tid / NQ][tid % NQ] = 0.f;
        sh->row_i[tid / NQ][tid % NQ] = 0;
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
    // Table entries and scales of 32 blocks of the unit's part at a time, one
    // per lane of warp 0; the first ones while the CTA is still setting up.
    int my_row = 0;
    float my_ks = 0.f, my_vs = 0.f;
    bool my_block = false;
    auto fetch = [&](int base) {
        my_row = p.num_blocks * p.H_kv * kBlockSize;           // behind the pool: zeros
        my_block = false;
        if (base + lane < walk.len) {
            const int phys = p.block_table[(size_t)walk.w.b * p.max_blocks +
                                           walk.w.slot(walk.w.blk_off + base + lane)];
            if (phys >= 0 && phys < p.num_blocks) {
                const size_t at = (size_t)phys * p.H_kv + walk.w.unit / p.chunks;
                my_row = (int)at * kBlockSize;
                my_ks = p.k_scale[at];
                my_vs = p.v_scale[at];
                my_block = true;
            } else {
                raise_error(p.err, kErrBadBlock);
            }
        }
    };
    if (warp == 0 && !walk.done()) fetch(0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem_base;

    if (warp >= 3) {
        // The first unit's queries: all warps that have nothing else to do yet.
        if (!walk.done())
            fb_prepare_q<D, NQ>(p, walk.w.b, fb_unit(p, walk.w.unit), sQ, sh->qsc[0],
                                sh->row_i[0], warp - 3, kFbThreads / 32 - 3);
        fence_proxy_async_smem();
        named_barrier(1, kFbThreads - 96);
    }
    if (warp < 4) {
    if constexpr (C::kSplitRegs) regs_decrease<C::kRegsLoad>();
    if (warp == 0) {
        // ============================================================ loads
        const uint64_t pol = l2_policy_evict_first();
        int tile = 0, n_k = 0, n_v = 0;         // tiles; copies of K and V issued (lane 0)
        bool ok = true;
        for (bool first = true; ok && !walk.done(); walk.next()) {
            for (int base = 0; ok && base < walk.len; base += 32, first = false) {
                if (!first) fetch(base);
                for (int j = 0; ok && j < 32 && base + j < walk.len; j += 2, ++tile) {
                    const int row0 = __shfl_sync(0xffffffffu, my_row, j);
                    const int row1 = __shfl_sync(0xffffffffu, my_row, j + 1);
                    const bool two = base + j + 1 < walk.len;
                    const uint32_t bytes = (two ? 2 : 1) * kBlockSize * D;
                    const int ks = tile % C::kKStages, vs = tile % C::kVStages;
                    if (lane == 0) {
                        ok = tile < C::kKStages ||
                             mbar_wait(&sh->k_empty[ks], (uint32_t)((tile / C::kKStages - 1) & 1),
                                       p.timeout_ns, p.err, abort_flag);
                        if (ok) {
                            mbar_arrive_expect_tx(&sh->k_full[ks], bytes);
#pragma unroll
                            for (int x = 0; x < C::kBoxes; ++x) {
                                unsigned char *dst = sK + ks * C::kSlot + x * C::kBoxBytes;
                                tma_load_2d(dst, &tm_k, x * C::kRowBytes, row0, &sh->k_full[ks],
                                            pol);
                                if (two)
                                    tma_load_2d(dst + kBlockSize * C::kRowBytes, &tm_k,
                                                x * C::kRowBytes, row1, &sh->k_full[ks], pol);
                            }
                            n_k = tile + 1;
                            ok = tile < C::kVStages ||
                                 mbar_wait(&sh->v_empty[vs],
                                           (uint32_t)((tile / C::kVStages - 1) & 1), p.timeout_ns,
                                           p.err, abort_flag);
                        }
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane == j || lane == j + 1) {
                        // A scale of 0 makes the values 0, not the weights: they
                        // enter the sum through any other scale.
                        const float vse = my_vs == 0.f ? 5.421010862427522e-20f /* 2^-64 */
                                                       : my_vs;
                        sh->info[vs][lane - j] =
                            my_block ? make_float4(my_ks * p.scale_log2, log2f(vse), 1.f / vse,
                                                   my_vs == 0.f ? 0.f : 1.f)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                    __syncwarp();
                    if (lane == 0) {
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
            }
        }
        // Copies still under way must land before the CTA ends.
        if (lane == 0) {
            for (int t = max(n_k - C::kKStages, 0); t < n_k; ++t)
                mbar_wait(&sh->k_full[t % C::kKStages], (uint32_t)((t / C::kKStages) & 1),
                          p.timeout_ns, p.err, nullptr);
            for (int t = max(n_v - C::kVStages, 0); t < n_v; ++t)
                mbar_wait(&sh->v_full[t % C::kVStages], (uint32_t)((t / C::kVStages) & 1),
                          p.timeout_ns, p.err, nullptr);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ===================================================== S^T = K Q^T
        if (lane == 0) {
            constexpr uint32_t idesc = fb_idesc(128, C::kN, 0, 0);
            constexpr int kLayout = C::kRowBytes == 128 ? 2 : 4;
            constexpr int kSteps = C::kRowBytes / 32;
            const uint64_t dk = fb_desc(smem_u32(sK), 16, C::kRowBytes * 8, kLayout);
            const uint64_t dq = fb_desc(smem_u32(sQ), 16, C::kRowBytes * 8, kLayout);
            int n = 0, seg = 0, ks = 0, turn = 0;          // slot of the ring, its round
            bool ok = true;
            for (; ok && !walk.done(); walk.next(), ++seg) {
                ok = mbar_poll(&sh->q_full[seg & 1], (uint32_t)((seg >> 1) & 1), p.timeout_ns,
                               p.err, abort_flag);
                for (int t = walk.tiles(); ok && t > 0; --t, ++n) {
                    ok = (n < 2 || mbar_poll(&sh->s_free[n & 1], (uint32_t)((n / 2 - 1) & 1),
                                             p.timeout_ns, p.err, abort_flag)) &&
                         mbar_poll(&sh->k_full[ks], (uint32_t)(turn & 1), p.timeout_ns, p.err,
                                   abort_flag);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int s = 0; s < C::kBoxes * kSteps; ++s) {
                        const int x = s / kSteps, o = (s % kSteps) * 32;
                        // addresses count in 16 bytes
                        umma_f8(tmem + C::kTmemS + (n & 1) * C::kN,
                                dk + ((ks * C::kSlot + x * C::kBoxBytes + o) >> 4),
                                dq + (((seg & 1) * C::kQBytes + x * C::kN * C::kRowBytes + o) >>
                                      4),
                                idesc, s != 0);
                    }
                    umma_commit(&sh->s_full[n & 1]);
                    umma_commit(&sh->k_empty[ks]);
                    if (++ks == C::kKStages) {
                        ks = 0;
                        ++turn;
                    }
                }
                if (ok) umma_commit(&sh->q_empty[seg & 1]);
            }
            umma_commit(&sh->mma_final);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ====================================================== O^T = V^T P
        if (lane == 0) {
            constexpr uint32_t idesc = fb_idesc(C::kM, C::kN, 1, 1);
            constexpr int kLayout = C::kRowBytes == 128 ? 2 : 4;
            const uint64_t dv = fb_desc(smem_u32(sV), 16, C::kRowBytes * 8, kLayout);
            const uint64_t dp = fb_desc(smem_u32(sP), 128, 2048, 0);
            int n = 0, vs = 0, turn = 0;
            bool ok = true;
            for (; ok && !walk.done(); walk.next()) {
                for (int t = walk.tiles(); ok && t > 0; --t, ++n) {
                    ok = mbar_poll(&sh->v_full[vs], (uint32_t)(turn & 1), p.timeout_ns, p.err,
                                   abort_flag) &&
                         (n < 2 || mbar_poll(&sh->o_free[n & 1], (uint32_t)((n / 2 - 1) & 1),
                                             p.timeout_ns, p.err, abort_flag)) &&
                         mbar_poll(&sh->p_full[n & 1], (uint32_t)((n >> 1) & 1), p.timeout_ns,
                                   p.err, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                        for (int s = 0; s < kFbTile / 32; ++s)
                            umma_f8(tmem + C::kTmemO + ((n & 1) * C::kHalves + h) * C::kN,
                                    dv + ((vs * C::kSlot + h * C::kBoxBytes +
                                           s * 32 * C::kRowBytes) >> 4),
                                    dp + (((n & 1) * C::kPBytes + s * 512) >> 4), idesc, s != 0);
                    umma_commit(&sh->o_full[n & 1]);
                    umma_commit(&sh->v_empty[vs]);
                    if (++vs == C::kVStages) {
                        vs = 0;
                        ++turn;
                    }
                }
            }
            umma_commit(&sh->mma_final);
            // Both issuers' products are done before tensor memory is freed.
            mbar_wait(&sh->mma_final, 0, p.timeout_ns, p.err, nullptr);
        }
        __syncwarp();
    } else {
            // ================================================== next queries
            int seg = 0;
            bool cut = false;          // the range's last unit goes on in the next CTA
            for (; !walk.done(); ++seg) {
                const int buf = seg & 1;
                if (seg > 0) {
                    const bool ok =
                        seg < 2 || mbar_wait(&sh->q_empty[buf], (uint32_t)((seg / 2 - 1) & 1),
                                             p.timeout_ns, p.err, abort_flag);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    fb_prepare_q<D, NQ>(p, walk.w.b, fb_unit(p, walk.w.unit),
                                        sQ + buf * C::kQBytes, sh->qsc[buf], sh->row_i[buf], 0,
                                        1);
                    fence_proxy_async_smem();
                }
                mbar_arrive_warp(&sh->q_full[buf]);
                cut = walk.w.blk_off + walk.len < walk.w.nb;
                walk.next();
            }
            // What the second kernel has to join at this CTA's end: the CTAs
            // that hold the unit, the first one's slot, sequence and unit.
            if (!p.whole_units && lane == 0 && (int)blockIdx.x + 1 < p.num_ctas) {
                FbCut c{0, -1, 0, 0, 0};
                if (cut) {
                    const int P = working_ctas(W, p.num_ctas);
                    const long long su = cta_bound(blockIdx.x + 1, W, P) - walk.w.blk_off;
                    c.first = cta_of(su, W, P);
                    c.last = cta_of(su + walk.w.nb - 1, W, P);
                    c.slot = 2 * c.first + (cta_bound(c.first, W, P) == su ? 0 : 1);
                    c.b = walk.w.b;
                    c.unit = walk.w.unit;
                }
                p.ws_cut[blockIdx.x] = c;
            }
    }
    } else if (warp < 12) {
            if constexpr (C::kSplitRegs) regs_increase<C::kRegsSoftmax>();
            // ======================================================= softmax
            const int grp = (warp - 4) >> 2, w = warp & 3, half = w >> 1;
            const int key = 32 * w + lane;                     // of the tile
            const uint32_t tlane = (uint32_t)(32 * w) << 16;
            const int L = p.q_len;
            float2 *ref = sh->ref[warp - 4];
            float *grow = sh->grow[warp - 4];
            int n = 0, seg = 0;                                // n: tiles before this unit's part
            bool ok = true;
            // Where a wait gives up, the warp goes on without waiting: the four
            // warps meet in a barrier at every tile, and none may miss it.
            auto wait = [&](uint64_t *bar, int phase) {
                if (ok && !mbar_test(bar, (uint32_t)(phase & 1)))
                    ok = mbar_wait(bar, (uint32_t)(phase & 1), p.timeout_ns, p.err, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
            };
            for (; !walk.done(); n += walk.tiles(), walk.next(), ++seg) {
                const int T = walk.w.T, tiles = walk.tiles();
                const bool global = G && global_query(p.vis, walk.w.b, T);
                const int window = global ? 0 : p.vis.window, sink = p.vis.sink;
                float2 l[NQ / 2];
                float top = -INFINITY;                         // of row `lane`
#pragma unroll
                for (int q = 0; q < NQ / 2; ++q) l[q] = make_float2(0.f, 0.f);
                wait(&sh->q_full[seg & 1], seg >> 1);
                const float *qsc = sh->qsc[seg & 1];
                for (int t = (n & 1) ^ grp; t < tiles; t += 2) {
                    const int at_tile = n + t, round = at_tile >> 1;
                    const int vs = at_tile % C::kVStages;
                    const bool there = 2 * t + half < walk.len;     // this warp's block
                    const int blk = walk.w.logical(walk.w.blk_off + 2 * t + (there ? half : 0));
                    const int first = blk * kBlockSize + 32 * (w & 1), pos = first + lane;
                    unsigned long long gmask = 0ull;
                    if (G && window > 0 && first <= T - 1 - window)
                        gmask = global_mask(p.vis, walk.w.b, blk, lane);
                    // every key of the warp seen by every query
                    const bool all = there && first + 31 <= T - L &&
                                     (window <= 0 || first > T - 1 - window || first + 31 < sink);
                    wait(&sh->v_full[vs], at_tile / C::kVStages);
                    const float4 info = sh->info[vs][half];
                    if (!all || info.w == 0.f) {
                        // Rows that no query sees may hold NaN codes: they are
                        // zeroed, since 0 x NaN would reach every row's sum.  So
                        // are those whose scale is 0.
                        const bool any = there && pos < T && info.w != 0.f &&
                                         (window <= 0 || pos > T - L - window || pos < sink ||
                                          ((gmask >> (pos & 63)) & 1ull));
                        if (!any) {
                            unsigned char *v = sV + vs * C::kSlot + key * C::kRowBytes;
#pragma unroll
                            for (int x = 0; x < C::kBoxes; ++x)
#pragma unroll
                                for (int c = 0; c < C::kRowBytes / 16; ++c)
                                    reinterpret_cast<uint4 *>(v + x * C::kBoxBytes)[c] =
                                        make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    wait(&sh->s_full[grp], round);
                    tc_fence_after();
                    float2 s[NQ / 2];
                    {
                        float x[NQ], y[NQ];
                        const uint32_t at = tmem + C::kTmemS + grp * C::kN + tlane;
                        if constexpr (NQ == 8) {
                            float xy[16];
                            tmem_ld16(at, xy);
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                x[q] = xy[q];
                                y[q] = xy[8 + q];
                            }
                        } else {
                            fb_tmem_ld<NQ>(at, x);
                            fb_tmem_ld<NQ>(at + NQ, y);
                        }
                        tc_fence_before();
                        mbar_arrive_warp(&sh->s_free[grp]);
                        // scores in log2 units, the V scale's exponent among them
                        const float2 k2 = make_float2(info.x, info.x);
                        const float2 v2 = make_float2(info.y, info.y);
                        const float2 part = make_float2(0.03125f, 0.03125f);
#pragma unroll
                        for (int q = 0; q < NQ; q += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(qsc + q);
                            s[q / 2] = __ffma2_rn(
                                __ffma2_rn(make_float2(y[q], y[q + 1]), part,
                                           make_float2(x[q], x[q + 1])),
                                __fmul2_rn(make_float2(f.x, f.y), k2), v2);
                            s[q / 2 + 1] = __ffma2_rn(
                                __ffma2_rn(make_float2(y[q + 2], y[q + 3]), part,
                                           make_float2(x[q + 2], x[q + 3])),
                                __fmul2_rn(make_float2(f.z, f.w), k2), v2);
                        }
                    }
                    if (!all) {
                        auto seen = [&](int q) {
                            const int at = T - L + (L > 1 ? sh->row_i[seg & 1][q] : 0);
                            return there && pos <= at &&
                                   (window <= 0 || pos > at - window || pos < sink ||
                                    ((gmask >> (pos & 63)) & 1ull));
                        };
#pragma unroll
                        for (int q = 0; q < NQ; q += 2) {
                            if (!seen(q)) s[q / 2].x = -INFINITY;
                            if (!seen(q + 1)) s[q / 2].y = -INFINITY;
                        }
                    }
                    // largest of the tile, per row
                    {
                        float mine = 0.f;
#pragma unroll
                        for (int q = 0; q < NQ; ++q) {
                            const float m = warp_max(q & 1 ? s[q / 2].y : s[q / 2].x);
                            if (lane == q) mine = m;
                        }
                        // The P buffer and what goes with it are free again: the
                        // group's last tile is through, wmax read by all.
                        if (round >= 1) wait(&sh->o_free[grp], round - 1);
                        if (lane < NQ) sh->wmax[grp][w][lane] = mine;
                    }
                    named_barrier(2 + grp, 128);
                    bool grew = false;
                    if (lane < NQ) {
                        const float m = fmaxf(fmaxf(sh->wmax[grp][0][lane], sh->wmax[grp][1][lane]),
                                              fmaxf(sh->wmax[grp][2][lane],
                                                    sh->wmax[grp][3][lane]));
                        const float now = m != m ? m : fmaxf(top, m);
                        // factor of this tile's weights (2^8 in them) in the sum
                        const float c = m == -INFINITY ? 0.f : exp2_approx(m - now - 8.f);
                        const float a = top == now ? 1.f : exp2_approx(top - now);
                        ref[lane] = make_float2(m == -INFINITY ? 0.f : 8.f - m, c * info.z);
                        grow[lane] = a;
                        grew = a != 1.f;
                        top = now;
                        if (w == 0) sh->top[grp][lane] = m;
                    }
                    grew = __any_sync(0xffffffffu, grew);
                    __syncwarp();
                    if (grew) {
#pragma unroll
                        for (int q = 0; q < NQ; q += 2)
                            l[q / 2] = __fmul2_rn(l[q / 2],
                                                  *reinterpret_cast<const float2 *>(grow + q));
                    }
                    uint32_t hi[NQ / 4], lo[NQ / 4];
#pragma unroll
                    for (int q = 0; q < NQ; q += 2) {
                        const float4 r = *reinterpret_cast<const float4 *>(&ref[q]);
                        float2 x = __fadd2_rn(s[q / 2], make_float2(r.x, r.z));
                        x.x = exp2_approx(x.x);
                        x.y = exp2_approx(x.y);
                        l[q / 2] = __ffma2_rn(x, make_float2(r.y, r.w), l[q / 2]);
                        uint32_t h2, l2;
                        e4m3_split2(x.x, x.y, h2, l2);
                        if (q % 4 == 0) {
                            hi[q / 4] = h2;
                            lo[q / 4] = l2;
                        } else {
                            hi[q / 4] |= h2 << 16;
                            lo[q / 4] |= l2 << 16;
                        }
                    }
                    // 16 columns of a key are 16 bytes, keys one after another
                    unsigned char *pk = sP + grp * C::kPBytes + key * 16;
                    if constexpr (NQ == 8) {
                        *reinterpret_cast<uint4 *>(pk) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
                    } else {
#pragma unroll
                        for (int g = 0; g < NQ / 16; ++g) {
                            *reinterpret_cast<uint4 *>(pk + g * 2048) = make_uint4(
                                hi[4 * g], hi[4 * g + 1], hi[4 * g + 2], hi[4 * g + 3]);
                            *reinterpret_cast<uint4 *>(pk + (NQ / 16 + g) * 2048) = make_uint4(
                                lo[4 * g], lo[4 * g + 1], lo[4 * g + 2], lo[4 * g + 3]);
                        }
                    }
                    if (t + 2 >= tiles) {              // the group's last of the unit
                        float v[NQ];
#pragma unroll
                        for (int q = 0; q < NQ; ++q) v[q] = q & 1 ? l[q / 2].y : l[q / 2].x;
                        const float sum = warp_sums<NQ>(v, lane);
                        if (lane < NQ) {
                            sh->lsum[seg & 1][grp][w][lane] = sum;
                            if (w == 0) sh->ltop[seg & 1][grp][lane] = top;
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive_warp(&sh->p_full[grp]);
                }
                mbar_arrive_warp(&sh->q_empty[seg & 1]);
            }
    } else {
            if constexpr (C::kSplitRegs) regs_increase<C::kRegsOutput>();
            // ======================================================== output
            const int w = warp & 3;
            const uint32_t tlane = (uint32_t)(32 * w) << 16;
            const int col = C::kM == 64 ? 16 * w + lane : 32 * w + lane;
            const bool mine = C::kM == 128 || lane < 16;
            float2 *join = sh->join[w];
            int n = 0, seg = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, int phase) {
                if (ok && !mbar_test(bar, (uint32_t)(phase & 1)))
                    ok = mbar_wait(bar, (uint32_t)(phase & 1), p.timeout_ns, p.err, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
            };
            for (; ok && !walk.done(); walk.next(), ++seg) {
                float2 o[C::kHalves][NQ / 2];
                float top = -INFINITY;
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                    for (int q = 0; q < NQ / 2; ++q) o[h][q] = make_float2(0.f, 0.f);
                const int tiles = walk.tiles(), n0 = n;
                for (int t = 0; ok && t < tiles; ++t, ++n) {
                    const int buf = n & 1;
                    wait(&sh->p_full[buf], n >> 1);
                    if (lane < NQ) {
                        const float m = sh->top[buf][lane];
                        const float now = m != m ? m : fmaxf(top, m);
                        // a tile that the row does not see adds nothing
                        join[lane] = make_float2(
                            m == -INFINITY ? 0.f : exp2_approx(m - now - 8.f),
                            top == now ? 1.f : exp2_approx(top - now));
                        top = now;
                    }
                    __syncwarp();
                    wait(&sh->o_full[buf], n >> 1);
                    if (!ok) break;
                    tc_fence_after();
                    constexpr int kCols = NQ < 16 ? NQ : 16;
                    const float2 part = make_float2(0.03125f, 0.03125f);
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                        for (int q0 = 0; q0 < NQ; q0 += kCols) {
                            float xy[2 * kCols];
                            const uint32_t at =
                                tmem + C::kTmemO + (buf * C::kHalves + h) * C::kN + tlane;
                            if constexpr (NQ <= 16) {
                                fb_tmem_ld<2 * kCols>(at, xy);
                            } else {
                                tmem_ld16(at + q0, xy);
                                tmem_ld16(at + NQ + q0, xy + 16);
                            }
#pragma unroll
                            for (int q = 0; q < kCols; q += 2) {
                                const float4 f =
                                    *reinterpret_cast<const float4 *>(&join[q0 + q]);
                                float2 &d = o[h][(q0 + q) / 2];
                                const float2 v = __ffma2_rn(
                                    make_float2(xy[kCols + q], xy[kCols + q + 1]), part,
                                    make_float2(xy[q], xy[q + 1]));
                                d = __ffma2_rn(v, make_float2(f.x, f.z),
                                               __fmul2_rn(d, make_float2(f.y, f.w)));
                            }
                        }
                    if (t == tiles - 1) {
                        const FbUnit u = fb_unit(p, walk.w.unit);
                        float sum = 0.f;               // of row `lane`
                        int out_row = 0;
                        if (lane < u.rows) {
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                // the group has a tile of this part
                                if (tiles < 2 && (n0 & 1) != g) continue;
                                const float lt = sh->ltop[seg & 1][g][lane];
                                const float *ls = &sh->lsum[seg & 1][g][0][lane];
                                const float s = (ls[0] + ls[NQ]) + (ls[2 * NQ] + ls[3 * NQ]);
                                if (lt != -INFINITY) sum = fmaf(s, exp2_approx(lt - top), sum);
                            }
                            const int row = u.row0 + lane, i = row / p.group;
                            out_row = (walk.w.b * p.q_len + i) * p.H_q + u.kvh * p.group +
                                      (row - i * p.group);
                        }
                        if (walk.whole()) {
                            const float by = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
                            for (int q = 0; q < NQ; ++q) {
                                const float f = __shfl_sync(0xffffffffu, by, q);
                                __nv_bfloat16 *dst =
                                    p.out +
                                    (size_t)__shfl_sync(0xffffffffu, out_row, q) * D + col;
                                if (q < u.rows && mine) {
#pragma unroll
                                    for (int h = 0; h < C::kHalves; ++h)
                                        dst[h * 128] = __float2bfloat16_rn(
                                            (q & 1 ? o[h][q / 2].y : o[h][q / 2].x) * f);
                                }
                            }
                        } else {
                            const int slot = 2 * blockIdx.x + (seg == 0 ? 0 : 1);
                            float *part_o = p.ws_o + (size_t)slot * NQ * D + col;
#pragma unroll
                            for (int q = 0; q < NQ; ++q)
                                if (q < u.rows && mine) {
#pragma unroll
                                    for (int h = 0; h < C::kHalves; ++h)
                                        part_o[q * D + h * 128] =
                                            q & 1 ? o[h][q / 2].y : o[h][q / 2].x;
                                }
                            if (w == 0 && lane < u.rows)
                                p.ws_ml[slot * NQ + lane] = make_float2(top, sum);
                        }
                    }
                    tc_fence_before();
                    mbar_arrive_warp(&sh->o_free[buf]);
                }
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

// Joins the partials of the unit that is cut between main CTAs i and i + 1
// (i = blockIdx.x), if one is.  The CTAs of a unit's cuts share its values;
// splits are added in order, so a result does not depend on which CTA came
// first.
constexpr int kFbJoinThreads = 256;
template <int D, int NQ>
__global__ void __launch_bounds__(kFbJoinThreads)
gqa_fp8_block_join_kernel(const GqaFp8BlockParams p) {
    constexpr int kWarps = kFbJoinThreads / 32;
    constexpr int kC = D / 4;                  // float4 of a row
    constexpr int kPer = D == 256 ? 2 : 1;     // of a lane
    constexpr int kPar = D == 64 ? 2 : 1;      // splits that a warp adds at a time
    constexpr int kAhead = 4;
    __shared__ float4 s_o[kWarps][kC * kPar];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait_primary();
    const FbCut cut = p.ws_cut[blockIdx.x];
    if (cut.last < cut.first) return;
    const FbUnit u = fb_unit(p, cut.unit);
    const int n = cut.last - cut.first + 1;    // splits
    const int sub = kPar == 2 ? lane >> 4 : 0, c = kPar == 2 ? lane & 15 : lane;
    auto slot = [&](int k) { return k == 0 ? cut.slot : 2 * (cut.first + k); };
    for (int q = (int)blockIdx.x - cut.first; q < u.rows; q += n - 1) {
        // Warp w adds splits w, w + 8, ... (two at once where a row is short),
        // each lane its columns, relative to the largest reference of them.
        float top = -INFINITY, sum = 0.f;
        float4 o[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = warp * kPar + sub; k0 < n; k0 += kAhead * kWarps * kPar) {
            float2 ml[kAhead];
            float4 v[kAhead][kPer];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int k = k0 + a * kWarps * kPar;
                ml[a] = make_float2(-INFINITY, 0.f);
                if (k < n) {
                    const size_t at = (size_t)slot(k) * NQ + q;
                    ml[a] = p.ws_ml[at];
#pragma unroll
                    for (int j = 0; j < kPer; ++j)
                        v[a][j] = *reinterpret_cast<const float4 *>(p.ws_o + at * D +
                                                                    (j * 32 + c) * 4);
                }
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                // a split whose keys the row does not see adds nothing
                if (ml[a].x == -INFINITY) continue;
                const float now = ml[a].x != ml[a].x ? ml[a].x : fmaxf(top, ml[a].x);
                const float f = exp2f(ml[a].x - now);
                const float g = top == now ? 1.f : exp2f(top - now);
                top = now;
                sum = fmaf(sum, g, ml[a].y * f);
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    o[j].x = fmaf(o[j].x, g, v[a][j].x * f);
                    o[j].y = fmaf(o[j].y, g, v[a][j].y * f);
                    o[j].z = fmaf(o[j].z, g, v[a][j].z * f);
                    o[j].w = fmaf(o[j].w, g, v[a][j].w * f);
                }
            }
        }
        // ... and the warps' sums, in order
        __shared__ float s_top[kWarps * kPar];
        __shared__ float s_part[kWarps * kPar];
        __syncthreads();                       // the last row's are read
        if (c == 0) {
            s_top[warp * kPar + sub] = top;
            s_part[warp * kPar + sub] = sum;
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) s_o[warp][(kPar == 2 ? sub * kC : j * 32) + c] = o[j];
        __syncthreads();
        if (tid < kC) {
            float all = -INFINITY;
            bool nan = false;
#pragma unroll
            for (int k = 0; k < kWarps * kPar; ++k) {
                nan |= s_top[k] != s_top[k];
                all = fmaxf(all, s_top[k]);
            }
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
            float total = nan ? NAN : 0.f;
#pragma unroll
            for (int k = 0; k < kWarps * kPar; ++k) {
                const float f = s_top[k] == -INFINITY ? 0.f : exp2f(s_top[k] - all);
                const float4 x = s_o[k / kPar][(k % kPar) * kC + tid];
                total = fmaf(f, s_part[k], total);
                r.x = fmaf(f, x.x, r.x);
                r.y = fmaf(f, x.y, r.y);
                r.z = fmaf(f, x.z, r.z);
                r.w = fmaf(f, x.w, r.w);
            }
            const float by = total != 0.f ? 1.f / total : 0.f;
            const int row = u.row0 + q, i = row / p.group, g = row % p.group;
            __nv_bfloat162 w[2] = {__floats2bfloat162_rn(r.x * by, r.y * by),
                                   __floats2bfloat162_rn(r.z * by, r.w * by)};
            *reinterpret_cast<uint2 *>(p.out + ((size_t)(cut.b * p.q_len + i) * p.H_q +
                                                u.kvh * p.group + g) * D + tid * 4) =
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

int64_t fp8_block_workspace_bytes(int num_ctas, int rows, int d) {
    const int64_t nq = fb_columns(fp8_block_rows(rows));
    return 2ll * num_ctas * nq * (d * 4 + 8) + num_ctas * (int64_t)sizeof(FbCut);
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
cudaError_t fb_launch(const GqaFp8BlockParams &p, cudaStream_t stream) {
    using C = FbCfg<D, NQ>;
    static PerDeviceFlag configured;
    cudaError_t e = configure_once_per_device(configured, [] {
        // The shares of a register split must fit in what the kernel is
        // launched with, or the increase would never be granted.
        cudaFuncAttributes fa;
        const cudaError_t r = cudaFuncGetAttributes(&fa, gqa_fp8_block_kernel<D, NQ, G>);
        if (r != cudaSuccess) return r;
        if (C::kSplitRegs && fa.numRegs < 128) return cudaErrorInvalidConfiguration;
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
    e = cudaLaunchKernelEx(&cfg, gqa_fp8_block_kernel<D, NQ, G>, tk, tv, p);
    if (e != cudaSuccess || p.whole_units || p.num_ctas == 1) return e;
    cfg.gridDim = dim3((unsigned)p.num_ctas - 1);
    cfg.blockDim = dim3(kFbJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, gqa_fp8_block_join_kernel<D, NQ>, p);
}

template <int D>
cudaError_t fb_launch_d(const GqaFp8BlockParams &p, cudaStream_t s) {
    const bool g = p.vis.n_g > 0;
    switch (fb_columns(p.chunk_rows)) {
        case 8: return g ? fb_launch<D, 8, true>(p, s) : fb_launch<D, 8, false>(p, s);
        case 16: return g ? fb_launch<D, 16, true>(p, s) : fb_launch<D, 16, false>(p, s);
        default: return g ? fb_launch<D, 32, true>(p, s) : fb_launch<D, 32, false>(p, s);
    }
}

}  // namespace

cudaError_t launch_gqa_fp8_block(const GqaFp8BlockParams &given, int d, void *workspace,
                                 cudaStream_t stream) {
    GqaFp8BlockParams p = given;
    const int rows = p.group * p.q_len;
    p.chunk_rows = fp8_block_rows(rows);
    p.chunks = (rows + p.chunk_rows - 1) / p.chunk_rows;
    const size_t slots = 2 * (size_t)p.num_ctas * fb_columns(p.chunk_rows);
    p.ws_o = static_cast<float *>(workspace);
    p.ws_ml = reinterpret_cast<float2 *>(p.ws_o + slots * d);
    p.ws_cut = reinterpret_cast<FbCut *>(p.ws_ml + slots);
    // Where no sequence can be long and there is an SM for every unit, a unit
    // is not split: that saves the second kernel.
    p.whole_units = p.max_blocks <= kFbWholeBlocks &&
                    (long long)p.B * p.H_kv * p.chunks <= p.num_ctas;
    p.small_plan = p.B <= 32 &&
                   (double)p.B * p.H_kv * p.chunks * p.max_blocks * (p.num_ctas + 1.0) < 4e9;
    switch (d) {
        case 64: return fb_launch_d<64>(p, stream);
        case 128: return fb_launch_d<128>(p, stream);
        default: return fb_launch_d<256>(p, stream);
    }
}

}  // namespace attn
