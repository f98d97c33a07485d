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
// Roles (one CTA per SM, 12 warps): warp 0 loads tiles of two blocks by TMA
// (swizzled as the MMA reads them) into two rings, with the block scales;
// warps 1 and 2 issue the two products; warp 3 prepares the next unit's
// queries; warps 4-7 are the softmax, warps 8-11 keep the output.  S, P and O
// are double-buffered.  Every wait is bounded, and tensor memory always freed.
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

constexpr int kFbThreads = 384;
constexpr int kFbMaxStages = 8;
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
    static constexpr int kFixed = 2 * kQBytes + 2 * kPBytes + 8 * 1024 + 1024 /*align*/;
    static constexpr int kSlots = (227 * 1024 - kFixed) / kSlot;
    static constexpr int kKStages = kSlots / 2 > kFbMaxStages ? kFbMaxStages : kSlots / 2;
    static constexpr int kVStages =
        kSlots - kKStages > kFbMaxStages ? kFbMaxStages : kSlots - kKStages;
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + kKStages * kSlot;
    static constexpr int kOffQ = kOffV + kVStages * kSlot;
    static constexpr int kOffP = kOffQ + 2 * kQBytes;
    static constexpr int kOffBar = kOffP + 2 * kPBytes;
    static constexpr int kSmem = kOffBar + 8 * 1024 + 1024;
    static constexpr uint32_t kTmemS = 0, kTmemO = 2 * kN;
    static constexpr uint32_t kTmemUsed = 2 * kN + 2 * kHalves * kN;
    static constexpr uint32_t kTmemCols =
        kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
    static_assert(kKStages >= 2 && kVStages >= 2, "at least two stages per ring");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

template <int NQ>
struct FbShared {
    uint64_t k_full[kFbMaxStages], k_empty[kFbMaxStages];
    uint64_t v_full[kFbMaxStages], v_empty[kFbMaxStages];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], s_free[2];
    uint64_t p_full[2], o_full[2], o_free[2];
    uint64_t mma_final;
    // Per V slot and block of the tile: K scale x softmax scale (log2 units),
    // log2 of the V scale, its reciprocal, whether V counts (scale not 0).
    alignas(16) float4 info[kFbMaxStages][2];
    alignas(16) float qsc[2][NQ];              // power-of-two scale of each query row
    int row_i[2][NQ];              // query position of each row
    float wmax[2][4][NQ];          // a tile's largest score per warp
    alignas(16) float2 ref[4][NQ];             // per warp: the tile's reference - 8, its factor
    float grow[4][NQ];             // per warp: factor of what was added before
    alignas(16) float2 join[2][NQ];            // for the output warps: factor of the tile, of the rest
    float lsum[2][4][NQ];          // at a unit's end: sums of weights per warp
    float top[2][NQ];              // and the reference they are relative to
    uint32_t tmem_base;
    int abort;
    PlanScratch plan;
};
static_assert(sizeof(FbShared<32>) <= 8 * 1024, "shared block");

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

// The part of the work list that a CTA takes, walked unit by unit.
template <bool G>
struct FbWalk {
    SegmentWalkerT<G> w;
    int len;
    __device__ void init(const PlanArgs &pa, long long lo, long long hi, int seq,
                         long long base) {
        w.init(pa, lo, hi, seq, base);
        len = w.done() ? 0 : w.seg_len();
    }
    __device__ bool done() const { return w.done(); }
    __device__ int tiles() const { return (len + 1) / 2; }
    __device__ void next() {
        w.advance(len);
        len = w.done() ? 0 : w.seg_len();
    }
};

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

    if (tid == 0) {
        for (int s = 0; s < C::kKStages; ++s) {
            mbar_init(&sh->k_full[s], 1);
            mbar_init(&sh->k_empty[s], 1);
        }
        for (int s = 0; s < C::kVStages; ++s) {
            mbar_init(&sh->v_full[s], 1);
            mbar_init(&sh->v_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh->q_full[s], 1);
            mbar_init(&sh->q_empty[s], 5);      // the S products' commit, four softmax warps
            mbar_init(&sh->s_full[s], 1);
            mbar_init(&sh->s_free[s], 4);
            mbar_init(&sh->p_full[s], 4);
            mbar_init(&sh->o_full[s], 1);
            mbar_init(&sh->o_free[s], 4);
        }
        mbar_init(&sh->mma_final, 2);
        sh->abort = 0;
        fence_barrier_init();
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
    }
    if (warp == 1) tmem_alloc(&sh->tmem_base, C::kTmemCols);
    // Rows of Q behind a unit's stay what they are: zeros from here on, or an
    // earlier unit's rows (their columns are never written out).
    for (int i = tid; i < 2 * C::kQBytes / 16; i += kFbThreads)
        reinterpret_cast<uint4 *>(sQ)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < 2 * NQ; i += kFbThreads) {
        sh->qsc[i / NQ][i % NQ] = 0.f;
        sh->row_i[i / NQ][i % NQ] = 0;
    }

    // What came before on the stream wrote the inputs.
    pdl_wait_primary();
    pdl_launch_dependents();

    // The visible blocks of any of a sequence's queries.
    Visibility vis = p.vis;
    if (vis.window > 0) vis.window += p.q_len - 1;
    const int units = p.H_kv * p.chunks;
    PlanArgs pa{p.seq_lens, p.B, units, vis, p.max_blocks, p.num_ctas};
    plan_locate(pa, blockIdx.x, &sh->plan, nullptr, p.err);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem_base;
    const long long W = sh->plan.total;
    const int P = working_ctas(W, p.num_ctas);
    const bool works = (int)blockIdx.x < P;
    const long long lo = works ? cta_bound(blockIdx.x, W, P) : 0;
    const long long hi = works ? cta_bound(blockIdx.x + 1, W, P) : 0;
    FbWalk<G> walk;
    walk.init(pa, lo, hi, sh->plan.seq, sh->plan.base);

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

    if (warp == 0) {
        // ============================================================ loads
        const uint64_t pol = l2_policy_evict_first();
        int tile = 0, n_k = 0, n_v = 0;         // tiles; copies of K and V issued (lane 0)
        bool ok = true;
        for (; ok && !walk.done(); walk.next()) {
            const FbUnit u = fb_unit(p, walk.w.unit);
            // Table entries and scales of 32 blocks at a time, one per lane.
            for (int base = 0; ok && base < walk.len; base += 32) {
                int row = p.num_blocks * p.H_kv * kBlockSize;       // behind the pool: zeros
                float4 info = make_float4(0.f, 0.f, 0.f, 0.f);
                if (base + lane < walk.len) {
                    const int phys = p.block_table[(size_t)walk.w.b * p.max_blocks +
                                                   walk.w.slot(walk.w.blk_off + base + lane)];
                    if (phys >= 0 && phys < p.num_blocks) {
                        const size_t at = (size_t)phys * p.H_kv + u.kvh;
                        row = (int)at * kBlockSize;
                        const float vs = p.v_scale[at];
                        // A scale of 0 makes the values 0, not the weights: they
                        // enter the sum through any other scale.
                        const float vse = vs == 0.f ? 5.421010862427522e-20f /* 2^-64 */ : vs;
                        info = make_float4(p.k_scale[at] * p.scale_log2, log2f(vse), 1.f / vse,
                                           vs == 0.f ? 0.f : 1.f);
                    } else {
                        raise_error(p.err, kErrBadBlock);
                    }
                }
                for (int j = 0; ok && j < 32 && base + j < walk.len; j += 2, ++tile) {
                    const int row0 = __shfl_sync(0xffffffffu, row, j);
                    const int row1 = __shfl_sync(0xffffffffu, row, j + 1);
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
                    if (lane == j || lane == j + 1) sh->info[vs][lane - j] = info;
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
            int n = 0, seg = 0;
            bool ok = true;
            for (; ok && !walk.done(); walk.next(), ++seg) {
                ok = mbar_wait(&sh->q_full[seg & 1], (uint32_t)((seg >> 1) & 1), p.timeout_ns,
                               p.err, abort_flag);
                const uint32_t qb = smem_u32(sQ) + (seg & 1) * C::kQBytes;
                for (int t = walk.tiles(); ok && t > 0; --t, ++n) {
                    const int ks = n % C::kKStages;
                    ok = mbar_wait(&sh->k_full[ks], (uint32_t)((n / C::kKStages) & 1),
                                   p.timeout_ns, p.err, abort_flag) &&
                         (n < 2 || mbar_wait(&sh->s_free[n & 1], (uint32_t)((n / 2 - 1) & 1),
                                             p.timeout_ns, p.err, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t kb = smem_u32(sK) + ks * C::kSlot;
#pragma unroll
                    for (int s = 0; s < C::kBoxes * kSteps; ++s) {
                        const int x = s / kSteps, o = (s % kSteps) * 32;
                        umma_f8(tmem + C::kTmemS + (n & 1) * C::kN,
                                fb_desc(kb + x * C::kBoxBytes + o, 16, C::kRowBytes * 8, kLayout),
                                fb_desc(qb + x * C::kN * C::kRowBytes + o, 16, C::kRowBytes * 8,
                                        kLayout),
                                idesc, s != 0);
                    }
                    umma_commit(&sh->s_full[n & 1]);
                    umma_commit(&sh->k_empty[ks]);
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
            int n = 0;
            bool ok = true;
            for (; ok && !walk.done(); walk.next()) {
                for (int t = walk.tiles(); ok && t > 0; --t, ++n) {
                    const int vs = n % C::kVStages;
                    ok = mbar_wait(&sh->v_full[vs], (uint32_t)((n / C::kVStages) & 1),
                                   p.timeout_ns, p.err, abort_flag) &&
                         (n < 2 || mbar_wait(&sh->o_free[n & 1], (uint32_t)((n / 2 - 1) & 1),
                                             p.timeout_ns, p.err, abort_flag)) &&
                         mbar_wait(&sh->p_full[n & 1], (uint32_t)((n >> 1) & 1), p.timeout_ns,
                                   p.err, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t vb = smem_u32(sV) + vs * C::kSlot;
                    const uint32_t pb = smem_u32(sP) + (n & 1) * C::kPBytes;
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                        for (int s = 0; s < kFbTile / 32; ++s)
                            umma_f8(tmem + C::kTmemO + ((n & 1) * C::kHalves + h) * C::kN,
                                    fb_desc(vb + h * C::kBoxBytes + s * 32 * C::kRowBytes, 16,
                                            C::kRowBytes * 8, kLayout),
                                    fb_desc(pb + s * 512, 128, 2048, 0), idesc, s != 0);
                    umma_commit(&sh->o_full[n & 1]);
                    umma_commit(&sh->v_empty[vs]);
                }
            }
            umma_commit(&sh->mma_final);
            // Both issuers' products are done before tensor memory is freed.
            mbar_wait(&sh->mma_final, 0, p.timeout_ns, p.err, nullptr);
        }
        __syncwarp();
    } else {
        // The first unit's queries: all warps that have nothing else to do yet.
        if (!walk.done())
            fb_prepare_q<D, NQ>(p, walk.w.b, fb_unit(p, walk.w.unit), sQ, sh->qsc[0],
                                sh->row_i[0], warp - 3, kFbThreads / 32 - 3);
        fence_proxy_async_smem();
        named_barrier(1, kFbThreads - 96);
        if (warp == 3) {
            // ================================================== next queries
            for (int seg = 0; !walk.done(); ++seg) {
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
                walk.next();
            }
        } else if (warp < 8) {
            // ======================================================= softmax
            const int w = warp - 4, half = w >> 1;
            const int key = 32 * w + lane;                     // of the tile
            const uint32_t tlane = (uint32_t)(32 * w) << 16;
            const int L = p.q_len;
            int n = 0, seg = 0;
            bool ok = true;
            // Where a wait gives up, the warp goes on without waiting: the four
            // warps meet in a barrier at every tile, and none may miss it.
            auto wait = [&](uint64_t *bar, int phase) {
                if (ok)
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(bar, (uint32_t)(phase & 1), p.timeout_ns, p.err,
                                              abort_flag));
            };
            for (; !walk.done(); walk.next(), ++seg) {
                const int b = walk.w.b, T = walk.w.T;
                const bool global = G && global_query(p.vis, b, T);
                const int window = global ? 0 : p.vis.window, sink = p.vis.sink;
                float l[NQ], top = -INFINITY;                  // top: of row lane
#pragma unroll
                for (int q = 0; q < NQ; ++q) l[q] = 0.f;
                wait(&sh->q_full[seg & 1], seg >> 1);
                const float *qsc = sh->qsc[seg & 1];
                const int tiles = walk.tiles();
                for (int t = 0; t < tiles; ++t, ++n) {
                    const int vs = n % C::kVStages, buf = n & 1;
                    const bool there = 2 * t + half < walk.len;     // this warp's block
                    const int blk = walk.w.logical(walk.w.blk_off + 2 * t + (there ? half : 0));
                    const int first = blk * kBlockSize + 32 * (w & 1), pos = first + lane;
                    unsigned long long gmask = 0ull;
                    if (G && window > 0 && first <= T - 1 - window)
                        gmask = global_mask(p.vis, b, blk, lane);
                    // every key of the warp seen by every query
                    const bool all = there && first + 31 <= T - L &&
                                     (window <= 0 || first > T - 1 - window || first + 31 < sink);
                    wait(&sh->v_full[vs], n / C::kVStages);
                    const float4 info = sh->info[vs][half];
                    if (!all) {
                        // Rows that no query sees may hold NaN codes: they are
                        // zeroed, since 0 x NaN would reach every row's sum.
                        const bool any = there && pos < T &&
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
                    wait(&sh->s_full[buf], n >> 1);
                    tc_fence_after();
                    float s[C::kN];
                    fb_tmem_ld<C::kN>(tmem + C::kTmemS + buf * C::kN + tlane, s);
                    tc_fence_before();
                    mbar_arrive_warp(&sh->s_free[buf]);

                    // scores in log2 units, the V scale's exponent among them
#pragma unroll
                    for (int q = 0; q < NQ; q += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(qsc + q);
                        s[q] = fmaf(fmaf(s[NQ + q], 0.03125f, s[q]), f.x * info.x, info.y);
                        s[q + 1] =
                            fmaf(fmaf(s[NQ + q + 1], 0.03125f, s[q + 1]), f.y * info.x, info.y);
                        s[q + 2] =
                            fmaf(fmaf(s[NQ + q + 2], 0.03125f, s[q + 2]), f.z * info.x, info.y);
                        s[q + 3] =
                            fmaf(fmaf(s[NQ + q + 3], 0.03125f, s[q + 3]), f.w * info.x, info.y);
                    }
                    if (!all) {
#pragma unroll
                        for (int q = 0; q < NQ; ++q) {
                            const int at = T - L + (L > 1 ? sh->row_i[seg & 1][q] : 0);
                            const bool seen =
                                there && pos <= at &&
                                (window <= 0 || pos > at - window || pos < sink ||
                                 ((gmask >> (pos & 63)) & 1ull));
                            if (!seen) s[q] = -INFINITY;
                        }
                    }
                    // largest of the tile, per row
                    {
                        float mine = 0.f;
#pragma unroll
                        for (int q = 0; q < NQ; ++q) {
                            const float m = warp_max(s[q]);
                            if (lane == q) mine = m;
                        }
                        if (lane < NQ) sh->wmax[buf][w][lane] = mine;
                    }
                    // the P buffer and what goes with it are free again
                    if (n >= 2) wait(&sh->o_free[buf], n / 2 - 1);
                    named_barrier(2, 128);
                    bool grew = false;
                    if (lane < NQ) {
                        const float m = fmaxf(fmaxf(sh->wmax[buf][0][lane], sh->wmax[buf][1][lane]),
                                              fmaxf(sh->wmax[buf][2][lane],
                                                    sh->wmax[buf][3][lane]));
                        const float now = m != m ? m : fmaxf(top, m);
                        // factor of this tile (2^8 in its weights), of what came before
                        const float c = m == -INFINITY ? 0.f : exp2f(m - now - 8.f);
                        const float a = top == now ? 1.f : exp2f(top - now);
                        sh->ref[w][lane] = make_float2(m == -INFINITY ? 0.f : m - 8.f, c);
                        sh->grow[w][lane] = a;
                        grew = a != 1.f;
                        top = now;
                        if (w == 0) sh->join[buf][lane] = make_float2(c, a);
                    }
                    grew = __any_sync(0xffffffffu, grew);
                    __syncwarp();
                    if (grew) {
#pragma unroll
                        for (int q = 0; q < NQ; ++q) l[q] *= sh->grow[w][q];
                    }
                    uint32_t hi[NQ / 4], lo_[NQ / 4];
#pragma unroll
                    for (int q = 0; q < NQ; q += 2) {
                        const float4 r = *reinterpret_cast<const float4 *>(&sh->ref[w][q]);
                        const float a = exp2_approx(s[q] - r.x), c = exp2_approx(s[q + 1] - r.z);
                        l[q] = fmaf(a, r.y * info.z, l[q]);
                        l[q + 1] = fmaf(c, r.w * info.z, l[q + 1]);
                        uint32_t h2, l2;
                        e4m3_split2(a * info.w, c * info.w, h2, l2);
                        if (q % 4 == 0) {
                            hi[q / 4] = h2;
                            lo_[q / 4] = l2;
                        } else {
                            hi[q / 4] |= h2 << 16;
                            lo_[q / 4] |= l2 << 16;
                        }
                    }
                    // 16 columns of a key are 16 bytes, keys one after another
                    unsigned char *pk = sP + buf * C::kPBytes + key * 16;
                    if constexpr (NQ == 8) {
                        *reinterpret_cast<uint4 *>(pk) = make_uint4(hi[0], hi[1], lo_[0], lo_[1]);
                    } else {
#pragma unroll
                        for (int g = 0; g < NQ / 16; ++g) {
                            *reinterpret_cast<uint4 *>(pk + g * 2048) = make_uint4(
                                hi[4 * g], hi[4 * g + 1], hi[4 * g + 2], hi[4 * g + 3]);
                            *reinterpret_cast<uint4 *>(pk + (NQ / 16 + g) * 2048) = make_uint4(
                                lo_[4 * g], lo_[4 * g + 1], lo_[4 * g + 2], lo_[4 * g + 3]);
                        }
                    }
                    if (t == tiles - 1) {
                        const float sum = warp_sums<NQ>(l, lane);
                        if (lane < NQ) {
                            sh->lsum[buf][w][lane] = sum;
                            if (w == 0) sh->top[buf][lane] = top;
                        }
                        mbar_arrive_warp(&sh->q_empty[seg & 1]);
                    }
                    fence_proxy_async_smem();
                    mbar_arrive_warp(&sh->p_full[buf]);
                }
            }
        } else {
            // ======================================================== output
            const int w = warp & 3;
            const uint32_t tlane = (uint32_t)(32 * w) << 16;
            const int col = C::kM == 64 ? 16 * w + lane : 32 * w + lane;
            const bool mine = C::kM == 128 || lane < 16;
            int n = 0;
            bool ok = true, first_seg = true;
            auto wait = [&](uint64_t *bar, int phase) {
                return __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)(phase & 1), p.timeout_ns,
                                                         p.err, abort_flag));
            };
            for (; ok && !walk.done(); walk.next(), first_seg = false) {
                float o[C::kHalves][NQ];
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                    for (int q = 0; q < NQ; ++q) o[h][q] = 0.f;
                const int tiles = walk.tiles();
                for (int t = 0; ok && t < tiles; ++t, ++n) {
                    const int buf = n & 1;
                    ok = wait(&sh->p_full[buf], n >> 1) && wait(&sh->o_full[buf], n >> 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h) {
                        float x[C::kN];
                        fb_tmem_ld<C::kN>(
                            tmem + C::kTmemO + (buf * C::kHalves + h) * C::kN + tlane, x);
#pragma unroll
                        for (int q = 0; q < NQ; q += 2) {
                            const float4 f = *reinterpret_cast<const float4 *>(&sh->join[buf][q]);
                            o[h][q] = fmaf(fmaf(x[NQ + q], 0.03125f, x[q]), f.x, o[h][q] * f.y);
                            o[h][q + 1] = fmaf(fmaf(x[NQ + q + 1], 0.03125f, x[q + 1]), f.z,
                                               o[h][q + 1] * f.w);
                        }
                    }
                    if (t == tiles - 1) {
                        const FbUnit u = fb_unit(p, walk.w.unit);
                        const bool whole = walk.w.blk_off == 0 && walk.len == walk.w.nb;
                        const int slot = 2 * blockIdx.x + (first_seg ? 0 : 1);
                        float *part = p.ws_o + (size_t)slot * NQ * D;
#pragma unroll
                        for (int q = 0; q < NQ; ++q) {
                            if (q >= u.rows) break;
                            const float sum = (sh->lsum[buf][0][q] + sh->lsum[buf][1][q]) +
                                              (sh->lsum[buf][2][q] + sh->lsum[buf][3][q]);
                            if (!whole) {
#pragma unroll
                                for (int h = 0; h < C::kHalves; ++h)
                                    if (mine) part[q * D + h * 128 + col] = o[h][q];
                                if (w == 0 && lane == 0)
                                    p.ws_ml[slot * NQ + q] = make_float2(sh->top[buf][q], sum);
                            } else {
                                const int row = u.row0 + q, i = row / p.group, g = row % p.group;
                                __nv_bfloat16 *dst =
                                    p.out + ((size_t)(walk.w.b * p.q_len + i) * p.H_q +
                                             u.kvh * p.group + g) * D;
#pragma unroll
                                for (int h = 0; h < C::kHalves; ++h)
                                    if (mine)
                                        dst[h * 128 + col] = __float2bfloat16_rn(
                                            sum != 0.f ? o[h][q] / sum : 0.f);
                            }
                        }
                    }
                    tc_fence_before();
                    mbar_arrive_warp(&sh->o_free[buf]);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// Joins the partials of the unit that holds the boundary between main CTAs i
// and i + 1 (i = blockIdx.x), if it lies inside one.  The CTAs of a unit's
// boundaries share its values; splits are added in order, so a result does
// not depend on which CTA came first.
constexpr int kFbJoinThreads = 256;
template <int D, int NQ>
__global__ void __launch_bounds__(kFbJoinThreads)
gqa_fp8_block_join_kernel(const GqaFp8BlockParams p) {
    __shared__ PlanScratch sc;
    const int tid = threadIdx.x;
    Visibility vis = p.vis;
    if (vis.window > 0) vis.window += p.q_len - 1;
    const int units = p.H_kv * p.chunks;
    const PlanArgs pa{p.seq_lens, p.B, units, vis, p.max_blocks, p.num_ctas};
    // the lengths were there before the main kernel began
    plan_locate(pa, blockIdx.x + 1, &sc, nullptr, nullptr);
    const long long W = sc.total;
    const int P = working_ctas(W, p.num_ctas);
    pdl_wait_primary();
    if ((int)blockIdx.x + 1 >= P) return;
    const long long x = cta_bound(blockIdx.x + 1, W, P);
    int fb, sb;
    bool bad;
    const int b = sc.seq;
    const int nb = visible_blocks(p.seq_lens[b], vis, p.max_blocks, &fb, &sb, &bad, b);
    const int unit = (int)((x - sc.base) / nb);
    const long long su = sc.base + (long long)unit * nb, eu = su + nb;
    if (x == su) return;
    const int c0 = cta_of(su, W, P), c1 = cta_of(eu - 1, W, P);
    const int slot0 = 2 * c0 + (cta_bound(c0, W, P) == su ? 0 : 1);
    const FbUnit u = fb_unit(p, unit);
    // float4 items of the unit, dealt out over its boundaries' CTAs
    const int items = u.rows * (D / 4), n = c1 - c0;
    for (int it = ((int)blockIdx.x - c0) * kFbJoinThreads + tid; it < items;
         it += n * kFbJoinThreads) {
        const int q = it / (D / 4), c = (it % (D / 4)) * 4;
        float top = -INFINITY;
        for (int k = c0; k <= c1; ++k)
            top = fmaxf(top, p.ws_ml[(k == c0 ? slot0 : 2 * k) * NQ + q].x);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 4
        for (int k = c0; k <= c1; ++k) {
            const int slot = k == c0 ? slot0 : 2 * k;
            const float2 ml = p.ws_ml[slot * NQ + q];
            const float4 v =
                *reinterpret_cast<const float4 *>(p.ws_o + ((size_t)slot * NQ + q) * D + c);
            // a split whose keys the row does not see has top -inf and sum 0
            const float a = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
            sum = fmaf(a, ml.y, sum);
            o.x = fmaf(a, v.x, o.x);
            o.y = fmaf(a, v.y, o.y);
            o.z = fmaf(a, v.z, o.z);
            o.w = fmaf(a, v.w, o.w);
        }
        const float by = sum != 0.f ? 1.f / sum : 0.f;
        const int row = u.row0 + q, i = row / p.group, g = row % p.group;
        __nv_bfloat162 r[2] = {__floats2bfloat162_rn(o.x * by, o.y * by),
                               __floats2bfloat162_rn(o.z * by, o.w * by)};
        *reinterpret_cast<uint2 *>(p.out + ((size_t)(b * p.q_len + i) * p.H_q + u.kvh * p.group +
                                            g) * D + c) = *reinterpret_cast<const uint2 *>(r);
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
    return 2ll * num_ctas * nq * (d * 4 + 8) + 256;
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
    cfg.gridDim = dim3((unsigned)p.num_ctas);
    cfg.blockDim = dim3(kFbThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gqa_fp8_block_kernel<D, NQ, G>, tk, tv, p);
    if (e != cudaSuccess || p.num_ctas == 1) return e;
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
    switch (d) {
        case 64: return fb_launch_d<64>(p, stream);
        case 128: return fb_launch_d<128>(p, stream);
        default: return fb_launch_d<256>(p, stream);
    }
}

}  // namespace attn
