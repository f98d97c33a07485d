// kv_fp8_block.cu -- append to and read back the block-scaled fp8 cache.
//
// Append: one CTA per (64-token block that a run touches, head, K or V).  A
// block's scale is the power of two that its largest new value asks for, so
// one CTA sees every new row of the block, holds them in registers between
// finding the maximum and writing the codes, and reads each input once.
// Read-back: one CTA per (block, up to 8 heads, K or V), 16-byte stores; 128 MiB
// of codes to bf16 take 70 us, 0.88 of the copy rate (152 us with one head a CTA
// and a thread's 16 values in two stores).
// Both are bound by memory; what is left beside that is the chain of dependent
// loads that finds a CTA its rows (offsets and positions, block table, data).
#include <cuda_fp8.h>

#include "fp8_block.cuh"

namespace attn {

constexpr int kRunThreads = 256;      // of the read-back

// Part of a run that falls into one block.
struct BlockRun {
    int b;          // sequence
    int src;        // row of the block's first new row among the call's rows
    int r0, r1;     // rows [r0, r1) of the block
    int slot;       // table slot, -1: not one of the sequence's blocks
    bool replaced;  // a later block of the run takes the slot
};

// First global slot of sequence b that names block blk (the first position of
// its global set in it), -1: none.  One warp, all 32 lanes; rows of up to 64.
__device__ __forceinline__ int named_slot(const Visibility &v, int b, int blk) {
    const int32_t *g = global_row(v, b);
    const int lane = threadIdx.x & 31;
    int prev = -1;                             // the entry before the 32 looked at
    for (int k0 = 0; k0 < v.n_g; k0 += 32) {
        const int pos = k0 + lane < v.n_g ? g[k0 + lane] : -1;
        const int up = __shfl_up_sync(0xffffffffu, pos, 1);
        // the row ends at the first entry that does not exceed the one before
        const unsigned stop = __ballot_sync(0xffffffffu, pos <= (lane ? up : prev));
        const unsigned hit = __ballot_sync(0xffffffffu, pos / kBlockSize == blk) &
                             (stop ? (stop & (0u - stop)) - 1u : 0xffffffffu);
        if (hit) return k0 + __ffs(hit) - 1;
        if (stop) return -1;
        prev = __shfl_sync(0xffffffffu, pos, 31);
    }
    return -1;
}

// The part of a run that CTA column x of the grid works on.  Sequence b owns
// columns offsets[b] / 64 + 2 b and on, up to the next sequence's: a run of n
// rows touches at most (n + 62) / 64 + 1 blocks, which is never more than the
// floor(o' / 64) - floor(o / 64) + 2 columns between o and o' = o + n.  So the
// columns need no prefix sum over block counts; 32 lanes probe the offsets at
// once to find b (one round for up to 32 sequences, two for 1024), and the
// last round brings the run's end and position along.  (Offsets that decrease
// are reported, and may hide columns of other sequences from the search: their
// blocks are left out, never written twice.)  Every thread of the
// CTA gets the same answer; false where the column has no work.  flag: this
// thread reports what is wrong with the run.  rest: the rows behind the last
// sequence are handed out as a run without blocks.
//
// In a ring with a global set a block that holds a global position has a slot
// of its own, which names it also when the ring has moved past it.  A reader
// goes there.  A writer goes there for the blocks that lie before the window
// when the run is done (the decode then reads them there, and a run longer than
// the ring replaces them itself), else through the ring like kv_append_ext.
// G: the call has such a table (compiled out of the other kernels, which it
// would cost 5 % of a ragged append's time: 14.4 against 13.7 us).
template <bool G>
__device__ __forceinline__ bool locate_run(const KvRunParams &p, int x, bool flag, bool rest,
                                           bool reading, BlockRun *out) {
    const int lane = threadIdx.x & 31;
    int b, o0, n, ord, pos;
    if (p.offsets) {
        // the first column reports offsets that are wrong: the search below may
        // not meet the sequence that has them
        if (x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
            for (int i = threadIdx.x; i < p.B; i += blockDim.x) {
                const int a = p.offsets[i], e = p.offsets[i + 1];
                if (a < 0 || e < a || e > p.n_tokens) raise_error(p.err, kErrBadSeqLen);
            }
        int lo = 0, hi = p.B + (rest ? 1 : 0), o1;
        for (;;) {
            const int step = (hi - lo + 31) / 32;
            const int i = lo + lane * step;
            const bool in = i < hi;
            const int o = in ? p.offsets[i] : 0;
            int end = 0, at = -1;
            if (step == 1 && in) {
                end = i < p.B ? p.offsets[i + 1] : p.n_tokens;
                if (i < p.B) at = p.positions[i];
            }
            const unsigned m =
                __ballot_sync(0xffffffffu, in && (long long)o / 64 + 2ll * i <= x);
            if (m == 0) return false;              // before the first row
            const int sel = 31 - __clz(m);
            if (step == 1) {
                b = lo + sel;
                o0 = __shfl_sync(0xffffffffu, o, sel);
                o1 = __shfl_sync(0xffffffffu, end, sel);
                pos = __shfl_sync(0xffffffffu, at, sel);
                break;
            }
            lo += sel * step;
            hi = min(hi, lo + step);
        }
        if (o0 < 0 || o1 < o0 || o1 > p.n_tokens) return false;
        n = o1 - o0;
        ord = (int)(x - ((long long)o0 / 64 + 2ll * b));
    } else {
        b = x;
        o0 = b;
        n = 1;
        ord = 0;
        pos = p.positions[b];
    }
    if (n == 0 || ord < 0) return false;
    if (pos < 0 || (long long)pos + n > (1ll << 31) - 64) {
        if (flag && ord == 0 && b < p.B) raise_error(p.err, kErrBadBlock);
        // a run that starts before the sequence has no block of its own: its
        // rows are handed out 64 at a time so that a reader can zero them
        if ((long long)ord * 64 >= n) return false;
        *out = BlockRun{b, o0 + ord * 64, 0, min(64, n - ord * 64), -1, false};
        return true;
    }
    const int lead = pos % kBlockSize, blk = pos / kBlockSize + ord;
    const int last = (int)(((long long)pos + n - 1) / kBlockSize);
    if (blk > last) return false;
    int slot = table_slot(p.vis, blk);
    bool replaced = p.vis.ring > 0 && slot >= ring_base(p.vis) && blk + p.vis.ring <= last;
    if (G && (reading || blk < window_lo(p.vis, pos + n) / kBlockSize)) {
        const int named = named_slot(p.vis, b, blk);
        if (named >= 0) {
            slot = named;
            replaced = false;
        }
    }
    *out = BlockRun{b,
                    o0 + (ord == 0 ? 0 : ord * kBlockSize - lead),
                    ord == 0 ? lead : 0,
                    min(kBlockSize, lead + n - ord * kBlockSize),
                    slot < p.max_blocks ? slot : -1,
                    replaced};
    return true;
}

// Physical block of a part, -1 where there is none.  A reader reports replaced
// blocks too; a writer just leaves them out.
__device__ __forceinline__ int run_block(const KvRunParams &p, const BlockRun &br, bool flag,
                                         bool reading) {
    int phys = -1;
    if (br.slot >= 0 && !br.replaced) {
        phys = p.block_table[(size_t)br.b * p.max_blocks + br.slot];
        if (phys < 0 || phys >= p.num_blocks) phys = -1;
    }
    if (phys < 0 && flag && br.b < p.B && (reading || !br.replaced))
        raise_error(p.err, kErrBadBlock);
    return phys;
}

// Smallest power of two s >= 2^-126 with amax <= 448 s; 0 for amax = 0.
// 448 = 1.75 x 2^8: for amax = m 2^e with 1 <= m < 2 that is 2^(e - 8) up to
// m = 1.75 and 2^(e - 7) above, read off the bits.
__device__ __forceinline__ float block_scale(float amax) {
    if (!(amax > 0.f)) return 0.f;
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;        // infinities and NaN: 0
}

// Values of a 16-byte chunk.
template <typename T> struct In {
    static constexpr int kE = 16 / sizeof(T);
};

// Values times `by` as E4M3 codes: nearest even, saturated, NaN kept.
__device__ __forceinline__ uint32_t four_codes(const float *f, float by) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0] * by, f[1] * by),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2] * by, f[3] * by),
                                                 __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
__device__ __forceinline__ void to_codes(const float *f, float by, uint4 *c) {
    *c = make_uint4(four_codes(f, by), four_codes(f + 4, by), four_codes(f + 8, by),
                    four_codes(f + 12, by));
}

// The numbers that codes are (every E4M3 number is an f16 number).
__device__ __forceinline__ void four_values(uint32_t w, float *f) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
}
__device__ __forceinline__ void from_codes(const uint2 &c, float *f) {
    four_values(c.x, f);
    four_values(c.y, f + 4);
}
__device__ __forceinline__ void from_codes(const uint32_t &c, float *f) { four_values(c, f); }
__device__ __forceinline__ void from_codes(const uint4 &c, float *f) {
    four_values(c.x, f);
    four_values(c.y, f + 4);
    four_values(c.z, f + 8);
    four_values(c.w, f + 12);
}

template <int E> struct CodesOf;
template <> struct CodesOf<4> { using type = uint32_t; };
template <> struct CodesOf<8> { using type = uint2; };
template <> struct CodesOf<16> { using type = uint4; };

// D threads; thread t takes 16 values of input rows t / (D / 16) + 16 k.  Few
// threads with much in flight each: what bounds the kernel beside HBM is the
// time of a CTA (three loads that wait for one another), so the bytes that all
// resident CTAs hold together count.  Measured: 256 MiB of fp32 rows of d = 64
// 106 to 109 us (0.94 to 0.97 of the copy rate; 124 with 256 threads of 4 values), 107 MB of
// bf16 rows of d = 64 32 us (0.76; 47 with 256 threads of 8 values).
template <typename T, int D, bool G>
__global__ void __launch_bounds__(D, (sizeof(T) == 2 ? 1024 : 640) / D)
kv_append_fp8_block_kernel(const KvAppendBlockParams p) {
    constexpr int kE = 16, kC = sizeof(T);                 // values, 16-byte chunks of them
    constexpr int kTpr = D / kE, kRows = D / kTpr, kPasses = kBlockSize / kRows;
    using Codes = typename CodesOf<kE>::type;
    __shared__ float s_max[D / 32];
    const int tid = threadIdx.x, h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    pdl_wait_primary();
    pdl_launch_dependents();
    BlockRun br;
    const bool flag = tid == 0 && h == 0 && !is_v;
    if (!locate_run<G>(p.run, blockIdx.x, flag, false, false, &br)) return;
    const T *src = static_cast<const T *>(is_v ? p.v_new : p.k_new);
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const int col = (tid % kTpr) * kE, row0 = tid / kTpr;

    // the inputs need the run only, not the block: their loads go out together
    // with the table's
    uint4 x[kPasses][kC];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int r = row0 + kRows * k;
        const bool in = r >= br.r0 && r < br.r1;
        const uint4 *at = reinterpret_cast<const uint4 *>(src + (br.src + (r - br.r0)) * stride +
                                                          h * D + col);
#pragma unroll
        for (int c = 0; c < kC; ++c) x[k][c] = in ? __ldg(at + c) : make_uint4(0u, 0u, 0u, 0u);
    }
    auto values = [&](int k, float *f) {
#pragma unroll
        for (int c = 0; c < kC; ++c) Chunk<T>::unpack(x[k][c], f + c * In<T>::kE);
    };
    const int phys = run_block(p.run, br, flag, false);
    if (phys < 0) return;
    const size_t tile = (size_t)phys * p.run.H_kv + h;
    float *scale = (is_v ? p.v_scale : p.k_scale) + tile;
    uint8_t *dst = (is_v ? p.v_cache : p.k_cache) + tile * (kBlockSize * D);
    const float held = br.r0 > 0 ? *scale : 0.f;
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        float f[kE];
        values(k, f);
#pragma unroll
        for (int i = 0; i < kE; ++i) amax = fmaxf(amax, finite_abs(f[i]));
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));   // not negative
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < D / 32; ++w) amax = fmaxf(amax, s_max[w]);

    const float old = held > 0.f ? held : 0.f;
    const float s = fmaxf(old, block_scale(amax));
    const float by = s > 0.f ? 1.f / s : 1.f;          // exact: a power of two
    if (br.r0 > 0 && s != old) {
        // the rows begun earlier, under the larger scale
        const float ratio = old * by;
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
            const int r = row0 + kRows * k;
            if (r < br.r0) {
                Codes *at = reinterpret_cast<Codes *>(dst + r * D + col);
                float f[kE];
                from_codes(*at, f);
                to_codes(f, ratio, at);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int r = row0 + kRows * k;
        if (r >= br.r0 && r < br.r1) {
            float f[kE];
            values(k, f);
            to_codes(f, by, reinterpret_cast<Codes *>(dst + r * D + col));
        }
    }
    if (tid == 0) *scale = s;
}

__device__ __forceinline__ uint4 out_chunk(const float *f, __nv_bfloat16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 out_chunk(const float *f, float) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
}

// A CTA reads 1 << heads_log2 heads of a block; a thread keeps to one head and
// one 16-byte chunk of the output row, so that its scale stays in a register
// and neighbours write neighbouring chunks.
template <typename T, int D, bool G>
__global__ void __launch_bounds__(kRunThreads)
kv_read_fp8_block_kernel(const KvReadBlockParams p, int heads_log2) {
    constexpr int kE = In<T>::kE, kTpr = D / kE, kUnits = kRunThreads / kTpr;
    constexpr int kAhead = 4;
    using Codes = typename CodesOf<kE>::type;
    const int tid = threadIdx.x, unit = tid / kTpr;
    const int h = (blockIdx.y << heads_log2) + (unit & ((1 << heads_log2) - 1));
    const int col = (tid % kTpr) * kE, row0 = unit >> heads_log2, rows = kUnits >> heads_log2;
    const bool is_v = blockIdx.z != 0;
    const size_t pitch = (size_t)p.run.H_kv * D;
    T *dst = static_cast<T *>(is_v ? p.v_out : p.k_out) + (size_t)h * D + col;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (p.zero_rest && p.run.offsets && blockIdx.x == 0) {
        const int n = min(p.run.offsets[0], p.run.n_tokens);        // rows before the first
        for (int r = row0; r < n; r += rows)
            *reinterpret_cast<uint4 *>(dst + r * pitch) = make_uint4(0u, 0u, 0u, 0u);
    }
    BlockRun br;
    const bool flag = tid == 0 && blockIdx.y == 0 && !is_v;
    if (!locate_run<G>(p.run, blockIdx.x, flag, p.zero_rest, true, &br)) return;
    const int phys = run_block(p.run, br, flag, true);
    dst += ((int64_t)br.src - br.r0) * (int64_t)pitch;
    if (phys < 0) {
        for (int r = br.r0 + row0; r < br.r1; r += rows)
            *reinterpret_cast<uint4 *>(dst + r * pitch) = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const size_t tile = (size_t)phys * p.run.H_kv + h;
    const float s = (is_v ? p.v_scale : p.k_scale)[tile];
    const uint8_t *src = (is_v ? p.v_cache : p.k_cache) + tile * (kBlockSize * D) + col;
    for (int r = br.r0 + row0; r < br.r1; r += kAhead * rows) {
        Codes c[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (r + k * rows < br.r1)
                c[k] = __ldg(reinterpret_cast<const Codes *>(src + (r + k * rows) * D));
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (r + k * rows >= br.r1) break;
            float f[kE];
            from_codes(c[k], f);
#pragma unroll
            for (int i = 0; i < kE; ++i) f[i] *= s;
            *reinterpret_cast<uint4 *>(dst + (r + k * rows) * pitch) = out_chunk(f, T());
        }
    }
}

namespace {

// CTA columns: one per sequence without offsets, else to the end of the last
// sequence (see locate_run), and of the rows behind it.
unsigned run_columns(const KvRunParams &r, bool rest) {
    return (unsigned)(r.offsets ? (long long)r.n_tokens / 64 + 2ll * r.B + (rest ? 1 : 0) : r.B);
}

// Programmatic launch: the kernels wait for what came before themselves, and
// what comes next may be set up while they run.
template <typename K, typename... A>
cudaError_t launch_run(K kernel, dim3 grid, int threads, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A ring with a global set: see locate_run.
bool has_global_slots(const Visibility &v) { return v.ring > 0 && v.n_g > 0; }

template <typename T, bool G>
cudaError_t append_d(const KvAppendBlockParams &p, int d, cudaStream_t s) {
    const dim3 g(run_columns(p.run, false), (unsigned)p.run.H_kv, 2u);
    switch (d) {
        case 64: return launch_run(kv_append_fp8_block_kernel<T, 64, G>, g, 64, s, p);
        case 128: return launch_run(kv_append_fp8_block_kernel<T, 128, G>, g, 128, s, p);
        default: return launch_run(kv_append_fp8_block_kernel<T, 256, G>, g, 256, s, p);
    }
}
template <typename T>
cudaError_t append_t(const KvAppendBlockParams &p, int d, cudaStream_t s) {
    return has_global_slots(p.run.vis) ? append_d<T, true>(p, d, s) : append_d<T, false>(p, d, s);
}

template <typename T, bool G>
cudaError_t read_d(const KvReadBlockParams &p, int d, cudaStream_t s) {
    // Heads of a CTA: the largest power of two that divides them, up to 32 KB
    // of codes, so that finding the rows is paid once for many.
    int lg = 0;
    while ((2 << lg) * kBlockSize * d <= 32768 && p.run.H_kv % (2 << lg) == 0) ++lg;
    const dim3 g(run_columns(p.run, p.zero_rest), (unsigned)(p.run.H_kv >> lg), 2u);
    switch (d) {
        case 64: return launch_run(kv_read_fp8_block_kernel<T, 64, G>, g, kRunThreads, s, p, lg);
        case 128: return launch_run(kv_read_fp8_block_kernel<T, 128, G>, g, kRunThreads, s, p, lg);
        default: return launch_run(kv_read_fp8_block_kernel<T, 256, G>, g, kRunThreads, s, p, lg);
    }
}
template <typename T>
cudaError_t read_t(const KvReadBlockParams &p, int d, cudaStream_t s) {
    return has_global_slots(p.run.vis) ? read_d<T, true>(p, d, s) : read_d<T, false>(p, d, s);
}

}  // namespace

cudaError_t launch_kv_append_fp8_block(const KvAppendBlockParams &p, int d, bool bf16,
                                       cudaStream_t stream) {
    return bf16 ? append_t<__nv_bfloat16>(p, d, stream) : append_t<float>(p, d, stream);
}

cudaError_t launch_kv_read_fp8_block(const KvReadBlockParams &p, int d, bool bf16,
                                     cudaStream_t stream) {
    return bf16 ? read_t<__nv_bfloat16>(p, d, stream) : read_t<float>(p, d, stream);
}

}  // namespace attn
