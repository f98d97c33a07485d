// kv_fp8_block.cu -- append to and read back the block-scaled fp8 cache.
//
// One CTA per (64-token block that a run touches, head, K or V): a block's
// scale is the power of two that its largest new value asks for, so one CTA
// sees every new row of the block, holds them in registers between finding
// the maximum and writing the codes, and reads each input once.
#include <cuda_fp8.h>

#include "fp8_block.cuh"

namespace attn {

// Part of a run that falls into one block.
struct BlockRun {
    int src;        // input row of the block's first new row
    int r0, r1;     // rows [r0, r1) of the block
    int phys;       // physical block, -1: not there (flagged) or nothing to do
};

// The part of a run that CTA column x of the grid works on.  Sequence b owns
// columns offsets[b] / 64 + 2 b and on, up to the next sequence's: a run of n
// rows touches at most (n + 62) / 64 + 1 blocks, which is never more than the
// floor(o' / 64) - floor(o / 64) + 2 columns between o and o' = o + n.  So the
// columns need no prefix sum over block counts; 32 lanes probe the offsets at
// once to find b (two rounds for up to 1024 sequences).  Every thread of the
// CTA gets the same answer; false where the column has no work.  flag: this
// thread reports what is wrong with the run.  reading: rows whose ring slot a
// later block of the run holds are an error (a writer just leaves them out).
__device__ __forceinline__ bool locate_run(const KvRunParams &p, int x, bool flag, bool reading,
                                           BlockRun *out) {
    const int lane = threadIdx.x & 31;
    int b, o0, n, ord;
    if (p.offsets) {
        // the first column reports offsets that are wrong: the search below may
        // not meet the sequence that has them
        if (x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
            for (int i = threadIdx.x; i < p.B; i += blockDim.x) {
                const int a = p.offsets[i], e = p.offsets[i + 1];
                if (a < 0 || e < a || e > p.n_tokens) raise_error(p.err, kErrBadSeqLen);
            }
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int i = lo + lane * step;
            const bool below = i < hi && (long long)p.offsets[i] / 64 + 2ll * i <= x;
            const unsigned m = __ballot_sync(0xffffffffu, below);
            if (m == 0) return false;              // before the first row
            lo += (31 - __clz(m)) * step;
            hi = min(hi, lo + step);
        }
        b = lo;
        o0 = p.offsets[b];
        const int o1 = p.offsets[b + 1];
        if (o0 < 0 || o1 < o0 || o1 > p.n_tokens) return false;
        n = o1 - o0;
        const long long first = (long long)o0 / 64 + 2ll * b;
        if (x < first) return false;
        ord = (int)(x - first);
    } else {
        b = x;
        o0 = b;
        n = 1;
        ord = 0;
    }
    if (n == 0) return false;
    const int pos = p.positions[b];
    if (pos < 0 || (long long)pos + n > (1ll << 31) - 64) {
        if (flag && ord == 0) raise_error(p.err, kErrBadBlock);
        // a run that starts before the sequence has no block of its own: its
        // rows are handed out 64 at a time so that a reader can zero them
        if (ord * 64 >= n) return false;
        *out = BlockRun{o0 + ord * 64, 0, min(64, n - ord * 64), -1};
        return true;
    }
    const int lead = pos % kBlockSize, blk = pos / kBlockSize + ord;
    const int last = (int)(((long long)pos + n - 1) / kBlockSize);
    if (blk > last) return false;
    const int r0 = ord == 0 ? lead : 0;
    const int r1 = min(kBlockSize, lead + n - ord * kBlockSize);
    int phys = -1;
    const int slot = table_slot(p.vis, blk);
    // a later block of this run takes the same ring slot
    const bool replaced = p.vis.ring > 0 && slot >= ring_base(p.vis) && blk + p.vis.ring <= last;
    if (slot >= 0 && slot < p.max_blocks && !replaced) {
        phys = p.block_table[(size_t)b * p.max_blocks + slot];
        if (phys < 0 || phys >= p.num_blocks) phys = -1;
    }
    if (phys < 0 && flag && (reading || !replaced)) raise_error(p.err, kErrBadBlock);
    *out = BlockRun{o0 + (ord == 0 ? 0 : ord * kBlockSize - lead), r0, r1, phys};
    return true;
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

// 16 consecutive input values.
template <typename T> struct In16;
template <> struct In16<__nv_bfloat16> {
    uint4 v[2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        v[0] = __ldg(reinterpret_cast<const uint4 *>(p));
        v[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float *f) const {
        Chunk<__nv_bfloat16>::unpack(v[0], f);
        Chunk<__nv_bfloat16>::unpack(v[1], f + 8);
    }
};
template <> struct In16<float> {
    uint4 v[4];
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(float *f) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) Chunk<float>::unpack(v[i], f + 4 * i);
    }
};

// 16 values times `by` as E4M3 codes: nearest even, saturated, NaN kept.
__device__ __forceinline__ uint4 to_codes(const float *f, float by) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(f[4 * i] * by, f[4 * i + 1] * by), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(f[4 * i + 2] * by, f[4 * i + 3] * by), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The numbers that 16 codes are (every E4M3 number is an f16 number).
__device__ __forceinline__ void from_codes(const uint4 &c, float *f) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
}

// D threads; thread t takes 16 values of rows t / (D / 16) + 16 k, k < 4.
template <typename T, int D>
__global__ void __launch_bounds__(D) kv_append_fp8_block_kernel(const KvAppendBlockParams p) {
    constexpr int kTpr = D / 16, kRows = D / kTpr, kPasses = kBlockSize / kRows;
    __shared__ float s_max[D / 32];
    const int tid = threadIdx.x, h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    BlockRun br;
    if (!locate_run(p.run, blockIdx.x, tid == 0 && h == 0 && !is_v, false, &br)) return;
    if (br.phys < 0) return;
    const T *src = static_cast<const T *>(is_v ? p.v_new : p.k_new);
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const size_t tile = (size_t)br.phys * p.run.H_kv + h;
    float *scale = (is_v ? p.v_scale : p.k_scale) + tile;
    uint8_t *dst = (is_v ? p.v_cache : p.k_cache) + tile * (kBlockSize * D);
    const float held = *scale;
    const int col = (tid % kTpr) * 16, row0 = tid / kTpr;

    In16<T> x[kPasses];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int r = row0 + kRows * k;
        if (r >= br.r0 && r < br.r1)
            x[k].load(src + (br.src + (r - br.r0)) * stride + h * D + col);
        else
            x[k].zero();
    }
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        float f[16];
        x[k].get(f);
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(f[i]));
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < D / 32; ++w) amax = fmaxf(amax, s_max[w]);

    const float old = br.r0 > 0 && held > 0.f ? held : 0.f;
    const float s = fmaxf(old, block_scale(amax));
    const float by = s > 0.f ? 1.f / s : 1.f;          // exact: a power of two
    if (br.r0 > 0 && s != old) {
        // the rows begun earlier, under the larger scale
        const float ratio = old * by;
#pragma unroll
        for (int k = 0; k < kPasses; ++k) {
            const int r = row0 + kRows * k;
            if (r < br.r0) {
                uint4 *at = reinterpret_cast<uint4 *>(dst + r * D + col);
                float f[16];
                from_codes(*at, f);
                *at = to_codes(f, ratio);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int r = row0 + kRows * k;
        if (r >= br.r0 && r < br.r1) {
            float f[16];
            x[k].get(f);
            *reinterpret_cast<uint4 *>(dst + r * D + col) = to_codes(f, by);
        }
    }
    if (tid == 0) *scale = s;
}

__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float *f) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void store16(float *p, const float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4 *>(p)[i] =
            make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(D) kv_read_fp8_block_kernel(const KvReadBlockParams p) {
    constexpr int kTpr = D / 16, kRows = D / kTpr, kPasses = kBlockSize / kRows;
    const int tid = threadIdx.x, h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    BlockRun br;
    if (!locate_run(p.run, blockIdx.x, tid == 0 && h == 0 && !is_v, true, &br)) return;
    const bool gone = br.phys < 0;
    const size_t tile = (size_t)(gone ? 0 : br.phys) * p.run.H_kv + h;
    const float s = gone ? 0.f : (is_v ? p.v_scale : p.k_scale)[tile];
    const uint8_t *src = (is_v ? p.v_cache : p.k_cache) + tile * (kBlockSize * D);
    T *dst = static_cast<T *>(is_v ? p.v_out : p.k_out);
    const int col = (tid % kTpr) * 16, row0 = tid / kTpr;
    uint4 c[kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int r = row0 + kRows * k;
        c[k] = !gone && r >= br.r0 && r < br.r1
                   ? __ldg(reinterpret_cast<const uint4 *>(src + r * D + col))
                   : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
        const int r = row0 + kRows * k;
        if (r < br.r0 || r >= br.r1) continue;
        float f[16];
        from_codes(c[k], f);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] *= s;
        store16(dst + ((size_t)(br.src + (r - br.r0)) * p.run.H_kv + h) * D + col, f);
    }
}

namespace {

// CTA columns: one per sequence without offsets, else the last sequence's end
// (see locate_run).
dim3 run_grid(const KvRunParams &r) {
    const long long cols = r.offsets ? (long long)r.n_tokens / 64 + 2ll * r.B : r.B;
    return dim3((unsigned)cols, (unsigned)r.H_kv, 2u);
}

template <typename T>
void append_d(const KvAppendBlockParams &p, int d, cudaStream_t s) {
    const dim3 g = run_grid(p.run);
    switch (d) {
        case 64: kv_append_fp8_block_kernel<T, 64><<<g, 64, 0, s>>>(p); break;
        case 128: kv_append_fp8_block_kernel<T, 128><<<g, 128, 0, s>>>(p); break;
        default: kv_append_fp8_block_kernel<T, 256><<<g, 256, 0, s>>>(p); break;
    }
}

template <typename T>
void read_d(const KvReadBlockParams &p, int d, cudaStream_t s) {
    const dim3 g = run_grid(p.run);
    switch (d) {
        case 64: kv_read_fp8_block_kernel<T, 64><<<g, 64, 0, s>>>(p); break;
        case 128: kv_read_fp8_block_kernel<T, 128><<<g, 128, 0, s>>>(p); break;
        default: kv_read_fp8_block_kernel<T, 256><<<g, 256, 0, s>>>(p); break;
    }
}

}  // namespace

cudaError_t launch_kv_append_fp8_block(const KvAppendBlockParams &p, int d, bool bf16,
                                       cudaStream_t stream) {
    if (bf16)
        append_d<__nv_bfloat16>(p, d, stream);
    else
        append_d<float>(p, d, stream);
    return cudaGetLastError();
}

cudaError_t launch_kv_read_fp8_block(const KvReadBlockParams &p, int d, bool bf16,
                                     cudaStream_t stream) {
    if (bf16)
        read_d<__nv_bfloat16>(p, d, stream);
    else
        read_d<float>(p, d, stream);
    return cudaGetLastError();
}

}  // namespace attn
