// gqa_fp8_block.cu -- decode attention over the block-scaled fp8 cache.
//
// One CTA per (sequence, query position, query head); its four warps take the
// visible keys in turn, each lane D / 32 values of a row, with the running
// maximum and sum of a one-pass softmax, merged over the warps at the end.
#include <cuda_fp8.h>

#include "fp8_block.cuh"

namespace attn {

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half *>(&h));
}

template <int D>
__global__ void __launch_bounds__(128) gqa_fp8_block_kernel(const GqaFp8BlockParams p) {
    constexpr int kE = D / 32;
    __shared__ float s_m[4], s_l[4], s_o[4][D];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hq = blockIdx.x % p.H_q, bi = blockIdx.x / p.H_q;
    const int b = bi / p.q_len, i = bi % p.q_len, h = hq / p.group;
    Visibility vis = p.vis;
    if (vis.window > 0) vis.window += p.q_len - 1;        // what any query sees
    int first, sink_blks;
    bool bad;
    const int T = p.seq_lens[b];
    const int nb = visible_blocks(T, vis, p.max_blocks, &first, &sink_blks, &bad, b);
    if (bad && tid == 0) raise_error(p.err, kErrBadSeqLen);
    const int at = T - p.q_len + i;
    const bool global = global_query(p.vis, b, T);
    const int lo = p.vis.window > 0 && !global ? at - p.vis.window + 1 : 0;
    float q[kE], o[kE], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        q[e] = __bfloat162float(p.q[(int64_t)bi * p.q_stride + hq * D + lane * kE + e]);
        o[e] = 0.f;
    }
    for (int v = 0; v < nb; ++v) {
        const bool early = v < sink_blks;
        const int blk = !early ? first + v - sink_blks
                               : (p.vis.n_g > 0 ? global_block(vis, b, v) : v);
        const int slot = early && p.vis.n_g > 0 && p.vis.ring > 0 ? global_slot(vis, b, v)
                                                                  : table_slot(vis, blk);
        const int phys = p.block_table[(size_t)b * p.max_blocks + slot];
        if (phys < 0 || phys >= p.num_blocks) {
            if (tid == 0) raise_error(p.err, kErrBadBlock);
            continue;
        }
        const unsigned long long gmask = p.vis.n_g > 0 ? global_mask(vis, b, blk, lane) : 0ull;
        const size_t tile = (size_t)phys * p.H_kv + h;
        const float ks = p.k_scale[tile] * p.scale_log2, vs = p.v_scale[tile];
        for (int t = warp; t < kBlockSize; t += 4) {
            const int pos = blk * kBlockSize + t;
            if (pos > at) break;
            if (pos < lo && pos >= p.vis.sink && !((gmask >> t) & 1ull)) continue;
            const uint8_t *kr = p.k_cache + (tile * kBlockSize + t) * D + lane * kE;
            const uint8_t *vr = p.v_cache + (tile * kBlockSize + t) * D + lane * kE;
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < kE; ++e) s += q[e] * e4m3_value(kr[e]);
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
            s *= ks;
            const float m2 = fmaxf(m, s);
            const float a = m == m2 ? 1.f : exp2f(m - m2), w = exp2f(s - m2);
            l = l * a + w;
#pragma unroll
            for (int e = 0; e < kE; ++e) o[e] = o[e] * a + w * vs * e4m3_value(vr[e]);
            m = m2;
        }
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) s_o[warp][lane * kE + e] = o[e];
    __syncthreads();
    const float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    float total = 0.f, w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        w[k] = s_m[k] == -INFINITY ? 0.f : exp2f(s_m[k] - top);
        total += w[k] * s_l[k];
    }
    for (int c = tid; c < D; c += 128) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) x += w[k] * s_o[k][c];
        p.out[((size_t)bi * p.H_q + hq) * D + c] =
            __float2bfloat16_rn(total != 0.f ? x / total : 0.f);
    }
}

cudaError_t launch_gqa_fp8_block(const GqaFp8BlockParams &p, int d, cudaStream_t stream) {
    const unsigned grid = (unsigned)((long long)p.B * p.q_len * p.H_q);
    switch (d) {
        case 64: gqa_fp8_block_kernel<64><<<grid, 128, 0, stream>>>(p); break;
        case 128: gqa_fp8_block_kernel<128><<<grid, 128, 0, stream>>>(p); break;
        default: gqa_fp8_block_kernel<256><<<grid, 128, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace attn
