// fp8_block.cuh -- the block-scaled fp8 cache: E4M3 codes [num_blocks][H_kv]
// [64][d] with one fp32 scale per (block, head); parameters and launches of
// its append, read-back and decode kernels.
#pragma once

#include <cuda.h>

#include "plan.cuh"

namespace attn {

// The driver's tensor-map encoder (null where it cannot be had), looked up
// once by gqa_tc.cu.
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);
EncodeTiledFn tc_encode_fn();

struct KvRunParams {
    const int32_t *positions;     // [B] first position of sequence b's run
    const int32_t *offsets;       // [B + 1] rows of sequence b, or null: row b
    const int32_t *block_table;
    unsigned *err;
    int B, n_tokens, H_kv, max_blocks, num_blocks;
    Visibility vis;
};

struct KvAppendBlockParams {
    KvRunParams run;
    const void *k_new, *v_new;    // [n_tokens][H_kv][d], rows k_stride / v_stride apart
    int64_t k_stride, v_stride;   // elements
    uint8_t *k_cache, *v_cache;
    float *k_scale, *v_scale;
};

struct KvReadBlockParams {
    KvRunParams run;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    void *k_out, *v_out;          // [n_tokens][H_kv][d]
    bool zero_rest;               // rows that no sequence owns become zeros
};

cudaError_t launch_kv_append_fp8_block(const KvAppendBlockParams &p, int d, bool bf16,
                                       cudaStream_t stream);
cudaError_t launch_kv_read_fp8_block(const KvReadBlockParams &p, int d, bool bf16,
                                     cudaStream_t stream);

// Most CTAs of a decode launch: its workspace begins with a cut for each.
constexpr int kFp8BlockMaxCtas = 512;

// A unit cut at the end of a CTA's range: the CTAs that hold it, the first
// one's partial, sequence and unit; last < first where nothing is cut.
struct FbCut {
    int first, last, slot, b, unit;
};

struct GqaFp8BlockParams {
    const __nv_bfloat16 *q;       // [B][q_len][H_q][d], q_stride elements between positions
    int64_t q_stride;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *seq_lens, *block_table;
    __nv_bfloat16 *out;           // [B][q_len][H_q][d]
    unsigned *err;
    float scale_log2;             // softmax scale x log2(e)
    int B, q_len, H_q, H_kv, group, max_blocks, num_blocks;
    Visibility vis;               // of a single query; the kernels widen the window by q_len - 1
    int num_ctas;
    unsigned long long timeout_ns;
    int force_timeout;            // testing: each CTA waits for something that never comes
    // filled by the launch: the query rows of a K/V head (group x q_len) in
    // chunks of chunk_rows; partials [2 num_ctas][columns][d] with what they
    // are relative to, the largest score, and the sum of weights relative to it
    int chunk_rows, chunks;
    float *ws_o;
    float4 *ws_ml;
    FbCut *ws_cut;                // the unit cut at each CTA's end
    bool whole_units;             // one CTA per unit, nothing split
    bool small_plan;              // few sequences, a list that 32 bits count
};

// Workspace of a launch over num_ctas CTAs with `rows` query rows per K/V head.
int64_t fp8_block_workspace_bytes(int num_ctas, int rows, int d);

// Events that a caller wants recorded around the main kernel (null: none).
struct FbEvents {
    cudaEvent_t start, stop;
};

cudaError_t launch_gqa_fp8_block(const GqaFp8BlockParams &p, int d, void *workspace,
                                 const FbEvents &events, cudaStream_t stream);

}  // namespace attn
