// Internal declarations of the append calls and the 8-bit KV cache.
#pragma once

#include "sv_internal.h"

namespace sv {

// ------------------------------- append -------------------------------------
struct AppendParams {
    const uint16_t *q, *k, *v;     // bf16 bits
    int64_t q_stride, kv_stride;   // elements between rows
    const int32_t *positions;      // [B][N] or null
    const int32_t *new_lens;       // [B] or null
    const float *cos_sin;          // [max_position][R]
    const int32_t *block_table, *ctx_lens;
    uint16_t *q_out;
    void *k_pool, *v_pool;         // bf16 or e4m3
    float *scales;                 // [num_blocks][Hkv][2] (8-bit cache)
    int32_t *status;
    int B, N, Hq, Hkv, D, R, interleaved, max_position, max_blocks, num_blocks;
    int slots;                     // of a head (set by launch_append)
};
cudaError_t launch_append(const AppendParams &p, bool q8, cudaStream_t stream);

// --------------------------- commit, 8-bit ----------------------------------
struct CommitQ8Launch {
    const int32_t *block_table, *ctx_lens, *accept_len, *accept_path;
    int32_t *new_ctx, *status;
    int B, N, Hkv, D, max_blocks, num_blocks, L;
    sv_kv_q8 layer[SV_COMMIT_MAX_LAYERS];
};
cudaError_t launch_kv_commit_q8(const CommitQ8Launch &c, cudaStream_t stream);

// -------------------------- attention, 8-bit --------------------------------
// p.k_pool and p.v_pool hold the e4m3 pools.
size_t attention_q8_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int num_ctas);
cudaError_t launch_attention_q8(const AttnParams &p, const float *scales, cudaStream_t stream);

}  // namespace sv
