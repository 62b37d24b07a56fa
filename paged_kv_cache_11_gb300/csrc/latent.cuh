// latent.cuh -- a cache of one latent row a token: the row's shape, and the launch parameters of its write and of the
// attention of prompts (those of its attention in the absorbed form are in drafted.cuh).
#pragma once

#include "pkv_internal.cuh"

namespace pkv {

// A row of a latent cache: the latent and the key part with the position.
constexpr int kLatentDim = 512, kLatentRope = 64, kLatentRow = kLatentDim + kLatentRope;

// Write into a paged latent cache (latent_append.cu); strides in elements.
struct LatentAppendParams {
    int* err;
    const uint16_t* q;           // 64 values a head
    const uint16_t* kv;          // 512 + 64 values a token
    const int64_t* positions;
    const float* cos_sin;        // [max_position][64]; nullptr: no rotation
    const uint16_t* kv_norm;     // [512] or nullptr
    const int64_t* slot_mapping;
    uint16_t* q_out;
    uint16_t* kv_out;            // [num_tokens][576] or nullptr
    uint16_t* cache;             // [num_slots][576]
    int64_t num_tokens, num_slots, max_position;
    int64_t q_stride, q_head_stride, q_out_stride, q_out_head_stride, kv_stride;
    int num_heads, head_tasks, interleaved;
    float norm_eps;
};
cudaError_t launch_latent_append(const LatentAppendParams& p, int dtype, cudaStream_t stream, int* launches);

// Attention of prompts over expanded keys and values (latent_prompt.cu).
struct LatentPromptParams {
    int* err;
    const int32_t* query_starts; // [num_seqs + 1]
    const int32_t* key_starts;   // [num_seqs + 1]
    const void* values;          // expanded rows: 128 key values, 128 values a head
    void* out;                   // [query tokens][num_heads][128]
    int64_t kv_stride, kv_head_stride;  // elements
    int num_seqs, num_heads;
    int num_queries, num_keys;   // tokens of q; of kv and k_rope
    int max_query_len;
    int sms;
    bool claims;                 // CTAs take the places of others that have not begun
    float scale_log2;
};
cudaError_t launch_latent_prompt(const LatentPromptParams& p, int dtype, const CUtensorMap& tmq, const CUtensorMap& tmkv,
                                 const CUtensorMap& tmr, cudaStream_t stream, int* launches);

}  // namespace pkv
