/*
 * pagedkv.h -- C ABI of libpagedkv.so: the decode hot path of a paged KV
 * cache on one GPU (sm_103a).
 *
 * What the operations are (web pages on paged KV caches; page title, then
 * section):
 *   - tonho.wtf "vllm", "como funciona": the KV cache of a sequence is cut
 *     into fixed-size blocks (16 tokens by default) that are slices of one
 *     GPU pool; a per-sequence block table maps logical blocks to physical
 *     ones; a new physical block is taken only when the last one is full;
 *     decode attention takes the current token's query against the keys of
 *     one block at a time and accumulates the output against that block's
 *     values, so blocks need not be adjacent; sequences share blocks through
 *     reference counts, and a write into the last shared block copies that
 *     block and only it.
 *   - tonho.wtf "vllm", "o que isso custou": the three kernels the method
 *     needs -- block write, paged read fused with attention, batched block
 *     copy.  They are paged_kv_append, paged_attention_decode and
 *     copy_blocks below.
 *   - techtrendfeed "KV Cache Administration: PagedAttention &
 *     RadixAttention", "How PagedAttention Works", steps 1-4 (blocks of 16
 *     or 32 tokens; block table used by the kernel to gather K and V; growth
 *     one block at a time; copy-on-write), and "Why this modified LLM
 *     serving" (paging changes neither the attention result nor the model's
 *     outputs).
 *
 * Conventions shared by every call:
 *   - Cache layout: k_cache and v_cache are each
 *       [num_blocks][num_kv_heads][block_size][head_dim]
 *     row-major, elements of pkv_cache_desc.dtype.  Token position t of a
 *     sequence sits in logical block t / block_size at offset
 *     t % block_size; the (block, KV head) tile is contiguous.
 *   - A slot is physical_block * block_size + offset.
 *   - GQA: query head h reads KV head h / (num_q_heads / num_kv_heads).
 *   - Ownership: every data pointer is a caller-owned DEVICE pointer unless
 *     stated otherwise; the library keeps no pointer after a call returns,
 *     allocates no memory, and never synchronises except in
 *     pkv_check_device_error.
 *   - Streams: `stream` is a cudaStream_t passed as void* (NULL = legacy
 *     default stream).  Every call is asynchronous on it.
 *   - Errors found on the host (null or misaligned pointers, unsupported
 *     shapes, too small a workspace) return a status and launch nothing.
 *     Bad metadata that lives on the device (a slot, block id or context
 *     length outside the pool) never faults: the kernel skips the access,
 *     zero-fills the affected output, and records the first such error in a
 *     per-device error word that pkv_check_device_error reads and clears.
 *   - Kernels never wait on another kernel or CTA.  Waits inside one CTA
 *     (its copy pipeline) are bounded; a wait that runs out records
 *     PKV_DEVERR_TIMEOUT and the CTA returns.
 */
#ifndef PAGEDKV_H
#define PAGEDKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PKV_OK = 0,
    PKV_ERR_INVALID_ARG = 1,     /* null/misaligned pointer or bad size */
    PKV_ERR_UNSUPPORTED = 2,     /* valid but not implemented shape or dtype */
    PKV_ERR_WORKSPACE = 3,       /* workspace missing or too small */
    PKV_ERR_CUDA = 4,            /* a CUDA runtime or driver call failed */
    PKV_ERR_DEVICE_METADATA = 5  /* reported by pkv_check_device_error */
} pkv_status;

/* PKV_E4M3: 8-bit floats with 4 exponent and 3 mantissa bits, no infinity, largest value 448. */
typedef enum { PKV_BF16 = 0, PKV_FP16 = 1, PKV_FP32 = 2, PKV_E4M3 = 3 } pkv_dtype;

/* Codes stored in the device error word (first error wins). */
enum {
    PKV_DEVERR_NONE = 0,
    PKV_DEVERR_SLOT = 1,        /* append / append_rope / compact_tokens: slot >= num_blocks * block_size */
    PKV_DEVERR_COPY_ID = 2,     /* copy_blocks / copy_blocks_fp8 / swap_blocks: src or dst outside its pool */
    PKV_DEVERR_CONTEXT_LEN = 3, /* decode: context_lens[s] < 0, above the table's capacity, or above max_context_len */
    PKV_DEVERR_BLOCK_ID = 4,    /* decode: block_tables entry outside the pool */
    PKV_DEVERR_TIMEOUT = 5,     /* a bounded in-CTA wait ran out */
    PKV_DEVERR_PREFIX_LEN = 6,  /* grouped decode: prefix_lens[s] < 0, above context_lens[s] or
                                   max_prefix_len, or not a multiple of block_size */
    PKV_DEVERR_GROUP = 7,       /* grouped decode: group_starts out of order or range, or a sequence
                                   with a shared prefix in no group or beyond max_group_size members */
    PKV_DEVERR_POSITION = 8,    /* append_rope: positions[t] outside [0, max_position) */
    PKV_DEVERR_SCALE = 9,       /* append_rope_fp8: rows join a block whose scale is not finite and at least 2^-126 */
    PKV_DEVERR_QUERY = 10       /* attention of drafted tokens, prompts: query_starts (or key_starts) out of order or
                                   range, or more tokens of a sequence than the call takes */
};

/* Shape of one layer's paged cache (host struct, read during the call). */
typedef struct {
    int64_t num_blocks;  /* physical blocks in the pool, >= 1 */
    int32_t num_kv_heads;
    int32_t block_size;  /* tokens per block: 16 or 32 */
    int32_t head_dim;    /* 128 */
    int32_t dtype;       /* pkv_dtype: PKV_BF16 or PKV_FP16; PKV_E4M3 for the calls that end in _fp8 */
} pkv_cache_desc;

/* The new rows of paged_kv_append_rope and how they are rotated (host struct, read during the call). */
typedef struct {
    int32_t num_q_heads;  /* heads of q and q_out; 0: no queries */
    int32_t dtype;        /* of q, k, v, q_out and the norm weights: PKV_BF16 or PKV_FP16 */
    int64_t q_stride;     /* elements from one token's row to the next, a multiple of 8 */
    int64_t k_stride;
    int64_t v_stride;
    int64_t max_position; /* rows of cos_sin */
    int32_t rot_dim;      /* dims of each head that are rotated, its first ones: 0 (none) or a multiple of 16, <= head_dim */
    int32_t interleaved;  /* 0: pairs (i, i + rot_dim / 2); 1: pairs (2i, 2i + 1) */
    float norm_eps;       /* added to the mean square; >= 0 */
} pkv_rope_desc;

/* A paged latent cache, [num_blocks][block_size][latent_dim + rope_dim] (host struct, read during the call). */
typedef struct {
    int64_t num_blocks;  /* >= 1 */
    int32_t block_size;  /* tokens per block: 16 or 32 */
    int32_t latent_dim;  /* 512 */
    int32_t rope_dim;    /* 64 */
    int32_t dtype;       /* PKV_BF16 or PKV_FP16 */
} pkv_latent_desc;

/* The new rows of paged_latent_append_rope (host struct, read during the call); strides in elements, multiples of 8. */
typedef struct {
    int32_t num_heads;         /* query heads; 0: no queries */
    int32_t interleaved;       /* 0: pairs (i, i + rope_dim / 2); 1: pairs (2i, 2i + 1) */
    int64_t q_stride;          /* from one token's queries to the next */
    int64_t q_head_stride;     /* from one head to the next */
    int64_t q_out_stride;
    int64_t q_out_head_stride;
    int64_t kv_stride;
    int64_t max_position;      /* rows of cos_sin */
    float norm_eps;            /* added to the mean square; >= 0 */
} pkv_latent_rope_desc;

/* The prompts of latent_attention_prefill (host struct, read during the call); strides in elements, multiples of 8. */
typedef struct {
    int32_t num_heads;
    int32_t dtype;             /* of q, kv, k_rope and out: PKV_BF16 or PKV_FP16 */
    int32_t nope_dim;          /* 128 */
    int32_t rope_dim;          /* 64 */
    int32_t value_dim;         /* 128 */
    int64_t q_stride;          /* from one token to the next */
    int64_t q_head_stride;     /* from one head to the next */
    int64_t kv_stride;
    int64_t kv_head_stride;
    int64_t k_rope_stride;
} pkv_prompt_desc;

/* Human-readable name of a status. Never NULL. */
const char* pkv_status_string(pkv_status status);

/* Library version as 10000*major + 100*minor + patch. */
int pkv_version(void);

/*
 * Block write ("vllm", "como funciona" and "o que isso custou").
 * For every token t with slot_mapping[t] >= 0 and every KV head h:
 *     k_cache[slot / bs][h][slot % bs][:] = k[t][h][:]   (same for v)
 * k, v:          [num_tokens][num_kv_heads][head_dim], cache dtype, 16-byte
 *                aligned device memory.
 * slot_mapping:  [num_tokens] int64 device memory; a negative slot marks a
 *                padding token, which is skipped.
 * k_cache, v_cache: the pool (layout above), 16-byte aligned.
 * num_tokens == 0 is a no-op.  Two tokens with the same slot race (last
 * writer undefined).  A slot >= num_blocks * block_size is skipped and
 * recorded as PKV_DEVERR_SLOT.  The copy is bit-exact.
 */
pkv_status paged_kv_append(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens,
                           void* k_cache, void* v_cache, const pkv_cache_desc* cache, void* stream);

/*
 * Block write with the position rotation, and the norms of query and key
 * heads, on the way: one pass over a step's new rows.  For every token t with
 * slot_mapping[t] >= 0 and every query and key head x (head_dim values):
 *     x' = x / sqrt(mean(x^2) + norm_eps) * w   (w = q_norm or k_norm; x' = x where that is NULL)
 *     y  = x' with its first rot_dim dims turned by the token's position p = positions[t]:
 *          (y_a, y_b) = (x'_a c_i - x'_b s_i, x'_b c_i + x'_a s_i) for pair i = (a, b) of pkv_rope_desc,
 *          c_i = cos_sin[p][i], s_i = cos_sin[p][rot_dim / 2 + i], i < rot_dim / 2
 * y goes to q_out (queries) or to the token's slot of k_cache (keys, as
 * paged_kv_append writes them); v goes to v_cache unchanged, bit for bit.
 * Everything between the loads and the one rounding of y is in 32 bits.
 *
 * q, k, v:       row t at base + t * stride elements, [num_heads][head_dim]
 *                contiguous inside the row: slices of one fused projection
 *                are passed as they are.  16-byte aligned; the cache's dtype.
 *                q and q_out may be NULL when num_q_heads is 0.
 * positions:     [num_tokens] int64 device memory; not read, NULL allowed, when
 *                rot_dim is 0.
 * cos_sin:       [max_position][rot_dim] fp32 device memory, 16-byte
 *                aligned; NULL when rot_dim is 0.
 * q_norm, k_norm: [head_dim] device memory, 16-byte aligned, or NULL.
 * slot_mapping:  as for paged_kv_append.
 * q_out:         [num_tokens][num_q_heads][head_dim], 16-byte aligned; may be
 *                q itself when q_stride is num_q_heads * head_dim, and must
 *                not overlap it otherwise, nor the k and v rows.
 * A token with a negative slot is padding: its position and its rows may hold
 * anything, and its row of q_out keeps its contents.  A slot past the pool is recorded as
 * PKV_DEVERR_SLOT and a position outside [0, max_position) as
 * PKV_DEVERR_POSITION; such a token's K and V are not written and its q_out
 * row is zeros.  Two tokens with the same slot race (last writer undefined).
 * num_tokens == 0 is a no-op.  Supported: head_dim 128, any block size, bf16
 * or fp16, pools and tables of fewer than 2^31 slots and positions.
 */
pkv_status paged_kv_append_rope(const void* q, const void* k, const void* v, const int64_t* positions,
                                const float* cos_sin, const void* q_norm, const void* k_norm,
                                const int64_t* slot_mapping, int64_t num_tokens, void* q_out, void* k_cache,
                                void* v_cache, const pkv_cache_desc* cache, const pkv_rope_desc* rope, void* stream);

/*
 * paged_kv_append_rope into an 8-bit pool.  k_cache and v_cache hold e4m3
 * values, and each (block, KV head) of either has one fp32 scale: a stored
 * value b stands for b * scale.
 * k_scales, v_scales: [num_blocks][num_kv_heads] fp32 device memory.
 * For each block and KV head that rows are written to, for K and for V, with
 * a = the largest finite magnitude of those rows (K: after the rotation):
 *   - the block's first row is among them: the block starts afresh, and its
 *     scale becomes P(a), the smallest power of two >= a / 448, 2^-64 at least;
 *   - otherwise the rows join those that the block holds: the scale is kept
 *     while a <= 448 * scale; else it becomes P(a), and the rows below the
 *     first written one are moved to it, each value rounded once to the
 *     nearest e4m3 value of b * (old / new).  A scale that is not a finite
 *     number of at least 2^-126 is recorded as PKV_DEVERR_SCALE and replaced
 *     by P(a), with the held bytes left as they are.
 * The new rows are stored as the nearest e4m3 values of y / scale, ties to
 * even; infinities and NaN are stored as NaN.  A scale that is a power of two
 * loses nothing when it is applied and keeps the relative precision of e4m3
 * (half a step, 2^-4) down to 2^-15 of the largest magnitude it can hold; it
 * also makes a move to a larger scale exact but for the smallest values.
 * Rows above the first written one that the call does not write keep their
 * bytes: a block is filled from its first row up.
 * Tokens of one block stand together in slot_mapping, in any order, with
 * padding between them or not; where they do not, that block's contents and
 * scales are unspecified.
 * cache->dtype is PKV_E4M3 and block_size 16 or 32; the rest as for
 * paged_kv_append_rope.
 */
pkv_status paged_kv_append_rope_fp8(const void* q, const void* k, const void* v, const int64_t* positions,
                                    const float* cos_sin, const void* q_norm, const void* k_norm,
                                    const int64_t* slot_mapping, int64_t num_tokens, void* q_out, void* k_cache,
                                    void* v_cache, float* k_scales, float* v_scales, const pkv_cache_desc* cache,
                                    const pkv_rope_desc* rope, void* stream);

/*
 * Bytes of workspace paged_attention_decode needs for these sizes (0 when
 * the call runs in a single pass).  partition_size as for
 * paged_attention_decode; with 0 (automatic) the size covers the smallest
 * automatic partition, so it is enough whatever the call picks.  Returns 0
 * for invalid sizes.
 */
size_t paged_attention_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t head_dim,
                                       int32_t max_context_len, int32_t partition_size);

/* How paged_attention_decode divides the work (see paged_attention_plan). */
enum {
    PKV_PLAN_SINGLE = 0,       /* one CTA per (sequence, head group): no partials */
    PKV_PLAN_SPLIT = 1,        /* split-K, merged by the last partition of each row */
    PKV_PLAN_SPLIT_REDUCE = 2  /* split-K with more than 16 partitions, merged by a second kernel */
};

/*
 * The decomposition paged_attention_decode uses for these sizes on the
 * current device; -1 for invalid sizes.  block_size is the cache's.
 */
int32_t paged_attention_plan(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t block_size,
                             int32_t max_context_len, int32_t partition_size);

/*
 * The split-K partition size (tokens) paged_attention_decode uses for these
 * sizes on the current device: partition_size itself when it is non-zero,
 * else the automatic choice.  Returns 0 for invalid sizes.
 */
int32_t paged_attention_partition_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                       int32_t max_context_len, int32_t partition_size);

/*
 * Paged decode attention ("vllm", "como funciona": the query of the current
 * token against the keys of one block at a time, output accumulated against
 * the same block's values; blocks need not be adjacent).
 * For every sequence s and query head h, with L = context_lens[s] and
 * kvh = h / (num_q_heads / num_kv_heads):
 *     out[s][h][:] = sum_{t<L} softmax_t(scale * q[s][h] . K[t]) V[t]
 * where K[t], V[t] are row t % bs of tile (block_tables[s][t / bs], kvh).
 * L counts every attended token, including the one appended this step;
 * L == 0 gives zeros.
 *
 * q:               [num_seqs][num_q_heads][head_dim], cache dtype, 16-byte aligned.
 * k_cache, v_cache: the pool, 16-byte aligned.
 * block_tables:    [num_seqs][max_blocks_per_seq] int32; entries past
 *                  ceil(L / bs) are never read.
 * context_lens:    [num_seqs] int32, each in [0, min(max_context_len,
 *                  max_blocks_per_seq * bs)].
 * max_context_len: host-side upper bound of context_lens; it sizes the
 *                  split-K partitions and the workspace.
 * out:             [num_seqs][num_q_heads][head_dim] of out_dtype (PKV_FP32,
 *                  PKV_BF16 or PKV_FP16), 16-byte aligned.
 * partition_size:  tokens per split-K partition, a multiple of block_size;
 *                  0 picks 512, 1024, 2048 or 4096 from the amount of work
 *                  and the device's SM count (the largest that still gives
 *                  every resident decode CTA two work units).  When max_context_len > partition_size
 *                  each partition writes (o_p, lse_p) to the workspace and
 *                  they are merged through their log-sum-exp: by the last
 *                  partition of each (sequence, head group) to finish when a
 *                  sequence has at most 16 partitions, else by a second
 *                  kernel.  Otherwise one kernel writes out directly.
 * workspace:       device memory of at least
 *                  paged_attention_workspace_bytes(...) bytes, 256-byte
 *                  aligned (may be NULL when that is 0).  Contents on entry
 *                  are ignored: the merge's arrival counters carry the
 *                  epoch of the call that wrote them, and a counter of any
 *                  other epoch counts as zero.  Two calls whose kernels may
 *                  overlap on the GPU must not share a workspace.
 * Supported: head_dim 128; block_size 16 or 32; bf16 or fp16 caches;
 * num_q_heads a multiple of num_kv_heads; num_seqs <= 65535.
 * Results depend only on logical token order: permuting physical block ids
 * leaves the output bit-for-bit unchanged.
 */
pkv_status paged_attention_decode(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_tables, int32_t max_blocks_per_seq,
                                  const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                                  int32_t max_context_len, float scale, void* out, int32_t out_dtype,
                                  const pkv_cache_desc* cache, int32_t partition_size, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * paged_attention_decode over an 8-bit pool (paged_kv_append_rope_fp8): with
 * ks = k_scales[b][kvh], vs = v_scales[b][kvh] of the block b that holds t,
 *     out[s][h][:] = sum_{t<L} softmax_t(scale * ks * q[s][h] . K[t]) vs V[t]
 * q_dtype:   PKV_BF16 or PKV_FP16, the type of q.
 * k_scales, v_scales: [num_blocks][num_kv_heads] fp32 device memory; any
 *            finite values, powers of two or not, of either sign, or zero.
 *            The V scales that a head meets in one context, but for zeros,
 *            should lie within 2^64 of one another: beyond that, values of
 *            small scales may count as zeros where large ones have weight in
 *            some head.  scale * ks * (the largest q of a head) and the scores
 *            must lie in fp32's range.  Those of blocks outside the
 *            sequences' contexts are never read.
 * cache->dtype is PKV_E4M3.  The other arguments, the workspace
 * (paged_attention_workspace_bytes), the errors and the limits are those of
 * paged_attention_decode.  partition_size is the most tokens of a split-K
 * partition: a sequence with more is cut into as few equal parts as that
 * allows; 0 chooses 512 to 4096 tokens by num_seqs, the heads and
 * max_context_len, for this kernel's own resident CTAs, so
 * paged_attention_plan and paged_attention_partition_size need not agree
 * (a max_context_len near the longest context chooses best).  The values enter the products exactly (as 16-bit floats),
 * the scales as 32-bit factors, a token's weight to within 2^-20 of itself
 * and 2^-26 of its head's largest: one further below than that counts as
 * nothing, whatever the scale of its value.
 */
pkv_status paged_attention_decode_fp8(const void* q, int32_t q_dtype, const void* k_cache, const void* v_cache,
                                      const float* k_scales, const float* v_scales, const int32_t* block_tables,
                                      int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t num_seqs,
                                      int32_t num_q_heads, int32_t max_context_len, float scale, void* out,
                                      int32_t out_dtype, const pkv_cache_desc* cache, int32_t partition_size,
                                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Attention of several query tokens of each sequence, the drafted tokens of
 * a speculative step, over the paged cache.  Sequence s's query tokens are
 * rows query_starts[s] .. query_starts[s+1]-1 of q, n of them, and stand for
 * the last n positions of its context of L = context_lens[s] tokens, whose K
 * and V are in the cache already.  With base = L - n, query token i attends
 * every position before base, and of the drafted positions base + j those
 * with bit j of its mask set (a tree: itself and what it descends from), or,
 * without masks, those with j <= i (a chain):
 *     out[i][h][:] = sum_t softmax_t(scale * q[i][h] . K[t]) V[t]   over the attended t
 * A query token that attends nothing gets zeros, and so does every query
 * token of a sequence with L == 0.
 *
 * q:            [num_tokens][num_q_heads][head_dim], cache dtype, 16-byte aligned.
 * query_starts: [num_seqs + 1] int32 device memory, in order, n <= 64; NULL:
 *               one token a sequence (num_tokens == num_seqs).  Rows of q and
 *               out outside the sequences are left alone.
 * tree_masks:   [num_tokens] int64 device memory, bits n and above ignored; or
 *               NULL.
 * context_lens: [num_seqs] int32, L == 0 or n <= L <= max_blocks_per_seq * bs.
 * out:          [num_tokens][num_q_heads][head_dim], cache dtype, 16-byte
 *               aligned, not q.
 * workspace:    at least paged_attention_tree_workspace_bytes() bytes, 256-byte
 *               aligned; contents on entry are ignored.  Two calls whose
 *               kernels may overlap on the GPU must not share it.
 * K and V of positions that a token does not attend, and of the blocks' rows
 * behind the context, may hold anything.  Values that are not finite make
 * not finite the outputs of the tokens that attend them, and of no others.
 * Weights are rounded once to the cache's type for their product with V (half
 * a step, 2^-8 of a weight in bf16 and 2^-11 in fp16, and in fp16 by up to 2^-32
 * of the largest weight for the smallest ones; paged_attention_decode carries
 * what its weights lose along); everything else is in 32 bits.
 * The result does not depend on physical block ids, and is the same from run
 * to run.
 * Bad metadata never faults: query_starts out of order or range
 * (PKV_DEVERR_QUERY) leave the sequence's rows alone (sequences that lie over
 * one another write the rows in no certain order); more than 64 query
 * tokens (PKV_DEVERR_QUERY), a context length out of range or below n
 * (PKV_DEVERR_CONTEXT_LEN) and a block id outside the pool
 * (PKV_DEVERR_BLOCK_ID; the query heads of the KV heads that read it) get
 * zeros.
 * Supported: head_dim 128; block_size 16 or 32; bf16 or fp16;
 * num_q_heads a multiple of num_kv_heads; num_seqs <= 65535; tables of up to
 * 2^31 - 1024 positions.
 */
pkv_status paged_attention_tree(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                                int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_starts,
                                const int64_t* tree_masks, int32_t num_seqs, int32_t num_tokens, int32_t num_q_heads,
                                float scale, void* out, const pkv_cache_desc* cache, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Workspace bytes of paged_attention_tree on the current device (0: no device). */
size_t paged_attention_tree_workspace_bytes(void);

/*
 * Write into a paged latent cache: one row a token, a latent that every
 * head's keys and values are expanded from and a key part with the position
 * that all heads share.  For every token t with slot_mapping[t] >= 0, with c =
 * the first latent_dim values of its row of kv and r = the rope_dim behind
 * them:
 *     c' = c / sqrt(mean(c^2) + norm_eps) * kv_norm   (c' = c where that is NULL)
 *     r' = r turned by the position, as paged_kv_append_rope turns a head with rot_dim = rope_dim
 * and (c', r') goes to the token's slot of the cache, and to its row of
 * kv_out where that is given (the prompt's latents, to be expanded); every
 * head's rope_dim query values are turned by the same angles into q_out.
 * Everything between the loads and the one rounding is in 32 bits.
 *
 * q, q_out:     token t's head h at base + t * stride + h * head_stride
 *               elements, rope_dim contiguous values: slices of the query
 *               projection and of the absorbed queries are passed as they
 *               are.  q_out may be q with the same strides, and must not
 *               overlap it otherwise.  May be NULL when num_heads is 0.
 * kv:           row t at base + t * kv_stride.
 * kv_out:       [num_tokens][latent_dim + rope_dim] or NULL; may be kv when
 *               kv_stride is latent_dim + rope_dim, and must not overlap it
 *               otherwise.
 * positions:    [num_tokens] int64; not read, NULL allowed, when cos_sin is NULL.
 * cos_sin:      [max_position][rope_dim] fp32, or NULL: no rotation.
 * kv_norm:      [latent_dim] or NULL.
 * slot_mapping: [num_tokens] int64; negative: padding, whose rows of q_out and
 *               kv_out keep their contents.
 * All device memory, 16-byte aligned but for positions and slot_mapping (8).
 * A slot past the pool is recorded as PKV_DEVERR_SLOT and a position outside
 * [0, max_position) as PKV_DEVERR_POSITION; such a token's row is not written
 * and its rows of q_out and kv_out are zeros.  Two tokens with the same slot
 * race.  num_tokens == 0 is a no-op.  Supported: latent_dim 512, rope_dim 64,
 * bf16 or fp16, any block size.
 * copy_blocks, swap_blocks and compact_tokens take such pools under a
 * pkv_cache_desc of one KV head with head_dim latent_dim + rope_dim: the pools
 * of two layers as K and V, or one for both.
 */
pkv_status paged_latent_append_rope(const void* q, const void* kv, const int64_t* positions, const float* cos_sin,
                                    const void* kv_norm, const int64_t* slot_mapping, int64_t num_tokens, void* q_out,
                                    void* kv_out, void* latent_cache, const pkv_latent_desc* cache,
                                    const pkv_latent_rope_desc* rope, void* stream);

/*
 * Attention over a paged latent cache in its absorbed form: each head's query
 * has been taken through the key expansion, so that its score against a token
 * is a product over the whole cached row, whose first latent_dim values are
 * the value too (the caller takes the output through the value expansion):
 *     out[i][h][:] = sum_t softmax_t(scale * q[i][h] . row[t]) row[t][:latent_dim]
 * over the positions that query token i attends, which query_starts,
 * tree_masks and context_lens say as for paged_attention_tree; so do the
 * errors, the workspace (paged_latent_decode_workspace_bytes()), the
 * roundings and what may lie in places that are not attended.
 * q:            [num_tokens][num_heads][latent_dim + rope_dim], cache dtype, 16-byte aligned.
 * latent_cache: the pool, 16-byte aligned.
 * out:          [num_tokens][num_heads][latent_dim], cache dtype, 16-byte aligned.
 * Supported: latent_dim 512, rope_dim 64; block_size 16 or 32; bf16 or fp16;
 * num_seqs <= 65535; num_tokens * num_heads and num_blocks * block_size below
 * 2^31; tables of up to 2^31 - 1024 positions.
 */
pkv_status paged_latent_decode(const void* q, const void* latent_cache, const int32_t* block_tables,
                               int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_starts,
                               const int64_t* tree_masks, int32_t num_seqs, int32_t num_tokens, int32_t num_heads,
                               float scale, void* out, const pkv_latent_desc* cache, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Workspace bytes of paged_latent_decode on the current device (0: no device). */
size_t paged_latent_decode_workspace_bytes(void);

/*
 * Causal attention of whole prompts in the expanded form of latent attention:
 * each head has a key of nope_dim values and a value of value_dim values a
 * token, expanded from the token's latent and side by side in kv, and the
 * rope_dim turned key values of k_rope are shared by the heads.  Sequence s's
 * queries are tokens query_starts[s] .. query_starts[s+1]-1 of q, n of them,
 * its keys tokens key_starts[s] .. key_starts[s+1]-1 of kv and k_rope, m of
 * them; the queries are the last n positions of the m: query i attends keys j
 * <= i + m - n.
 *     s_ij = scale * (q[i][h][:nope] . kv[j][h][:nope] + q[i][h][nope:] . k_rope[j])
 *     out[i][h][:] = sum_j softmax_j(s_ij) kv[j][h][nope:]
 * A query that attends nothing (m < n) gets zeros.
 * q:        token t's head h at base + t * q_stride + h * q_head_stride, nope_dim + rope_dim values.
 * kv:       token t's head h at base + t * kv_stride + h * kv_head_stride, nope_dim + value_dim values.
 * k_rope:   token t at base + t * k_rope_stride: kv_out of paged_latent_append_rope behind its first latent_dim values.
 * query_starts, key_starts: [num_seqs + 1] int32 device memory, in order.
 *           Rows of q and out outside the sequences are left alone.
 * max_query_len: host-side upper bound of the sequences' n, at most
 *           num_query_tokens (which is always one; more is refused).
 * out:      [num_query_tokens][num_heads][value_dim], 16-byte aligned.
 * q, kv and k_rope are 16-byte aligned.  What is not finite stays with the
 * queries that attend it, and weights are rounded as for paged_attention_tree.
 * Bad metadata never faults: query_starts out of order or range leave the
 * sequence's rows alone (and may leave alone those of sequences that lie over
 * others), key_starts out of order or range and n > max_query_len get zeros
 * (PKV_DEVERR_QUERY).
 * Supported: nope_dim 128, rope_dim 64, value_dim 128; bf16 or fp16; num_heads and num_seqs <= 65535.
 */
pkv_status latent_attention_prefill(const void* q, const void* kv, const void* k_rope, const int32_t* query_starts,
                                    const int32_t* key_starts, int32_t num_seqs, int32_t num_query_tokens,
                                    int32_t num_key_tokens, int32_t max_query_len, float scale, void* out,
                                    const pkv_prompt_desc* prompt, void* stream);

/*
 * A decode step in one launch: the block write of one new token per
 * sequence ("vllm", "o que isso custou": block write) fused into
 * paged_attention_decode.  The result, and the cache afterwards, are those
 * of paged_kv_append(k_new, v_new, slot_mapping, num_seqs, ...) followed by
 * paged_attention_decode(...), provided that each sequence's new token is its
 * last context position: slot_mapping[s] must be the slot of position
 * context_lens[s] - 1 of sequence s (block_tables[s][(L-1)/bs] * bs +
 * (L-1) % bs), or negative when sequence s has no new token, and no other
 * sequence may read that slot in this call.  A slot that is not that position
 * is not written and is recorded as PKV_DEVERR_SLOT.
 * k_new, v_new:  [num_seqs][num_kv_heads][head_dim], cache dtype, 16-byte
 *                aligned device memory.
 * slot_mapping:  [num_seqs] int64 device memory.
 * Other arguments as for paged_attention_decode; k_cache and v_cache are
 * written.
 */
pkv_status paged_attention_append_decode(const void* q, const void* k_new, const void* v_new,
                                         const int64_t* slot_mapping, void* k_cache, void* v_cache,
                                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                                         const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                                         int32_t max_context_len, float scale, void* out, int32_t out_dtype,
                                         const pkv_cache_desc* cache, int32_t partition_size, void* workspace,
                                         size_t workspace_bytes, void* stream);

/*
 * paged_attention_decode for batches whose sequences share prompt blocks
 * (samples forked from one prompt, a common system prompt).  Forked
 * sequences map the prompt's logical blocks to the same physical blocks,
 * counted by reference ("vllm", "como funciona"; techtrendfeed "KV Cache
 * Administration", "How PagedAttention Works", step 4), and a shared prefix
 * is read once and reused (aitalk.it "PagedAttention e RadixAttention").
 * Here each shared block is read from HBM once per (group, KV head) and
 * attended by every member's query heads together; each member's own
 * blocks are attended as in paged_attention_decode, and the two parts are
 * merged through their log-sum-exp.
 *
 * The result is paged_attention_decode's on the same q, cache, tables and
 * lengths, provided that for every member s of group g, positions
 * 0 .. prefix_lens[s]-1 of s sit in the same physical blocks as the same
 * positions of the group's first member (block_tables rows agree there).
 *
 * group_starts:   [num_groups + 1] int32 device memory: the members of group
 *                 g are sequences group_starts[g] .. group_starts[g+1]-1, in
 *                 order; groups must not overlap.
 * max_group_size: host-side upper bound of group_starts[g+1] - group_starts[g].
 * prefix_lens:    [num_seqs] int32 device memory: tokens of s attended through
 *                 its group's first member's block table, a multiple of
 *                 block_size in [0, min(context_lens[s], max_prefix_len)].
 *                 Members of one group may differ.  A sequence with
 *                 prefix_lens[s] == 0 need not be in any group.
 * max_prefix_len: host-side upper bound of prefix_lens, <= max_context_len.
 * workspace:      at least paged_attention_grouped_workspace_bytes(...)
 *                 bytes, 256-byte aligned; always needed.  Contents on entry
 *                 are ignored.
 * Other arguments as for paged_attention_decode.  Supported: as for
 * paged_attention_decode, with num_q_heads / num_kv_heads <= 64 and
 * num_groups <= 65535.  Bad metadata never faults: a prefix length out of
 * range (PKV_DEVERR_PREFIX_LEN), or a sequence with a nonzero prefix length
 * that lies in no group or in a group beyond max_group_size members
 * (PKV_DEVERR_GROUP), zeroes that sequence's output.  A group whose range
 * is out of order or out of bounds is skipped (PKV_DEVERR_GROUP); the
 * groups on either side of it may then overlap, and a sequence in two of
 * them gets a finite but unspecified output.  The pages describe the
 * sharing, not this kernel: the grouped read is an addition of this
 * library.
 */
pkv_status paged_attention_decode_grouped(const void* q, const void* k_cache, const void* v_cache,
                                          const int32_t* block_tables, int32_t max_blocks_per_seq,
                                          const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                                          int32_t max_context_len, const int32_t* group_starts,
                                          int32_t num_groups, int32_t max_group_size, const int32_t* prefix_lens,
                                          int32_t max_prefix_len, float scale, void* out, int32_t out_dtype,
                                          const pkv_cache_desc* cache, int32_t partition_size, void* workspace,
                                          size_t workspace_bytes, void* stream);

/*
 * A grouped decode step in one call: the block write of one new token per
 * sequence (as paged_attention_append_decode) fused into
 * paged_attention_decode_grouped.  The result, and the cache afterwards, are
 * those of paged_kv_append(k_new, v_new, slot_mapping, num_seqs, ...)
 * followed by paged_attention_decode_grouped(...), provided that each
 * sequence's new token is its last context position and lies past its
 * shared prefix (prefix_lens[s] < context_lens[s]; a write into a shared
 * block is preceded by its copy, "vllm", "como funciona"): slot_mapping[s]
 * must be the slot of position context_lens[s] - 1, or negative when
 * sequence s has no new token.  A slot that is not that position is not
 * written and is recorded as PKV_DEVERR_SLOT.  Arguments as for
 * paged_attention_append_decode and paged_attention_decode_grouped.
 */
pkv_status paged_attention_append_decode_grouped(const void* q, const void* k_new, const void* v_new,
                                                 const int64_t* slot_mapping, void* k_cache, void* v_cache,
                                                 const int32_t* block_tables, int32_t max_blocks_per_seq,
                                                 const int32_t* context_lens, int32_t num_seqs,
                                                 int32_t num_q_heads, int32_t max_context_len,
                                                 const int32_t* group_starts, int32_t num_groups,
                                                 int32_t max_group_size, const int32_t* prefix_lens,
                                                 int32_t max_prefix_len, float scale, void* out, int32_t out_dtype,
                                                 const pkv_cache_desc* cache, int32_t partition_size,
                                                 void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes paged_attention_decode_grouped needs (0 for invalid sizes). */
size_t paged_attention_grouped_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t head_dim,
                                               int32_t max_context_len, int32_t max_prefix_len,
                                               int32_t partition_size);

/*
 * paged_attention_decode without a workspace argument, for callers that
 * cannot allocate device memory: a process whose device memory is all owned
 * by another allocator (such as a serving engine that reserved nearly all of
 * HBM for its KV pool at start-up), or a latency-critical loop that must not
 * call cudaMalloc because it can implicitly synchronise the device.  The
 * pages have no counterpart to this call; it is an addition of this library.
 *
 * Arguments and results are those of paged_attention_decode.  The split-K
 * partials live in a file-scope device array of 16 MiB that every GPU which
 * loads the library holds until the process exits; a call whose
 * paged_attention_workspace_bytes(...) exceeds 16 MiB is rejected with
 * PKV_ERR_WORKSPACE before anything is launched.  The call allocates nothing.
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture.  The array is shared by every call on the
 * device and keeps the last call's contents; nothing in it needs to start at
 * zero.  Calls whose kernels overlap on the GPU race on the array: the caller
 * must serialise them.
 */
pkv_status paged_attention_decode_static(const void* q, const void* k_cache, const void* v_cache,
                                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                                         const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads,
                                         int32_t max_context_len, float scale, void* out, int32_t out_dtype,
                                         const pkv_cache_desc* cache, int32_t partition_size, void* stream);

/*
 * Batched copy-on-write block copy ("vllm", "como funciona": a write into
 * the last shared block copies that block and only it; "o que isso
 * custou": batched block copy).
 * For each pair i and each layer l:
 *     k_caches[l][dst] = k_caches[l][src], v_caches[l][dst] = v_caches[l][src]
 * (whole blocks: every KV head and slot), with (src, dst) =
 * (src_dst_pairs[2i], src_dst_pairs[2i+1]).
 * k_caches, v_caches: HOST arrays of num_layers device pointers (each
 *                  16-byte aligned), all layers of the shape in `cache`.
 * src_dst_pairs:   [num_pairs][2] int64 DEVICE memory.
 * Destinations must be distinct and no destination may also be a source
 * (otherwise the result depends on block scheduling); an id outside the
 * pool skips that pair and records PKV_DEVERR_COPY_ID.  Bit-exact.
 */
pkv_status copy_blocks(void* const* k_caches, void* const* v_caches, int32_t num_layers,
                       const int64_t* src_dst_pairs, int32_t num_pairs, const pkv_cache_desc* cache,
                       void* stream);

/*
 * copy_blocks for 8-bit pools: the copy takes a block's scales along, for
 * each pair i and each layer l also
 *     k_scales[l][dst][:] = k_scales[l][src][:]   (and the V scales)
 * k_scales, v_scales: HOST arrays of num_layers device pointers to
 *                  [num_blocks][num_kv_heads] fp32, 4-byte aligned.
 * cache->dtype is PKV_E4M3; the rest as for copy_blocks.
 */
pkv_status copy_blocks_fp8(void* const* k_caches, void* const* v_caches, float* const* k_scales,
                           float* const* v_scales, int32_t num_layers, const int64_t* src_dst_pairs,
                           int32_t num_pairs, const pkv_cache_desc* cache, void* stream);

/*
 * Swap-out / swap-in of whole blocks between two pools ("vllm", "como
 * funciona": a preempted sequence's blocks go to CPU RAM and come back).
 * For each pair i and each layer l:
 *     dst_k_caches[l][dst] = src_k_caches[l][src]   (and the V caches)
 * with (src, dst) = (src_dst_pairs[2i], src_dst_pairs[2i+1]), src a block of
 * the source pool (src_num_blocks blocks) and dst one of the destination
 * pool (dst_num_blocks blocks).  Either pool may be GPU memory or page-locked
 * host memory that the GPU addresses directly (cudaHostAlloc, or
 * cudaHostRegister'ed memory, on a unified-addressing system; on GB300 the
 * copy runs over NVLink-C2C).  Both pools have the per-block shape of
 * `cache` (its num_blocks is not used).
 * src_k_caches, ...: HOST arrays of num_layers pointers, 16-byte aligned.
 * src_dst_pairs:    [num_pairs][2] int64, GPU-addressable memory.
 * An id outside its pool skips that pair and records PKV_DEVERR_COPY_ID.
 * Destinations must be distinct.  Bit-exact.
 */
pkv_status swap_blocks(void* const* src_k_caches, void* const* src_v_caches, int64_t src_num_blocks,
                       void* const* dst_k_caches, void* const* dst_v_caches, int64_t dst_num_blocks,
                       int32_t num_layers, const int64_t* src_dst_pairs, int32_t num_pairs,
                       const pkv_cache_desc* cache, void* stream);

/*
 * Token-level compaction into fresh target blocks (gist.science "Zipage",
 * Compressed PagedAttention: once a request holds N_max blocks and the last
 * one is full, the tokens it keeps are rewritten into new target blocks --
 * the first N_max - 1 of its new table -- so that prefix blocks shared with
 * other requests stay intact).  For each i with both slots >= 0:
 *     k_cache[dst slot row of head h] = k_cache[src slot row of head h]
 * for every KV head h, and the same for v_cache.  The caller chooses the
 * kept tokens (their scoring is not part of this library) and the target
 * blocks.  No destination slot may also be a source slot, and destinations
 * must be distinct.  A slot >= num_blocks * block_size skips the token and
 * records PKV_DEVERR_SLOT.  src_slots, dst_slots: [num_tokens] int64 device
 * memory.  Bit-exact.
 */
pkv_status compact_tokens(const int64_t* src_slots, const int64_t* dst_slots, int64_t num_tokens, void* k_cache,
                          void* v_cache, const pkv_cache_desc* cache, void* stream);

/*
 * Synchronises `stream`, then reads and clears the current device's error
 * word.  Returns PKV_OK (and *first_error_code = 0) when no kernel recorded
 * an error since the last check, PKV_ERR_DEVICE_METADATA with the first
 * PKV_DEVERR_* code otherwise, or PKV_ERR_CUDA.  first_error_code may be
 * NULL.
 * The word is one per device, shared by the library's calls on every stream,
 * and only `stream` is synchronised: an error recorded by a kernel still
 * running on another stream is not seen by this check, and is reported by a
 * later one (or, if it lands between the read and the clear, lost).  To check
 * the calls of several streams, synchronise all of them (or the device)
 * before calling this.
 */
pkv_status pkv_check_device_error(void* stream, int32_t* first_error_code);

/*
 * Self-test of the bounded-wait error path, with no fault and no hang.
 * Launches one CTA that waits, through the same bounded mbarrier wait the
 * copy pipelines use but with a limit of limit_us microseconds, on a phase
 * that nothing completes.  The wait runs out, the CTA records
 * PKV_DEVERR_TIMEOUT in the device error word (as a stalled pipeline would)
 * and returns; the context stays usable.  limit_us: 1 .. 2,000,000, else
 * PKV_ERR_INVALID_ARG with nothing launched.  Asynchronous on `stream`.
 */
pkv_status pkv_wait_selftest(int32_t limit_us, void* stream);

/* Number of kernels this library has launched in this process. */
uint64_t pkv_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_H */
