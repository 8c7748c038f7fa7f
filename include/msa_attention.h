/*
 * msa_attention.h -- attention over the paged K/V caches the MSA producer writes, as a
 * C ABI, for NVIDIA GB300 (sm_103a).
 *
 * Two operators, both grouped-query attention of the producer's compact queries
 * (q_out) over strided, paged K/V caches (msa_cache_desc, FP8 E4M3 or bf16):
 *
 *   msa_sparse_attention_forward   each query attends the tokens of the blocks an
 *                                  indexer selected for it (msa_indexer_forward's
 *                                  topk_ids): the consumer of the indexer in an MSA
 *                                  layer ("[None][perf] Fuse MiniMax-M3 QKV and index
 *                                  projection", TensorRT-LLM PR 18205, AFTER diagram:
 *                                  score, max-pool, top-k block ids, sparse attention);
 *   msa_prefix_attention_forward   dense attention in which groups of queries share a
 *                                  prefix, whose keys and values are read and
 *                                  multiplied once for each tile of 128 of the group's
 *                                  rows (queries times heads on a K/V head) within
 *                                  windows of up to 384 queries; with no group it is
 *                                  plain dense paged attention.
 *
 * Per query t and query head h, with c = h / (num_q_heads / num_kv_heads):
 *
 *     s_j      = softmax_scale * (q[t,h,:] . (ks[c] * K[j,c,:]))      j visible to t
 *     out[t,h] = sum_j exp(s_j) * vs[c] * V[j,c,:] / sum_j exp(s_j)   (bf16)
 *     lse[t,h] = ln sum_j exp(s_j)                                    (fp32)
 *
 * where ks, vs are the dequantisation scales of an FP8 cache (1 for bf16).  A query
 * that sees no token gets out = 0 and lse = -inf.  Values behind a token that a query
 * does not see (unwritten cache cells, NaN or infinity among them) never reach its
 * result.  A token whose score is -infinity (an infinite key of a bf16 cache) has no
 * weight, as one that is not visible.  A row of q that is not finite and sees a token has
 * no result of its own: over E4M3 keys NaN (out and lse), over bf16 keys what its scores
 * give.
 *
 * The token of a history at index j lies in page page_table[offset + j / page_size],
 * row j % page_size; a token whose table index falls outside [0, page_table_len) or
 * whose page falls outside either cache is not visible.
 *
 * Arithmetic: scores, the running maximum, the sum and the output are accumulated in
 * fp32.  Where the products run on the tensor cores, bf16 caches take the queries as
 * they are and the weights exp(s - max) rounded to bf16; E4M3 caches are multiplied as
 * stored, against the queries split into two E4M3 halves hi + lo under a power-of-two
 * scale (reproduced exactly except elements below 2^-9 of the largest of their row) and
 * the weights split into three E5M2 parts (a weight to 2^-9 + 2^-11 of itself or 2^-28 of
 * the largest).  Results do not depend on which other calls run, and a call repeated with
 * the same arguments gives the same bits.
 *
 * Ownership and threading: as for msa_producer_forward.  The caller owns every buffer,
 * the workspace among them; the library allocates nothing, never synchronises, reads
 * no device memory on the host, and enqueues its kernels on `stream` alone, so a call
 * is stream-ordered and can be captured into a CUDA graph.  The stream must belong to
 * the current device.  A workspace need not be initialised and carries nothing from
 * one call to the next; calls (or graph replays) that may run at the same time need
 * separate workspaces.
 *
 * Errors: every argument check runs on the host before any launch; a call that
 * returns an error has enqueued nothing and written nothing (MSA_ERR_CUDA from a
 * launch that the CUDA runtime refused: earlier launches of the call may run).  Waits
 * inside the kernels are bounded (2 s); rows that a kernel could not finish are NaN.
 */
#ifndef MSA_ATTENTION_H
#define MSA_ATTENTION_H

#include <stdint.h>

#include "msa_producer.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t num_q_heads;     /* Hq: a positive multiple of num_kv_heads, at most 128 times it */
    int32_t num_kv_heads;    /* Hkv: 1..1024 */
    int32_t head_dim;        /* 64 or 128 */
    int32_t page_size;       /* tokens per page of both caches, > 0 */
    int32_t block_tokens;    /* sparse: tokens per selected block, a multiple of 32, 32..1024 */
    int32_t topk;            /* sparse: ids per query, 1..64 */
    float softmax_scale;     /* > 0, finite */
    int32_t scale_mode;      /* msa_scale_mode of `scales` */
    int32_t reserved[2];     /* must be 0 */
} msa_attention_cfg;

/*
 * Bytes of workspace that either operator needs for num_queries queries in num_groups
 * groups (0 for the sparse operator) under cfg.  However many queries:
 *   without groups  less than 4 MB, and up to 26 MB more where a sparse call with
 *                   MSA_LAUNCH_QUERY_RUNS would split its tiles of queries (a few hundred
 *                   queries or fewer, block_tokens a multiple of 128; nothing more where
 *                   topk is 0, as a cfg for prefix attention may have it);
 *   with groups     less than 55 MB, and two rows of (head_dim + 4) * 4 bytes for each
 *                   query head of min(num_queries, 384, max(1, 65536 / num_q_heads))
 *                   queries: 27 MB for 64 heads of 128 dims, at most 70 MB up to 65,536
 *                   heads.
 * Host-side; enqueues nothing.
 */
msa_status msa_attention_workspace_bytes(const msa_attention_cfg *cfg, int64_t num_queries,
                                         int64_t num_groups, int64_t *bytes);

/*
 * Sparse attention: query t sees the tokens j < kv_len[t] of the blocks topk_ids[t, :]
 * (block b: tokens [b * block_tokens, (b + 1) * block_tokens)).  Ids below 0 or past
 * the history are skipped; an id given twice counts once; the order of the ids does
 * not matter.
 *
 * q              device bf16 [num_queries, Hq, D], 16-byte aligned.
 * kv_len         device int32 [num_queries]: visible tokens (< 0 as 0).
 * table_offset   device int64 [num_queries]: start of the query's row in page_table.
 * page_table     device int32 [page_table_len].
 * topk_ids       device int32 [num_queries, topk].
 * k_cache, v_cache  Hkv-head descriptors; any mix of dtypes.
 * scales         device fp32, as the producer's: per tensor {k, v, ...}, per head Hkv
 *                K scales then Hkv V scales.  Read only by FP8 caches; may be NULL when
 *                neither is FP8.
 * out            device bf16 [num_queries, Hq, D], 16-byte aligned.
 * lse            device fp32 [num_queries, Hq], or NULL.
 * workspace      device, 16-byte aligned, msa_attention_workspace_bytes(cfg,
 *                num_queries, 0) bytes; NULL only where that is 0.
 * launch_flags   MSA_LAUNCH_PDL: accepted; the kernels are launched with programmatic
 *                dependent launch in any case, since they read and write memory only
 *                after waiting for the kernels ahead of them on the stream, and let the
 *                next one start as soon as they have waited.
 *                MSA_LAUNCH_QUERY_RUNS: consecutive queries mostly belong to one
 *                sequence (the same table_offset) and agree on many blocks, as in a
 *                prefill chunk, so tiles of consecutive queries share the blocks that
 *                any of them selected.  A hint: any queries are answered rightly.
 *
 * num_queries == 0 returns MSA_OK and launches nothing.
 */
msa_status msa_sparse_attention_forward(const msa_attention_cfg *cfg, int64_t num_queries,
                                        const void *q, const int32_t *kv_len,
                                        const int64_t *table_offset, const int32_t *page_table,
                                        int64_t page_table_len, const int32_t *topk_ids,
                                        const msa_cache_desc *k_cache,
                                        const msa_cache_desc *v_cache, const float *scales,
                                        void *out, float *lse, void *workspace,
                                        int64_t workspace_bytes, int32_t launch_flags,
                                        cudaStream_t stream);

/*
 * Prefix attention: query t sees the prefix_len[g] tokens of its group's prefix, whose
 * table row starts at prefix_offset[g], and then the kv_len[t] tokens of its own row.
 * Query t belongs to group g when g + 1 is the first index i of group_start with
 * group_start[i] > t; a query before group_start[0], or one that no entry exceeds, has
 * no prefix.  (With group_start non-decreasing, group g holds the queries
 * group_start[g] .. group_start[g + 1] - 1.)
 *
 * num_groups     0..512; 0: no prefixes, and the three group arrays may be NULL.
 * group_start    device int32 [num_groups + 1].
 * prefix_len     device int32 [num_groups] (< 0 as 0); any length, whole pages or not.
 * prefix_offset  device int64 [num_groups].
 * kv_len         device int32 [num_queries]: tokens of the query's own row (< 0 as 0).
 * launch_flags   MSA_LAUNCH_PDL.
 * Other arguments, and errors, as above (block_tokens and topk are not used).
 */
msa_status msa_prefix_attention_forward(const msa_attention_cfg *cfg, int64_t num_queries,
                                        const void *q, int64_t num_groups,
                                        const int32_t *group_start, const int32_t *prefix_len,
                                        const int64_t *prefix_offset, const int32_t *kv_len,
                                        const int64_t *table_offset, const int32_t *page_table,
                                        int64_t page_table_len, const msa_cache_desc *k_cache,
                                        const msa_cache_desc *v_cache, const float *scales,
                                        void *out, float *lse, void *workspace,
                                        int64_t workspace_bytes, int32_t launch_flags,
                                        cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MSA_ATTENTION_H */
