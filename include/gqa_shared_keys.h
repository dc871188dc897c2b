/*
 * gqa_shared_keys.h -- C ABI of the GB300 (sm_103a) library, second part:
 * attention of many query rows over keys they share.
 *
 * gqa_decode.h serves one or a few new tokens per sequence, each sequence with
 * a cache of its own.  Here are the two serving operators whose query rows are
 * many: cross attention of a decoder's tokens to an encoder's states, and
 * decode attention of a batch whose sequences all begin with the same prefix,
 * held and read once.  Both compute
 *
 *     O[r,:] = sum_j softmax_j(scale * q[r,:] . K[j,:]) V[j,:]
 *     lse[r] = ln sum_j exp(scale * q[r,:] . K[j,:])
 *
 * per query row r over the keys j that it sees; a row that sees none yields
 * O = 0, lse = -inf.  Scores, softmax and sums are fp32, P enters the value
 * MMA in in_dtype, as in the decode kernel.  The MMA's fp32 accumulator
 * truncates: a CTA that adds up n blocks of 128 keys leaves O up to ~5e-7 n
 * (relative to the weighted |v|) too small, 2e-4 at 64000 keys.  Results are
 * bit-identical from run to run.
 *
 * A score of NaN makes its row NaN, O and lse; one of -inf is a key that is not
 * seen; one of +inf makes the row NaN.  V's infinities and NaN reach O of every
 * row that sees their key, and of those from which only the causal mask hides
 * it: their weight is 0, and 0 * NaN is NaN.  What lies past a length is never
 * used, whatever it is.
 *
 * The conventions of gqa_decode.h hold: device pointers, caller-owned memory,
 * dense row-major tensors, asynchronous on `stream`, checked before anything
 * is launched, on the current device; make one call outside stream capture
 * first.  Calls that may overlap on the GPU need a workspace each, and so do
 * captured graphs that may.  The library has no gradients: these are forward
 * operators of a serving path.
 */
#ifndef GQA_SHARED_KEYS_H
#define GQA_SHARED_KEYS_H

#include "gqa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Query heads that share a KV head: at most GQA_MAX_GROUP (the rows of one
 * query token must fit in one 128-row tile). */
#define GQA_MAX_GROUP 128

/*
 * Cross attention.  desc: batch, q_tokens (any number of query tokens),
 * q_heads, kv_heads, head_dim, max_seqlen (the capacity of k and v along the
 * encoder's positions), scale, out_dtype and in_dtype as in gqa_decode.h;
 * causal must be 0 (every token sees every valid key) and reduction
 * GQA_REDUCE_AUTO, else GQA_ERR_UNSUPPORTED.
 *   q        in_dtype [B, nq, Hq, d], 16-byte aligned
 *   k, v     in_dtype [B, S_max, Hkv, d], 16-byte aligned: the encoder's states
 *   kv_lens  int32 [B] device array; keys [0, L_b) of entry b are seen, L_b in
 *            [0, S_max] (values outside are clamped and flagged as
 *            GQA_ERR_BAD_SEQLEN by gqa_decode_get_error).  Positions from L_b
 *            on may hold any values, they are never used.
 *   out      [B, nq, Hq, d] of out_dtype, 16-byte aligned; written in full
 *   lse      fp32 [B, nq, Hq], or NULL
 *   workspace  >= gqa_cross_workspace_size() bytes, 256-byte aligned (may be
 *            NULL when that is 0); needs no initialisation
 * Up to GQA_MAX_QROWS rows per KV head (nq * Hq / Hkv: a decode step) run as
 * gqa_decode_attn does, with the results of that call; more rows run in
 * 128-row tiles.
 */
size_t gqa_cross_workspace_size(const gqa_desc_t* desc);
gqa_status_t gqa_cross_attn(const gqa_desc_t* desc, const void* q, const void* k, const void* v,
                            const int32_t* kv_lens, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * Decode attention behind a shared prefix.  Every sequence of the batch sees
 * the keys of the prefix, [0, P), and then its own, [0, L_b) of its cache; the
 * softmax runs over both together.  desc describes the decode step as in
 * gqa_decode_attn (max_seqlen: the capacity of the sequences' own caches;
 * q_tokens * q_heads / kv_heads <= GQA_MAX_QROWS, as there: the rows of a
 * sequence's own keys are then one tile, on which the causal mask and the split
 * of its keys rely); reduction must be GQA_REDUCE_AUTO.  The causal flag masks among a sequence's own keys (its nq
 * new tokens are the last of them; token t sees j <= L_b - nq + t); the prefix
 * is seen by every token.
 *   k_prefix, v_prefix  in_dtype [max_prefix, Hkv, d], 16-byte aligned
 *   prefix_len  int32 device scalar: P in [0, max_prefix] (clamped and flagged
 *            like a length).  Positions from P on are never used.
 *   k_cache, v_cache, seqlens  the sequences' own keys, as in gqa_decode_attn;
 *            L_b = 0 is a sequence with nothing but the prefix
 *   out, lse, workspace  as in gqa_cross_attn
 */
size_t gqa_prefix_workspace_size(const gqa_desc_t* desc, int max_prefix);
gqa_status_t gqa_prefix_attn(const gqa_desc_t* desc, const void* q, const void* k_prefix, const void* v_prefix,
                             const int32_t* prefix_len, int max_prefix, const void* k_cache, const void* v_cache,
                             const int32_t* seqlens, void* out, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * Host-side view of the tiled kernel's work decomposition, for inspection and
 * testing (the counterpart of gqa_decode_plan).  max_prefix = 0: the launch of
 * gqa_cross_attn(desc) with more than GQA_MAX_QROWS rows per KV head, one
 * section of batch entries; else that of gqa_prefix_attn, section 0 the prefix
 * (one entry, prefix_len keys), section 1 the sequences' own keys.  A triple
 * is an (entry, KV head, tile group).  kv_lens_host: int32 [B] in host memory;
 * sm_count: SMs to plan for (0: those of the current device).  Fills
 *   *num_ctas, *every_piece (whether every triple leaves partials),
 *   info     per section: query tokens of a tile, tile groups, whether both
 *            tiles hold the same rows with the keys in turn, pieces its part
 *            of the workspace holds (8 int in all)
 *   items    (if not NULL) up to max_items records of 9 int32 each: cta,
 *            section, b, h, tile group, blk_begin, blk_end, piece (-1 = final
 *            output), n_pieces (of the triple, in the item of its first block),
 *            in the order each CTA processes them; triples without keys of
 *            which there is only that to record come last
 *   *num_items  their total count
 * sm_count and lengths as gqa_decode_plan; any output but items may be NULL.
 */
gqa_status_t gqa_shared_keys_plan(const gqa_desc_t* desc, int prefix_len, int max_prefix, const int32_t* kv_lens_host,
                                  int sm_count, int* num_ctas, int* every_piece, int* info, int32_t* items,
                                  int64_t max_items, int64_t* num_items);

#ifdef __cplusplus
}
#endif

#endif /* GQA_SHARED_KEYS_H */
