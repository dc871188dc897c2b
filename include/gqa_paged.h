/*
 * gqa_paged.h -- C ABI of the GB300 (sm_103a) library, third part: serving
 * from a paged cache, with drafted tokens.
 *
 * A cache here is a pool of pages of page_size positions each, and a sequence's
 * positions lie in the pages that its row of page_table names, in their order.
 * One verification step of drafted tokens is
 *
 *     gqa_tree_from_parents   the drafts' tree as bits, and their positions
 *     gqa_paged_append        queries and keys rotated to their positions, keys
 *                             and values put into the cache
 *     gqa_tree_attn           attention of the drafts over the cache, each along
 *                             its own branch
 *     gqa_paged_keep          the accepted branch moved together in the cache
 *
 * and a step of one token, or a chunk of a prompt, gqa_paged_append and
 * gqa_tree_attn (which takes up to GQA_MAX_TREE_TOKENS tokens of a sequence a call:
 * longer chunks take several, see there).  gqa_rotary_apply rotates a tensor by itself.
 *
 * The conventions of gqa_decode.h hold: device pointers, caller-owned memory,
 * asynchronous on `stream`, checked before anything is launched, on the current
 * device; make one call outside stream capture first.  Calls of gqa_tree_attn
 * that may overlap on the GPU need a workspace each, and so do captured graphs
 * that may.  Results are bit-identical from run to run, but where two tokens are
 * put into one place of a cache (pages that two sequences share and both write):
 * which of them stays is not defined.
 *
 * What only the device can see -- page numbers, parents, branches, numbers of
 * new tokens -- is checked there: one that is out of its range is flagged as
 * GQA_ERR_BAD_INDEX by gqa_decode_get_error, and nothing outside the buffers is
 * read or written for it.
 */
#ifndef GQA_PAGED_H
#define GQA_PAGED_H

#include "gqa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* New tokens of a sequence in one call of gqa_tree_attn and
 * gqa_tree_from_parents, at most. */
#define GQA_MAX_TREE_TOKENS 256

/* The k and v caches: both have this layout.  Element (page, position, head, i)
 * lies page * page_stride + position * pos_stride + head * head_stride + i
 * elements from the start; strides are positive multiples of 8 and no two
 * elements share a place, so that pages may be [page_size, Hkv, d], [Hkv,
 * page_size, d], or every other one of a pool that holds K and V together. */
typedef struct {
  int num_pages;       /* >= 1: pages of the pool */
  int page_size;       /* positions of a page: a power of two, 16 to 65536 */
  int max_pages;       /* >= 1: columns of page_table */
  int64_t page_stride, pos_stride, head_stride;
} gqa_pages_t;

/* Rotation of the first `dim` elements of a head: pair i (of dim / 2) turns by
 * position * f_i radians,
 *     (a, b) -> magnitude * (a cos - b sin, a sin + b cos),
 * and the other elements stay.  A pair is elements (i, i + dim / 2), or with
 * `interleaved` (2i, 2i + 1).  `inverse` turns back (by minus the angle, with the
 * same magnitude): the transposed map, which is the gradient of the rotation. */
typedef struct {
  int dim;             /* even, 2 .. head_dim */
  int interleaved;
  int inverse;
  float magnitude;     /* >= 0; 0 selects 1 */
} gqa_rotary_t;

/* How gqa_rotary_turns stretches positions by `factor` >= 1:
 *   NONE    not at all: f_i = base^(-2i / dim); factor must be 1
 *   LINEAR  f_i / factor
 *   BASE    base becomes base * factor^(dim / (dim - 2)) (dim 2: nothing changes):
 *           the slowest pair turns factor times slower, the fastest as before
 *   PARTS   pairs that turn at most `slow` times over original_length positions
 *           are divided by factor, those of at least `fast` turns stay, and in
 *           between f_i ((1 - w) / factor + w), w = (turns - slow) / (fast - slow) */
typedef enum {
  GQA_ROTARY_NONE = 0, GQA_ROTARY_LINEAR = 1, GQA_ROTARY_BASE = 2, GQA_ROTARY_PARTS = 3
} gqa_rotary_scaling_t;

/*
 * The table that the kernels turn by, computed on the host into host memory:
 * turns[i] = f_i / (2 pi) as a fraction of a turn in units of 2^-64.  A position
 * times it, modulo 2^64, is the angle without its whole turns: the product is exact,
 * and the table, computed in fp64, is within 2^-54 of a turn, so that the angle is off
 * by position * 2^-54 turns at most (position 10^9: 3.5e-7 radians).  With PARTS that
 * holds where fast^2 <= original_length * (fast - slow) / 16; a steeper ramp loses bits
 * of w.  Copy the table to the device once.
 * base > 1; original_length >= 1 and 0 <= slow < fast with PARTS (else ignored).
 */
gqa_status_t gqa_rotary_turns(int dim, double base, int scaling, double factor, int original_length, double slow,
                              double fast, uint64_t* turns);

/*
 * Rotates every head of every token: x and out are of `dtype` (bf16, fp16 or
 * fp32) and [tokens, heads, head_dim] with x_stride / out_stride elements from
 * token to token (at least heads * head_dim, multiples of 8) and dense heads;
 * out may be x itself (with the same stride), but may not overlap it otherwise.
 *   turns      uint64 [dim / 2], 8-byte aligned
 *   positions  int32 [tokens], of any sign
 * x and out are 16-byte aligned.  fp32 arithmetic, one rounding.
 */
gqa_status_t gqa_rotary_apply(const gqa_rotary_t* rope, const uint64_t* turns, const int32_t* positions,
                              int64_t tokens, int heads, int head_dim, int dtype, const void* x, int64_t x_stride,
                              void* out, int64_t out_stride, void* stream);

/*
 * Puts each sequence's new keys and values into the paged cache, the keys (and,
 * into q_out, the queries) rotated on the way.  desc: batch, q_tokens (new tokens
 * of a sequence, at most; any number), q_heads, kv_heads, head_dim, max_seqlen
 * (positions of a sequence, at most max_pages * page_size), in_dtype; the rest is
 * not used, and neither are the limits on query rows.
 *   q, k, v     in_dtype [B, nq, Hq | Hkv, d], dense heads, with q_stride / ...
 *               elements from token to token (and nq times that from sequence to
 *               sequence), multiples of 8: views of one projection's output will do.
 *               q may be NULL (with q_out): only keys and values then
 *   q_out       in_dtype [B, nq, Hq, d], dense; q itself if that is dense
 *   rope, turns as above (inverse must be 0); both NULL: nothing is rotated
 *   positions   int32 [B, nq], what the tokens are rotated to; NULL: their place
 *               in the sequence
 *   page_table  int32 [B, max_pages], in [0, num_pages) as far as a sequence
 *               reaches, anything behind
 *   seqlens     int32 [B]: positions with the new tokens, L_b in [0, max_seqlen]
 *               (clamped and flagged)
 *   new_lens    int32 [B]: n_b in [0, nq] (clamped and flagged); NULL: nq.  At most
 *               L_b of them are there (an unused slot of a batch has L_b = 0)
 * Token t < n_b goes to position L_b - n_b + t; of tokens behind the last nothing
 * is used or written.  A token whose page is out of range is not put anywhere.
 * All of q, q_out, k, v and the caches are 16-byte aligned.
 */
gqa_status_t gqa_paged_append(const gqa_desc_t* desc, const gqa_pages_t* pages, const gqa_rotary_t* rope,
                              const uint64_t* turns, const int32_t* positions, const void* q, int64_t q_stride,
                              const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* q_out,
                              void* k_cache, void* v_cache, const int32_t* page_table, const int32_t* seqlens,
                              const int32_t* new_lens, void* stream);

/*
 * The tree of each sequence's drafted tokens, as gqa_tree_attn reads it.
 *   parents    int32 [batch, q_tokens]: the parent of token t, an earlier token or
 *              -1 for the last position before them (anything else is flagged and
 *              taken for -1); of tokens behind the last anything
 *   seqlens, max_seqlen, new_lens  as in gqa_paged_append
 *   tree       uint32 [batch, q_tokens, ceil(q_tokens / 32)], written in full: bit
 *              j % 32 of word j / 32 of token t's row says that j is t or one of
 *              its ancestors; 0 behind the last token
 *   positions  int32 [batch, q_tokens] or NULL, written in full: L_b - n_b + the
 *              number of t's ancestors; 0 behind the last token
 * 1 <= q_tokens <= GQA_MAX_TREE_TOKENS.
 */
gqa_status_t gqa_tree_from_parents(int batch, int q_tokens, int max_seqlen, const int32_t* parents,
                                   const int32_t* seqlens, const int32_t* new_lens, uint32_t* tree,
                                   int32_t* positions, void* stream);

/*
 * Attention of each sequence's new tokens over its positions in the paged
 * cache.  Token t < n_b sees every position before the new ones, [0, L_b - n_b),
 * and of the new ones
 *   those whose bit its row of `tree` has set (tree not NULL; desc->causal 0),
 *   the first to itself (tree NULL, desc->causal not 0: a chain of drafts or a
 *   chunk of a prompt), or
 *   all of them (tree NULL, desc->causal 0).
 * A row that sees nothing, and every row behind the last token, is O = 0,
 * lse = -inf.
 * A chain of n_b > GQA_MAX_TREE_TOKENS tokens, appended in one call, is seen in
 * several, each over the positions up to its own last token: for tokens [i, i + m)
 * of it, L_b - n_b + min(n_b, i + m) as the length and min(max(n_b - i, 0), m) as
 * the number of new tokens.
 * desc as in gqa_decode_attn, with q_tokens <= GQA_MAX_TREE_TOKENS,
 * at most 128 query heads to a KV head and max_seqlen <= max_pages * page_size;
 * reduction must be GQA_REDUCE_AUTO.
 *   q          in_dtype [B, nq, Hq, d], dense, 16-byte aligned
 *   k_cache, v_cache, page_table, seqlens, new_lens  as in gqa_paged_append; a
 *              page out of range reads as zeros
 *   tree       uint32 [B, nq, ceil(nq / 32)]: any bits (bits of new tokens that a
 *              sequence lacks are not looked at)
 *   out        [B, nq, Hq, d] of out_dtype, 16-byte aligned; written in full
 *   lse        fp32 [B, nq, Hq], or NULL
 *   workspace  >= gqa_tree_workspace_size() bytes, 256-byte aligned (may be NULL
 *              when that is 0); needs no initialisation
 * Rounding, infinities and NaN as gqa_shared_keys.h has them: what lies past L_b
 * is never used, a hidden key's K neither; a hidden key's V has weight 0, and
 * 0 * NaN is NaN.
 */
size_t gqa_tree_workspace_size(const gqa_desc_t* desc, const gqa_pages_t* pages);
gqa_status_t gqa_tree_attn(const gqa_desc_t* desc, const gqa_pages_t* pages, const void* q, const void* k_cache,
                           const void* v_cache, const int32_t* page_table, const int32_t* seqlens,
                           const int32_t* new_lens, const uint32_t* tree, void* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * Moves the keys and values of each sequence's accepted branch together behind
 * the positions before the new ones: token path[b][i] to position L_b - n_b + i,
 * i < m_b.  What a branch's keys were rotated to is then their place.
 *   desc       batch, q_tokens, kv_heads, head_dim, max_seqlen, in_dtype as in
 *              gqa_paged_append
 *   path       int32 [B, max_keep]: new tokens, each in [0, n_b) and past the one
 *              before it; the branch ends (and is flagged) at one that is not
 *   keep_lens  int32 [B]: m_b in [0, max_keep] (clamped and flagged)
 *   seqlens_out  int32 [B] or NULL: L_b - n_b + the branch's tokens; may be seqlens
 * A token whose page, or whose place's page, is out of range is not moved (and is
 * flagged); its place counts all the same.
 */
gqa_status_t gqa_paged_keep(const gqa_desc_t* desc, const gqa_pages_t* pages, void* k_cache, void* v_cache,
                            const int32_t* page_table, const int32_t* seqlens, const int32_t* new_lens,
                            const int32_t* path, int max_keep, const int32_t* keep_lens, int32_t* seqlens_out,
                            void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_PAGED_H */
