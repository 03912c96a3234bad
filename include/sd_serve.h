/*
 * sd_serve.h -- C ABI of the operators that a serving step of drafted trees
 * needs beside those of sd_tree.h on gfx950:
 *
 *   sd_qk_norm_rope        queries and keys out of a projection: the norm of
 *                          each head and the rotation by the token's position
 *   sd_quant_attention     attention of the tree's nodes over a paged cache
 *                          held in 8 bits, whole or through a sliding window
 *                          with sinks, and over each other
 *   sd_tree_verify_sample  the branch that keeps the target's distribution,
 *                          from the target's (and the draft's) probabilities
 *                          and given random numbers
 *   sd_quant_append        the kept branch, or a prompt, quantised and
 *                          appended to that cache
 *
 * The conventions of sd_verify.h and sd_tree.h hold: trees, page tables, status
 * bits, ownership, streams, workspaces and which outputs may be inputs.
 */
#ifndef SD_SERVE_H
#define SD_SERVE_H

#include "sd_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of a cache held in 8 bits. */
#define SD_I8   3            /* whole numbers -127 .. 127                      */
#define SD_E4M3 4            /* OCP e4m3: 1 sign, 4 exponent, 3 mantissa bits,
                                largest value 448                              */

#define SD_MIN_BLOCK 16      /* slots that share a scale, at least             */

/* Children of a node were drawn without replacement (sd_tree_verify_sample). */
#define SD_NO_REPLACEMENT 4u

/* Per-request status bit beside those of sd_tree.h. */
#define SD_ST_BAD_SCALE (1u << 14)  /* scales outside their range: their blocks count
                                       as absent                                    */

/* ------------------------------------------------------------------------
 * Norm and rotation of queries and keys.
 * Every head x of D elements of a token at position P becomes
 *   y = x / sqrt(mean(x^2) + eps) * weight      (y = x where weight is NULL)
 *   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),
 *   t = P * inv_freq[j],  j < rot / 2,
 * with (a, b) = (j, j + rot / 2), or (2 j, 2 j + 1) where `interleaved`;
 * elements at and past rot are not rotated.  All of it in fp32 (the angle in 64
 * bits, reduced to one turn), rounded once to the element type.
 * Outputs may be the inputs (the same pointer and strides); otherwise they
 * overlap neither them nor each other.
 * ------------------------------------------------------------------------ */
typedef struct sd_qk_norm_rope_args {
  const void    *q;              /* [N][H_q][D]; 16-byte aligned rows (pointers */
  const void    *k;              /* [N][H_k][D]   and strides, in elements and
                                    multiples of 8); NULL where H_k is 0        */
  void          *q_out, *k_out;
  int64_t        q_node, q_head, k_node, k_head;
  int64_t        q_out_node, q_out_head, k_out_node, k_out_head;   /* no two rows
                                    of an output share memory                   */
  const void    *q_weight;       /* [D] of the element type, 16-byte aligned, or
                                    NULL                                        */
  const void    *k_weight;
  const int32_t *positions;      /* [N]                                         */
  const float   *inv_freq;       /* [rot / 2]                                   */
  int32_t        dtype;          /* SD_BF16 or SD_F16                           */
  int32_t        N;              /* >= 1; from 2^24 on only with few heads      */
  int32_t        H_q;            /* >= 1; H_q + H_k <= 65535                    */
  int32_t        H_k;            /* >= 0                                        */
  int32_t        D;              /* 64, 128 or 256                              */
  int32_t        rot;            /* a multiple of 16, 16 .. D                   */
  int32_t        interleaved;
  float          eps;            /* finite, >= 0                                */
} sd_qk_norm_rope_args_t;

int sd_qk_norm_rope(const sd_qk_norm_rope_args_t *args, void *stream);

/* ------------------------------------------------------------------------
 * Cache in 8 bits.  Slots lie in pages as in sd_kv_cache_t, one byte an
 * element; `block` slots of one page and head share a scale: the value of an
 * element is its code times
 *   scale[page * scale_page + h * scale_head + place / block].
 * A scale is 0 (its block's values are 0) or within [2^-50, 2^50]; slots of a
 * block whose key or value scale is anything else count as absent and set
 * SD_ST_BAD_SCALE.  An e4m3 code that is not a number counts as 0.
 * ------------------------------------------------------------------------ */
typedef struct sd_quant_cache {
  void          *k, *v;          /* 16-byte aligned, the same strides           */
  float         *k_scale, *v_scale;
  int64_t        page_stride;    /* bytes, multiples of 16, >= 0                */
  int64_t        head_stride;
  int64_t        slot_stride;    /* >= D                                        */
  int64_t        scale_page;     /* entries, >= 0                               */
  int64_t        scale_head;
  const int32_t *page_table;     /* as in sd_kv_cache_t                         */
  int64_t        ld_table;
  const int32_t *context_lens;
  int32_t        code;           /* SD_I8 or SD_E4M3                            */
  int32_t        B;              /* 1 .. 65535                                  */
  int32_t        H_kv;           /* 1 .. 32767                                  */
  int32_t        D;              /* 64 or 128                                   */
  int32_t        page_size;      /* a power of two, 16 .. SD_MAX_PAGE_SIZE      */
  int32_t        block;          /* a power of two, SD_MIN_BLOCK .. page_size   */
  int32_t        num_pages;
  int32_t        max_pages;
} sd_quant_cache_t;

/* ------------------------------------------------------------------------
 * Attention over the 8-bit cache.
 * Query head g of node i of request b attends, with scores scale * q . k and
 * KV head g / (H_q / H_kv), the slots of its cache in use and, of its own tree,
 * itself and its ancestors (parents NULL: itself and the nodes before it).
 * The position of slot t is t, that of a node context_lens[b] + its depth (the
 * root's is 0).  With window > 0 a row at position P sees a key at position p
 * only if p < sinks or P - p < window.
 * k_new and v_new are of the queries' type and enter as they are.
 * out = softmax(scores) . v, rounded once to the queries' type; out_lse (may be
 * NULL) = log sum exp(scores).  A row that sees nothing gets zeros and -inf.
 * Keys and values that a row does not see never reach its result.  Pages and blocks
 * of slots outside the sinks and the root's window are not looked at and report
 * nothing.  Rows of a request of wrong length get zeros and -inf; rows of one whose
 * node offsets are wrong, and rows of packed nodes that belong to no request, are left
 * as they were.
 * out [N][H_q][D] and out_lse [N][H_q] are contiguous; out may be q where q is.
 * ------------------------------------------------------------------------ */
typedef struct sd_quant_attention_args {
  sd_quant_cache_t cache;
  const void     *q;             /* [N][H_q][D]; 16-byte aligned rows (this     */
  const void     *k_new;         /* [N][H_kv][D]   and the strides below in     */
  const void     *v_new;         /* [N][H_kv][D]   elements, multiples of 8)    */
  int64_t         q_node, q_head;
  int64_t         k_node, k_head;
  int64_t         v_node, v_head;
  const int32_t  *node_offsets;  /* [B + 1]                                     */
  const int32_t  *parents;       /* [N] or NULL                                 */
  int32_t         dtype;         /* SD_BF16 or SD_F16                           */
  int32_t         N;             /* packed nodes, >= 1                          */
  int32_t         max_nodes;     /* 1 .. SD_MAX_NODES                           */
  int32_t         H_q;           /* a multiple of H_kv, <= SD_MAX_GROUP * H_kv  */
  int32_t         window;        /* 0: every slot; else >= 1                    */
  int32_t         sinks;         /* >= 0; 0 without a window                    */
  float           scale;         /* finite                                      */
} sd_quant_attention_args_t;

/* Workspace bytes (depends on sizes only; 0 for short tables, then workspace may
 * be NULL). */
int sd_quant_attention_workspace_bytes(const sd_quant_attention_args_t *args, size_t *bytes);

int sd_quant_attention(const sd_quant_attention_args_t *args, void *workspace,
                       size_t workspace_bytes, void *out, float *out_lse,
                       uint32_t *out_status, void *stream);

/* ------------------------------------------------------------------------
 * Append to the 8-bit cache.  Row i of request b's new rows (node path[b *
 * ld_path + i] for i < path_lens[b], or with path NULL its i-th node, all of
 * them) becomes slot context_lens[b] + i of every KV head.  Per block of slots,
 * KV head and of keys and values each, all in fp32:
 *   scale = max(old, clamp(amax / M, 2^-50, 2^50)),  M = 127 (SD_I8) or 448,
 * amax over the new rows of the block (nothing where it is 0); old is the block's
 * scale where slots of it are in use already, else 0.  Codes are x * (1 / scale)
 * rounded to nearest, ties to even, and kept within +-M.  Where the scale of a
 * block in use grows, its codes are rounded again: (code * old) * (1 / scale).
 * Elements that are not finite do not enter amax; NaN becomes 0, infinities +-M,
 * and the request reports SD_ST_NONFINITE (it is not invalid for that).  An old
 * scale outside its range counts as 0.
 * out_context[b] = context_lens[b] + rows.  Rows of a bad page are not written.
 * An invalid request appends nothing: out_context[b] = context_lens[b].
 * The pages that hold the appended slots belong to one request only, and each
 * head's rows and scales are its own: strides of 0 are refused.
 * ------------------------------------------------------------------------ */
typedef struct sd_quant_append_args {
  sd_quant_cache_t cache;
  const void    *k_new;          /* [N][H_kv][D]; 16-byte aligned rows          */
  const void    *v_new;
  int64_t        k_node, k_head;
  int64_t        v_node, v_head;
  const int32_t *node_offsets;   /* [B + 1]                                     */
  const int32_t *path;           /* [B] rows of node indices within the request,
                                    or NULL                                     */
  int64_t        ld_path;        /* >= max_new                                  */
  const int32_t *path_lens;      /* [B] in [0, nodes of the request]            */
  int32_t        dtype;          /* of the new rows: SD_BF16 or SD_F16          */
  int32_t        N;
  int32_t        max_new;        /* nodes of a request, at most; with a path
                                    <= SD_MAX_NODES; less than 2^24 blocks      */
} sd_quant_append_args_t;

int sd_quant_append(const sd_quant_append_args_t *args, int32_t *out_context,
                    uint32_t *out_status, void *stream);

/* ------------------------------------------------------------------------
 * Verify of a tree against probabilities.  p = target_probs of node c, a row of
 * V fp32 numbers >= 0 whose sum is 1; q = draft_probs of c, the row that c's
 * children were drawn from (V_draft numbers; tokens past them have q = 0).  At
 * node c, from the root on, its children are tested in their order:
 *   cut = 0, Z = 1, r = 1;
 *   the child with token x and random number u = accept_uniforms[child] is
 *   accepted if  u * (q(x) * r) * Z < max(p(x) - cut * q(x), 0);
 *   otherwise  cut += Z * r,  Z = sum of max(p - cut * q, 0)  (and with
 *   SD_NO_REPLACEMENT r = 1 / (1 - the sum of q over the tokens rejected so far
 *   at c), 0 where nothing is left).
 * An accepted child is the next c.  Where none is (or there is none), the last
 * token is drawn from max(p - cut * q, 0): the first token whose cumulative sum
 * passes draw_uniforms[b] times the total.  The tokens emitted then have the
 * target's distribution.  A total of 0 after a rejection sets SD_ST_RESID_ZERO,
 * no further child is tested, and the token is drawn from p.  A tested child
 * with q(x) = 0 sets SD_ST_Q_ZERO.
 * draft_probs NULL: children are not drawn but given (a beam's).  A child with
 * token x is accepted if u * Z < p(x), where Z = 1 - the sum of p over the tokens
 * rejected so far at c (a rejected token has p = 0 from then on); the last token
 * is drawn from p without the rejected tokens.  Where they were all that p holds (its
 * numbers sum to 1 only within rounding, so even the last of them can be rejected),
 * SD_ST_RESID_ZERO is set and the token is drawn from p.
 * Arithmetic is in 64 bits, but the sums of up to 64 slices that a row is cut into
 * are kept to 46 bits (2^-45 of themselves).  Outputs as in sd_tree_verify_greedy: out_accepted
 * [B], out_path [B][max_nodes], out_tokens [B][max_nodes]; with SD_NO_BONUS the
 * last token is left out where the walk ends at a node without children.
 * Only what the walk uses is examined.  Invalid: SD_ST_BAD_NODES,
 * SD_ST_BAD_DRAFT_ID (a drafted token outside [0, V)), SD_ST_BAD_PARAM (a used
 * random number outside [0, 1)), SD_ST_NONFINITE (a used probability that is
 * negative or not finite, or a total of 0 of p itself), SD_ST_UNFINISHED:
 * -1 everywhere.
 * ------------------------------------------------------------------------ */
typedef struct sd_tree_sample_args {
  const float   *target_probs;   /* [N] rows, 16-byte aligned                   */
  const float   *draft_probs;    /* [N] rows, 16-byte aligned, or NULL; rows of
                                    nodes without children are not read         */
  int64_t        ld_target;      /* elements between rows, multiples of 4, >= V */
  int64_t        ld_draft;       /* >= V_draft                                  */
  const int32_t *tokens;         /* [N]; the root's is not used                 */
  const int32_t *parents;        /* [N]                                         */
  const int32_t *node_offsets;   /* [B + 1]                                     */
  const float   *accept_uniforms;   /* [N]; the root's is not used              */
  const float   *draw_uniforms;  /* [B]                                         */
  int32_t        B;              /* 1 .. 65535                                  */
  int32_t        N;              /* >= 1                                        */
  int32_t        V;              /* < 2^28                                      */
  int32_t        V_draft;        /* 1 .. V (not used without draft_probs)       */
  int32_t        max_nodes;      /* 1 .. SD_MAX_NODES                           */
  uint32_t       flags;          /* SD_NO_BONUS, SD_NO_REPLACEMENT              */
} sd_tree_sample_args_t;

int sd_tree_sample_workspace_bytes(const sd_tree_sample_args_t *args, size_t *bytes);

int sd_tree_verify_sample(const sd_tree_sample_args_t *args, void *workspace,
                          size_t workspace_bytes, int32_t *out_accepted,
                          int32_t *out_path, int32_t *out_tokens,
                          uint32_t *out_status, void *stream);

/* Test export: sd_tree_verify_sample with this many looks at a pass that is
 * waited for before its request is given up (SD_ST_UNFINISHED).  Negative: with the
 * usual number of them, and only half of the workgroups that share a request come: they
 * take the others' slices over. */
int sd_debug_tree_sample_polls(const sd_tree_sample_args_t *args, void *workspace,
                               size_t workspace_bytes, int32_t *out_accepted,
                               int32_t *out_path, int32_t *out_tokens,
                               uint32_t *out_status, int32_t polls, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SD_SERVE_H */
