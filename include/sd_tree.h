/*
 * sd_tree.h -- C ABI of the tree-drafting operators on gfx950: what a verify
 * step needs when the draft proposes a tree of tokens instead of a chain.
 *
 *   sd_beam_select, sd_beam_reorder   grow the tree: the best continuations
 *                                     over beams and vocabulary, and the
 *                                     draft's states moved to their beams
 *   sd_tree_attention                 attention of the tree's nodes over a
 *                                     paged key/value cache and each other
 *   sd_tree_verify_greedy             the branch that the target agrees with
 *   sd_cache_commit                   that branch's keys and values appended
 *                                     to the cache, and the attention weight
 *                                     its rows gave to every cached token
 *   sd_cache_evict                    the cache cut to a budget of tokens by
 *                                     that accumulated weight
 *
 * The conventions of sd_verify.h hold (device pointers owned by the caller,
 * asynchronous work on `stream`, host-checkable errors by return code,
 * data-dependent ones per request in out_status, no memory allocated,
 * workspaces that need no initialization and are not shared by calls that
 * overlap in time).  The device that owns the pointers is the current one.  An
 * output overlaps no input, no other output and not the workspace, except where
 * an operator says so; the same pointer for both is refused where that would
 * change results.
 *
 * Trees.  Request b has the nodes node_offsets[b] .. node_offsets[b + 1] - 1
 * of the packed node arrays, at most max_nodes (<= SD_MAX_NODES) of them.
 * Node 0 is the root: the last committed token, whose key and value are not
 * in the cache yet.  The others are drafted.  parents[i] is the index within
 * the request of node i's parent, -1 for the root; a parent comes before its
 * children.
 *
 * Cache.  Slot t of request b is place t % page_size of page
 * page_table[b * ld_table + t / page_size]; the D elements of KV head h there
 * are at page * page_stride + h * head_stride + place * slot_stride in k and
 * in v.  context_lens[b] slots are in use.  A table entry outside
 * [0, num_pages) is a bad page: it is never accessed, its slots count as
 * absent, and SD_ST_BAD_PAGE is reported.  Entries past the slots in use
 * (and, for a commit, the appended ones) are not read.
 */
#ifndef SD_TREE_H
#define SD_TREE_H

#include "sd_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of queries, keys and values beside SD_BF16. */
#define SD_F16 2

#define SD_MAX_NODES 64      /* nodes of one request's tree                  */
#define SD_MAX_BEAMS 64      /* beams of one request, before and after       */
#define SD_MAX_PAGE_SIZE 1024
#define SD_MAX_GROUP 32      /* query heads of one KV head                   */

/* Per-request status bits beside those of sd_verify.h. */
#define SD_ST_BAD_LEN   (1u << 8)   /* context length outside the table (or, for a
                                       commit, the table or the weight rows
                                       cannot hold the appended slots)  invalid */
#define SD_ST_BAD_NODES (1u << 9)   /* node offsets decreasing, beyond N or over
                                       max_nodes; no node at all where a root
                                       is needed                        invalid */
#define SD_ST_BAD_PAGE  (1u << 10)  /* bad pages were left out                  */
#define SD_ST_BAD_TREE  (1u << 11)  /* a parent outside [-1, own index) was taken
                                       as -1 (a node that no walk reaches)       */
#define SD_ST_BAD_PATH  (1u << 12)  /* path length outside [0, nodes], or a path
                                       node outside the request         invalid */
#define SD_ST_UNFINISHED (1u << 13) /* a walk was given up: calls that overlap in time
                                       shared its workspace              invalid */
#define SD_ST_TREE_INVALID_MASK (SD_ST_INVALID_MASK | SD_ST_BAD_LEN | SD_ST_BAD_NODES | SD_ST_BAD_PATH | \
                                 SD_ST_UNFINISHED)

typedef struct sd_kv_cache {
  void          *k, *v;          /* 16-byte aligned, the same strides           */
  int64_t        page_stride;    /* elements, multiples of 8, >= 0              */
  int64_t        head_stride;
  int64_t        slot_stride;    /* >= D                                        */
  const int32_t *page_table;     /* [B] rows of max_pages entries               */
  int64_t        ld_table;       /* entries between rows, >= max_pages          */
  const int32_t *context_lens;   /* [B] in [0, max_pages * page_size]           */
  int32_t        dtype;          /* SD_BF16 or SD_F16                           */
  int32_t        B;              /* requests, 1 .. 65535                        */
  int32_t        H_kv;           /* KV heads, 1 .. 65535                        */
  int32_t        D;              /* head size: 64 or 128                        */
  int32_t        page_size;      /* a power of two, <= SD_MAX_PAGE_SIZE         */
  int32_t        num_pages;      /* pages of the pool                           */
  int32_t        max_pages;      /* table entries of a request; at most 2^30
                                    slots                                       */
} sd_kv_cache_t;

/* ------------------------------------------------------------------------
 * Attention of drafted nodes over the cache.
 * Query head g of node i attends, with scores scale * q . k, the slots of
 * its request's cache in use and the nodes of its own tree that it sees, all
 * with KV head g / (H_q / H_kv):
 *   tree_mask != NULL   node j for every set bit j of tree_mask[i] (bits at
 *                       or past the request's node count are ignored);
 *   else parents != NULL  itself and its ancestors;
 *   else                itself and the nodes before it (a chain).
 * out = softmax(scores) . v, rounded once to the element type; out_lse (may
 * be NULL) = log sum exp(scores).  A row that sees nothing gets zeros and
 * -inf.  Keys and values that a row does not see never reach its result,
 * whatever they hold.  Rows of a request of wrong length get zeros and -inf;
 * rows of one whose node offsets are wrong, and rows of packed nodes that belong
 * to no request, are left as they were.
 * out [N][H_q][D] and out_lse [N][H_q] are contiguous; out may be q where q is.
 * ------------------------------------------------------------------------ */
typedef struct sd_tree_attention_args {
  sd_kv_cache_t   cache;
  const void     *q;             /* [N][H_q][D]; 16-byte aligned rows (this     */
  const void     *k_new;         /* [N][H_kv][D]   and the strides below in     */
  const void     *v_new;         /* [N][H_kv][D]   elements, multiples of 8)    */
  int64_t         q_node, q_head;       /* strides of nodes and heads           */
  int64_t         k_node, k_head;
  int64_t         v_node, v_head;
  const int32_t  *node_offsets;  /* [B + 1]                                     */
  const int32_t  *parents;       /* [N] or NULL                                 */
  const uint64_t *tree_mask;     /* [N] or NULL                                 */
  int32_t         N;             /* packed nodes, >= 1                          */
  int32_t         max_nodes;     /* 1 .. SD_MAX_NODES                           */
  int32_t         H_q;           /* a multiple of H_kv, <= SD_MAX_GROUP * H_kv  */
  float           scale;         /* finite                                      */
} sd_tree_attention_args_t;

/* Workspace bytes (depends on H_q / H_kv, D, max_nodes and the table's size
 * only; 0 for short tables, then workspace may be NULL).  SD_EUNSUPPORTED where
 * B * H_kv * (packed rows / 16) * (slots of a table / 64) could pass 2^31. */
int sd_tree_attention_workspace_bytes(const sd_tree_attention_args_t *args, size_t *bytes);

int sd_tree_attention(const sd_tree_attention_args_t *args, void *workspace,
                      size_t workspace_bytes, void *out, float *out_lse,
                      uint32_t *out_status, void *stream);

/* ------------------------------------------------------------------------
 * Greedy verify of a tree.  From the root, go from node c to the first child
 * whose token is argmax(logits row of c) (the lowest id among equal maxima)
 * as long as there is one.
 * out_accepted [B]: drafted nodes visited; out_path [B][max_nodes]: the nodes
 * visited, the root first, -1 padded; out_tokens [B][max_nodes]: the tokens of
 * the drafted nodes visited and the argmax of the last one's row, -1 padded
 * (with SD_NO_BONUS that last token is left out where the walk ended at a node
 * without children).  Rows of nodes that the walk does not visit do not enter
 * the results: a NaN there is not reported.  An invalid request (SD_ST_BAD_NODES,
 * SD_ST_BAD_DRAFT_ID: a drafted token outside [0, V), SD_ST_NONFINITE: a
 * NaN in a visited row, SD_ST_UNFINISHED) gets -1 everywhere.
 * ------------------------------------------------------------------------ */
typedef struct sd_tree_verify_args {
  const void    *logits;         /* [N] rows of V, SD_F32 or SD_BF16, 16-byte aligned rows */
  int64_t        ld;             /* elements between rows, >= V                 */
  const int32_t *tokens;         /* [N]; the root's is not used                 */
  const int32_t *parents;        /* [N]                                         */
  const int32_t *node_offsets;   /* [B + 1]                                     */
  int32_t        dtype;
  int32_t        B;              /* 1 .. 65535                                  */
  int32_t        N;              /* 1 .. 2^24 - 1                               */
  int32_t        V;              /* < 2^28                                      */
  int32_t        max_nodes;
  uint32_t       flags;          /* SD_NO_BONUS                                 */
} sd_tree_verify_args_t;

int sd_tree_verify_workspace_bytes(const sd_tree_verify_args_t *args, size_t *bytes);

int sd_tree_verify_greedy(const sd_tree_verify_args_t *args, void *workspace,
                          size_t workspace_bytes, int32_t *out_accepted,
                          int32_t *out_path, int32_t *out_tokens,
                          uint32_t *out_status, void *stream);

/* ------------------------------------------------------------------------
 * Append of the kept branch.  For i < path_lens[b] the keys and values of
 * node path[b * ld_path + i] become those of slot context_lens[b] + i;
 * positions (if given) of those slots, for every KV head, become seen[b] + i;
 * out_context[b] = context_lens[b] + path_lens[b].
 * With mass_out given, the attention weight of the branch is accumulated:
 *   w(t) = sum over i < path_lens[b] and the heads g of KV head h of
 *          exp(scale * q_i,g . k_t - lse_i,g),
 * where row i attends the slots in use and the branch's nodes 0..i, and
 *   mass_out[t] = decay * mass_in[t] + w(t)   for t < context_lens[b]
 *   mass_out[t] = w(t)                        for the appended slots;
 * slots behind them are left as they were.  With decay = 0 mass_in is not
 * read.  lse is what sd_tree_attention gave for these rows; one of -inf (the row
 * saw nothing) makes its row add no weight.  A slot of a bad
 * page has w = 0; an appended slot on one is not written.  mass_in may be
 * mass_out.  An invalid request appends
 * nothing: its mass and positions stay and out_context[b] = context_lens[b].
 * The pages that hold the appended slots belong to one request only.
 * ------------------------------------------------------------------------ */
typedef struct sd_cache_commit_args {
  sd_kv_cache_t  cache;
  const void    *k_new;          /* as in sd_tree_attention                     */
  const void    *v_new;
  int64_t        k_node, k_head;
  int64_t        v_node, v_head;
  const int32_t *node_offsets;
  const int32_t *path;           /* [B] rows of node indices within the request */
  int64_t        ld_path;        /* >= max_nodes                                */
  const int32_t *path_lens;      /* [B] in [0, nodes of the request]            */
  int32_t        N;
  int32_t        max_nodes;
  /* weights: all of these, or mass_out NULL */
  const void    *q;
  int64_t        q_node, q_head;
  const float   *lse;            /* [N][H_q]                                    */
  int32_t        H_q;
  float          scale;
  float          decay;          /* finite                                      */
  const float   *mass_in;        /* [B][H_kv] rows, ld_mass apart               */
  float         *mass_out;
  int64_t        ld_mass;        /* entries between rows, >= 1                  */
  /* positions: both or neither */
  int32_t       *positions;      /* [B][H_kv] rows, ld_mass apart               */
  const int32_t *seen;           /* [B] tokens that the request has had         */
} sd_cache_commit_args_t;

int sd_cache_commit(const sd_cache_commit_args_t *args, int32_t *out_context,
                    uint32_t *out_status, void *stream);

/* ------------------------------------------------------------------------
 * Eviction.  Every KV head of request b (B * H_kv < 2^31) keeps
 * min(context_lens[b], budget) of its slots: first those of positions < sinks or >= seen[b] - recent, then
 * those of the largest mass (a NaN counts as -inf), the lower slot first among
 * equals.  The kept slots end up as slots 0 .. budget - 1: those below the
 * budget stay, and the j-th kept slot at or past it moves (keys, values, mass,
 * position) to the j-th of the freed ones.  Attention does not depend on the
 * order of the slots, so only displaced rows are read and written.
 * mass_out and positions_out are written for the slots kept; they may be
 * mass_in and positions_in.  out_context[b] = min(context_lens[b], budget).
 * positions NULL: sinks = recent = 0, no slot comes first.  An invalid request is left as it was.
 * A bad page's slots are ranked like the others, and their masses and positions
 * move like the others', but their keys and values are neither read nor written:
 * the place that such a row would move to keeps the row that it held, under the
 * mass and position of the other.  So a request reported with SD_ST_BAD_PAGE has
 * a cache that is no longer that of its tokens.  The request's pages are its own,
 * and so are each head's rows of a page: strides of 0 are refused.
 * ------------------------------------------------------------------------ */
typedef struct sd_cache_evict_args {
  sd_kv_cache_t  cache;
  const float   *mass_in;        /* [B][H_kv] rows, ld_mass apart               */
  float         *mass_out;
  const int32_t *positions_in;   /* same layout, or NULL                        */
  int32_t       *positions_out;
  int64_t        ld_mass;        /* >= max_pages * page_size                    */
  const int32_t *seen;           /* [B]; NULL only without positions            */
  int32_t        budget;         /* >= 1                                        */
  int32_t        recent;         /* >= 0, sinks + recent <= budget              */
  int32_t        sinks;
} sd_cache_evict_args_t;

int sd_cache_evict_workspace_bytes(const sd_cache_evict_args_t *args, size_t *bytes);

int sd_cache_evict(const sd_cache_evict_args_t *args, void *workspace,
                   size_t workspace_bytes, int32_t *out_context,
                   uint32_t *out_status, void *stream);

/* ------------------------------------------------------------------------
 * Beam selection.  Candidate (w, v): scores[b][w] + logits[b][w][v] -
 * log sum exp(logits[b][w]); the n_out largest over all beams and tokens in
 * descending order, the lower w * V + v first among equals.  A beam with
 * ended[b][w] != 0 has one candidate, (w, eos_id) at scores[b][w]; a beam at
 * -inf has none.  Candidates at -inf are none either; places without a
 * candidate get score -inf, parent and token -1.  The logits of ended beams
 * and of beams at -inf are not examined.
 * out_ended (may be NULL) = ended[parent] or token == eos_id, 0 without one.
 * SD_ST_NONFINITE (a NaN or +inf logit, or only -inf, in an examined row) and
 * SD_ST_BAD_PARAM (a NaN or +inf score) are invalid: no candidates.
 * ------------------------------------------------------------------------ */
typedef struct sd_beam_select_args {
  const void    *logits;         /* [B][W] rows of V, SD_F32 or SD_BF16, 16-byte aligned */
  int64_t        ld;
  const float   *scores;         /* [B][W]                                      */
  const uint8_t *ended;          /* [B][W] or NULL                              */
  int32_t        dtype;
  int32_t        B;              /* 1 .. 2^20, B * W < 2^24                     */
  int32_t        W;              /* 1 .. SD_MAX_BEAMS                           */
  int32_t        V;              /* < 2^24                                      */
  int32_t        n_out;          /* 1 .. SD_MAX_BEAMS                           */
  int32_t        eos_id;         /* used where ended, and for out_ended         */
} sd_beam_select_args_t;

int sd_beam_select_workspace_bytes(const sd_beam_select_args_t *args, size_t *bytes);

int sd_beam_select(const sd_beam_select_args_t *args, void *workspace,
                   size_t workspace_bytes, float *out_scores, int32_t *out_parents,
                   int32_t *out_tokens, uint8_t *out_ended, uint32_t *out_status,
                   void *stream);

/* Reordering of beam states: row (l, b, w, s) of out becomes row
 * (l, b, parents[b][w], s) of in, for the first lengths[b] of max_units
 * units of unit_bytes each (all of them where lengths is NULL; a length
 * outside [0, max_units] is clamped).  Strides in bytes, rows contiguous.
 * Where out is in (the same pointer; W_in = W_out and equal strides), the rows are
 * permuted in place; otherwise the two must not overlap.  A parent outside
 * [0, W_in) leaves its row as it was.  Units past the length are left as they
 * were.  No two rows of out share memory (strides of 0 are refused; in may be
 * broadcast).  unit_bytes and all strides are multiples of 16, pointers 16-byte
 * aligned; W_in, W_out <= SD_MAX_BEAMS, B and layers * segs <= 65535. */
typedef struct sd_beam_reorder_args {
  const void    *in;
  void          *out;
  int64_t        in_layer, in_request, in_beam, in_seg;      /* strides in bytes */
  int64_t        out_layer, out_request, out_beam, out_seg;
  const int32_t *parents;        /* [B][W_out]                                  */
  const int32_t *lengths;        /* [B] or NULL                                 */
  int64_t        unit_bytes;
  int32_t        layers, B, W_in, W_out, segs, max_units;
} sd_beam_reorder_args_t;

int sd_beam_reorder(const sd_beam_reorder_args_t *args, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SD_TREE_H */
