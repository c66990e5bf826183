/*
 * spec_tree.h -- drafted trees verified over a paged key/value cache.
 *
 * The operations around a verification step whose drafts form a tree (or a
 * chain, or a single token) behind each sequence's cached context:
 *
 *   spec_tree_attention   attention of the drafted nodes over the cached
 *                         context and their own ancestors: the target's pass
 *                         that gives one row per node, each after the node's
 *                         own prefix (the rows "SpecTr-GBV", Methodology,
 *                         Algorithm 1 verifies drafts with).
 *   spec_verify_probs     verification of a chain from given probabilities
 *   spec_verify_tree      ... of a tree, with the caller's random numbers:
 *                         the form of "FlashSpec", Methodology s.1, whose
 *                         input is normalised, so only two numbers a
 *                         candidate are read until the final draw.
 *   spec_kv_slots         block tables and slot maps from request lengths,
 *                         on the device.
 *   spec_kv_append        keys and values written at their slots.
 *
 * One step: attention per layer -> probabilities -> verification -> slots of
 * the accepted path -> append.  The tree's own keys and values stay outside
 * the cache until they are accepted, so a rejected branch never occupies it.
 *
 * Trees.  The nodes of all sequences are packed: cu_nodes[B + 1] (int32,
 * non-decreasing, cu_nodes[0] >= 0) bounds sequence b's nodes, parents[i] is
 * the index of node i's parent within its sequence, or -1.  A node's parent
 * comes before it (parents[i] < i).  A sequence may have no nodes, and at
 * most SV_MAX_NODES.  For a verification node 0 is the root (the last token
 * that is already decided, parent -1) and every other node has a parent.
 *
 * Conventions (streams, errors, status codes, no allocation, nothing kept
 * between calls) are those of spec_verify.h.  Problems in device data mark
 * their own sequence only, as stated at each function.
 */
#ifndef SPEC_TREE_H
#define SPEC_TREE_H

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* fp16, taken by spec_tree_attention (beside SV_BF16) only. */
#define SV_F16 2
/* Largest number of nodes of one sequence's tree. */
#define SV_MAX_NODES 1024
/* Largest head width of spec_tree_attention. */
#define SV_MAX_HEAD_DIM 128

/*
 * spec_verify_probs -- a chain of gamma drafted tokens per sequence, verified
 * against given probabilities with given uniforms.
 *
 * Inputs (device):
 *   target_probs  [B, gamma+1, V]  target probabilities at the gamma draft
 *                                  positions and the one after them.
 *   draft_probs   [B, gamma, V]    the laws the drafts were drawn from, or
 *                                  NULL: point drafts (each drafted token
 *                                  had probability 1).
 *   draft_tokens  [B, gamma] int32
 *   uniforms      [B, gamma] fp32 in [0, 1), one per drafted token.
 *   draw_uniforms [B] fp32 in [0, 1), for the correction or bonus token.
 *   Probabilities are fp32 or bf16 (sv_dtype), dense, of any alignment of the
 *   element type; they are taken as they are (each row as a law of mass 1).
 * Outputs (device): out_accept_len [B], out_tokens [B, gamma+1] as
 * spec_verify.
 *
 * Rule: token x at position i is accepted when u q(x) < p(x).  The first
 * rejection's correction token is drawn from max(p - q, 0) (from p with that
 * token's entry cleared, for point drafts); from p itself where that has no
 * mass (for point drafts: that token); the bonus token, when all are accepted,
 * from target row gamma.  The draw from weights w is the lowest v whose
 * cumulative weight exceeds draw_uniform * sum(w).  Comparisons and sums are in
 * fp64.
 *
 * Marks (accept_len -1, tokens -1): a draft token outside [0, V), a uniform
 * outside [0, 1) or NaN, a drafted token's probability (target or draft) that
 * is negative or not finite, a sum of draw weights that is not finite or, with
 * no point drafts to draw from instead, zero.  Negative probabilities elsewhere
 * weigh nothing.
 */
int spec_verify_probs(const void* target_probs, const void* draft_probs,
                      const int32_t* draft_tokens, const float* uniforms,
                      const float* draw_uniforms, int B, int gamma, int V, int dtype,
                      int32_t* out_accept_len, int32_t* out_tokens, void* stream);

/*
 * spec_verify_tree -- drafted trees, verified against given probabilities.
 *
 * Inputs (device), N = number of packed nodes the buffers hold:
 *   target_probs  [N, V]  row i: the target's law of the token after node i.
 *   draft_probs   [N, V]  row i: the law node i's children were drawn from,
 *                         independently (rows of leaves are not read); or
 *                         NULL for point drafts.
 *   tokens        [N] int32 (the root's is not read)
 *   parents       [N] int32, cu_nodes [B + 1] int32 (see "Trees")
 *   uniforms      [N] fp32 (the root's is not read), draw_uniforms [B] fp32
 * Outputs (device):
 *   out_accept_len [B]            accepted drafted nodes, or -1.
 *   out_tokens     [B, max_nodes] their tokens, the drawn token, -1 padding.
 *   out_path       [B, max_nodes] 0 (the root), the accepted nodes' indices
 *                                 within the sequence, -1 padding; may be
 *                                 NULL.
 * Rule, from the root on: the children of the current node are tried in
 * index order against the node's law r, r = p at first: child x is accepted
 * when u q(x) < r(x), and becomes the current node; after a rejection
 * r <- norm(max(r - q, 0)), unchanged where that has no mass (point drafts: r
 * loses the child's entry, and a token rejected once at a node is not accepted
 * there again).  When no child is left the final token is drawn from r (point
 * drafts that took all of its mass, possible where p sums to less than 1: the
 * last of them that had any).  After k rejections r = max(p - c_k q, 0) / M_k
 * with c_0 = 0, M_0 = 1, c_{k+1} = c_k + M_k and
 * M_{k+1} = sum max(p - c_{k+1} q, 0), which is how it is computed.
 * Marks as spec_verify_probs (-1 in path too), and a sequence without nodes,
 * with more than max_nodes or SV_MAX_NODES of them, with a parent that does
 * not come before its node, with a second root, or whose cu_nodes bounds do
 * not lie in [0, N].
 */
int spec_verify_tree(const void* target_probs, const void* draft_probs, const int32_t* tokens,
                     const int32_t* parents, const int32_t* cu_nodes, const float* uniforms,
                     const float* draw_uniforms, int B, int N, int max_nodes, int V, int dtype,
                     int32_t* out_accept_len, int32_t* out_tokens, int32_t* out_path,
                     void* stream);

/*
 * spec_kv_slots -- block tables and slot maps from request lengths.
 *
 * Request b holds lens[b] tokens, in pages table[b][0 .. ceil(len/page)) of
 * page_size tokens; add[b] tokens join it.  Their pages are taken from the
 * stack of free pages (the last entry first, requests in order), and every
 * packed row of new keys and values gets its slot page * page_size + offset.
 *
 * Inputs (device): lens [B], add [B] (>= 0; -1 releases the request: its
 * pages go back on the stack, its length to 0), cu_rows [B + 1] (request b's
 * packed rows; as cu_nodes), path [B, path_width] or NULL: which of the
 * request's rows are kept, strictly increasing (the out_path of
 * spec_verify_tree); NULL keeps its first add[b] rows.
 * Updated in place (device): table [B, table_width] (row stride table_row
 * entries), free_pages [pool].
 * Outputs (device): slots [N] (-1 for rows that are not kept and rows outside
 * every request), start [B] (the position of the first new token; -1 for a
 * refused or released request), out_lens [B], out_free_count [1]; the last
 * two may be lens and free_count themselves.
 *
 * A request is refused (start -1, its rows' slots -1, length, table row and
 * stack as they were for it) when its table row is too short, when the pages
 * of the requests up to it exceed the free ones, or when its data is bad:
 * lens outside [0, table_width * page_size], add below -1, more rows asked
 * than it has, path entries out of range or order.  Requests that need no new
 * page are never refused for lack of pages.  Released pages can be taken from
 * the next call on; pages that would not fit in free_pages are dropped.
 */
int spec_kv_slots(const int32_t* lens, const int32_t* add, const int32_t* cu_rows,
                  const int32_t* path, int path_width, int32_t* table, int64_t table_row,
                  int table_width, int32_t* free_pages, int pool, const int32_t* free_count, int B,
                  int N, int page_size, int32_t* out_slots, int32_t* out_start,
                  int32_t* out_lens, int32_t* out_free_count, void* stream);

/*
 * spec_kv_append -- keys and values of packed rows written into the cache.
 *
 * Row i of every layer goes to slot slots[i] (page slot / page_size, token
 * slot % page_size) of that layer's cache; slots outside
 * [0, num_pages * page_size) skip the row.  Elements are copied as they are.
 * Two rows with one slot leave either row's values.  Strides are in elements
 * of elem_bytes (1, 2 or 4) bytes; the D elements of a head are contiguous.
 * [0] is the keys', [1] the values'.
 */
typedef struct {
  const void* src[2]; /* [layers, N, H, D]                       */
  void* cache[2];     /* [layers, num_pages, page_size, H, D]    */
  int64_t src_layer[2], src_row[2], src_head[2];
  int64_t cache_layer[2], cache_page[2], cache_token[2], cache_head[2];
  const int32_t* slots; /* [N] device */
  int layers, N, H, D, num_pages, page_size, elem_bytes;
} sv_kv_append_args;
int spec_kv_append(const sv_kv_append_args* args, void* stream);

/*
 * spec_tree_attention -- softmax attention of drafted nodes.
 *
 * Node i of sequence b, query head h (key head h / (Hq / Hkv)) attends to the
 * lens[b] cached tokens of its sequence and to itself and its ancestors:
 *   out[i, h] = sum_t softmax_t(scale q_i . k_t) v_t.
 * Inputs (device):
 *   q [N, Hq, D], k, v [N, Hkv, D]: the nodes' rows (packed as cu_nodes says).
 *   k_cache, v_cache [num_pages, page_size, Hkv, D]: the pages.
 *   block_table [B, table_width] int32 (row stride table_row): request b's
 *   token t lies in page block_table[b][t / page_size].
 *   lens [B] int32 (>= 0), parents [N], cu_nodes [B + 1] int32.
 * Outputs: out [N, Hq, D], dense; out_lse [N, Hq] fp32 or NULL: the natural
 * logarithm of the sum of exp(scale q . k).  Rows outside every sequence are
 * left as they were.
 * Types: SV_BF16 or SV_F16 throughout.  D a multiple of 8 up to
 * SV_MAX_HEAD_DIM, Hq a multiple of Hkv, Hq / Hkv <= 128; page_size 8, 16,
 * 32, 64 or a multiple of 128; strides (elements) multiples of 8, addresses
 * 16-byte aligned.  Products are accumulated in fp32, the softmax is fp32,
 * its weights are rounded to the input type for the second product: by 2^-8
 * (bf16) or 2^-11 (fp16) of themselves, in fp16 also by up to 2^-32 of their
 * row's largest.
 * Nothing a node may not see reaches its result, whatever it holds (other
 * branches, rest of the last page, neighbours' rows: infinities and NaN too).
 * Where all scores that a node sees are -inf, its out is NaN (0 / 0) and its
 * lse -inf; a score of +inf or NaN makes both NaN.
 * Marks: a sequence whose lens is negative or beyond its table row, which
 * has more than SV_MAX_NODES nodes, or one of whose pages (of those it uses)
 * lies outside [0, num_pages), gets NaN in its rows; so does a node one of
 * whose ancestors (itself included) has a parent outside [-1, own index).
 * The rows of a sequence whose cu_nodes bounds do not lie in [0, N] are left
 * as they were.
 * Workspace: spec_tree_attention_workspace_size bytes, 256-byte aligned, of
 * any content; nothing is kept in it between calls.
 */
typedef struct {
  const void *q, *k, *v, *k_cache, *v_cache;
  void* out;
  float* out_lse;
  const int32_t *block_table, *lens, *parents, *cu_nodes;
  int64_t q_node, q_head, k_node, k_head, v_node, v_head;
  int64_t kc_page, kc_token, kc_head, vc_page, vc_token, vc_head, table_row;
  int B, N, Hq, Hkv, D, num_pages, page_size, table_width, dtype;
  float scale;
} sv_tree_attention_args;
size_t spec_tree_attention_workspace_size(int Hq, int Hkv, int D);
int spec_tree_attention(const sv_tree_attention_args* args, void* workspace,
                        size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_TREE_H */
