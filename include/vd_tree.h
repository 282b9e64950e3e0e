/*
 * vd_tree.h -- token trees: verifying drafted continuations of many requests
 * in one step (libvd.so).
 *
 * A request's tree hangs below its cached_len = c cached tokens.  Node 0 is
 * its root (the token at position c); the parent of every other node is an
 * earlier node.  Node i stands at position c + depth(i) (the root's depth is
 * 0), keeps its K/V in the request's slot c + i, and sees the cached tokens
 * and the nodes from the root to itself.  Its row is bit for bit the row that
 * decoding that path token by token computes: the logits of vd_step_tree
 * equal those of vd_step on the history followed by the path, whatever the
 * rest of the tree and of the batch [B §二 Theorem 4.1], be it infinite or NaN
 * (cached K/V have to be finite where a window hides them from some of the
 * nodes only, as in a prefill chunk).  Trees are an addition of this library;
 * the pages verify single continuations [L, §4].
 *
 * Use, per step: vd_tree_plan() with the nodes of every request, then
 * vd_step_tree() (or the single ops per layer), a token choice for every node
 * (vd_sample / vd_sample_filtered with the row's state at the node's
 * position), and vd_tree_accept(), which follows the chosen tokens down the
 * tree and moves the K/V of the accepted nodes to consecutive slots.
 *
 * A vd_tree holds the plan in force and its own split partials, so two trees
 * of one model share neither; the calls on one tree (and the steps of its
 * model, whose activations vd_step_tree uses) are to be ordered by the
 * caller, on one stream or with events.  A tree belongs to the device of its
 * model, which has to be the current one.  Its calls cannot be captured into
 * a graph (VD_ERR_UNSUPPORTED): their plan changes from step to step.
 * Conventions and errors otherwise as in vd.h.
 */
#ifndef VD_TREE_H_
#define VD_TREE_H_

#include <stdint.h>

#include "vd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct vd_tree vd_tree;

/* The trees of one step.  All arrays are host memory. */
typedef struct vd_tree_batch {
  int32_t num_nodes;           /* T = cu_nodes[B]                                   */
  int32_t num_seqs;            /* B                                                 */
  int32_t page_table_stride;   /* columns of page_table                             */
  int32_t pad_;
  const int32_t* cu_nodes;     /* [B + 1], cu_nodes[0] = 0, strictly increasing     */
  const int32_t* parent;       /* [T]: -1 for a request's node 0, else the number,
                                  within the request, of an earlier node            */
  const int32_t* cached_len;   /* [B]                                               */
  const int32_t* page_table;   /* [B * page_table_stride], for cached_len + nodes
                                  slots per request                                 */
  const int32_t* token_ids;    /* [T] or null (vd_step_tree needs them)             */
} vd_tree_batch;

/* max_nodes: most nodes of one plan (at most the model's max_tokens; at most
 * 1024 per request).  Once its model is destroyed, vd_destroy_tree is the only
 * call that a tree takes.
 * Errors: VD_ERR_INVALID_ARG, VD_ERR_CAPACITY, VD_ERR_CUDA. */
int vd_tree_create(vd_model* m, int32_t max_nodes, vd_tree** out);
void vd_destroy_tree(vd_tree* t);

/* Validates the trees (parents, positions, page ids, capacities; no two nodes
 * share a KV slot), and uploads them on the stream; the later calls use this
 * plan until the next one.  The first plans allocate (device memory for the
 * plan and for split partials of num_nodes * n_heads * splits rows), which
 * may synchronise the device; a plan no larger than an earlier one does not.
 * A failed call keeps the plan before it, unless an allocation failed.
 * num_nodes = num_seqs = 0 is a plan without work.
 * Errors: VD_ERR_INVALID_ARG, VD_ERR_OUT_OF_RANGE, VD_ERR_CAPACITY, VD_ERR_CUDA. */
int vd_tree_plan(vd_tree* t, vd_kv_pool* pool, const vd_tree_batch* b, void* stream);

/* Attention of every node for `layer`: q dev bf16 [T][Hq][hd] (rotated), out
 * dev bf16 [T][Hq][hd].  The K/V of the nodes must already be in their slots.
 * The cached tiles that all nodes share are read once per request and KV head
 * for (up to 128 rows of) its nodes. */
int vd_op_tree_attention(vd_tree* t, vd_kv_pool* pool, int32_t layer, const void* q, void* out, void* stream);

/* RoPE at the nodes' positions + K/V write into their slots (vd_op_rope_kv
 * for trees): qkv dev bf16 [T][(Hq+2Hkv) hd] -> q_out dev bf16 [T][Hq][hd]. */
int vd_op_tree_rope_kv(vd_tree* t, vd_kv_pool* pool, int32_t layer, const void* qkv, void* q_out, void* stream);

/* The whole decoder forward of the planned nodes (the plan needs token_ids
 * and at most max_logit_rows nodes): writes their K/V and logits_out, dev
 * float32 [T][V], 16-byte aligned. */
int vd_step_tree(vd_tree* t, vd_kv_pool* pool, float* logits_out, void* stream);

/* Acceptance.  choices: dev int32 [T], the token chosen after each node;
 * node_tokens: dev int32 [T] or null (the plan's token_ids).  A request's path
 * starts at its root and goes on to the lowest-numbered child whose token is
 * the one chosen after the path's last node, while there is one and the path
 * has fewer than out_stride nodes.
 * accepted_len: dev int32 [B], the nodes of the path (at least 1).
 * out_tokens: dev int32 [B][out_stride], row b the tokens chosen along the
 * path (accepted_len of them: the accepted drafts and one new token), then
 * -1; out_stride at least 1 (a whole row holds the longest path of the plan).  The K/V of the path's
 * node at depth d is moved to slot cached_len + d, in every layer, so that
 * cached_len + accepted_len slots of the request then hold its history;
 * other slots are left as they are.  A plan is accepted once: the move
 * overwrites slots of nodes off the path, and of nodes that have moved.
 * Errors: VD_ERR_INVALID_ARG, VD_ERR_CAPACITY, VD_ERR_CUDA. */
int vd_tree_accept(vd_tree* t, vd_kv_pool* pool, const int32_t* node_tokens, const int32_t* choices,
                   int32_t* accepted_len, int32_t* out_tokens, int32_t out_stride, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* VD_TREE_H_ */
