/*
 * vd_kv8.h -- a KV cache held in 8 bits, attention over it, and the pages of
 * either cache (libvd.so).
 *
 * A vd_kv8 holds complete pages (16 tokens) in 8 bits, with one scale for each
 * page, K or V, and KV head.  Sealing copies a page of the bf16 pool into it.
 * With a = the largest magnitude of the 16 x head_dim values (at least 2^-80),
 *   VD_KV8_INT8  code = 127 x / a rounded to the nearest integer (ties to even),
 *                standing for code * a / 127;
 *   VD_KV8_E4M3  code = 448 x / a rounded to e4m3, standing for code * a / 448.
 * A block that holds an infinity or NaN has the scale NaN: every row that sees
 * a token of it is NaN.
 *
 * What a row sees.  The scale of a page depends on all its tokens, so a page
 * that is still being filled has none.  A row at position p sees the page of
 * its own position, floor(p / 16), in bf16 and every earlier page in 8 bits,
 * whether those pages were sealed long ago or by the same step.  That is a
 * function of the row's history alone, so rows stay what the rest of this
 * library makes them: bit for bit the same whatever the batch, the chunking of
 * prompts, the prefill/decode split, the reuse of complete pages and the
 * placement of pages [深入解析 Vosti §二 Theorem 4.1, §五 5.1].  The cache itself is
 * an addition of this library; the pages describe a 16-bit one.
 *
 * Use, per step: vd_kv8_plan_make() with the requests of the step, then
 * vd_step_kv8(), or per layer vd_op_kv8_rope_kv() (K/V of the new tokens into
 * the bf16 pool), vd_op_kv8_seal() (the pages that the step completes) and
 * vd_op_kv8_attention().  The bf16 pool holds the pages being filled and those
 * of the step's new tokens only; a completed one is free again after the step.
 *
 * Conventions and errors otherwise as in vd.h.  A cache, a plan and the pools
 * belong to the device of their model, which has to be the current one.
 */
#ifndef VD_KV8_H_
#define VD_KV8_H_

#include <stddef.h>
#include <stdint.h>

#include "vd.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { VD_KV8_INT8 = 0, VD_KV8_E4M3 = 1 };

typedef struct vd_kv8 vd_kv8;
typedef struct vd_kv8_plan vd_kv8_plan;
typedef struct vd_pages vd_pages;

/* ---- the cache ----
 * Memory: codes [layer][page][kv_head][32 * head_dim] bytes, then scales
 * [layer][page][kv_head][4] float32 (K's scale a / top; V's 1 / scale, log2 of
 * the scale, and the scale), vd_kv8_bytes() in all.  The codes of a (page, head)
 * are in the order in which the attention kernels feed them to the tensor cores,
 * K first:
 *   K, token j, dim c:  (c / 32) * 512 + ((j % 8) * 4 + (c % 8) / 2) * 16
 *                       + (c / 16 % 2) * 8 + (j / 8) * 4 + (c / 8 % 2) * 2 + c % 2
 *   V, token j, dim c:  16 * head_dim + (c / 32) * 512 + ((c % 8) * 4 + (j % 8) / 2) * 16
 *                       + (c / 8 % 4) * 4 + (j / 8) * 2 + j % 2
 * An int8 code is stored plus 128.  dev_mem as in vd_kv_pool_alloc; the memory is
 * zero-filled, and a page is to be sealed before a row sees it.
 * Errors: VD_ERR_INVALID_ARG, VD_ERR_CAPACITY, VD_ERR_CUDA. */
size_t vd_kv8_bytes(const vd_model* m, int32_t num_pages);
int vd_kv8_create(vd_model* m, int32_t format, int32_t num_pages, void* dev_mem, size_t bytes, vd_kv8** out);
void vd_destroy_kv8(vd_kv8* c);
void* vd_kv8_data(vd_kv8* c);

/* Pages src[i] of the bf16 pool -> pages dst[i] of the cache (host arrays [n]),
 * in one layer, or in all of them with layer = -1.  A page may be sealed into
 * several; two of one call's pages may not go to the same one.
 * Errors: VD_ERR_INVALID_ARG, VD_ERR_OUT_OF_RANGE, VD_ERR_CUDA. */
int vd_kv8_seal(vd_kv8* c, vd_kv_pool* pool, int32_t layer, int32_t n, const int32_t* src, const int32_t* dst,
                void* stream);
/* The reverse: the values that pages src[i] of the cache stand for, rounded to
 * bf16, into pages dst[i] of the bf16 pool (to run a request's steps or token
 * trees over that pool, or to read the values).  A block whose scale is NaN
 * gives NaN. */
int vd_kv8_unseal(vd_kv8* c, vd_kv_pool* pool, int32_t layer, int32_t n, const int32_t* src, const int32_t* dst,
                  void* stream);

/* ---- steps over the cache ----
 * The requests of a step, one after the other: request b's new tokens are cu_q[b] ..
 * cu_q[b + 1] - 1, at the positions from cached_len[b] on.
 * page_table[b * page_table_stride + i] is the page of the *cache* that holds
 * request b's logical page i, for the pages that are complete after the step,
 * i < (cached_len + q_len) / 16; of these the ones from cached_len / 16 on are
 * sealed by the step, the earlier ones have been.  open_table[b * open_stride + j]
 * is the page of the *bf16 pool* that holds logical page cached_len / 16 + j, up
 * to that of the last new token. */
typedef struct vd_kv8_batch {
  int32_t num_tokens;          /* T = cu_q[B]                                   */
  int32_t num_seqs;            /* B                                             */
  int32_t num_logit_rows;      /* R (vd_step_kv8)                               */
  int32_t page_table_stride;
  int32_t open_stride;
  int32_t pad_;
  const int32_t* cu_q;         /* [B + 1], cu_q[0] = 0, strictly increasing     */
  const int32_t* cached_len;   /* [B]                                           */
  const int32_t* page_table;   /* [B * page_table_stride] (may be null where no page is complete) */
  const int32_t* open_table;   /* [B * open_stride]                             */
  const int32_t* token_ids;    /* [T] or null (vd_step_kv8 needs them)          */
  const int32_t* logit_rows;   /* [R] token indices in [0, T)                   */
} vd_kv8_batch;

/* A plan in force and its split partials; max_tokens at most the model's.  The
 * calls on one plan (and the steps of its model, whose activations vd_step_kv8
 * uses) are to be ordered by the caller; two plans share nothing.  Its calls
 * cannot be captured into a graph (VD_ERR_UNSUPPORTED): a plan changes from step
 * to step.  Once the model is destroyed, vd_destroy_kv8_plan is the only call
 * that a plan takes (vd_destroy_kv8 that a cache takes). */
int vd_kv8_plan_create(vd_model* m, int32_t max_tokens, vd_kv8_plan** out);
void vd_destroy_kv8_plan(vd_kv8_plan* p);
/* Validates the batch (lengths, page ids, capacities; no two new tokens share a
 * slot; a page sealed by the step is sealed once and seen by no row as an earlier
 * one) and uploads it on the stream; the later calls use this plan until the next
 * one.  The first plans allocate, which may synchronise the device.  A failed
 * call keeps the plan before it, unless an allocation failed.  num_tokens =
 * num_seqs = 0 is a plan without work.
 * Errors: VD_ERR_INVALID_ARG, VD_ERR_OUT_OF_RANGE, VD_ERR_CAPACITY, VD_ERR_CUDA. */
int vd_kv8_plan_make(vd_kv8_plan* p, vd_kv8* c, vd_kv_pool* pool, const vd_kv8_batch* b, void* stream);

/* Kernel of the chunks of more than 16 rows (q_len * Hq / Hkv) in the plans made
 * after the call: 0 (default) chosen by their sizes, 1 mma.sync, 2 tcgen05.  The
 * same bits either way.  tcgen05 keeps fp16 images of its requests' histories in the
 * plan's memory, twice the bytes of their codes in one layer; the default takes it for
 * 8 GiB of them at most.  (A model set to mma.sync by vd_set_attention_prefill takes
 * that.)  Errors: VD_ERR_INVALID_ARG. */
int vd_kv8_set_prefill(vd_kv8_plan* p, int32_t kernel);

/* vd_op_rope_kv of the planned tokens: qkv dev bf16 [T][(Hq+2Hkv) hd] -> q_out
 * dev bf16 [T][Hq][hd], K/V into the bf16 pool. */
int vd_op_kv8_rope_kv(vd_kv8_plan* p, vd_kv8* c, vd_kv_pool* pool, int32_t layer, const void* qkv, void* q_out,
                      void* stream);
/* Seals, in one layer, the pages that the planned step completes. */
int vd_op_kv8_seal(vd_kv8_plan* p, vd_kv8* c, vd_kv_pool* pool, int32_t layer, void* stream);
/* Attention of the planned tokens: q, out dev bf16 [T][Hq][hd]; q has been
 * rotated, K/V of the new tokens are in the bf16 pool and the pages that the step
 * completes are sealed.  q and out may not overlap (VD_ERR_INVALID_ARG).  Slots of
 * the bf16 pool behind a row's position are not seen, whatever they hold.  Sums,
 * softmax statistics and outputs' partials are float32; weights enter the product
 * with V as fp16, at most 2^-11 of themselves (or, times their V scales, 2^-25 of the
 * largest such) off.  V of any sizes may stand beside each other.  Weights below 2^-126
 * of the row's largest may count as 0, and below 2^-36 in the sum of weights where their
 * V is 2^90 and more below another's. */
int vd_op_kv8_attention(vd_kv8_plan* p, vd_kv8* c, vd_kv_pool* pool, int32_t layer, const void* q, void* out,
                        void* stream);
/* The whole decoder forward of the planned tokens over the cache (vd_step with
 * these three in place of its own): writes their K/V, seals the pages that they
 * complete, in every layer, and logits_out, dev float32 [R][V], 16-byte aligned
 * (null if R = 0).  The plan needs token_ids. */
int vd_step_kv8(vd_kv8_plan* p, vd_kv8* c, vd_kv_pool* pool, float* logits_out, void* stream);

/* ---- pages ----
 * Copies, in every layer, pages src[i] to pages dst[i] (host arrays [n]; no page
 * twice among the dst, none both src and dst).  Stateless: calls of any threads
 * and streams, captured ones included, touch nothing but those pages.
 * Errors: VD_ERR_INVALID_ARG, VD_ERR_OUT_OF_RANGE, VD_ERR_CUDA. */
int vd_kv_copy_pages(vd_kv_pool* pool, int32_t n, const int32_t* src, const int32_t* dst, void* stream);
int vd_kv8_copy_pages(vd_kv8* c, int32_t n, const int32_t* src, const int32_t* dst, void* stream);

/* Reference counts of the pages of a pool or cache: host memory only, no device
 * work.  A call that fails has changed nothing.  Not thread-safe: one thread at a
 * time uses a vd_pages.
 * Errors: VD_ERR_INVALID_ARG, VD_ERR_OUT_OF_RANGE, VD_ERR_CAPACITY. */
int vd_pages_create(int32_t num_pages, vd_pages** out);
void vd_destroy_pages(vd_pages* p);
int32_t vd_pages_free(const vd_pages* p);               /* pages with no reference (-1: null) */
int32_t vd_pages_refs(const vd_pages* p, int32_t page); /* (-1: null or out of range)         */
/* The n lowest free pages, in ascending order, one reference each. */
int vd_pages_alloc(vd_pages* p, int32_t n, int32_t* out);
/* One reference more / less for each entry (a page may stand there several
 * times); a page without references is free. */
int vd_pages_retain(vd_pages* p, int32_t n, const int32_t* pages);
int vd_pages_release(vd_pages* p, int32_t n, const int32_t* pages);
/* Forks a request whose n pages are table[0..n) into `children` more of the same
 * history: row k of out [children][n] shares the first n_shared pages (the
 * complete ones, one reference more each) and has pages of its own for the rest,
 * whose copies are src[i] -> dst[i], children * (n - n_shared) of them. */
int vd_pages_fork(vd_pages* p, int32_t n, int32_t n_shared, const int32_t* table, int32_t children, int32_t* out,
                  int32_t* src, int32_t* dst);
/* Moves the highest pages in use to the lowest free ones, at most max_moves, until
 * the pages in use are the lowest: writes the moves src[i] -> dst[i], their
 * number to *n_moves, and rewrites the entries of `tables` (host [n_entries], the
 * page tables of every request that uses the pages; negative entries stand).  The
 * moves' copies are the caller's, ordered before the next use of the pages. */
int vd_pages_compact(vd_pages* p, int32_t max_moves, int32_t* src, int32_t* dst, int32_t* n_moves, int32_t n_entries,
                     int32_t* tables);

#ifdef __cplusplus
}
#endif
#endif /* VD_KV8_H_ */
