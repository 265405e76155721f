/*
 * tree_decode.h -- growing a rollout tree: a key/value cache in 8 bits that
 * stores every shared prefix once, and the attention of the decoding nodes' new
 * tokens over it (libtreeattn).
 *
 * The cache.  Rollouts share prefixes (AReaL-DTA abstract; TreePO, segment-level
 * tree sampling), so the keys and values of a node are kept once, whatever the
 * number of rollouts under it.  Every node owns whole pages of
 * TREE_DECODE_PAGE = 64 tokens of a pool that the caller allocates:
 *
 *   k8 [n_pages, hkv, 64, d]  e4m3 codes of the keys, a token's features together
 *   v8 [n_pages, hkv, d, 64]  e4m3 codes of the values, a feature's tokens together
 *   k_scale, v_scale [n_pages, hkv]  fp32, a power of two per page and kv-head
 *
 * A stored value is code * scale.  The scale of a page is the smallest 2^e with
 * |x| / 2^e <= 448 (the largest e4m3 value) for its tokens' finite values x, and
 * at least 2^-100; codes are rounded to nearest even, infinities saturate at
 * +-448, NaN stays NaN.  e4m3 is a floating format, so a power of two costs no
 * precision, and a page whose scale grows when a token is appended is brought to
 * the new scale exactly, except for values that leave the normal range (below
 * 2^-6 * scale), which are rounded again.  Slots behind a node's last token are
 * never read into a result and never written.
 *
 * The plan.  tree_attn_decode_plan() takes the tree, the tokens already in each
 * node, the tokens each node has room for, the pages and the nodes that decode.
 * It stays valid while nodes grow inside their room: the lengths in force are a
 * device array (`lens`, int32 [n_nodes] by node id) that every call reads, so a
 * whole segment can be decoded with one plan, or one captured graph.
 *
 * Conventions are those of tree_attn.h: status 0 = success, negative =
 * TREE_ATTN_ERR_*; host pointers are read during the call only; device pointers
 * belong to the caller and are used asynchronously on `stream` of the current
 * device; the plan's first call on a device uploads its tables (allocates and
 * synchronises; make it outside stream capture, or call
 * tree_attn_decode_plan_upload).  Calls of one plan may run on several streams
 * at once when they do not touch the same pages or workspace.  A call is ordered
 * with what came before on its own stream only: its inputs have to be there, and
 * their memory stays the call's until the stream has passed it.
 */
#ifndef TREE_DECODE_H
#define TREE_DECODE_H

#include <stddef.h>
#include <stdint.h>

#include "tree_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TREE_DECODE_PAGE 64

/* Device status only (tree_attn_get_device_status): a token was appended to a
 * node without room; it was dropped and the node's length left as it was. */
#define TREE_ATTN_ERR_CACHE_FULL -14

typedef struct tree_decode_plan_s* tree_decode_plan_t;

typedef struct {
    int32_t cta_pages;     /* most pages per CTA's work item of the attention (runs read by more
                              than 8 query rows), 1..128; 0 = automatic */
    int32_t warp_pages;    /* the same for a warp's item (at most 8 rows), 1..32; 0 = automatic */
} tree_attn_decode_opts_t;

typedef struct {
    int64_t n_fresh_tokens;   /* rows tree_attn_cache_write reads            */
    int64_t n_entries;        /* pages of the nodes on some query's path      */
    int64_t n_combine;        /* (query, work item) pairs                     */
    int64_t n_part_rows;      /* partial rows per kv-head                     */
    int64_t workspace_bytes;  /* device workspace tree_attn_decode needs      */
    int32_t n_write_jobs;     /* pages tree_attn_cache_write fills            */
    int32_t n_ctas;           /* CTAs of the attention, per kv-head           */
    int32_t n_live;           /* queries that are not padding                 */
    int32_t n_sub;            /* parts a query's head group is cut into       */
    int32_t rows_per_sub;     /* query heads per part                         */
    int32_t cta_pages;        /* pages per item in force                      */
    int32_t warp_pages;
} tree_attn_decode_info_t;

/* Caller-allocated destinations for tree_attn_decode_plan_export; any may be
 * NULL.  A "row group" is one part of one query's heads: row group s * n_sub + p
 * is part p of the query at place s of the depth-first query order. */
typedef struct {
    int32_t* entries;        /* [4 * n_entries]    {page, node, first token in node, room +
                                                   65536 if it holds tokens at plan time}   */
    int32_t* items;          /* [n_ctas * 6 * 8]  six items per CTA {first entry, entries, first
                                                   row group, end row group, first partial row, 1 if
                                                   the whole CTA's (then the only one), 0, 0}; no
                                                   entries: none */
    int32_t* query_order;    /* [n_live]           query index at each place                */
    int32_t* combine_ptr;    /* [n_live*n_sub + 1] CSR offsets into combine_row             */
    int32_t* combine_row;    /* [n_combine]        first partial row of each (row group, item) */
    int32_t* write_jobs;     /* [4 * n_write_jobs] {page, first source row, tokens, 0}      */
} tree_attn_decode_arrays_t;

/* Build a plan (host only, no GPU needed).
 *   parent[v]    parent node id, -1 for a root
 *   seg_len[v]   tokens in node v now (>= 0; a node that has just branched may be empty)
 *   capacity[v]  tokens node v has room for (>= seg_len[v]); NULL = seg_len
 *   pages        the nodes' pages, ceil(capacity[v] / 64) for each node in id order, all
 *                different and in [0, n_pages); NULL = 0, 1, 2, ...
 *   n_pages      pages of the pool; 0 where no node has room (the pool's pointers may then be NULL)
 *   fresh[v]     non-zero: tree_attn_cache_write brings node v's tokens; NULL = every node
 *   query_node   the node each query decodes in; a query attends to every token of its
 *                node and of the node's ancestors.  -1 marks a padding row: nothing of it
 *                is read or written.  Nodes may repeat, and may have descendants.
 *   hq, hkv, d   query heads, kv-heads (hq a multiple of hkv), head size 64 or 128
 * Errors: INVALID_ARG, INVALID_TREE (parent out of range, cycle, seg_len < 0, capacity <
 * seg_len), UNSUPPORTED (heads), TOO_LARGE, OUT_OF_MEMORY.  A page that is out of range
 * or given twice is INVALID_ARG. */
int tree_attn_decode_plan(const int32_t* parent, const int32_t* seg_len, const int32_t* capacity, int32_t n_nodes,
                          const int32_t* pages, int32_t n_pages, const uint8_t* fresh, const int32_t* query_node,
                          int32_t n_queries, int32_t hq, int32_t hkv, int32_t d,
                          const tree_attn_decode_opts_t* opts, tree_decode_plan_t* out);

int tree_attn_decode_plan_info(tree_decode_plan_t plan, tree_attn_decode_info_t* info);

int tree_attn_decode_plan_export(tree_decode_plan_t plan, const tree_attn_decode_arrays_t* dst);

int tree_attn_decode_plan_upload(tree_decode_plan_t plan);

/* Free the plan and its device copies (call after work using it finished, replays
 * of graphs that captured its calls included).  Allowed while another stream is
 * being captured. */
void tree_attn_decode_plan_destroy(tree_decode_plan_t plan);

/* Write the fresh nodes' tokens, e.g. what a prefill with tree_attn_fwd produced:
 * k, v bf16, row r at element r * k_stride (v_stride), [hkv, d] contiguous in it;
 * rows are the fresh nodes' tokens in depth-first pre-order (the packed order of
 * tree_attn.h).  Sets the codes of those tokens and the scales of their pages.
 * Strides are multiples of 8 elements and at least hkv * d. */
int tree_attn_cache_write(tree_decode_plan_t plan, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                          void* k8, void* v8, float* k_scale, float* v_scale, void* stream);

/* Append one token to each query's node: row r of k, v (bf16, as above, one row
 * per query) becomes token lens[u] of node u = query_node[r], the page's scales grow
 * where the token needs it, and lens_out[u] = lens[u] + 1 (other entries of lens_out
 * are left alone; lens_out may be lens).  A node without room drops the token,
 * records TREE_ATTN_ERR_CACHE_FULL and keeps its length.  Refused (INVALID_ARG)
 * when two queries have the same node. */
int tree_attn_cache_append(tree_decode_plan_t plan, const int32_t* lens, int32_t* lens_out, const void* k,
                           const void* v, int64_t k_stride, int64_t v_stride, void* k8, void* v8, float* k_scale,
                           float* v_scale, void* stream);

/* Attention of one new token per query over the cache:
 *   S_j = softmax_scale * q . k_j,  LSE = ln sum_j exp(S_j),  O = sum_j exp(S_j - LSE) v_j
 * over the tokens j of the query's node and its ancestors (lens[v] tokens of node
 * v, at most its room).  q bf16, row r at element r * q_stride (a multiple of 8, at
 * least hq * d); o [n_queries, hq, d] bf16; lse [hq, n_queries] fp32.  A query whose
 * path holds no token gets O = 0 and LSE = -inf.  Rows of padding queries are left as
 * they were.  The result is bitwise reproducible.
 * Precision: scores, statistics and sums are fp32; o is rounded once, to bf16.  A softmax
 * weight times its page's v_scale is rounded to f16 before it meets the codes: by 2^-11 of
 * itself, and where it is below 2^-26 of the row's largest such product by at most 2^-37
 * of that.  q is exact but for features below 2^-14 of their row's largest, which lose at
 * most 2^-25 of that.
 * workspace: workspace_bytes of device memory, 256-byte aligned, contents ignored; calls
 * that may overlap on the GPU need one each. */
int tree_attn_decode(tree_decode_plan_t plan, const int32_t* lens, const void* q, int64_t q_stride, const void* k8,
                     const void* v8, const float* k_scale, const float* v_scale, void* o, float* lse,
                     float softmax_scale, void* workspace, size_t ws_bytes, void* stream);

/* Copy whole pages inside one or several caches of the same shape (one per layer, say): page
 * src[i] to page dst[i] of every cache, codes and scales, in one launch for up to 32 caches and 1,024 pages.
 * A node branches at token s < its length without moving what others read: its full pages below
 * s stay, a new node gets a copy of the page that holds token s and the tokens of it below s as its
 * length; the old node's later pages become a node of their own beside it.  (Slots behind a
 * node's last token are never read; a copied page's scale covers all that was in it.)  The same
 * call moves pages when a pool is compacted.
 *   k8, v8, k_scale, v_scale   host arrays of n_caches device pointers, read during the call
 *   src, dst                   host arrays of n page numbers in [0, n_pages), read during the call.
 *                              dst are all different and none of them is a source: INVALID_ARG
 *                              otherwise.  A page may be copied to several.
 * No plan, no workspace; may be captured: a replay copies the pages of the captured call again.
 * Asynchronous on `stream`. */
int tree_attn_cache_copy(int32_t n_caches, void* const* k8, void* const* v8, float* const* k_scale,
                         float* const* v_scale, int32_t n_pages, int32_t hkv, int32_t d, const int32_t* src,
                         const int32_t* dst, int64_t n, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TREE_DECODE_H */
