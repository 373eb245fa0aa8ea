/*
 * attn_tree.h -- C ABI of a step that verifies drafted tokens over the paged
 * bf16 cache: page tables kept on the GPU, the append and the attention of a
 * tree of drafted tokens per sequence, and the accepted path's cache rows.
 * The layer shapes, pages, block tables, streams, workspaces, errors and
 * status bits are attn_decode.h's; this header states what differs.
 *
 * A step.  A drafting model proposes for sequence b a tree of n tokens behind
 * the ctx tokens that the cache keeps.  Its nodes are rows cu_q[b] ..
 * cu_q[b+1]-1 of the packed arrays, n = cu_q[b+1] - cu_q[b] <= ATTN_MAX_TREE,
 * and seq_lens[b] = ctx + n.  parents[cu_q[b] + i] is the node that node i
 * continues, counted from 0 within the sequence and below i, or -1 where it
 * continues the context itself (node 0 always does; several may).  A chain,
 * parents i - 1, is a chunk of consecutive tokens.
 *   depth_i  its number of ancestors; node i stands at position ctx + depth_i
 *            of the text it belongs to, which is where it is rotated
 *   slot     its key and value are cached at position ctx + i of the table
 * Then: attn_pages_assign (tables and lengths), and per layer
 * attn_kv_append_*_tree and attn_decode_*_tree; the caller picks the path that
 * the target model agrees with; attn_kv_commit_* moves its rows to ctx, ctx +
 * 1, ..., where each node's position then is its slot.
 * A parent outside [-1, i) raises ATTN_DEV_BAD_TREE and counts as -1.
 */
#ifndef ATTN_TREE_H
#define ATTN_TREE_H

#include "attn_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_MAX_TREE 64   /* nodes of a sequence's tree                          */
#define ATTN_MAX_LAYERS 64 /* layers of one attn_kv_commit_* call                 */

/* further device status bits */
#define ATTN_DEV_BAD_TREE 16 /* a parent or a path entry outside its range        */
#define ATTN_DEV_NO_PAGES 32 /* attn_pages_assign: fewer free pages than needed   */

/*
 * attn_decode_sliding_tree / attn_decode_global_tree -- attention of the
 * nodes over the context and their own ancestors:
 *
 *   o[i,h] = sum over visible l of softmax_l( <q[i,h], k_l> ) * v_l,
 *
 * node i seeing the context's positions l < ctx and the nodes j that are its
 * ancestors or itself; with a window w only those less than w positions
 * behind it: ctx + depth_i - l < w, depth_i - depth_j < w.
 *
 * q            bf16 [total_q, 16, D], as attn_kv_append_*_tree leaves it
 * k_pool, v_pool, block_table, num_pages, max_blocks: as for the decode calls;
 *              the nodes' own keys and values are in the cache
 * seq_lens     int32 [batch], nodes included, n <= L <= max_blocks*16
 * cu_q         int32 [batch + 1], cu_q[0] = 0, non-decreasing, cu_q[batch] <=
 *              total_q; rows of o behind it are left as they are
 * parents      int32 [total_q]
 * o            [total_q, 16, D], bf16 or fp32 per out_dtype
 * max_q        host bound on n, 0 .. ATTN_MAX_TREE (shapes the tiles); with max_q
 *              or total_q 0 the lengths are checked, where there is a status,
 *              and nothing else is done
 * max_seq_len  host bound on seq_lens; it only sizes the launch
 * window       sliding: > 0 (the node's is 1024); global: <= 0 none, > 0 a window
 * num_splits   thread blocks the keys are cut among: 0 = one per SM (fewer for
 *              small calls); > 0 forces that many, 16 to 1024
 * workspace    attn_decode_tree_workspace_size(...) bytes for the call's
 *              arguments or larger ones (or attn_decode_tree_plan's for exactly
 *              its arguments); no initialisation; not shared by calls that may
 *              overlap
 * status       a sequence with n > L, n > max_q, L beyond the table or rows past
 *              total_q raises ATTN_DEV_BAD_SEQ_LEN and its rows are not
 *              written; a cu_q that decreases anywhere raises it too and nothing
 *              of the call is written; a visible page id outside [0, num_pages)
 *              raises ATTN_DEV_BAD_PAGE and reads as zeros
 *
 * Products run on the tensor cores on bf16 with fp32 sums; weights are rounded
 * to bf16 for their product with the values.  A visible NaN gives NaN outputs;
 * an infinity among the values gives itself, or NaN (next to one of the other
 * sign, or where every node sees it with a weight below fp32's range); what a
 * node does not see is not used for it, whatever it holds.  Every array 16
 * bytes aligned, the int32 ones 4.  One or two kernels.
 */
int32_t attn_decode_sliding_tree(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_table,
                                 const int32_t* seq_lens, const int32_t* cu_q, const int32_t* parents, void* o,
                                 int32_t batch, int32_t total_q, int32_t max_q, int32_t max_blocks, int64_t num_pages,
                                 int32_t max_seq_len, int32_t window, int32_t out_dtype, int32_t num_splits,
                                 void* workspace, size_t workspace_bytes, int32_t* status, void* stream);
int32_t attn_decode_global_tree(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_table,
                                const int32_t* seq_lens, const int32_t* cu_q, const int32_t* parents, void* o,
                                int32_t batch, int32_t total_q, int32_t max_q, int32_t max_blocks, int64_t num_pages,
                                int32_t max_seq_len, int32_t window, int32_t out_dtype, int32_t num_splits,
                                void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/*
 * attn_decode_tree_plan -- the launch plan of the calls above, as pure host
 * arithmetic: thread blocks, kernels launched (1 or 2) and workspace bytes (any
 * of the three may be NULL) on a device of num_sms multiprocessors.  A call of
 * fewer or shorter sequences may need more than one of many that are not cut.
 * attn_decode_tree_workspace_size -- a workspace for the current CUDA device
 * that serves these arguments and any smaller batch, max_q or max_seq_len (same
 * window and num_splits; 0, with attn_last_error, on bad arguments or when no
 * device can be queried).
 */
int32_t attn_decode_tree_plan(int32_t kind, int32_t batch, int32_t max_q, int32_t max_seq_len, int32_t window,
                              int32_t num_splits, int32_t num_sms, int32_t* out_num_splits, int32_t* out_launches,
                              size_t* out_workspace_bytes);
size_t attn_decode_tree_workspace_size(int32_t kind, int32_t batch, int32_t max_q, int32_t max_seq_len, int32_t window,
                                       int32_t num_splits);

/*
 * attn_kv_append_sliding_tree / attn_kv_append_global_tree --
 * attn_kv_append_*_chunk for the nodes of trees: node i's key and value go to
 * slot ctx + i, and its query and key are rotated at position ctx + depth_i.
 * parents int32 [total_q]; a sequence of more than ATTN_MAX_TREE nodes raises
 * ATTN_DEV_BAD_SEQ_LEN and nothing of it is written.  Every other argument is
 * attn_kv_append_*_chunk's; k_pool is required.
 */
int32_t attn_kv_append_sliding_tree(const void* qkv, const void* w_q, const void* w_k, const int32_t* block_table,
                                    const int32_t* seq_lens, const int32_t* cu_q, const int32_t* parents, void* q_out,
                                    void* k_pool, void* v_pool, int32_t batch, int32_t total_q, int32_t max_blocks,
                                    int64_t num_pages, int32_t* status, void* stream);
int32_t attn_kv_append_global_tree(const void* qkv, const void* w_q, const void* w_k, const int32_t* block_table,
                                   const int32_t* seq_lens, const int32_t* cu_q, const int32_t* parents, void* q_out,
                                   void* k_pool, void* v_pool, int32_t batch, int32_t total_q, int32_t max_blocks,
                                   int64_t num_pages, int32_t* status, void* stream);

/*
 * attn_kv_commit_sliding / attn_kv_commit_global -- the accepted path of every
 * sequence moved to the front of its nodes, in all layers of one type at once:
 * the key and value rows at slot ctx + path[b][j] go to slot ctx + j, j <
 * path_len[b].  Rows behind the path keep what they hold (the next step's nodes
 * overwrite them).
 *
 * k_pools, v_pools  host arrays of `layers` device pointers, each a pool as
 *              for the decode calls, all of num_pages pages; read during the call
 * seq_lens, cu_q  the tree's: ctx = seq_lens[b] - (cu_q[b+1] - cu_q[b])
 * path         int32 [batch, max_path]: node indices, increasing, in [0, n)
 * path_len     int32 [batch], 0 .. min(max_path, n)
 * new_lens     int32 [batch] (written): ctx + path_len[b], what the cache then
 *              keeps; none of the other arrays
 * max_path     1 .. ATTN_MAX_TREE
 * status       lengths that do not fit together raise ATTN_DEV_BAD_SEQ_LEN and
 *              nothing of the sequence is written, its new_lens neither; a bad
 *              path or path_len raises ATTN_DEV_BAD_TREE, no row of it moves
 *              and new_lens is ctx; a page id outside [0, num_pages) raises
 *              ATTN_DEV_BAD_PAGE and that row does not move
 * Pools 16 bytes aligned, the int32 arrays 4.  One kernel.
 */
int32_t attn_kv_commit_sliding(const void* const* k_pools, const void* const* v_pools, int32_t layers,
                               const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q,
                               const int32_t* path, const int32_t* path_len, int32_t* new_lens, int32_t batch,
                               int32_t max_path, int32_t max_blocks, int64_t num_pages, int32_t* status, void* stream);
int32_t attn_kv_commit_global(const void* const* k_pools, const void* const* v_pools, int32_t layers,
                              const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q,
                              const int32_t* path, const int32_t* path_len, int32_t* new_lens, int32_t batch,
                              int32_t max_path, int32_t max_blocks, int64_t num_pages, int32_t* status, void* stream);

/*
 * attn_pages_assign -- the tables of a step from its requests' lengths, on the
 * GPU: request b keeps cached_lens[b] tokens and brings new_tokens[b].
 *
 *   seq_lens[b] = cached_lens[b] + new_tokens[b],  cu_q = the running sum of new_tokens
 *   b's pages   = logical pages [first, end): first = max(0, cached_lens[b] - window
 *                 + 1) / 16 (0 without a window), end = ceil(seq_lens[b] / 16), at
 *                 least first
 *
 * Pages that b held and no longer needs go to the back of the free list, in the
 * order of b and of the logical page; pages that it needs and did not hold come
 * from its front, in the same order, and are entered into block_table.  (A page
 * given back by this call is not handed out again by it.)  A finished request
 * has cached_lens = new_tokens = 0 and gives back all its pages; one with
 * cached_lens 0 may follow it in the same row at once (and takes over the pages
 * that lie where it needs some).
 *
 * block_table  int32 [batch, max_blocks]: entries of new pages are written,
 *              others (those of pages given back, too) kept
 * held         int32 [batch][2]: logical pages [first, end) that b holds
 * free_list    int32 [num_pages]: a ring; the free pages are entries head,
 *              head + 1, ..., head + count - 1, modulo num_pages
 * free_state   int32 [2]: head, count
 * held_out, free_state_out  where the new ones are written; may be held and
 *              free_state themselves
 * seq_lens     int32 [batch], cu_q int32 [batch + 1] (written); none of the
 *              other arrays
 * status       lengths below 0 or beyond the table (or ATTN_MAX_SEQ_LEN), pages
 *              held outside the table, kept tokens in front of the pages held, a
 *              free list whose numbers do not fit: ATTN_DEV_BAD_SEQ_LEN; fewer
 *              free pages than needed: ATTN_DEV_NO_PAGES.  Then nothing of the
 *              state changes (held_out, free_state_out take the old one), cu_q is
 *              0 throughout and seq_lens is cached_lens, clamped into the table:
 *              the calls behind it have no new tokens.
 * Arrays 4 bytes aligned, held, held_out, free_state and free_state_out 8.  One
 * kernel.
 */
int32_t attn_pages_assign(const int32_t* cached_lens, const int32_t* new_tokens, int32_t* block_table,
                          const int32_t* held, int32_t* free_list, const int32_t* free_state, int32_t* held_out,
                          int32_t* free_state_out, int32_t* seq_lens, int32_t* cu_q, int32_t batch, int32_t max_blocks,
                          int64_t num_pages, int32_t window, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_TREE_H */
