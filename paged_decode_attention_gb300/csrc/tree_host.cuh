// tree_host.cuh -- host side of include/attn_tree.h (the tree append's is
// serving.cuh's run_chunk).  Included in attn_decode.cu, whose validation helpers,
// tensor-map encoder and launch recording it shares.
#pragma once

#include "attn_tree.h"
#include "kv_commit.cuh"
#include "pages.cuh"
#include "tree_decode.cuh"

namespace {

// ---------------------------------------------------------------------------
// Attention of trees
// ---------------------------------------------------------------------------
// Every (sequence, group, KV head) in a block of its own, and no merge kernel, where there are blocks enough and cutting
// gains less than it costs: the longest takes its pages' time, and cut up the share of r = items / blocks of the pages of
// all (half of the longest's, on average), but as well the merge (kTreeWholePages' time) and r further starts and ends a
// block (kTreeWholeStarts).  us a call, whole and cut: global trees of 4 nodes, 8 behind 200 positions 13.4 and 14.9,
// behind 380 18.0 and 14.8, 60 behind 380 18.9 and 24.8; sliding ones of 8, 4 behind 300 11.9 and 14.0, behind 600 15.6 and
// 15.9, 16 behind 600 17.9 and 22.8.
constexpr int kTreeWholePages = 16, kTreeWholeStarts = 32;
// What a sequence's start and end cost a block, in pages: its Q, its masks, the sums, the stores, some 12 us in all.
// Where few sequences are spread over many blocks they pay it side by side, and a large weight would only leave blocks
// without pages.  Weights 4, 12, 24 and 48 in us: 64 sliding trees of up to 45 nodes 127, 122, 123, 125; 8 of 26 nodes
// 26.5, 24.8, 24.5, 27.4; 4 short ones 14.9, 16.6, 17.0, 18.5; 8 ragged global trees 42.1, 40.5, 41.1, 42.9.
constexpr int kTreeSegWeight = 12, kTreeSegWeightFew = 4;

struct TreePlan {
  int rows;      // of the configuration's groups
  int lists;     // of pages, per KV head: a group of rows each
  int grid;
  int seg_weight;
  bool whole;
  bool merge;    // a sequence may be cut (however low the caller's bound on the lengths): a second kernel
  size_t part_o_bytes, part_ml_bytes, workspace_bytes;
  size_t covering_bytes;  // workspace of calls with these arguments or smaller batch, max_q or max_seq_len
};

// Rows of the configuration that holds a whole tree of max_q nodes, or the widest.  us a call with 32, 64 and 128 rows: 200
// sliding trees of 5 nodes 276, 277, 293; 64 of 16 nodes 102, 103, 107; 4 behind 600 positions 17.4, 18.4, 18.3; 64 of 32
// nodes with 64 and 128 rows 110 and 116.
int tree_rows(int32_t kind, int32_t max_q) {
  namespace tr = pda::tree;
  if (kind == ATTN_KIND_GLOBAL) return tr::GlobalConfig::kN;
  return max_q <= tr::SlidingNarrow::kQueries ? tr::SlidingNarrow::kN
         : max_q <= tr::SlidingMid::kQueries  ? tr::SlidingMid::kN
                                            : tr::SlidingWide::kN;
}

int32_t make_tree_plan(int32_t kind, int32_t batch, int32_t max_q, int32_t max_seq_len, int32_t window,
                       int32_t num_splits, int32_t num_sms, TreePlan* out) {
  namespace tr = pda::tree;
  if (kind != ATTN_KIND_SLIDING && kind != ATTN_KIND_GLOBAL) return fail(ATTN_ERR_INVALID_ARG, "unknown kind %d", kind);
  if (batch < 1 || batch > ATTN_MAX_BATCH) return fail(ATTN_ERR_INVALID_ARG, "batch %d outside [1, %d]", batch, ATTN_MAX_BATCH);
  if (max_q < 0 || max_q > ATTN_MAX_TREE) return fail(ATTN_ERR_INVALID_ARG, "max_q %d outside [0, %d]", max_q, ATTN_MAX_TREE);
  if (max_seq_len < 0 || max_seq_len > ATTN_MAX_SEQ_LEN)
    return fail(ATTN_ERR_INVALID_ARG, "max_seq_len %d outside [0, %d]", max_seq_len, ATTN_MAX_SEQ_LEN);
  if (num_sms < 1) return fail(ATTN_ERR_INVALID_ARG, "num_sms must be >= 1");
  if (num_splits < 0 || (num_splits > 0 && num_splits < tr::kMaxGroups) || num_splits > tr::kMaxGrid)
    return fail(ATTN_ERR_INVALID_ARG, "num_splits must be 0 or in [%d, %d]", tr::kMaxGroups, tr::kMaxGrid);
  const bool sliding = kind == ATTN_KIND_SLIDING;
  const int d = sliding ? ATTN_SLIDING_D : ATTN_GLOBAL_D;
  const int hkv = sliding ? ATTN_SLIDING_HKV : ATTN_GLOBAL_HKV;
  out->rows = tree_rows(kind, max_q);
  const int nodes = out->rows * hkv / 16;  // of a group; 16 query heads
  out->lists = std::max(1, (max_q + nodes - 1) / nodes);
  // pages of one sequence: with a window those of window + max_q - 1 positions
  const int64_t span = window > 0 ? std::min<int64_t>(max_seq_len, static_cast<int64_t>(window) + max_q - 1) : max_seq_len;
  const int64_t pages = std::max<int64_t>(1, std::min<int64_t>((span + 2 * ATTN_PAGE_SIZE - 2) / ATTN_PAGE_SIZE,
                                                               (static_cast<int64_t>(max_seq_len) + ATTN_PAGE_SIZE - 1) / ATTN_PAGE_SIZE));
  // Whole sequences take an even number of blocks where they have several groups, as their plans always had; one without
  // nodes leaves at once.
  const int whole_lists = out->lists > 1 ? (out->lists + 1) & ~1 : 1;
  const int64_t whole_items = static_cast<int64_t>(batch) * whole_lists * hkv;
  const int64_t items = static_cast<int64_t>(batch) * out->lists * hkv;
  out->seg_weight = 4 * items >= num_sms ? kTreeSegWeight : kTreeSegWeightFew;
  out->whole = num_splits == 0 && whole_items <= num_sms &&
               pages * (2 * num_sms - whole_items) <= 2 * (kTreeWholePages * num_sms + kTreeWholeStarts * whole_items);
  out->merge = !out->whole;
  const int64_t useful = (items * (pages + out->seg_weight) + tr::kMinPer - 1) / tr::kMinPer;
  const int64_t least = tr::kMaxGroups;  // a run for every list
  const int cut_grid = num_splits > 0 ? num_splits
                                      : static_cast<int>(std::max<int64_t>(least, std::min<int64_t>({num_sms, useful, tr::kMaxGrid})));
  out->grid = cut_grid;
  if (out->whole) {
    out->lists = whole_lists;
    out->grid = static_cast<int>(whole_items);
  }
  const auto part_o = [&](int grid) { return align256(2 * static_cast<size_t>(grid) * out->rows * d * sizeof(float)); };
  const auto part_ml = [&](int grid) { return align256(2 * static_cast<size_t>(grid) * out->rows * sizeof(float2)); };
  const auto cuts = [](int grid) { return align256(static_cast<size_t>(grid) * sizeof(int4)); };
  out->part_o_bytes = out->merge ? part_o(out->grid) : 0;
  out->part_ml_bytes = out->merge ? part_ml(out->grid) : 0;
  out->workspace_bytes = out->part_o_bytes + out->part_ml_bytes + cuts(out->grid);
  // A call of fewer or shorter sequences may be cut where this one is not.  Rows, pages, items and the start weight grow
  // with every argument, so the cut plan of these covers the cut plans of smaller ones, and any whole one.
  out->covering_bytes = std::max(part_o(cut_grid) + part_ml(cut_grid) + cuts(cut_grid), cuts(num_sms));
  return ATTN_OK;
}

// Q [total_q, Hq, D] as {64 dims, D/64 chunks, Hq heads, total_q nodes}: a box {64, 1, G,
// nq} copies one 64-dim chunk of nq consecutive nodes' G heads of a KV head as
// [node][head][128 B], 128-byte swizzled; nodes past total_q read as zeros.
int32_t encode_tree_q_map(CUtensorMap* map, const void* q, int32_t total_q, int hq, int d, int g, int nq) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(d / 64), static_cast<cuuint64_t>(hq),
                              static_cast<cuuint64_t>(total_q)};
  const cuuint64_t strides[3] = {128, static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(hq) * d * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(g), static_cast<cuuint32_t>(nq)};
  const cuuint32_t elem_strides[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, elem_strides,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled (tree q map) failed (%d)", static_cast<int>(r));
  return ATTN_OK;
}

template <typename C>
int32_t launch_tree(const char* name, const void* q, const void* k_pool, const void* v_pool, int32_t total_q,
                    const TreePlan& plan, int dev, int num_sms, pda::tree::TreeParams& p, cudaStream_t s) {
  namespace tr = pda::tree;
  // nodes a copy brings: no more than the longest tree's, whole groups of 16 rows
  constexpr int kUnit = C::kG < 16 ? 16 / C::kG : 1;
  p.q_box = std::min(C::kQueries, (p.max_q + kUnit - 1) / kUnit * kUnit);
  CUtensorMap tm_q, tm_k, tm_v;
  int32_t st;
  if ((st = encode_tree_q_map(&tm_q, q, total_q, C::kHq, C::kD, C::kG, p.q_box)) ||
      (st = encode_chunk_map(&tm_k, k_pool, p.num_pages, C::kHkv * C::kD, 1)) ||
      (st = encode_chunk_map(&tm_v, v_pool, p.num_pages, C::kHkv * C::kD, C::kChunks)))
    return st;
  const auto kernel = tr::tree_kernel<C>;
  static bool main_set[kMaxDevices] = {false}, merge_set[kMaxDevices] = {false};
  if ((st = ensure_smem(kernel, C::kSmemBytes, dev, main_set)) ||
      (st = ensure_smem(tr::merge_kernel<C>, 0, dev, merge_set)))
    return st;
  cudaError_t e = launch_pdl(kernel, dim3(plan.grid), tr::kThreads, C::kSmemBytes, s, tm_q, tm_k, tm_v, p);
  if (e == cudaSuccess && plan.merge) {
    tr::MergeParams mp;
    mp.t = p;
    mp.grid = plan.grid;
    const int64_t rows = static_cast<int64_t>(p.batch) * p.max_q * C::kHq;  // a block per row's 128 dims, at most
    const int blocks = static_cast<int>(std::min<int64_t>(rows * C::kTiles, static_cast<int64_t>(num_sms) * tr::kMergeBlocksPerSm));
    e = launch_pdl(tr::merge_kernel<C>, dim3(blocks), tr::kMergeWarps * 32, 0, s, mp);
  }
  return launched(name, e);
}

int32_t run_tree(int32_t kind, const void* q, const void* k_pool, const void* v_pool, const int32_t* block_table,
                 const int32_t* seq_lens, const int32_t* cu_q, const int32_t* parents, void* o, int32_t batch,
                 int32_t total_q, int32_t max_q, int32_t max_blocks, int64_t num_pages, int32_t max_seq_len,
                 int32_t window, int32_t out_dtype, int32_t num_splits, void* workspace, size_t workspace_bytes,
                 int32_t* status, void* stream) {
  g_err[0] = '\0';
  const bool sliding = kind == ATTN_KIND_SLIDING;
  const char* name = sliding ? "attn_decode_sliding_tree" : "attn_decode_global_tree";
  if (!k_pool || !v_pool || !block_table || !seq_lens || !cu_q || (total_q > 0 && (!q || !parents || !o)))
    return fail(ATTN_ERR_INVALID_ARG, "%s: null array pointer", name);
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(o) || !aligned_to(block_table, 4) ||
      !aligned_to(seq_lens, 4) || !aligned_to(cu_q, 4) || !aligned_to(parents, 4) || !aligned_to(status, 4))
    return fail(ATTN_ERR_INVALID_ARG, "%s: misaligned pointer (q, o and the pools 16 bytes, tables 4)", name);
  int32_t st;
  if ((st = check_batch(name, batch, max_blocks)) || (st = check_pages(name, "num_pages", num_pages)) ||
      (st = check_max_seq_len(name, max_seq_len, max_blocks)))
    return st;
  if (total_q < 0) return fail(ATTN_ERR_INVALID_ARG, "%s: total_q must be >= 0", name);
  if (max_q < 0) return fail(ATTN_ERR_INVALID_ARG, "%s: max_q must be >= 0", name);
  if (max_q > ATTN_MAX_TREE)
    return fail(ATTN_ERR_UNSUPPORTED, "%s: max_q %d beyond %d nodes", name, max_q, ATTN_MAX_TREE);
  if (sliding && window <= 0)
    return fail(ATTN_ERR_INVALID_ARG, "%s: window must be > 0 (the node's is 1024)", name);
  if (out_dtype != ATTN_OUT_BF16 && out_dtype != ATTN_OUT_F32)
    return fail(ATTN_ERR_INVALID_ARG, "%s: out_dtype must be ATTN_OUT_BF16 or ATTN_OUT_F32", name);
  if (num_splits < 0 || (num_splits > 0 && num_splits < pda::tree::kMaxGroups) || num_splits > pda::tree::kMaxGrid)
    return fail(ATTN_ERR_INVALID_ARG, "%s: num_splits must be 0 or in [%d, %d]", name, pda::tree::kMaxGroups,
                pda::tree::kMaxGrid);
  int dev = 0, num_sms = 0;
  if ((st = current_device(&dev, &num_sms)) != ATTN_OK) return st;
  TreePlan plan;
  if ((st = make_tree_plan(kind, batch, max_q, max_seq_len, window, num_splits, num_sms, &plan)) != ATTN_OK) return st;
  if (!workspace || workspace_bytes < plan.workspace_bytes)
    return fail(ATTN_ERR_WORKSPACE, "%s: workspace of %zu bytes required (got %zu)", name, plan.workspace_bytes,
                workspace ? workspace_bytes : size_t{0});
  if (!aligned16(workspace)) return fail(ATTN_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", name);
  const bool idle = total_q == 0 || max_q == 0;  // no nodes, by the caller: there are only the lengths to check
  g_last_launches = idle ? (status ? 1 : 0) : plan.merge ? 2 : 1;
  if (g_last_launches == 0 || g_validate_only) return ATTN_OK;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  pda::tree::TreeParams p{};
  p.v_pool = static_cast<const __nv_bfloat16*>(v_pool);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q;
  p.parents = parents;
  p.o = o;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + plan.part_o_bytes);
  p.cuts = reinterpret_cast<int4*>(ws + plan.part_o_bytes + plan.part_ml_bytes);
  p.status = status;
  p.num_pages = num_pages;
  p.batch = batch;
  p.max_blocks = max_blocks;
  p.window = window;
  p.total_q = total_q;
  p.max_q = max_q;
  p.lists = plan.lists;
  p.out_f32 = out_dtype == ATTN_OUT_F32;
  p.seg_weight = plan.seg_weight;
  p.whole = plan.whole;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  namespace tr = pda::tree;
  if (idle) return launched(name, launch_pdl(tr::check_kernel, dim3(1), pda::kMaxBatch, 0, s, p));
  const auto launch = [&](auto config) {
    return launch_tree<decltype(config)>(name, q, k_pool, v_pool, total_q, plan, dev, num_sms, p, s);
  };
  if (!sliding) return launch(tr::GlobalConfig{});
  return plan.rows == tr::SlidingNarrow::kN ? launch(tr::SlidingNarrow{})
         : plan.rows == tr::SlidingMid::kN  ? launch(tr::SlidingMid{})
                                            : launch(tr::SlidingWide{});
}

// ---------------------------------------------------------------------------
// Commit of accepted paths
// ---------------------------------------------------------------------------
int32_t run_commit(int32_t kind, const void* const* k_pools, const void* const* v_pools, int32_t layers,
                   const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q, const int32_t* path,
                   const int32_t* path_len, int32_t* new_lens, int32_t batch, int32_t max_path, int32_t max_blocks,
                   int64_t num_pages, int32_t* status, void* stream) {
  g_err[0] = '\0';
  const bool sliding = kind == ATTN_KIND_SLIDING;
  const char* name = sliding ? "attn_kv_commit_sliding" : "attn_kv_commit_global";
  if (!k_pools || !v_pools || !block_table || !seq_lens || !cu_q || !path || !path_len || !new_lens)
    return fail(ATTN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (!aligned_to(block_table, 4) || !aligned_to(seq_lens, 4) || !aligned_to(cu_q, 4) || !aligned_to(path, 4) ||
      !aligned_to(path_len, 4) || !aligned_to(new_lens, 4) || !aligned_to(status, 4) ||
      !aligned_to(k_pools, alignof(void*)) || !aligned_to(v_pools, alignof(void*)))
    return fail(ATTN_ERR_INVALID_ARG, "%s: misaligned pointer (tables 4 bytes)", name);
  if (layers < 1) return fail(ATTN_ERR_INVALID_ARG, "%s: layers must be >= 1", name);
  if (layers > ATTN_MAX_LAYERS)
    return fail(ATTN_ERR_UNSUPPORTED, "%s: %d layers, at most %d a call", name, layers, ATTN_MAX_LAYERS);
  int32_t st;
  if ((st = check_batch(name, batch, max_blocks)) || (st = check_pages(name, "num_pages", num_pages))) return st;
  if (max_path < 1) return fail(ATTN_ERR_INVALID_ARG, "%s: max_path must be >= 1", name);
  if (max_path > ATTN_MAX_TREE)
    return fail(ATTN_ERR_UNSUPPORTED, "%s: max_path %d beyond %d nodes", name, max_path, ATTN_MAX_TREE);
  pda::commit::CommitParams p{};
  for (int i = 0; i < layers; ++i) {
    if (!k_pools[i] || !v_pools[i]) return fail(ATTN_ERR_INVALID_ARG, "%s: null pool of layer %d", name, i);
    if (!aligned16(k_pools[i]) || !aligned16(v_pools[i]))
      return fail(ATTN_ERR_INVALID_ARG, "%s: pool of layer %d not 16-byte aligned", name, i);
    p.pool[2 * i] = static_cast<uint8_t*>(const_cast<void*>(k_pools[i]));
    p.pool[2 * i + 1] = static_cast<uint8_t*>(const_cast<void*>(v_pools[i]));
  }
  // the blocks of other layers read the lengths and paths while those of the first write new_lens
  const auto apart = [&](const int32_t* in, int64_t count) { return new_lens + batch <= in || in + count <= new_lens; };
  if (!apart(seq_lens, batch) || !apart(cu_q, batch + 1) || !apart(path, static_cast<int64_t>(batch) * max_path) ||
      !apart(path_len, batch) || !apart(block_table, static_cast<int64_t>(batch) * max_blocks))
    return fail(ATTN_ERR_INVALID_ARG, "%s: new_lens overlaps an input", name);
  for (int i = 0; i < 2 * layers; ++i)  // a row moved twice would be moved wrongly
    for (int j = 0; j < i; ++j)
      if (p.pool[i] == p.pool[j]) return fail(ATTN_ERR_INVALID_ARG, "%s: a pool is given twice", name);
  g_last_launches = 1;
  if (g_validate_only) return ATTN_OK;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q;
  p.path = path;
  p.path_len = path_len;
  p.new_lens = new_lens;
  p.status = status;
  p.num_pages = num_pages;
  p.max_path = max_path;
  p.max_blocks = max_blocks;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(batch, layers);
  constexpr int kSlidingRow = ATTN_SLIDING_HKV * ATTN_SLIDING_D * 2, kGlobalRow = ATTN_GLOBAL_HKV * ATTN_GLOBAL_D * 2;
  return launched(name, sliding ? launch_pdl(pda::commit::commit_kernel<kSlidingRow>, grid, kSlidingRow / 16, 0, s, p)
                                : launch_pdl(pda::commit::commit_kernel<kGlobalRow>, grid, kGlobalRow / 16, 0, s, p));
}

}  // namespace

extern "C" {

int32_t attn_decode_sliding_tree(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_table,
                                 const int32_t* seq_lens, const int32_t* cu_q, const int32_t* parents, void* o,
                                 int32_t batch, int32_t total_q, int32_t max_q, int32_t max_blocks, int64_t num_pages,
                                 int32_t max_seq_len, int32_t window, int32_t out_dtype, int32_t num_splits,
                                 void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  return run_tree(ATTN_KIND_SLIDING, q, k_pool, v_pool, block_table, seq_lens, cu_q, parents, o, batch, total_q, max_q,
                  max_blocks, num_pages, max_seq_len, window, out_dtype, num_splits, workspace, workspace_bytes, status,
                  stream);
}

int32_t attn_decode_global_tree(const void* q, const void* k_pool, const void* v_pool, const int32_t* block_table,
                                const int32_t* seq_lens, const int32_t* cu_q, const int32_t* parents, void* o,
                                int32_t batch, int32_t total_q, int32_t max_q, int32_t max_blocks, int64_t num_pages,
                                int32_t max_seq_len, int32_t window, int32_t out_dtype, int32_t num_splits,
                                void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  return run_tree(ATTN_KIND_GLOBAL, q, k_pool, v_pool, block_table, seq_lens, cu_q, parents, o, batch, total_q, max_q,
                  max_blocks, num_pages, max_seq_len, window, out_dtype, num_splits, workspace, workspace_bytes, status,
                  stream);
}

int32_t attn_decode_tree_plan(int32_t kind, int32_t batch, int32_t max_q, int32_t max_seq_len, int32_t window,
                              int32_t num_splits, int32_t num_sms, int32_t* out_num_splits, int32_t* out_launches,
                              size_t* out_workspace_bytes) {
  g_err[0] = '\0';
  TreePlan plan;
  const int32_t st = make_tree_plan(kind, batch, max_q, max_seq_len, window, num_splits, num_sms, &plan);
  if (st != ATTN_OK) return st;
  if (out_num_splits) *out_num_splits = plan.grid;
  if (out_launches) *out_launches = plan.merge ? 2 : 1;
  if (out_workspace_bytes) *out_workspace_bytes = plan.workspace_bytes;
  return ATTN_OK;
}

size_t attn_decode_tree_workspace_size(int32_t kind, int32_t batch, int32_t max_q, int32_t max_seq_len, int32_t window,
                                       int32_t num_splits) {
  g_err[0] = '\0';
  int dev = 0, num_sms = 0;
  if (current_device(&dev, &num_sms) != ATTN_OK) return 0;
  TreePlan plan;
  if (make_tree_plan(kind, batch, max_q, max_seq_len, window, num_splits, num_sms, &plan) != ATTN_OK) return 0;
  return plan.covering_bytes;
}

int32_t attn_kv_append_sliding_tree(const void* qkv, const void* w_q, const void* w_k, const int32_t* block_table,
                                    const int32_t* seq_lens, const int32_t* cu_q, const int32_t* parents, void* q_out,
                                    void* k_pool, void* v_pool, int32_t batch, int32_t total_q, int32_t max_blocks,
                                    int64_t num_pages, int32_t* status, void* stream) {
  return run_chunk(ATTN_KIND_SLIDING, Chunk::kTree, qkv, w_q, w_k, parents, block_table, seq_lens, cu_q, q_out, k_pool,
                   v_pool, nullptr, nullptr, batch, total_q, max_blocks, num_pages, status, stream);
}

int32_t attn_kv_append_global_tree(const void* qkv, const void* w_q, const void* w_k, const int32_t* block_table,
                                   const int32_t* seq_lens, const int32_t* cu_q, const int32_t* parents, void* q_out,
                                   void* k_pool, void* v_pool, int32_t batch, int32_t total_q, int32_t max_blocks,
                                   int64_t num_pages, int32_t* status, void* stream) {
  return run_chunk(ATTN_KIND_GLOBAL, Chunk::kTree, qkv, w_q, w_k, parents, block_table, seq_lens, cu_q, q_out, k_pool,
                   v_pool, nullptr, nullptr, batch, total_q, max_blocks, num_pages, status, stream);
}

int32_t attn_kv_commit_sliding(const void* const* k_pools, const void* const* v_pools, int32_t layers,
                               const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q,
                               const int32_t* path, const int32_t* path_len, int32_t* new_lens, int32_t batch,
                               int32_t max_path, int32_t max_blocks, int64_t num_pages, int32_t* status, void* stream) {
  return run_commit(ATTN_KIND_SLIDING, k_pools, v_pools, layers, block_table, seq_lens, cu_q, path, path_len, new_lens,
                    batch, max_path, max_blocks, num_pages, status, stream);
}

int32_t attn_kv_commit_global(const void* const* k_pools, const void* const* v_pools, int32_t layers,
                              const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q,
                              const int32_t* path, const int32_t* path_len, int32_t* new_lens, int32_t batch,
                              int32_t max_path, int32_t max_blocks, int64_t num_pages, int32_t* status, void* stream) {
  return run_commit(ATTN_KIND_GLOBAL, k_pools, v_pools, layers, block_table, seq_lens, cu_q, path, path_len, new_lens,
                    batch, max_path, max_blocks, num_pages, status, stream);
}

int32_t attn_pages_assign(const int32_t* cached_lens, const int32_t* new_tokens, int32_t* block_table,
                          const int32_t* held, int32_t* free_list, const int32_t* free_state, int32_t* held_out,
                          int32_t* free_state_out, int32_t* seq_lens, int32_t* cu_q, int32_t batch, int32_t max_blocks,
                          int64_t num_pages, int32_t window, int32_t* status, void* stream) {
  g_err[0] = '\0';
  const char* name = "attn_pages_assign";
  if (!cached_lens || !new_tokens || !block_table || !held || !free_list || !free_state || !held_out ||
      !free_state_out || !seq_lens || !cu_q)
    return fail(ATTN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (!aligned_to(cached_lens, 4) || !aligned_to(new_tokens, 4) || !aligned_to(block_table, 4) ||
      !aligned_to(free_list, 4) || !aligned_to(seq_lens, 4) || !aligned_to(cu_q, 4) || !aligned_to(status, 4) ||
      !aligned_to(held, 8) || !aligned_to(free_state, 8) || !aligned_to(held_out, 8) || !aligned_to(free_state_out, 8))
    return fail(ATTN_ERR_INVALID_ARG, "%s: misaligned pointer (held, free_state and their outputs 8 bytes, others 4)",
                name);
  int32_t st;
  if ((st = check_batch(name, batch, max_blocks)) || (st = check_pages(name, "num_pages", num_pages))) return st;
  g_last_launches = 1;
  if (g_validate_only) return ATTN_OK;
  pda::pages::PagesParams p{};
  p.cached = cached_lens;
  p.fresh = new_tokens;
  p.block_table = block_table;
  p.held = reinterpret_cast<const int2*>(held);
  p.free_list = free_list;
  p.free_state = reinterpret_cast<const int2*>(free_state);
  p.held_out = reinterpret_cast<int2*>(held_out);
  p.free_state_out = reinterpret_cast<int2*>(free_state_out);
  p.seq_lens = seq_lens;
  p.cu_q = cu_q;
  p.status = status;
  p.num_pages = static_cast<int32_t>(num_pages);
  p.batch = batch;
  p.max_blocks = max_blocks;
  p.window = window;
  return launched(name, launch_pdl(pda::pages::assign_kernel, dim3(pda::pages::kBlocks), pda::pages::kThreads, 0,
                                   static_cast<cudaStream_t>(stream), p));
}

}  // extern "C"
