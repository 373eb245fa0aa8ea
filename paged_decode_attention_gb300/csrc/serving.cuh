// serving.cuh -- host side of the chunk appends, the 8-bit cache
// (include/attn_fp8.h) and the decode behind a shared prefix.  Included in attn_decode.cu, whose
// validation helpers, plan, tensor-map encoder and launch recording it shares.
#pragma once

#include "attn_fp8.h"
#include "fp8_read.cuh"
#include "global_fp8.cuh"
#include "joined.cuh"
#include "kv_chunk.cuh"
#include "prefix.cuh"
#include "sliding_fp8.cuh"

namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// num_pages of a pool whose row coordinate (16 rows per page) is an int32
int32_t check_pages(const char* name, const char* what, int64_t num_pages) {
  if (num_pages < 1 || num_pages > (int64_t{1} << 31) / ATTN_PAGE_SIZE - 1)
    return fail(ATTN_ERR_INVALID_ARG, "%s: %s %lld out of range", name, what, static_cast<long long>(num_pages));
  return ATTN_OK;
}

int32_t check_batch(const char* name, int32_t batch, int32_t max_blocks) {
  if (batch < 1) return fail(ATTN_ERR_INVALID_ARG, "%s: batch must be >= 1 (got %d)", name, batch);
  if (batch > ATTN_MAX_BATCH)
    return fail(ATTN_ERR_UNSUPPORTED, "%s: batch %d outside [1, %d]", name, batch, ATTN_MAX_BATCH);
  if (max_blocks < 1) return fail(ATTN_ERR_INVALID_ARG, "%s: max_blocks must be >= 1", name);
  return ATTN_OK;
}

int32_t check_max_seq_len(const char* name, int32_t max_seq_len, int32_t max_blocks) {
  if (max_seq_len < 0 || static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_blocks) * ATTN_PAGE_SIZE)
    return fail(ATTN_ERR_INVALID_ARG, "%s: max_seq_len %d not in [0, max_blocks*16 = %lld]", name, max_seq_len,
                static_cast<long long>(max_blocks) * ATTN_PAGE_SIZE);
  if (max_seq_len > ATTN_MAX_SEQ_LEN)
    return fail(ATTN_ERR_UNSUPPORTED, "%s: max_seq_len %d beyond the model's domain (%d)", name, max_seq_len,
                ATTN_MAX_SEQ_LEN);
  return ATTN_OK;
}

int32_t launched(const char* name, cudaError_t e) {
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(ATTN_ERR_CUDA, "%s: launch failed: %s", name, cudaGetErrorString(e));
  return ATTN_OK;
}

// Pages that a sequence of up to max_len positions shows, at most.
int64_t visible_pages_bound(int32_t max_len, int32_t window) {
  const int64_t pages = (static_cast<int64_t>(max_len) + ATTN_PAGE_SIZE - 1) / ATTN_PAGE_SIZE;
  if (window <= 0) return pages;
  return std::min<int64_t>(pages, (static_cast<int64_t>(window) + ATTN_PAGE_SIZE - 1) / ATTN_PAGE_SIZE + 1);
}

// ---------------------------------------------------------------------------
// Launch plan of the 8-bit decode and of the own positions behind a prefix:
// make_plan's, but for the smallest spans.  A sequence that a block starts costs
// it some 2 us (its q, its end), so many short sequences want a block each: the
// grid has a virtual page per sequence in its count, and the smallest span is two
// pages.  A span cut off a long sequence costs the merge a partial row, so where a
// sequence may have many pages the smallest is longer.
// The kernels cut by the weights of their own parameters (4, sliding 12, fp8.cuh),
// which were measured on these grids: spans come out longer and some blocks find
// virtual pages only (global layers, one sequence of 250 pages: 63 blocks, spans
// of 5, 51 at work).  Likewise merge_in_grid is make_plan's, for its own spans: a
// choice between two ways of merging, either of which is right for any schedule.
// Global layers, automatic plan, two-page and four-page spans: 30 sequences of up
// to 15 positions 7.9 and 11.7 us (19.0 with make_plan's four pages per block), 4 of
// up to 600 8.2 and 10.9 us, one of 4000 11.0 and 9.3 us.
// ---------------------------------------------------------------------------
int32_t make_serving_plan(int32_t kind, int32_t batch, int32_t max_seq_len, int32_t window, int32_t forced_blocks,
                          int32_t num_sms, Plan* out) {
  const int32_t st = make_plan(kind, batch, max_seq_len, window, forced_blocks, num_sms, out);
  if (st != ATTN_OK) return st;
  const bool sliding = kind == ATTN_KIND_SLIDING;
  const int64_t pages = visible_pages_bound(max_seq_len, window);
  constexpr int kPartials = 32;  // per sequence, before spans grow
  out->min_pages = static_cast<int>(std::min<int64_t>(4, std::max<int64_t>(2, (pages + kPartials - 1) / kPartials)));
  if (forced_blocks == 0) {
    const int64_t resident = sliding ? static_cast<int64_t>(num_sms) * pda::sliding::kBlocksPerSm / ATTN_SLIDING_HKV
                                     : static_cast<int64_t>(num_sms) * pda::global::kBlocksPerSm;
    const int64_t useful = ((pages + pda::DecodeParams::kSeqWeight) * batch + out->min_pages - 1) / out->min_pages;
    out->grid_x = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({resident, useful, pda::kMaxSplits})));
  }
  const int d = sliding ? ATTN_SLIDING_D : ATTN_GLOBAL_D;
  const size_t rows = (static_cast<size_t>(out->grid_x) + batch) * (sliding ? ATTN_SLIDING_HQ : ATTN_GLOBAL_HQ);
  out->part_o_bytes = align256(rows * d * sizeof(float));
  out->workspace_bytes = ATTN_WORKSPACE_ZERO_BYTES + out->part_o_bytes + align256(rows * sizeof(float2));
  return ATTN_OK;
}

// Visible pages up to which every sequence gets a block of its own (per KV
// head): no partials and no merge kernel, but a sequence's pages one after
// another.  One call in us, in balanced spans and by sequence:
//   8-bit, global: 1 sequence of 64 positions 7.4 and 6.8, of 128 8.6 and 9.6; 4 of
//     16 7.3 and 5.0, of 128 10.2 and 9.7, of 256 9.9 and 15.4; 64 of 256 16.6 and
//     16.2, of 512 18.8 and 27.1; 128 of 128 21.9 and 11.0, of 512 32.3 and 27.5; 256
//     of 16 19.2 and 10.3, of 512 58.2 and 36.0;
//   8-bit, sliding: 1 of 128 6.6 and 6.0; 4 of 256 8.2 and 9.6; 32 of 128 13.1 and 8.2;
//     64 of 64 13.7 and 12.3, of 128 15.5 and 15.9; 128 of 32 14.3 and 19.7 (the
//     blocks of 57 sequences are resident at once on 152 SMs, which is the limit
//     taken: a second wave wins for the shortest only);
//   bf16 behind a prefix, both in one list: 1 of 32 positions 6.3 and 4.8, of 80 8.1
//     and 10.4; 4 of 56 8.4 and 7.7, of 128 7.9 and 9.8; 16 of 128 12.0 and 10.9; 32 of
//     120 16.8 and 12.2.
// Uneven lengths favour the spans, so long sequences take them unless the batch
// has eight for every page of the longest.
enum class Serving { kSlidingFp8, kGlobalFp8, kJoined };

int64_t whole_pages(Serving call, int32_t batch, int32_t num_sms) {
  switch (call) {
    case Serving::kSlidingFp8:
      return batch <= static_cast<int64_t>(num_sms) * pda::sliding::kBlocksPerSm / ATTN_SLIDING_HKV ? 8 : 0;
    case Serving::kGlobalFp8: return batch >= 64 ? std::max(16, batch / 8) : batch >= 4 ? 8 : 4;
    default: return batch >= 16 ? 8 : 4;
  }
}

// make_serving_plan's, or a block per sequence (its workspace is not used then).
int32_t make_whole_plan(Serving call, int32_t batch, int32_t max_seq_len, int32_t window, int32_t forced_blocks,
                        int32_t num_sms, Plan* out, bool* whole) {
  const int32_t kind = call == Serving::kSlidingFp8 ? ATTN_KIND_SLIDING : ATTN_KIND_GLOBAL;
  const int32_t st = make_serving_plan(kind, batch, max_seq_len, window, forced_blocks, num_sms, out);
  if (st != ATTN_OK) return st;
  *whole = forced_blocks == 0 && visible_pages_bound(max_seq_len, window) <= whole_pages(call, batch, num_sms);
  if (*whole) {
    out->grid_x = batch;
    out->merge_in_grid = true;  // (nothing to merge)
  }
  return ATTN_OK;
}

// ---------------------------------------------------------------------------
// Norms, RoPE and cache append of a chunk of tokens per sequence
// ---------------------------------------------------------------------------
enum class Chunk { kBf16, kFp8, kBehindPrefix };

int32_t run_chunk(int32_t kind, Chunk form, const void* qkv, const void* w_q, const void* w_k, const int32_t* prefix_len,
                  const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q, void* q_out, void* k_pool,
                  void* v_pool, uint8_t* k_scale, uint8_t* v_scale, int32_t batch, int32_t total_q, int32_t max_blocks,
                  int64_t num_pages, int32_t* status, void* stream) {
  g_err[0] = '\0';
  const bool sliding = kind == ATTN_KIND_SLIDING;
  const bool fp8 = form == Chunk::kFp8, behind = form == Chunk::kBehindPrefix;
  const char* name = fp8      ? (sliding ? "attn_kv_append_sliding_fp8" : "attn_kv_append_global_fp8")
                     : behind ? "attn_kv_append_global_prefix"
                              : (sliding ? "attn_kv_append_sliding_chunk" : "attn_kv_append_global_chunk");
  const bool values_only = !sliding && form == Chunk::kBf16;  // may leave the keys out
  if (!w_q || !w_k || !block_table || !seq_lens || !cu_q || (total_q > 0 && (!qkv || !q_out)) ||
      (!k_pool && !values_only) || !v_pool || (fp8 && (!k_scale || !v_scale)) || (behind && !prefix_len))
    return fail(ATTN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (!aligned_to(qkv, 16) || !aligned_to(w_q, 16) || !aligned_to(w_k, 16) || !aligned_to(q_out, 16) ||
      !aligned_to(k_pool, 16) || !aligned_to(v_pool, 16) || !aligned_to(k_scale, 16) || !aligned_to(v_scale, 16) ||
      !aligned_to(prefix_len, 4) || !aligned_to(block_table, 4) || !aligned_to(seq_lens, 4) || !aligned_to(cu_q, 4) ||
      !aligned_to(status, 4))
    return fail(ATTN_ERR_INVALID_ARG, "%s: misaligned pointer (qkv, w_q, w_k, q_out, pools and scales 16 bytes, "
                "tables 4)", name);
  int32_t st;
  if ((st = check_batch(name, batch, max_blocks)) || (st = check_pages(name, "num_pages", num_pages))) return st;
  if (total_q < 0) return fail(ATTN_ERR_INVALID_ARG, "%s: total_q must be >= 0", name);
  if (total_q > 1 << 28) return fail(ATTN_ERR_UNSUPPORTED, "%s: total_q %d too large", name, total_q);
  g_last_launches = total_q > 0 ? 1 : 0;
  if (total_q == 0) return ATTN_OK;  // no tokens
  int dev = 0, num_sms = 0;
  if ((st = current_device(&dev, &num_sms)) != ATTN_OK) return st;
  if (g_validate_only) return ATTN_OK;

  const int D = sliding ? ATTN_SLIDING_D : ATTN_GLOBAL_D;
  const double theta = sliding ? ATTN_SLIDING_ROPE_THETA : ATTN_GLOBAL_ROPE_THETA;
  pda::chunk::ChunkParams p{};
  p.qkv = static_cast<const __nv_bfloat16*>(qkv);
  p.w_q = static_cast<const __nv_bfloat16*>(w_q);
  p.w_k = static_cast<const __nv_bfloat16*>(w_k);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q;
  p.prefix_len = prefix_len;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.status = status;
  p.num_pages = num_pages;
  p.batch = batch;
  p.total_q = total_q;
  p.max_blocks = max_blocks;
  p.eps = 1e-6f;
  p.inv_pi = split_float_pair(0.31830988618379067154);
  for (int k = 0; k < pda::chunk::kPairBits; ++k)
    p.bit_factor[k] = split_float_pair(std::pow(theta, -2.0 * (1 << k) / D));

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  namespace ch = pda::chunk;
  const int blocks = std::min(total_q, num_sms * ch::kBlocksPerSm);
  const auto kernels = [&](auto fp8_c) {
    constexpr bool kFp8 = decltype(fp8_c)::value;
    if (sliding)
      return launch_pdl(ch::chunk_kernel<ATTN_SLIDING_D, ATTN_SLIDING_HQ, ATTN_SLIDING_HKV, ATTN_SLIDING_ROPE_PAIRS,
                                         false, kFp8>,
                        dim3(blocks), ch::kThreads<false>, 0, s, p);
    return launch_pdl(ch::chunk_kernel<ATTN_GLOBAL_D, ATTN_GLOBAL_HQ, ATTN_GLOBAL_HKV, ATTN_GLOBAL_ROPE_PAIRS, true,
                                       kFp8>,
                      dim3(blocks), ch::kThreads<true>, 0, s, p);
  };
  const cudaError_t e = fp8 ? kernels(std::true_type{}) : kernels(std::false_type{});
  return launched(name, e);
}

// ---------------------------------------------------------------------------
// 8-bit cache: read back into bf16 pages
// ---------------------------------------------------------------------------
int32_t run_read(int32_t kind, const void* k_pool, const void* v_pool, const uint8_t* k_scale, const uint8_t* v_scale,
                 const int32_t* block_table, const int32_t* seq_lens, void* k_out, void* v_out,
                 const int32_t* out_table, int32_t batch, int32_t max_blocks, int64_t num_pages, int64_t out_pages,
                 int32_t max_seq_len, int32_t span, int32_t* status, void* stream) {
  g_err[0] = '\0';
  const bool sliding = kind == ATTN_KIND_SLIDING;
  const char* name = sliding ? "attn_kv_read_sliding_fp8" : "attn_kv_read_global_fp8";
  if (!k_pool || !v_pool || !k_scale || !v_scale || !block_table || !seq_lens || !k_out || !v_out || !out_table)
    return fail(ATTN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (!aligned_to(k_pool, 16) || !aligned_to(v_pool, 16) || !aligned_to(k_scale, 16) || !aligned_to(v_scale, 16) ||
      !aligned_to(k_out, 16) || !aligned_to(v_out, 16) || !aligned_to(block_table, 4) || !aligned_to(seq_lens, 4) ||
      !aligned_to(out_table, 4) || !aligned_to(status, 4))
    return fail(ATTN_ERR_INVALID_ARG, "%s: misaligned pointer (pools and scales 16 bytes, tables 4)", name);
  int32_t st;
  if ((st = check_batch(name, batch, max_blocks)) || (st = check_pages(name, "num_pages", num_pages)) ||
      (st = check_pages(name, "out_pages", out_pages)) || (st = check_max_seq_len(name, max_seq_len, max_blocks)))
    return st;
  int dev = 0, num_sms = 0;
  if ((st = current_device(&dev, &num_sms)) != ATTN_OK) return st;
  g_last_launches = 1;
  if (g_validate_only) return ATTN_OK;

  pda::fp8_read::ReadParams p{};
  p.d.block_table = block_table;
  p.d.seq_lens = seq_lens;
  p.d.status = status;
  p.d.num_pages = num_pages;
  p.d.batch = batch;
  p.d.max_blocks = max_blocks;
  p.d.window = span;
  p.d.min_pages = 1;
  p.src[0] = static_cast<const uint8_t*>(k_pool);
  p.src[1] = static_cast<const uint8_t*>(v_pool);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.dst[0] = static_cast<__nv_bfloat16*>(k_out);
  p.dst[1] = static_cast<__nv_bfloat16*>(v_out);
  p.out_table = out_table;
  p.out_pages = out_pages;
  // no more blocks than the (weighted) pages that max_seq_len allows
  const int64_t want = (visible_pages_bound(max_seq_len, span) + pda::DecodeParams::kSeqWeight) * batch;
  p.d.grid_x = static_cast<int32_t>(
      std::max<int64_t>(1, std::min<int64_t>(want, num_sms * pda::fp8_read::kGridPerSm)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(p.d.grid_x, 2);
  const cudaError_t e =
      sliding ? launch_pdl(pda::fp8_read::read_kernel<ATTN_SLIDING_HKV, ATTN_SLIDING_D>, grid, pda::fp8_read::kThreads, 0,
                           s, p)
              : launch_pdl(pda::fp8_read::read_kernel<ATTN_GLOBAL_HKV, ATTN_GLOBAL_D>, grid, pda::fp8_read::kThreads, 0,
                           s, p);
  return launched(name, e);
}

// ---------------------------------------------------------------------------
// The merge of global layers' partials where rows are few: combine.cuh's four
// blocks per row, of 128 threads, which start beside the decode blocks, and
// hold 32 partials in flight per round.  Where a sequence may have more than
// two rounds of them, 16 blocks per row with 128 in flight.  One call over the
// 8-bit cache in us, 4 blocks and 16: one sequence of 38656 (152 partials)
// 28.8 and 21.2, one of 4000 (63) 9.2 and 9.8, 8 of 4700 17.2 and 21.2.
// ---------------------------------------------------------------------------
constexpr int kMergeDims = 32;  // of a row, per block of the second kind
constexpr int kMergeThreads = 128;

template <typename Params>
constexpr auto kWideMerge = pda::prefix::merge_kernel<ATTN_GLOBAL_D, 0, 1, kMergeDims, kMergeThreads * 4 / kMergeDims, Params>;

template <typename Params>
int32_t ensure_merge(int dev) {
  static bool comb_set[kMaxDevices] = {false}, wide_set[kMaxDevices] = {false};
  const int32_t st = ensure_smem(pda::combine_kernel<ATTN_GLOBAL_D, Params>, 0, dev, comb_set);
  return st != ATTN_OK ? st : ensure_smem(kWideMerge<Params>, 0, dev, wide_set);
}

template <typename Params>
cudaError_t launch_merge(const Params& p, cudaStream_t s) {
  if (p.grid_x > 64 * p.batch) {
    pda::prefix::MergeParams<Params> mp{};
    mp.d = p;
    return launch_pdl(kWideMerge<Params>, dim3(ATTN_GLOBAL_HQ * (ATTN_GLOBAL_D / kMergeDims), p.batch), kMergeThreads, 0,
                      s, mp);
  }
  return launch_pdl(pda::combine_kernel<ATTN_GLOBAL_D, Params>,
                    dim3(ATTN_GLOBAL_HQ * (ATTN_GLOBAL_D / pda::kCombineCols), p.batch), pda::kCombineWarps * 32, 0, s,
                    p);
}

// ---------------------------------------------------------------------------
// Decode over an 8-bit cache
// ---------------------------------------------------------------------------

// An e4m3 pool [num_pages*16 rows][row_bytes] as a 3-D tensor (x: 128 dims
// of a chunk, y: row, z: chunk): a box {128, 16, chunks} copies one KV head of
// a page as 128-byte-swizzled [16 rows][128 dims] tiles.
int32_t encode_fp8_map(CUtensorMap* map, const void* pool, int64_t num_pages, int row_bytes, int chunks) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(num_pages) * ATTN_PAGE_SIZE,
                              static_cast<cuuint64_t>(row_bytes / 128)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_bytes), 128};
  const cuuint32_t box[3] = {128, ATTN_PAGE_SIZE, static_cast<cuuint32_t>(chunks)};
  const cuuint32_t elem_strides[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool), dims, strides, box, elem_strides,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled (e4m3 map) failed (%d)", static_cast<int>(r));
  return ATTN_OK;
}

// A scale pool as rows of 16 bytes, one per (page, KV head).
int32_t encode_scale_map(CUtensorMap* map, const void* scales, int64_t rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[2] = {ATTN_PAGE_SIZE, static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {ATTN_PAGE_SIZE};
  const cuuint32_t box[2] = {ATTN_PAGE_SIZE, 1};
  const cuuint32_t elem_strides[2] = {1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(scales), dims, strides, box, elem_strides,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled (scale map) failed (%d)", static_cast<int>(r));
  return ATTN_OK;
}

int32_t run_decode_fp8(int32_t kind, const void* q, const void* k_pool, const void* v_pool, const uint8_t* k_scale,
                       const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens, void* o,
                       int32_t batch, int32_t max_blocks, int64_t num_pages, int32_t max_seq_len, int32_t window,
                       int32_t out_dtype, int32_t num_splits, void* workspace, size_t workspace_bytes, int32_t* status,
                       void* stream) {
  g_err[0] = '\0';
  const bool sliding = kind == ATTN_KIND_SLIDING;
  const char* name = sliding ? "attn_decode_sliding_fp8" : "attn_decode_global_fp8";
  if (!q || !k_pool || !v_pool || !k_scale || !v_scale || !block_table || !seq_lens || !o)
    return fail(ATTN_ERR_INVALID_ARG, "%s: null array pointer", name);
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_scale) || !aligned16(v_scale) ||
      !aligned16(block_table) || !aligned16(seq_lens) || !aligned16(o))
    return fail(ATTN_ERR_INVALID_ARG, "%s: every array must be 16-byte aligned", name);
  if (!aligned_to(status, 4)) return fail(ATTN_ERR_INVALID_ARG, "%s: status must be 4-byte aligned", name);
  int32_t st;
  if ((st = check_batch(name, batch, max_blocks)) || (st = check_pages(name, "num_pages", num_pages)) ||
      (st = check_max_seq_len(name, max_seq_len, max_blocks)))
    return st;
  if (sliding && window <= 0)
    return fail(ATTN_ERR_INVALID_ARG, "%s: window must be > 0 (the node's is 1024)", name);
  if (out_dtype != ATTN_OUT_BF16 && out_dtype != ATTN_OUT_F32)
    return fail(ATTN_ERR_INVALID_ARG, "%s: out_dtype must be ATTN_OUT_BF16 or ATTN_OUT_F32", name);
  if (num_splits < 0) return fail(ATTN_ERR_INVALID_ARG, "%s: num_splits must be >= 0", name);

  int dev = 0, num_sms = 0;
  if ((st = current_device(&dev, &num_sms)) != ATTN_OK) return st;
  Plan plan;
  bool whole = false;
  st = make_whole_plan(sliding ? Serving::kSlidingFp8 : Serving::kGlobalFp8, batch, max_seq_len, window, num_splits,
                       num_sms, &plan, &whole);
  if (st != ATTN_OK) return st;
  if (!workspace || workspace_bytes < plan.workspace_bytes)
    return fail(ATTN_ERR_WORKSPACE, "%s: workspace of %zu bytes required (got %zu)", name, plan.workspace_bytes,
                workspace ? workspace_bytes : size_t{0});
  if (!aligned16(workspace)) return fail(ATTN_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", name);
  g_last_launches = plan.merge_in_grid ? 1 : 2;
  if (g_validate_only) return ATTN_OK;

  pda::Fp8WholeParams all{};
  pda::DecodeParams& p = all;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_pool = static_cast<const __nv_bfloat16*>(k_pool);  // bytes; addressed as such by the kernels
  p.v_pool = static_cast<const __nv_bfloat16*>(v_pool);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.o = o;
  p.counters = static_cast<int32_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ATTN_WORKSPACE_ZERO_BYTES);
  p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + ATTN_WORKSPACE_ZERO_BYTES +
                                        plan.part_o_bytes);
  p.status = status;
  p.num_pages = num_pages;
  p.batch = batch;
  p.max_blocks = max_blocks;
  p.window = window;
  p.grid_x = plan.grid_x;
  p.min_pages = plan.min_pages;
  p.out_f32 = out_dtype == ATTN_OUT_F32;
  p.part_rows = (static_cast<int64_t>(plan.grid_x) + batch) * (sliding ? ATTN_SLIDING_HQ : ATTN_GLOBAL_HQ);
  p.merge_in_grid = plan.merge_in_grid;

  const int hkv = sliding ? ATTN_SLIDING_HKV : ATTN_GLOBAL_HKV;
  const int d = sliding ? ATTN_SLIDING_D : ATTN_GLOBAL_D;
  CUtensorMap tm_k, tm_v, tm_ks, tm_vs;
  if ((st = encode_fp8_map(&tm_k, k_pool, num_pages, hkv * d, d / 128)) ||
      (st = encode_fp8_map(&tm_v, v_pool, num_pages, hkv * d, d / 128)) ||
      (st = encode_scale_map(&tm_ks, k_scale, num_pages * hkv)) ||
      (st = encode_scale_map(&tm_vs, v_scale, num_pages * hkv)))
    return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (sliding) {
    pda::Fp8SlidingParams cut{};
    static_cast<pda::DecodeParams&>(cut) = p;
    namespace sl = pda::sliding_fp8;
    const auto decode = sl::decode_kernel<pda::Fp8SlidingParams>;
    const auto decode_whole = sl::decode_kernel<pda::Fp8WholeParams>;
    const auto combine = pda::combine_kernel<ATTN_SLIDING_D, pda::Fp8SlidingParams>;
    static bool smem_set[kMaxDevices] = {false}, whole_set[kMaxDevices] = {false}, comb_set[kMaxDevices] = {false};
    if ((st = ensure_smem(decode, sl::kSmemBytes, dev, smem_set)) ||
        (st = ensure_smem(decode_whole, sl::kSmemBytes, dev, whole_set)) ||
        (st = ensure_smem(combine, 0, dev, comb_set)))
      return st;
    const dim3 grid(ATTN_SLIDING_HKV, plan.grid_x);
    e = whole ? launch_pdl(decode_whole, grid, sl::kThreads, sl::kSmemBytes, s, tm_k, tm_v, tm_ks, tm_vs, all)
              : launch_pdl(decode, grid, sl::kThreads, sl::kSmemBytes, s, tm_k, tm_v, tm_ks, tm_vs, cut);
    if (e == cudaSuccess && !plan.merge_in_grid)
      e = launch_pdl(combine, dim3(ATTN_SLIDING_HQ * (ATTN_SLIDING_D / pda::kCombineCols), batch),
                     pda::kCombineWarps * 32, 0, s, cut);
  } else {
    pda::Fp8GlobalParams cut{};
    static_cast<pda::DecodeParams&>(cut) = p;
    namespace gl = pda::global_fp8;
    const auto decode = gl::decode_kernel<pda::Fp8GlobalParams>;
    const auto decode_whole = gl::decode_kernel<pda::Fp8WholeParams>;
    // Many rows: one merge block per row (64 sequences of 500: 22.5 us a call,
    // against 29.4 with launch_merge's four).
    const bool few_rows = batch * ATTN_GLOBAL_HQ <= 2 * num_sms;
    const auto row_kernel = pda::prefix::merge_kernel<ATTN_GLOBAL_D, 0, 1, ATTN_GLOBAL_D, 2, pda::Fp8GlobalParams>;
    static bool smem_set[kMaxDevices] = {false}, whole_set[kMaxDevices] = {false}, row_set[kMaxDevices] = {false};
    if ((st = ensure_smem(decode, gl::kSmemBytes, dev, smem_set)) ||
        (st = ensure_smem(decode_whole, gl::kSmemBytes, dev, whole_set)) ||
        (st = ensure_smem(row_kernel, 0, dev, row_set)) || (st = ensure_merge<pda::Fp8GlobalParams>(dev)))
      return st;
    if (whole) {
      e = launch_pdl(decode_whole, dim3(plan.grid_x), gl::kThreads, gl::kSmemBytes, s, tm_k, tm_v, tm_ks, tm_vs, all);
    } else {
      pda::prefix::MergeParams<pda::Fp8GlobalParams> mp{};
      mp.d = cut;
      e = launch_pdl(decode, dim3(plan.grid_x), gl::kThreads, gl::kSmemBytes, s, tm_k, tm_v, tm_ks, tm_vs, cut);
      if (e == cudaSuccess)
        e = few_rows ? launch_merge(cut, s) : launch_pdl(row_kernel, dim3(ATTN_GLOBAL_HQ, batch), 256, 0, s, mp);
    }
  }
  return launched(name, e);
}

// ---------------------------------------------------------------------------
// Decode behind a prefix that the batch shares
// ---------------------------------------------------------------------------
using PrefixConfig = pda::prefill_pair::GlobalPairConfig;
constexpr int kMaxPrefixSplits = 128;
// Whether every sequence reads the prefix for itself (joined.cuh).  That costs
// a pass of L2 over the prefix per sequence and saves a kernel and a merge of
// spans.  One call in us, joined and in spans: 1 sequence, 16 positions 8.2 and
// 12.1, 32768 18.9 and 36.7, 262144 88 and 202; 2 sequences, 16384 17.0 and 25.7,
// 262144 160 and 197; 3 of 65536 51 and 62; 4 of 22000 30.0 and 32.4; 8 of 2000 14.1
// and 19.5, 8000 24.2 and 24.6, 10500 28.6 and 26.5; 12 of 2000 15.9 and 20.2,
// 6500 27.6 and 23.4; 16 of 1000 16.5 and 19.2, 3000 24.1 and 21.4; 24 of 500 18.2
// and 20.4, 2500 27.9 and 22.7; 32 of 100 17.8 and 19.8, 500 21.7 and 20.6.  The
// rule runs through the crossings of 8 to 32 sequences; for 3, and 4 as far as
// measured, it takes spans before the crossing (3 from 61923 positions on).
bool join_prefix(int32_t batch, int32_t max_prefix_len) {
  return batch <= 2 || static_cast<int64_t>(batch) * batch * (static_cast<int64_t>(max_prefix_len) + 300) <= 560000;
}
constexpr int kPrefixMinSteps = 2;  // steps of 64 keys a span is given at least (32 sequences, 2000 positions: 28.8 us)

struct PrefixPlan {
  bool joined;        // prefix and own pages as one list per sequence (joined.cuh): two kernels
  bool whole;         // joined, a block per sequence: one kernel
  Plan own;           // the decode over the own positions, or over the joined list
  int splits;         // spans of the prefix; 0 when joined
  size_t part_o_off, part_ml_off, workspace_bytes;
};

int32_t make_prefix_plan(int32_t batch, int32_t max_prefix_len, int32_t max_seq_len, int32_t num_splits,
                         int32_t prefix_splits, int32_t num_sms, PrefixPlan* out) {
  if (max_prefix_len < 0) return fail(ATTN_ERR_INVALID_ARG, "max_prefix_len must be >= 0");
  if (prefix_splits < 0) return fail(ATTN_ERR_INVALID_ARG, "prefix_splits must be >= 0");
  if (max_seq_len < 0) return fail(ATTN_ERR_INVALID_ARG, "max_seq_len must be >= 0");
  out->joined = prefix_splits == 0 && join_prefix(batch, max_prefix_len);
  const int64_t joined_len =
      (static_cast<int64_t>(max_prefix_len) + ATTN_PAGE_SIZE - 1) / ATTN_PAGE_SIZE * ATTN_PAGE_SIZE + max_seq_len;
  const int32_t len = static_cast<int32_t>(std::min<int64_t>(joined_len, INT32_MAX));
  out->whole = false;
  const int32_t st =
      out->joined ? make_whole_plan(Serving::kJoined, batch, len, 0, num_splits, num_sms, &out->own, &out->whole)
                  : make_serving_plan(ATTN_KIND_GLOBAL, batch, max_seq_len, 0, num_splits, num_sms, &out->own);
  if (st != ATTN_OK) return st;
  out->splits = 0;
  out->part_o_off = out->part_ml_off = 0;
  out->workspace_bytes = out->own.workspace_bytes;
  if (out->joined) return ATTN_OK;
  // One CTA pair per SM pair: 2 query tiles (of kQ sequences each) and one
  // slice of the output dims per cluster, the rest of the GPU by spans.
  const int64_t pairs = (batch + 2 * PrefixConfig::kQ - 1) / (2 * PrefixConfig::kQ) * PrefixConfig::kSlices;
  const int64_t steps = (static_cast<int64_t>(max_prefix_len) + PrefixConfig::kKeys - 1) / PrefixConfig::kKeys;
  int64_t splits = prefix_splits;
  if (splits == 0) {
    splits = num_sms / 2 / pairs;
    if (splits > steps / kPrefixMinSteps) splits = steps / kPrefixMinSteps;
  }
  out->splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(splits, kMaxPrefixSplits)));
  const size_t rows = static_cast<size_t>(out->splits) * batch * ATTN_GLOBAL_HQ;
  out->part_o_off = out->own.workspace_bytes;
  out->part_ml_off = out->part_o_off + align256(rows * ATTN_GLOBAL_D * sizeof(float));
  out->workspace_bytes = out->part_ml_off + align256(rows * PrefixConfig::kSlices * sizeof(float2));
  return ATTN_OK;
}

int32_t run_prefix(const void* q, const void* k_pool, const void* v_pool, const int32_t* prefix_table,
                   const int32_t* prefix_len, const int32_t* block_table, const int32_t* seq_lens, void* o,
                   int32_t batch, int32_t prefix_blocks, int32_t max_blocks, int64_t num_pages, int32_t max_prefix_len,
                   int32_t max_seq_len, int32_t out_dtype, int32_t num_splits, int32_t prefix_splits, void* workspace,
                   size_t workspace_bytes, int32_t* status, void* stream) {
  g_err[0] = '\0';
  const char* name = "attn_decode_global_prefix";
  if (!q || !k_pool || !v_pool || !prefix_table || !prefix_len || !block_table || !seq_lens || !o)
    return fail(ATTN_ERR_INVALID_ARG, "%s: null array pointer", name);
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(block_table) || !aligned16(seq_lens) ||
      !aligned16(o) || !aligned_to(prefix_table, 4) || !aligned_to(prefix_len, 4) || !aligned_to(status, 4))
    return fail(ATTN_ERR_INVALID_ARG, "%s: misaligned pointer (arrays 16 bytes; prefix_table, prefix_len, status 4)",
                name);
  int32_t st;
  if ((st = check_batch(name, batch, max_blocks)) || (st = check_pages(name, "num_pages", num_pages)) ||
      (st = check_max_seq_len(name, max_seq_len, max_blocks)))
    return st;
  if (prefix_blocks < 1) return fail(ATTN_ERR_INVALID_ARG, "%s: prefix_blocks must be >= 1", name);
  if (max_prefix_len < 0 || static_cast<int64_t>(max_prefix_len) > static_cast<int64_t>(prefix_blocks) * ATTN_PAGE_SIZE)
    return fail(ATTN_ERR_INVALID_ARG, "%s: max_prefix_len %d not in [0, prefix_blocks*16 = %lld]", name, max_prefix_len,
                static_cast<long long>(prefix_blocks) * ATTN_PAGE_SIZE);
  if (max_prefix_len > ATTN_MAX_SEQ_LEN)
    return fail(ATTN_ERR_UNSUPPORTED, "%s: max_prefix_len %d beyond the model's domain (%d)", name, max_prefix_len,
                ATTN_MAX_SEQ_LEN);
  if (out_dtype != ATTN_OUT_BF16 && out_dtype != ATTN_OUT_F32)
    return fail(ATTN_ERR_INVALID_ARG, "%s: out_dtype must be ATTN_OUT_BF16 or ATTN_OUT_F32", name);
  if (num_splits < 0 || prefix_splits < 0)
    return fail(ATTN_ERR_INVALID_ARG, "%s: num_splits and prefix_splits must be >= 0", name);
  int dev = 0, num_sms = 0;
  if ((st = current_device(&dev, &num_sms)) != ATTN_OK) return st;
  PrefixPlan plan;
  st = make_prefix_plan(batch, max_prefix_len, max_seq_len, num_splits, prefix_splits, num_sms, &plan);
  if (st != ATTN_OK) return st;
  if (!workspace || workspace_bytes < plan.workspace_bytes)
    return fail(ATTN_ERR_WORKSPACE, "%s: workspace of %zu bytes required (got %zu)", name, plan.workspace_bytes,
                workspace ? workspace_bytes : size_t{0});
  if (!aligned16(workspace)) return fail(ATTN_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", name);
  g_last_launches = plan.whole ? 1 : plan.joined ? 2 : 3;
  if (g_validate_only) return ATTN_OK;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  pda::JoinedParams jp{};
  pda::DecodeParams& p = jp;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_pool = static_cast<const __nv_bfloat16*>(k_pool);
  p.v_pool = static_cast<const __nv_bfloat16*>(v_pool);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.o = o;
  p.counters = static_cast<int32_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws + ATTN_WORKSPACE_ZERO_BYTES);
  p.part_ml = reinterpret_cast<float2*>(ws + ATTN_WORKSPACE_ZERO_BYTES + plan.own.part_o_bytes);
  p.status = status;
  p.num_pages = num_pages;
  p.batch = batch;
  p.max_blocks = max_blocks;
  p.grid_x = plan.own.grid_x;
  p.min_pages = plan.own.min_pages;
  p.out_f32 = out_dtype == ATTN_OUT_F32;
  p.part_rows = (static_cast<int64_t>(plan.own.grid_x) + batch) * ATTN_GLOBAL_HQ;
  jp.prefix_table = prefix_table;
  jp.prefix_len = prefix_len;
  jp.prefix_blocks = prefix_blocks;
  jp.whole_sequences = plan.whole;
  CUtensorMap tm_k, tm_v;
  if ((st = encode_global_page_map(&tm_k, k_pool, num_pages)) || (st = encode_global_page_map(&tm_v, v_pool, num_pages)))
    return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (plan.joined) {
    const auto decode = pda::global::decode_kernel_listed<pda::JoinedParams>;
    static bool dec_set[kMaxDevices] = {false};
    if ((st = ensure_smem(decode, pda::global::kSmemBytes, dev, dec_set)) || (st = ensure_merge<pda::JoinedParams>(dev)))
      return st;
    cudaError_t e = launch_pdl(decode, dim3(plan.own.grid_x), pda::global::kThreads, pda::global::kSmemBytes, s, tm_k,
                               tm_v, jp);
    if (e == cudaSuccess && !plan.whole) e = launch_merge(jp, s);
    return launched(name, e);
  }
  pda::prefill_pair::PrefixParams pp{};
  pp.q = p.q;
  pp.block_table = prefix_table;
  pp.seq_lens = prefix_len;
  pp.status = status;
  pp.num_pages = num_pages;
  pp.batch = 1;
  pp.max_blocks = prefix_blocks;
  pp.total_q = batch;
  pp.max_q = batch;
  pp.part_o = reinterpret_cast<float*>(ws + plan.part_o_off);
  pp.part_ml = reinterpret_cast<float2*>(ws + plan.part_ml_off);
  pp.splits = plan.splits;

  pda::prefix::OwnParams own{};
  static_cast<pda::DecodeParams&>(own) = p;
  pda::prefix::MergeParams<pda::prefix::OwnParams> mp{};
  mp.d = own;
  mp.part_o = pp.part_o;
  mp.part_ml = pp.part_ml;
  mp.prefix_len = prefix_len;
  mp.prefix_blocks = prefix_blocks;
  mp.splits = plan.splits;

  using C = PrefixConfig;
  const auto prefix_kernel = pda::prefill_pair::prefill_pair_kernel<C, pda::prefill_pair::PrefixParams>;
  const bool few_rows = batch * ATTN_GLOBAL_HQ <= 2 * num_sms;  // the merge's blocks are resident at once
  const auto merge_kernel =
      few_rows ? pda::prefix::merge_kernel<ATTN_GLOBAL_D, C::kSlices, C::kPPS, ATTN_GLOBAL_D, 4, pda::prefix::OwnParams>
               : pda::prefix::merge_kernel<ATTN_GLOBAL_D, C::kSlices, C::kPPS, ATTN_GLOBAL_D, 2, pda::prefix::OwnParams>;
  const auto own_kernel = pda::global::decode_kernel_partial<pda::prefix::OwnParams>;
  static bool pre_set[kMaxDevices] = {false}, dec_set[kMaxDevices] = {false}, merge_set[2][kMaxDevices] = {{false}};
  if ((st = ensure_smem(prefix_kernel, C::kSmemBytes, dev, pre_set)) ||
      (st = ensure_smem(own_kernel, pda::global::kSmemBytes, dev, dec_set)) ||
      (st = ensure_smem(merge_kernel, 0, dev, merge_set[few_rows])))
    return st;
  CUtensorMap tm_pk, tm_pv;
  if ((st = encode_chunk_map(&tm_pk, k_pool, num_pages, C::kHkv * C::kD, C::kKBoxChunks)) ||
      (st = encode_chunk_map(&tm_pv, v_pool, num_pages, C::kHkv * C::kD, C::kDS / 128)))
    return st;
  int tiles = (batch + C::kQ - 1) / C::kQ;
  tiles += tiles & 1;  // whole clusters of two query tiles
  cudaError_t e = launch_pdl(prefix_kernel, dim3(tiles, C::kHkv * C::kSlices, plan.splits), C::kThreads, C::kSmemBytes, s,
                             tm_pk, tm_pv, pp);
  if (e == cudaSuccess)
    e = launch_pdl(own_kernel, dim3(plan.own.grid_x), pda::global::kThreads,
                   pda::global::kSmemBytes, s, tm_k, tm_v, own);
  if (e == cudaSuccess)
    e = launch_pdl(merge_kernel, dim3(ATTN_GLOBAL_HQ, batch), few_rows ? 512 : 256, 0, s, mp);
  return launched(name, e);
}

}  // namespace

extern "C" {

int32_t attn_decode_global_prefix(const void* q, const void* k_pool, const void* v_pool, const int32_t* prefix_table,
                                  const int32_t* prefix_len, const int32_t* block_table, const int32_t* seq_lens,
                                  void* o, int32_t batch, int32_t prefix_blocks, int32_t max_blocks, int64_t num_pages,
                                  int32_t max_prefix_len, int32_t max_seq_len, int32_t out_dtype, int32_t num_splits,
                                  int32_t prefix_splits, void* workspace, size_t workspace_bytes, int32_t* status,
                                  void* stream) {
  return run_prefix(q, k_pool, v_pool, prefix_table, prefix_len, block_table, seq_lens, o, batch, prefix_blocks,
                    max_blocks, num_pages, max_prefix_len, max_seq_len, out_dtype, num_splits, prefix_splits, workspace,
                    workspace_bytes, status, stream);
}

int32_t attn_decode_fp8_plan(int32_t kind, int32_t batch, int32_t max_seq_len, int32_t window, int32_t num_splits,
                             int32_t num_sms, int32_t* out_num_splits, int32_t* out_launches,
                             size_t* out_workspace_bytes) {
  g_err[0] = '\0';
  Plan plan;
  bool whole = false;
  int32_t st = make_serving_plan(kind, batch, max_seq_len, window, num_splits, num_sms, &plan);  // (refuses a bad kind)
  if (st != ATTN_OK) return st;
  st = make_whole_plan(kind == ATTN_KIND_SLIDING ? Serving::kSlidingFp8 : Serving::kGlobalFp8, batch, max_seq_len,
                       window, num_splits, num_sms, &plan, &whole);
  if (st != ATTN_OK) return st;
  if (out_num_splits) *out_num_splits = plan.grid_x;
  if (out_launches) *out_launches = plan.merge_in_grid ? 1 : 2;
  if (out_workspace_bytes) *out_workspace_bytes = plan.workspace_bytes;
  return ATTN_OK;
}

size_t attn_decode_fp8_workspace_size(int32_t kind, int32_t batch, int32_t max_seq_len, int32_t window,
                                      int32_t num_splits) {
  g_err[0] = '\0';
  int dev = 0, num_sms = 0;
  if (current_device(&dev, &num_sms) != ATTN_OK) return 0;
  Plan plan;
  if (make_serving_plan(kind, batch, max_seq_len, window, num_splits, num_sms, &plan) != ATTN_OK) return 0;
  return plan.workspace_bytes;
}

int32_t attn_decode_prefix_plan(int32_t batch, int32_t max_prefix_len, int32_t max_seq_len, int32_t num_splits,
                                int32_t prefix_splits, int32_t num_sms, int32_t* out_num_splits,
                                int32_t* out_prefix_splits, size_t* out_workspace_bytes) {
  g_err[0] = '\0';
  PrefixPlan plan;
  const int32_t st = make_prefix_plan(batch, max_prefix_len, max_seq_len, num_splits, prefix_splits, num_sms, &plan);
  if (st != ATTN_OK) return st;
  if (out_num_splits) *out_num_splits = plan.own.grid_x;
  if (out_prefix_splits) *out_prefix_splits = plan.splits;
  if (out_workspace_bytes) *out_workspace_bytes = plan.workspace_bytes;
  return ATTN_OK;
}

size_t attn_decode_prefix_workspace_size(int32_t batch, int32_t max_prefix_len, int32_t max_seq_len,
                                         int32_t num_splits, int32_t prefix_splits) {
  g_err[0] = '\0';
  int dev = 0, num_sms = 0;
  if (current_device(&dev, &num_sms) != ATTN_OK) return 0;
  PrefixPlan plan;
  if (make_prefix_plan(batch, max_prefix_len, max_seq_len, num_splits, prefix_splits, num_sms, &plan) != ATTN_OK)
    return 0;
  return plan.workspace_bytes;
}

int32_t attn_kv_append_sliding_chunk(const void* qkv, const void* w_q, const void* w_k, const int32_t* block_table,
                                     const int32_t* seq_lens, const int32_t* cu_q, void* q_out, void* k_pool,
                                     void* v_pool, int32_t batch, int32_t total_q, int32_t max_blocks,
                                     int64_t num_pages, int32_t* status, void* stream) {
  return run_chunk(ATTN_KIND_SLIDING, Chunk::kBf16, qkv, w_q, w_k, nullptr, block_table, seq_lens, cu_q, q_out, k_pool,
                   v_pool, nullptr, nullptr, batch, total_q, max_blocks, num_pages, status, stream);
}

int32_t attn_kv_append_global_chunk(const void* qkv, const void* w_q, const void* w_k, const int32_t* block_table,
                                    const int32_t* seq_lens, const int32_t* cu_q, void* q_out, void* k_pool,
                                    void* v_pool, int32_t batch, int32_t total_q, int32_t max_blocks,
                                    int64_t num_pages, int32_t* status, void* stream) {
  return run_chunk(ATTN_KIND_GLOBAL, Chunk::kBf16, qkv, w_q, w_k, nullptr, block_table, seq_lens, cu_q, q_out, k_pool,
                   v_pool, nullptr, nullptr, batch, total_q, max_blocks, num_pages, status, stream);
}

int32_t attn_kv_append_global_prefix(const void* qkv, const void* w_q, const void* w_k, const int32_t* prefix_len,
                                     const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q,
                                     void* q_out, void* k_pool, void* v_pool, int32_t batch, int32_t total_q,
                                     int32_t max_blocks, int64_t num_pages, int32_t* status, void* stream) {
  return run_chunk(ATTN_KIND_GLOBAL, Chunk::kBehindPrefix, qkv, w_q, w_k, prefix_len, block_table, seq_lens, cu_q, q_out,
                   k_pool, v_pool, nullptr, nullptr, batch, total_q, max_blocks, num_pages, status, stream);
}

int32_t attn_kv_append_sliding_fp8(const void* qkv, const void* w_q, const void* w_k, const int32_t* block_table,
                                   const int32_t* seq_lens, const int32_t* cu_q, void* q_out, void* k_pool,
                                   void* v_pool, uint8_t* k_scale, uint8_t* v_scale, int32_t batch, int32_t total_q,
                                   int32_t max_blocks, int64_t num_pages, int32_t* status, void* stream) {
  return run_chunk(ATTN_KIND_SLIDING, Chunk::kFp8, qkv, w_q, w_k, nullptr, block_table, seq_lens, cu_q, q_out, k_pool,
                   v_pool, k_scale, v_scale, batch, total_q, max_blocks, num_pages, status, stream);
}

int32_t attn_kv_append_global_fp8(const void* qkv, const void* w_q, const void* w_k, const int32_t* block_table,
                                  const int32_t* seq_lens, const int32_t* cu_q, void* q_out, void* k_pool, void* v_pool,
                                  uint8_t* k_scale, uint8_t* v_scale, int32_t batch, int32_t total_q,
                                  int32_t max_blocks, int64_t num_pages, int32_t* status, void* stream) {
  return run_chunk(ATTN_KIND_GLOBAL, Chunk::kFp8, qkv, w_q, w_k, nullptr, block_table, seq_lens, cu_q, q_out, k_pool,
                   v_pool, k_scale, v_scale, batch, total_q, max_blocks, num_pages, status, stream);
}

int32_t attn_kv_read_sliding_fp8(const void* k_pool, const void* v_pool, const uint8_t* k_scale, const uint8_t* v_scale,
                                 const int32_t* block_table, const int32_t* seq_lens, void* k_out, void* v_out,
                                 const int32_t* out_table, int32_t batch, int32_t max_blocks, int64_t num_pages,
                                 int64_t out_pages, int32_t max_seq_len, int32_t span, int32_t* status, void* stream) {
  return run_read(ATTN_KIND_SLIDING, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, k_out, v_out, out_table,
                  batch, max_blocks, num_pages, out_pages, max_seq_len, span, status, stream);
}

int32_t attn_kv_read_global_fp8(const void* k_pool, const void* v_pool, const uint8_t* k_scale, const uint8_t* v_scale,
                                const int32_t* block_table, const int32_t* seq_lens, void* k_out, void* v_out,
                                const int32_t* out_table, int32_t batch, int32_t max_blocks, int64_t num_pages,
                                int64_t out_pages, int32_t max_seq_len, int32_t span, int32_t* status, void* stream) {
  return run_read(ATTN_KIND_GLOBAL, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, k_out, v_out, out_table,
                  batch, max_blocks, num_pages, out_pages, max_seq_len, span, status, stream);
}

int32_t attn_decode_sliding_fp8(const void* q, const void* k_pool, const void* v_pool, const uint8_t* k_scale,
                                const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens, void* o,
                                int32_t batch, int32_t max_blocks, int64_t num_pages, int32_t max_seq_len,
                                int32_t window, int32_t out_dtype, int32_t num_splits, void* workspace,
                                size_t workspace_bytes, int32_t* status, void* stream) {
  return run_decode_fp8(ATTN_KIND_SLIDING, q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, o, batch,
                        max_blocks, num_pages, max_seq_len, window, out_dtype, num_splits, workspace, workspace_bytes,
                        status, stream);
}

int32_t attn_decode_global_fp8(const void* q, const void* k_pool, const void* v_pool, const uint8_t* k_scale,
                               const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens, void* o,
                               int32_t batch, int32_t max_blocks, int64_t num_pages, int32_t max_seq_len,
                               int32_t window, int32_t out_dtype, int32_t num_splits, void* workspace,
                               size_t workspace_bytes, int32_t* status, void* stream) {
  return run_decode_fp8(ATTN_KIND_GLOBAL, q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, o, batch,
                        max_blocks, num_pages, max_seq_len, window, out_dtype, num_splits, workspace, workspace_bytes,
                        status, stream);
}

}  // extern "C"
