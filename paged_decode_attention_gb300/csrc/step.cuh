// step.cuh -- host side of include/attn_step.h: the attention calls of a
// decode step recorded once and replayed with one call, either as one CUDA
// graph or as the recorded kernel launches enqueued back to back.  Included
// at the end of attn_decode.cu, whose validation (g_validate_only), launch
// recording (g_record) and error reporting it shares.
#pragma once

#include <array>
#include <functional>
#include <new>
#include <utility>
#include <vector>

#include "attn_step.h"

struct attn_step {
  std::vector<std::function<int32_t(void*)>> calls;  // each enqueues one call on the given stream
  int32_t kernels = 0;
  int32_t mode = ATTN_STEP_LAUNCH_AUTO;  // as requested; resolved by attn_step_finalize
  bool finalized = false;
  int device = -1;                       // the device the step was finalized on
  std::vector<RecordedLaunch> launches;  // every kernel launch of the step, arguments bound
  cudaGraph_t graph = nullptr;           // ATTN_STEP_LAUNCH_GRAPH only
  cudaGraphExec_t exec = nullptr;
};

namespace {

// Validates `call` (its launches suppressed) and, if it passes, appends it
// with the number of kernels it launches.
template <typename Call>
int32_t record(attn_step* step, const Call& call, const char* name) {
  g_err[0] = '\0';
  if (!step) return fail(ATTN_ERR_INVALID_ARG, "%s: null step", name);
  if (step->finalized) return fail(ATTN_ERR_INVALID_ARG, "%s: the step is already finalized", name);
  g_validate_only = true;
  g_last_launches = 0;
  const int32_t st = call(nullptr);
  g_validate_only = false;
  if (st != ATTN_OK) return st;
  const int32_t kernels = g_last_launches;
  try {
    step->calls.emplace_back(call);  // the std::function is made here, so that its allocation is caught too
  } catch (...) {  // no exception may leave the C ABI
    return fail(ATTN_ERR_INVALID_ARG, "%s: out of host memory", name);
  }
  step->kernels += kernels;
  return ATTN_OK;
}

// The same for a commit, whose pool pointers are kept with the step.
template <typename Call>
int32_t record_commit(attn_step* step, const void* const* k_pools, const void* const* v_pools, int32_t layers,
                      const Call& call, const char* name) {
  g_err[0] = '\0';
  using Pools = std::array<const void*, ATTN_MAX_LAYERS>;
  if (!k_pools || !v_pools) return fail(ATTN_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (!aligned_to(k_pools, alignof(void*)) || !aligned_to(v_pools, alignof(void*)))
    return fail(ATTN_ERR_INVALID_ARG, "%s: misaligned pointer", name);
  Pools k{}, v{};
  for (int i = 0; i < layers && i < ATTN_MAX_LAYERS; ++i) {  // (the call refuses other numbers of layers)
    k[i] = k_pools[i];
    v[i] = v_pools[i];
  }
  return record(step, [=](void* s) { return call(k, v, s); }, name);
}

}  // namespace

extern "C" {

int32_t attn_step_create(attn_step** out) {
  g_err[0] = '\0';
  if (!out) return fail(ATTN_ERR_INVALID_ARG, "attn_step_create: null out");
  *out = new (std::nothrow) attn_step();
  if (!*out) return fail(ATTN_ERR_INVALID_ARG, "attn_step_create: out of host memory");
  return ATTN_OK;
}

void attn_step_destroy(attn_step* step) {
  if (!step) return;
  if (step->exec) cudaGraphExecDestroy(step->exec);
  if (step->graph) cudaGraphDestroy(step->graph);
  delete step;
}

int32_t attn_step_add_decode_sliding(attn_step* step, const void* q, const void* k_pool, const void* v_pool,
                                     const int32_t* block_table, const int32_t* seq_lens, void* o, int32_t batch,
                                     int32_t max_blocks, int64_t num_pages, int32_t max_seq_len, int32_t window,
                                     int32_t out_dtype, int32_t num_splits, void* workspace, size_t workspace_bytes,
                                     int32_t* status) {
  return record(step, [=](void* s) {
    return attn_decode_sliding(q, k_pool, v_pool, block_table, seq_lens, o, batch, max_blocks, num_pages,
                               max_seq_len, window, out_dtype, num_splits, workspace, workspace_bytes, status, s);
  }, "attn_step_add_decode_sliding");
}

int32_t attn_step_add_decode_global(attn_step* step, const void* q, const void* k_pool, const void* v_pool,
                                    const int32_t* block_table, const int32_t* seq_lens, void* o, int32_t batch,
                                    int32_t max_blocks, int64_t num_pages, int32_t max_seq_len, int32_t window,
                                    int32_t out_dtype, int32_t num_splits, void* workspace, size_t workspace_bytes,
                                    int32_t* status) {
  return record(step, [=](void* s) {
    return attn_decode_global(q, k_pool, v_pool, block_table, seq_lens, o, batch, max_blocks, num_pages,
                              max_seq_len, window, out_dtype, num_splits, workspace, workspace_bytes, status, s);
  }, "attn_step_add_decode_global");
}

int32_t attn_step_add_decode_global_shared(attn_step* step, const void* q, const void* kv_pool, const void* w_k,
                                           const int32_t* block_table, const int32_t* seq_lens, void* o,
                                           int32_t batch, int32_t max_blocks, int64_t num_pages,
                                           int32_t max_seq_len, int32_t window, int32_t out_dtype,
                                           int32_t num_splits, void* workspace, size_t workspace_bytes,
                                           int32_t* status) {
  return record(step, [=](void* s) {
    return attn_decode_global_shared(q, kv_pool, w_k, block_table, seq_lens, o, batch, max_blocks, num_pages,
                                     max_seq_len, window, out_dtype, num_splits, workspace, workspace_bytes,
                                     status, s);
  }, "attn_step_add_decode_global_shared");
}

int32_t attn_step_add_kv_append_sliding(attn_step* step, const void* qkv, const void* w_q, const void* w_k,
                                        const int32_t* block_table, const int32_t* positions, void* q_out,
                                        void* k_pool, void* v_pool, int32_t batch, int32_t max_blocks,
                                        int64_t num_pages, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_kv_append_sliding(qkv, w_q, w_k, block_table, positions, q_out, k_pool, v_pool, batch, max_blocks,
                                  num_pages, status, s);
  }, "attn_step_add_kv_append_sliding");
}

int32_t attn_step_add_kv_append_global(attn_step* step, const void* qkv, const void* w_q, const void* w_k,
                                       const int32_t* block_table, const int32_t* positions, void* q_out,
                                       void* k_pool, void* v_pool, int32_t batch, int32_t max_blocks,
                                       int64_t num_pages, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_kv_append_global(qkv, w_q, w_k, block_table, positions, q_out, k_pool, v_pool, batch, max_blocks,
                                 num_pages, status, s);
  }, "attn_step_add_kv_append_global");
}

int32_t attn_step_add_kv_append_sliding_chunk(attn_step* step, const void* qkv, const void* w_q, const void* w_k,
    const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q, void* q_out, void* k_pool, void* v_pool,
    int32_t batch, int32_t total_q, int32_t max_blocks, int64_t num_pages, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_kv_append_sliding_chunk(qkv, w_q, w_k, block_table, seq_lens, cu_q, q_out, k_pool, v_pool, batch, total_q,
        max_blocks, num_pages, status, s);
  }, "attn_step_add_kv_append_sliding_chunk");
}

int32_t attn_step_add_kv_append_sliding_fp8(attn_step* step, const void* qkv, const void* w_q, const void* w_k,
    const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q, void* q_out, void* k_pool, void* v_pool,
    uint8_t* k_scale, uint8_t* v_scale, int32_t batch, int32_t total_q, int32_t max_blocks, int64_t num_pages, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_kv_append_sliding_fp8(qkv, w_q, w_k, block_table, seq_lens, cu_q, q_out, k_pool, v_pool, k_scale, v_scale, batch, total_q,
        max_blocks, num_pages, status, s);
  }, "attn_step_add_kv_append_sliding_fp8");
}

int32_t attn_step_add_decode_sliding_fp8(attn_step* step, const void* q, const void* k_pool, const void* v_pool,
    const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens, void* o,
    int32_t batch, int32_t max_blocks, int64_t num_pages, int32_t max_seq_len, int32_t window, int32_t out_dtype,
    int32_t num_splits, void* workspace, size_t workspace_bytes, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_decode_sliding_fp8(q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, o, batch, max_blocks,
        num_pages, max_seq_len, window, out_dtype, num_splits, workspace, workspace_bytes, status, s);
  }, "attn_step_add_decode_sliding_fp8");
}

int32_t attn_step_add_kv_append_global_chunk(attn_step* step, const void* qkv, const void* w_q, const void* w_k,
    const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q, void* q_out, void* k_pool, void* v_pool,
    int32_t batch, int32_t total_q, int32_t max_blocks, int64_t num_pages, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_kv_append_global_chunk(qkv, w_q, w_k, block_table, seq_lens, cu_q, q_out, k_pool, v_pool, batch, total_q,
        max_blocks, num_pages, status, s);
  }, "attn_step_add_kv_append_global_chunk");
}

int32_t attn_step_add_kv_append_global_prefix(attn_step* step, const void* qkv, const void* w_q, const void* w_k,
    const int32_t* prefix_len, const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q, void* q_out,
    void* k_pool, void* v_pool, int32_t batch, int32_t total_q, int32_t max_blocks, int64_t num_pages, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_kv_append_global_prefix(qkv, w_q, w_k, prefix_len, block_table, seq_lens, cu_q, q_out, k_pool, v_pool,
        batch, total_q, max_blocks, num_pages, status, s);
  }, "attn_step_add_kv_append_global_prefix");
}

int32_t attn_step_add_kv_append_global_fp8(attn_step* step, const void* qkv, const void* w_q, const void* w_k,
    const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q, void* q_out, void* k_pool, void* v_pool,
    uint8_t* k_scale, uint8_t* v_scale, int32_t batch, int32_t total_q, int32_t max_blocks, int64_t num_pages, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_kv_append_global_fp8(qkv, w_q, w_k, block_table, seq_lens, cu_q, q_out, k_pool, v_pool, k_scale, v_scale, batch, total_q,
        max_blocks, num_pages, status, s);
  }, "attn_step_add_kv_append_global_fp8");
}

int32_t attn_step_add_decode_global_fp8(attn_step* step, const void* q, const void* k_pool, const void* v_pool,
    const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens, void* o,
    int32_t batch, int32_t max_blocks, int64_t num_pages, int32_t max_seq_len, int32_t window, int32_t out_dtype,
    int32_t num_splits, void* workspace, size_t workspace_bytes, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_decode_global_fp8(q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, o, batch, max_blocks,
        num_pages, max_seq_len, window, out_dtype, num_splits, workspace, workspace_bytes, status, s);
  }, "attn_step_add_decode_global_fp8");
}

int32_t attn_step_add_kv_read_sliding_fp8(attn_step* step, const void* k_pool, const void* v_pool,
    const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens, void* k_out,
    void* v_out, const int32_t* out_table, int32_t batch, int32_t max_blocks, int64_t num_pages, int64_t out_pages,
    int32_t max_seq_len, int32_t span, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_kv_read_sliding_fp8(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, k_out, v_out, out_table, batch,
        max_blocks, num_pages, out_pages, max_seq_len, span, status, s);
  }, "attn_step_add_kv_read_sliding_fp8");
}

int32_t attn_step_add_kv_read_global_fp8(attn_step* step, const void* k_pool, const void* v_pool,
    const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens, void* k_out,
    void* v_out, const int32_t* out_table, int32_t batch, int32_t max_blocks, int64_t num_pages, int64_t out_pages,
    int32_t max_seq_len, int32_t span, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_kv_read_global_fp8(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, k_out, v_out, out_table, batch,
        max_blocks, num_pages, out_pages, max_seq_len, span, status, s);
  }, "attn_step_add_kv_read_global_fp8");
}

int32_t attn_step_add_decode_global_prefix(attn_step* step, const void* q, const void* k_pool, const void* v_pool,
    const int32_t* prefix_table, const int32_t* prefix_len, const int32_t* block_table, const int32_t* seq_lens,
    void* o, int32_t batch, int32_t prefix_blocks, int32_t max_blocks, int64_t num_pages, int32_t max_prefix_len,
    int32_t max_seq_len, int32_t out_dtype, int32_t num_splits, int32_t prefix_splits, void* workspace,
    size_t workspace_bytes, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_decode_global_prefix(q, k_pool, v_pool, prefix_table, prefix_len, block_table, seq_lens, o, batch,
        prefix_blocks, max_blocks, num_pages, max_prefix_len, max_seq_len, out_dtype, num_splits, prefix_splits,
        workspace, workspace_bytes, status, s);
  }, "attn_step_add_decode_global_prefix");
}

int32_t attn_step_add_decode_sliding_tree(attn_step* step, const void* q, const void* k_pool, const void* v_pool,
                                          const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q,
                                          const int32_t* parents, void* o, int32_t batch, int32_t total_q,
                                          int32_t max_q, int32_t max_blocks, int64_t num_pages, int32_t max_seq_len,
                                          int32_t window, int32_t out_dtype, int32_t num_splits, void* workspace,
                                          size_t workspace_bytes, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_decode_sliding_tree(q, k_pool, v_pool, block_table, seq_lens, cu_q, parents, o, batch, total_q,
                                    max_q, max_blocks, num_pages, max_seq_len, window, out_dtype, num_splits,
                                    workspace, workspace_bytes, status, s);
  }, "attn_step_add_decode_sliding_tree");
}

int32_t attn_step_add_decode_global_tree(attn_step* step, const void* q, const void* k_pool, const void* v_pool,
                                         const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q,
                                         const int32_t* parents, void* o, int32_t batch, int32_t total_q,
                                         int32_t max_q, int32_t max_blocks, int64_t num_pages, int32_t max_seq_len,
                                         int32_t window, int32_t out_dtype, int32_t num_splits, void* workspace,
                                         size_t workspace_bytes, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_decode_global_tree(q, k_pool, v_pool, block_table, seq_lens, cu_q, parents, o, batch, total_q, max_q,
                                   max_blocks, num_pages, max_seq_len, window, out_dtype, num_splits, workspace,
                                   workspace_bytes, status, s);
  }, "attn_step_add_decode_global_tree");
}

int32_t attn_step_add_kv_append_sliding_tree(attn_step* step, const void* qkv, const void* w_q, const void* w_k,
                                             const int32_t* block_table, const int32_t* seq_lens,
                                             const int32_t* cu_q, const int32_t* parents, void* q_out, void* k_pool,
                                             void* v_pool, int32_t batch, int32_t total_q, int32_t max_blocks,
                                             int64_t num_pages, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_kv_append_sliding_tree(qkv, w_q, w_k, block_table, seq_lens, cu_q, parents, q_out, k_pool, v_pool,
                                       batch, total_q, max_blocks, num_pages, status, s);
  }, "attn_step_add_kv_append_sliding_tree");
}

int32_t attn_step_add_kv_append_global_tree(attn_step* step, const void* qkv, const void* w_q, const void* w_k,
                                            const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_q,
                                            const int32_t* parents, void* q_out, void* k_pool, void* v_pool,
                                            int32_t batch, int32_t total_q, int32_t max_blocks, int64_t num_pages,
                                            int32_t* status) {
  return record(step, [=](void* s) {
    return attn_kv_append_global_tree(qkv, w_q, w_k, block_table, seq_lens, cu_q, parents, q_out, k_pool, v_pool,
                                      batch, total_q, max_blocks, num_pages, status, s);
  }, "attn_step_add_kv_append_global_tree");
}

int32_t attn_step_add_kv_commit_sliding(attn_step* step, const void* const* k_pools, const void* const* v_pools,
                                        int32_t layers, const int32_t* block_table, const int32_t* seq_lens,
                                        const int32_t* cu_q, const int32_t* path, const int32_t* path_len,
                                        int32_t* new_lens, int32_t batch, int32_t max_path, int32_t max_blocks,
                                        int64_t num_pages, int32_t* status) {
  return record_commit(step, k_pools, v_pools, layers, [=](const auto& k, const auto& v, void* s) {
    return attn_kv_commit_sliding(k.data(), v.data(), layers, block_table, seq_lens, cu_q, path, path_len, new_lens,
                                  batch, max_path, max_blocks, num_pages, status, s);
  }, "attn_step_add_kv_commit_sliding");
}

int32_t attn_step_add_kv_commit_global(attn_step* step, const void* const* k_pools, const void* const* v_pools,
                                       int32_t layers, const int32_t* block_table, const int32_t* seq_lens,
                                       const int32_t* cu_q, const int32_t* path, const int32_t* path_len,
                                       int32_t* new_lens, int32_t batch, int32_t max_path, int32_t max_blocks,
                                       int64_t num_pages, int32_t* status) {
  return record_commit(step, k_pools, v_pools, layers, [=](const auto& k, const auto& v, void* s) {
    return attn_kv_commit_global(k.data(), v.data(), layers, block_table, seq_lens, cu_q, path, path_len, new_lens,
                                 batch, max_path, max_blocks, num_pages, status, s);
  }, "attn_step_add_kv_commit_global");
}

int32_t attn_step_add_pages_assign(attn_step* step, const int32_t* cached_lens, const int32_t* new_tokens,
                                   int32_t* block_table, const int32_t* held, int32_t* free_list,
                                   const int32_t* free_state, int32_t* held_out, int32_t* free_state_out,
                                   int32_t* seq_lens, int32_t* cu_q, int32_t batch, int32_t max_blocks,
                                   int64_t num_pages, int32_t window, int32_t* status) {
  return record(step, [=](void* s) {
    return attn_pages_assign(cached_lens, new_tokens, block_table, held, free_list, free_state, held_out,
                             free_state_out, seq_lens, cu_q, batch, max_blocks, num_pages, window, status, s);
  }, "attn_step_add_pages_assign");
}

int32_t attn_step_num_calls(const attn_step* step) { return step ? static_cast<int32_t>(step->calls.size()) : 0; }

int32_t attn_step_num_kernels(const attn_step* step) { return step ? step->kernels : 0; }

int32_t attn_step_set_launch_mode(attn_step* step, int32_t mode) {
  g_err[0] = '\0';
  const char* name = "attn_step_set_launch_mode";
  if (!step) return fail(ATTN_ERR_INVALID_ARG, "%s: null step", name);
  if (step->finalized) return fail(ATTN_ERR_INVALID_ARG, "%s: the step is already finalized", name);
  if (mode != ATTN_STEP_LAUNCH_AUTO && mode != ATTN_STEP_LAUNCH_GRAPH && mode != ATTN_STEP_LAUNCH_DIRECT)
    return fail(ATTN_ERR_INVALID_ARG, "%s: unknown mode %d", name, mode);
  step->mode = mode;
  return ATTN_OK;
}

int32_t attn_step_launch_mode(const attn_step* step) { return step ? step->mode : -1; }

int32_t attn_step_finalize(attn_step* step) {
  g_err[0] = '\0';
  const char* name = "attn_step_finalize";
  if (!step) return fail(ATTN_ERR_INVALID_ARG, "%s: null step", name);
  if (step->finalized) return fail(ATTN_ERR_INVALID_ARG, "%s: already finalized", name);
  if (step->calls.empty()) return fail(ATTN_ERR_INVALID_ARG, "%s: no calls recorded", name);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(ATTN_ERR_CUDA, "%s: cudaGetDevice: %s", name, cudaGetErrorString(e));

  // Run every call once more with its launches recorded instead of enqueued:
  // host validation, tensor maps and kernel attributes are done here, once.
  std::vector<RecordedLaunch> launches;
  int32_t st = ATTN_OK;
  g_record = &launches;
  for (size_t i = 0; i < step->calls.size() && st == ATTN_OK; ++i) st = step->calls[i](nullptr);
  g_record = nullptr;
  if (st != ATTN_OK) return st;
  if (launches.size() != static_cast<size_t>(step->kernels))
    return fail(ATTN_ERR_INVALID_ARG, "%s: recorded %zu launches for %d kernels", name, launches.size(),
                step->kernels);

  int32_t mode = step->mode;
  if (mode == ATTN_STEP_LAUNCH_AUTO)
    mode = step->kernels <= ATTN_STEP_DIRECT_MAX_KERNELS ? ATTN_STEP_LAUNCH_DIRECT : ATTN_STEP_LAUNCH_GRAPH;
  cudaGraph_t graph = nullptr;
  cudaGraphExec_t exec = nullptr;
  if (mode == ATTN_STEP_LAUNCH_GRAPH) {
    cudaStream_t cs = nullptr;
    e = cudaStreamCreateWithFlags(&cs, cudaStreamNonBlocking);
    if (e != cudaSuccess) return fail(ATTN_ERR_CUDA, "%s: cudaStreamCreate: %s", name, cudaGetErrorString(e));
    e = cudaStreamBeginCapture(cs, cudaStreamCaptureModeRelaxed);
    if (e != cudaSuccess) {
      cudaStreamDestroy(cs);
      return fail(ATTN_ERR_CUDA, "%s: cudaStreamBeginCapture: %s", name, cudaGetErrorString(e));
    }
    // The kernels keep their programmatic-serialisation attribute, so the
    // graph holds programmatic edges between consecutive kernels.
    for (size_t i = 0; i < launches.size() && st == ATTN_OK; ++i) {
      const cudaError_t le = launches[i](cs);
      if (le != cudaSuccess) st = fail(ATTN_ERR_CUDA, "%s: launch %zu: %s", name, i, cudaGetErrorString(le));
    }
    e = cudaStreamEndCapture(cs, &graph);
    if (st == ATTN_OK && e != cudaSuccess)
      st = fail(ATTN_ERR_CUDA, "%s: cudaStreamEndCapture: %s", name, cudaGetErrorString(e));
    if (st == ATTN_OK) {
      e = cudaGraphInstantiate(&exec, graph, 0);
      if (e != cudaSuccess) st = fail(ATTN_ERR_CUDA, "%s: cudaGraphInstantiate: %s", name, cudaGetErrorString(e));
    }
    cudaStreamDestroy(cs);
    if (st != ATTN_OK) {
      if (graph) cudaGraphDestroy(graph);
      cudaGetLastError();  // a failed capture leaves no sticky error; clear the non-sticky one
      return st;
    }
  }
  step->launches = std::move(launches);
  step->graph = graph;
  step->exec = exec;
  step->mode = mode;
  step->device = dev;
  step->finalized = true;
  return ATTN_OK;
}

int32_t attn_step_launch(attn_step* step, void* stream) {
  g_err[0] = '\0';
  if (!step) return fail(ATTN_ERR_INVALID_ARG, "attn_step_launch: null step");
  if (!step->finalized) return fail(ATTN_ERR_INVALID_ARG, "attn_step_launch: the step is not finalized");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (step->exec) {
    const cudaError_t e = cudaGraphLaunch(step->exec, s);
    if (e != cudaSuccess) return fail(ATTN_ERR_CUDA, "attn_step_launch: %s", cudaGetErrorString(e));
    return ATTN_OK;
  }
  // Direct mode: the recorded launches, back to back, on the step's device.
  int cur = 0;
  cudaError_t e = cudaGetDevice(&cur);
  if (e == cudaSuccess && cur != step->device) e = cudaSetDevice(step->device);
  for (size_t i = 0; i < step->launches.size() && e == cudaSuccess; ++i) e = step->launches[i](s);
  if (cur != step->device) cudaSetDevice(cur);
  if (e != cudaSuccess) return fail(ATTN_ERR_CUDA, "attn_step_launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

}  // extern "C"
