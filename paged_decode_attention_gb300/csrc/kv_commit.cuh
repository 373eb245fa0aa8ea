// kv_commit.cuh -- the accepted path's cache rows moved to the front of their
// sequence's nodes, in every layer of a type (attn_kv_commit_*): slot ctx +
// path[j] to slot ctx + j.
//
// A path increases, so path[j] >= j, and every row that is written, at j, lies in
// front of every row still to be read, at path[j'] > path[j] >= j.  A block takes one
// sequence in one layer, each thread 16 bytes of the row of both pools for all j in
// order, kInFlight rows read before they are written; no row is read by one thread and
// written by another.  Bound by memory where paths and batches are long (two passes over a
// row's bytes): 64 sequences in 40 sliding layers, 92 MB, 18.3 us, 0.74 of the copy rate (12.6
// with the rows in L2); a block for one pool or for two layers took 18.9 and 19.7.  One
// sequence in 8 global layers 5.0: the chain of lengths, path, table, row.
#pragma once

#include "attn_tree.h"
#include "common.cuh"

namespace pda {
namespace commit {

constexpr int kInFlight = 4;  // rows of each pool (in L2: 2 12.9 us, 8 16.7 instead of 12.6)

struct CommitParams {
  uint8_t* pool[2 * ATTN_MAX_LAYERS];  // k and v of every layer
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  const int32_t* path;
  const int32_t* path_len;
  int32_t* new_lens;
  int32_t* status;
  int64_t num_pages;
  int32_t max_path;
  int32_t max_blocks;
};

// kRow bytes of a row, kRow / 16 threads.
template <int kRow>
__global__ void __launch_bounds__(kRow / 16) commit_kernel(const __grid_constant__ CommitParams p) {
  __shared__ int32_t s_src[ATTN_MAX_TREE], s_dst[ATTN_MAX_TREE];  // pool rows; src < 0: left alone
  __shared__ int32_t s_count;
  const int b = blockIdx.x;
  const int tid = threadIdx.x;
  wait_for_primary_grid();
  allow_dependent_launch();
  if (tid < 32) {
    const int n = p.cu_q[b + 1] - p.cu_q[b];
    const int L = p.seq_lens[b];
    const int cap = p.max_blocks < ATTN_MAX_SEQ_LEN / kPage ? p.max_blocks * kPage : ATTN_MAX_SEQ_LEN;
    const bool reporter = tid == 0 && blockIdx.y == 0;
    int count = 0;
    if (n < 0 || L < n || L > cap) {
      if (reporter) report(p.status, ATTN_DEV_BAD_SEQ_LEN);
    } else {
      const int ctx = L - n;
      count = p.path_len[b];
      bool bad = count < 0 || count > p.max_path || count > n;
      if (!bad) {
        const int32_t* path = p.path + static_cast<int64_t>(b) * p.max_path;
        for (int j = tid; j < count; j += 32) {
          const int at = path[j];
          bad |= at < 0 || at >= n || (j > 0 && at <= path[j - 1]);
          s_src[j] = at;
        }
        bad = __any_sync(0xffffffffu, bad);
      }
      if (bad) {
        if (reporter) report(p.status, ATTN_DEV_BAD_TREE);
        count = 0;
      }
      const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
      for (int j = tid; j < count; j += 32) {
        const int src = ctx + s_src[j], dst = ctx + j;
        const int sp = table[src / kPage], dp = table[dst / kPage];
        const bool ok = sp >= 0 && sp < p.num_pages && dp >= 0 && dp < p.num_pages;
        if (!ok && src != dst && blockIdx.y == 0) report(p.status, ATTN_DEV_BAD_PAGE);
        s_src[j] = ok && src != dst ? sp * kPage + src % kPage : -1;
        s_dst[j] = dp * kPage + dst % kPage;
      }
      if (reporter) p.new_lens[b] = ctx + count;
    }
    if (tid == 0) s_count = count;
  }
  __syncthreads();
  const int count = s_count;
  uint8_t* const k = p.pool[2 * blockIdx.y] + 16 * tid;
  uint8_t* const v = p.pool[2 * blockIdx.y + 1] + 16 * tid;
  for (int j0 = 0; j0 < count; j0 += kInFlight) {
    uint4 x[kInFlight], y[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int j = j0 + u;
      if (j < count && s_src[j] >= 0) {
        x[u] = *reinterpret_cast<const uint4*>(k + static_cast<int64_t>(s_src[j]) * kRow);
        y[u] = *reinterpret_cast<const uint4*>(v + static_cast<int64_t>(s_src[j]) * kRow);
      }
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int j = j0 + u;
      if (j < count && s_src[j] >= 0) {
        *reinterpret_cast<uint4*>(k + static_cast<int64_t>(s_dst[j]) * kRow) = x[u];
        *reinterpret_cast<uint4*>(v + static_cast<int64_t>(s_dst[j]) * kRow) = y[u];
      }
    }
  }
}

}  // namespace commit
}  // namespace pda
