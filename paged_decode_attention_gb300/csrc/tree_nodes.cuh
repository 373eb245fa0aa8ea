// tree_nodes.cuh -- the tree of a sequence's drafted tokens (include/attn_tree.h)
// in the registers of one warp: lane l holds nodes l and l + 32.
//
// Ancestors by pointer doubling: after k rounds a node knows its nearest 2^k - 1
// ancestors and jumps to the next one beyond, so a tree of depth d takes
// log2(d) + 1 rounds of a few shuffles, where walking up would take d dependent
// loads.
#pragma once

#include "attn_tree.h"
#include "common.cuh"

namespace pda {
namespace tree {

static_assert(ATTN_MAX_TREE == 64, "two nodes per lane, one 64-bit word of ancestors");

// The value that node `i`'s lane holds for it.
template <typename T>
__device__ __forceinline__ T of_node(const T (&v)[2], int i) {
  const T a = __shfl_sync(0xffffffffu, v[0], i & 31);
  const T b = __shfl_sync(0xffffffffu, v[1], i & 31);
  return i & 32 ? b : a;
}

// The parents of n <= ATTN_MAX_TREE nodes, as they are ...
__device__ __forceinline__ void read_parents(const int32_t* parents, int n, int (&parent)[2]) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = (threadIdx.x & 31) + 32 * u;
    parent[u] = i < n ? parents[i] : -1;
  }
}
// ... and those outside [-1, i) made -1.  Returns whether there was one (the same in every lane).
__device__ __forceinline__ bool check_parents(int n, int (&parent)[2]) {
  bool bad = false;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = (threadIdx.x & 31) + 32 * u;
    if (parent[u] < -1 || parent[u] >= i) {
      bad |= i < n;
      parent[u] = -1;
    }
  }
  return __any_sync(0xffffffffu, bad);
}

// Ancestors of every node, itself included, as bits: one more than its depth.
__device__ __forceinline__ void ancestors(const int (&parent)[2], unsigned long long (&mask)[2]) {
  int jump[2] = {parent[0], parent[1]};
#pragma unroll
  for (int u = 0; u < 2; ++u) mask[u] = 1ull << ((threadIdx.x & 31) + 32 * u);
#pragma unroll 1
  while (__any_sync(0xffffffffu, jump[0] >= 0 || jump[1] >= 0)) {
    unsigned long long m[2];
    int up[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      m[u] = of_node(mask, jump[u]);
      up[u] = of_node(jump, jump[u]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (jump[u] < 0) continue;
      mask[u] |= m[u];
      jump[u] = up[u];
    }
  }
}

// The same for at most 32 nodes, one a lane.
__device__ __forceinline__ uint32_t ancestors32(int parent) {
  const int lane = threadIdx.x & 31;
  uint32_t mask = 1u << lane;
  int jump = parent;
#pragma unroll 1
  while (__any_sync(0xffffffffu, jump >= 0)) {
    const uint32_t m = __shfl_sync(0xffffffffu, mask, jump & 31);
    const int up = __shfl_sync(0xffffffffu, jump, jump & 31);
    if (jump >= 0) {
      mask |= m;
      jump = up;
    }
  }
  return mask;
}

// Depth of node i of n.
__device__ __forceinline__ int depth_of(int n, const int (&parent)[2], int i) {
  if (n <= 32) return __popc(__shfl_sync(0xffffffffu, ancestors32(parent[0]), i)) - 1;
  unsigned long long mask[2];
  ancestors(parent, mask);
  return __popcll(of_node(mask, i)) - 1;
}

}  // namespace tree
}  // namespace pda
