// tree_decode.cuh -- attention of a tree of drafted tokens per sequence over the
// paged cache (attn_decode_*_tree) on the 5th-generation tensor cores.
//
// Node i of a sequence of n nodes behind ctx cached positions sees position l < ctx
// and the slots ctx + j of its ancestors and itself, within the window where there is
// one (include/attn_tree.h).  A node brings 16 query heads, so a tree is n * G rows
// over each KV head: 16 to 1024, where a tensor-core tile has 128.  The products are
// therefore turned round, keys and dims in the tile's 128 rows, query rows in its
// columns, of which any multiple of 16 will do:
//   S^T = K Q^T     M = 128 keys (eight pages), N = rows, K = D: A = the step's K, one
//                   64-dim chunk [128 keys][128 B] after another, B = Q; one key per
//                   tensor-memory lane;
//   P^T = softmax   a thread per key (two warpgroups, half of the columns each):
//                   masks, weights to bf16 in shared memory, [64 rows][keys] atoms;
//   O^T += V^T P^T  M = 128 dims (D / 128 tiles), N = rows, K = 16 keys: A = a page of V as
//                   it was copied, dims contiguous, B = P^T; one dim per lane.
// So all D dims of the output fit tensor memory at 64 rows (D = 512) or 128 (D =
// 256): no logit is computed twice, and a chain of few tokens costs few columns.
//
// Running max.  A row's (column's) reference max m is shared by all keys of a step.
// It moves only when a score exceeds it by more than kSlack, and then to kHeadroom
// above (prefill_tc.cuh has the bounds); a thread compares its own scores with the
// bounds, and one barrier with an OR tells whether any row moves.  So in nearly all
// steps nothing is reduced across lanes: each thread sums the weights of its own keys,
// and the 128 sums per row meet once, at the end of a segment.  A first step whose
// keys all nodes see takes one key's scores for the first references, which the same
// bounds then correct.
//
// Schedule.  Rows come in groups of kQueries nodes; kCluster groups of KV head c of
// all sequences that have them are a list of pages, with kSegWeight virtual pages in
// front of every sequence (its Q, its end).  All lists are cut into runs of `per`
// pages, the fewest that give no more runs than clusters: every cluster has the same
// work whatever the lengths, and those of neighbouring lists walk the same keys at the
// same time.  A sequence inside one run is finished there; of a cut one every block
// leaves a partial (O, m, sum), and merge_kernel joins them.
//
// Clusters.  On global layers a tree of more than four nodes has several groups, and
// every group reads all keys.  Two CTAs walk a run together, a group each: each copies
// half of the pages of K and V into both (multicast), so that L2 is read once for both;
// a stage is free again when both have used it.
//
// What a node does not see.  Scores are masked, and rows of V that no node sees are
// zeroed in shared memory.  A row that some nodes see and others do not (a node of the
// tree, the window's edge) may hold an infinity or NaN, and 0 * inf would reach the
// others: such elements are zeroed too, and the epilogue adds them to the rows that do
// see them.
//
// Roles: warps 0-7 softmax and epilogue, 8 copies Q and K, 9 copies V, 10 issues S^T,
// 11 issues O^T.  Every wait is bounded.
#pragma once

#include "attn_tree.h"
#include "common.cuh"
#include "prefill_tc.cuh"
#include "tcgen05.cuh"
#include "tree_nodes.cuh"

namespace pda {
namespace tree {

constexpr int kKeys = 128;                  // per step
constexpr int kStepPages = kKeys / kPage;
constexpr int kMaxGroups = 16;              // of rows, per KV head
constexpr int kSegWeight = 4;               // virtual pages charged per sequence
constexpr int kMinPer = 4;                  // pages of the smallest run
constexpr int kSoftmaxThreads = 256;
constexpr int kThreads = 384;
constexpr int kMaxGrid = kMaxSplits;

struct TreeParams {
  const __nv_bfloat16* v_pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  const int32_t* parents;
  void* o;
  float* part_o;    // [2 grid][kN][D]: a block's first segment, and its last
  float2* part_ml;  // [2 grid][kN]: (reference max in log2 units, sum)
  int4* cuts;       // [grid]: the sequence that is cut first in this block: first node, (nodes, KV head), first
                    // partial, partials; 0 partials: none
  int32_t* status;
  int64_t num_pages;
  int32_t batch;
  int32_t max_blocks;
  int32_t window;
  int32_t total_q;
  int32_t max_q;
  int32_t lists;    // per KV head: ceil(max_q / (kQueries * kCluster))
  int32_t q_box;    // nodes that a copy of Q brings
  int32_t out_f32;
  int32_t whole;    // a block per (sequence, group, KV head) instead of runs
};

template <int kD_, int kG_, int kHkv_, int kN_, int kPBufs_, int kKStages_, int kVStages_, int kCluster_ = 1>
struct Config {
  static constexpr int kCluster = kCluster_;   // CTAs that share their copies of K and V
  static constexpr int kD = kD_, kG = kG_, kHkv = kHkv_, kHq = kG * kHkv;
  static constexpr int kN = kN_;               // rows per group, at most
  static constexpr int kHalf = kN / 2;         // columns per softmax warpgroup
  static constexpr int kBlock = kHalf < 32 ? kHalf : 32;  // columns at a time
  static constexpr int kQueries = kN / kG;
  static constexpr int kChunks = kD / 64;
  static constexpr int kTiles = kD / 128;      // of 128 output dims
  static constexpr int kPBufs = kPBufs_;
  static constexpr int kKStages = kKStages_;   // K chunks
  static constexpr int kVStages = kVStages_;   // V pages
  static constexpr int kKChunk = kKeys * 128;  // bytes: [128 keys][64 dims]
  static constexpr int kVPage = kPage * kD * 2;
  static constexpr int kPChunk = kKeys * 128;  // P^T of 64 rows
  static constexpr int kPBytes = (kN + 63) / 64 * kPChunk;
  static constexpr uint32_t kSCol = kTiles * kN;  // O^T first, then two S^T buffers
  static constexpr uint32_t kUsedCols = kSCol + 2 * kN;
  static constexpr uint32_t kTmemCols = kUsedCols <= 128 ? 128 : kUsedCols <= 256 ? 256 : 512;
  static_assert(kUsedCols <= 512 && kN % 16 == 0 && kN <= 256, "tensor memory");
  static_assert(kBlock == 16 || kBlock == 32, "column reductions");
  static_assert(kCluster == 1 || kCluster == 2, "pages by rank");

  struct Smem {
    alignas(1024) uint8_t q[kChunks][kN * 128];
    alignas(1024) uint8_t p[kPBufs][kPBytes];
    alignas(1024) uint8_t k[kKStages][kKChunk];
    alignas(1024) uint8_t v[kVStages][kVPage];
    alignas(16) float neg_m[kN];      // minus the reference max (log2 units), 0 before there is one
    alignas(16) float bound[kN];      // a score above this moves it; -inf before there is one
    alignas(16) float f[kN];          // factor of a moved reference; 1 / sum at the end
    alignas(16) float red[8][kN / 2]; // per softmax warp and column: max, sum
    alignas(8) unsigned long long below[ATTN_MAX_TREE];    // nodes that see node j by ancestry
    alignas(8) unsigned long long shallow[ATTN_MAX_TREE];  // nodes of depth <= x
    int32_t depth[ATTN_MAX_TREE];
    int32_t pre[kMaxBatch + 1];       // pages (virtual ones included) before sequence b in this block's list
    int32_t cu_q[kMaxBatch + 1], len[kMaxBatch];
    int32_t sched[4];                 // list, KV head, per, run
    int32_t refused;                  // the call as a whole
    int32_t poison;                   // this segment: an element was zeroed that some row sees
    alignas(8) uint64_t k_full[kKStages], k_empty[kKStages];
    alignas(8) uint64_t v_full[kVStages], v_empty[kVStages];
    alignas(8) uint64_t s_full[2], s_free[2];
    alignas(8) uint64_t p_full[kPBufs], p_empty[kPBufs];
    alignas(8) uint64_t q_ready, q_empty;
    alignas(8) uint64_t o_full, o_free;
    alignas(8) uint64_t mma_done;
    uint32_t tmem_base;
  };
  static constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "one CTA per SM within the 227 KB a CTA may have");
};

// One sequence as the schedule sees it.
struct Sequence {
  int q0, n, L, ctx, lo, page0, pages;  // pages 0: nothing to do
};

__device__ __forceinline__ Sequence make_sequence(const TreeParams& p, int q0, int q1, int L, bool& refused) {
  Sequence s{};
  s.q0 = q0;
  s.L = L;
  const int64_t n = static_cast<int64_t>(q1) - q0;
  const int cap = p.max_blocks < ATTN_MAX_SEQ_LEN / kPage ? p.max_blocks * kPage : ATTN_MAX_SEQ_LEN;
  refused = n < 0 || q0 < 0 || q1 > p.total_q || n > p.max_q || n > L || L > cap;
  if (refused || n == 0) return s;
  s.n = static_cast<int>(n);
  s.ctx = L - s.n;
  s.lo = p.window > 0 && s.ctx >= p.window ? s.ctx - p.window + 1 : 0;
  s.page0 = s.lo / kPage;
  s.pages = (L - 1) / kPage - s.page0 + 1;
  return s;
}

// Positions below are not seen by every node.
__device__ __forceinline__ int all_from(const Sequence& q, int window) {
  return window > 0 ? q.ctx + (q.n - 1) - window + 1 : 0;  // (a depth is at most n - 1)
}

// A part of one sequence's pages for one group of rows.
struct Segment {
  Sequence q;
  int b, row0, nodes, cols, N;  // first node of the group (packed), its nodes, rows, columns of the products
  int p0, p1, steps;            // pages, and steps of kStepPages
  bool whole;
  int slot;                     // of its partial
};

// Walks a block's segments; every role does it for itself, with the same result.
template <typename C>
struct Walk {
  int b, w0, w1, group, kv, index;
  template <typename S>
  __device__ __forceinline__ void start(const TreeParams& p, const S& s) {
    group = s.sched[0] * C::kCluster + static_cast<int>(blockIdx.x % C::kCluster);
    kv = s.sched[1];
    index = 0;
    const int per = s.sched[2], run = s.sched[3];
    if (p.whole) {
      b = run;
      w0 = s.pre[b];
      w1 = s.pre[b + 1];
      return;
    }
    const int total = s.pre[p.batch];
    const long long u0 = static_cast<long long>(run) * per;
    w0 = run < 0 || u0 >= total ? total : static_cast<int>(u0);
    w1 = total - w0 < per ? total : w0 + per;
    int lo = 0, hi = p.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.pre[mid] <= w0) lo = mid; else hi = mid - 1;
    }
    b = lo;
  }
  template <typename S>
  __device__ __forceinline__ bool next(const TreeParams& p, const S& s, Segment& g) {
    for (; b < p.batch && s.pre[b] < w1; ++b) {
      const int pages = s.pre[b + 1] - s.pre[b] - kSegWeight;
      if (pages <= 0) continue;
      const int first = s.pre[b] + kSegWeight;
      g.p0 = w0 > first ? w0 - first : 0;
      g.p1 = w1 - first < pages ? w1 - first : pages;
      if (g.p1 <= g.p0) continue;
      bool refused;
      g.q = make_sequence(p, s.cu_q[b], s.cu_q[b + 1], s.len[b], refused);
      g.b = b;
      g.row0 = g.q.q0 + group * C::kQueries;
      g.nodes = max(0, min(C::kQueries, g.q.n - group * C::kQueries));  // (0: only the cluster's other groups have any)
      g.cols = g.nodes * C::kG;
      g.N = max(16, (g.cols + 15) & ~15);
      g.steps = (g.p1 - g.p0 + kStepPages - 1) / kStepPages;
      g.whole = g.p0 == 0 && g.p1 == pages;
      g.slot = 2 * static_cast<int>(blockIdx.x) + (index > 0);
      ++index;
      ++b;
      return true;
    }
    return false;
  }
};

// Reduces kW values of every lane across the warp, column by column: lane l gets
// column l (kW = 32) or l / 2 (kW = 16).
template <int kW, typename Op>
__device__ __forceinline__ float reduce_columns(float (&v)[kW], Op op) {
  const int lane = threadIdx.x & 31;
  int off = 16;
#pragma unroll
  for (int w = kW / 2; w >= 1; w /= 2, off /= 2) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float send = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
    }
  }
  if constexpr (kW == 16) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
  return v[0];
}

// All columns of a softmax thread into its warp's row of `red`.
template <int kHalf, typename Op>
__device__ __forceinline__ void reduce_into(const float (&v)[kHalf], float* red, Op op) {
  const int lane = threadIdx.x & 31;
  if constexpr (kHalf == 16) {
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = v[i];
    const float r = reduce_columns<16>(t, op);
    red[lane >> 1] = r;  // (two lanes, one value)
  } else {
#pragma unroll
    for (int c0 = 0; c0 < kHalf; c0 += 32) {
      float t[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) t[i] = v[c0 + i];
      red[c0 + lane] = reduce_columns<32>(t, op);
    }
  }
}

__device__ __forceinline__ bool barrier_or(uint32_t id, uint32_t threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// The nodes (bits) that see position pos.  (The masks are there where a segment holds positions that not all nodes see.)
template <typename S>
__device__ __forceinline__ unsigned long long seen_by(const Sequence& q, int window, const S& s, int pos) {
  if (pos >= all_from(q, window) && pos < q.ctx) return ~0ull;
  if (pos < q.lo || pos >= q.L) return 0;
  if (pos < q.ctx) return s.shallow[min(pos - (q.ctx - window + 1), ATTN_MAX_TREE - 1)];
  const int j = pos - q.ctx;
  const unsigned long long m = s.below[j];
  return window > 0 && window < ATTN_MAX_TREE ? m & s.shallow[min(s.depth[j] + window - 1, ATTN_MAX_TREE - 1)] : m;
}

// bf16 pairs: nonzero where a half is an infinity or NaN (its exponent all ones).
__device__ __forceinline__ uint32_t nonfinite_bf16x2(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// A page of V as this lane sees it (16 bytes of every fourth chunk of a row): the rows in `none` zeroed, and every
// element of the rows in `some` that is not finite.  Returns whether there was one.  Eight rows are read before any is
// looked at: one after the other they would cost a shared-memory round trip each.
template <typename C>
__device__ __forceinline__ bool clean_page(uint32_t at, uint32_t none, uint32_t some) {
  bool found = false;
#pragma unroll 1
  for (int r0 = 0; r0 < kPage; r0 += 8) {
    if (((none | some) >> r0 & 0xffu) == 0) continue;
#pragma unroll
    for (int c0 = 0; c0 < C::kChunks; c0 += 4) {
      const uint32_t a = at + c0 * (kPage * 128) + r0 * 128;
      uint4 x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) x[r] = ld_shared_v4(a + r * 128);
      uint32_t bad = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const uint32_t any = nonfinite_bf16x2(x[r].x) | nonfinite_bf16x2(x[r].y) | nonfinite_bf16x2(x[r].z) |
                             nonfinite_bf16x2(x[r].w);
        bad |= (any != 0 ? 1u : 0u) << r;
        if (none >> (r0 + r) & 1) st_shared_v4(a + r * 128, make_uint4(0, 0, 0, 0));
      }
      bad &= some >> r0;
      if (bad == 0) continue;
      found = true;
#pragma unroll 1
      for (int r = 0; r < 8; ++r) {
        if (!(bad >> r & 1)) continue;
        const uint4 y = ld_shared_v4(a + r * 128);
        uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t z = nonfinite_bf16x2(w[e]);
          w[e] &= (z & 0x8000u ? 0u : 0xffffu) | (z & 0x80000000u ? 0u : 0xffff0000u);
        }
        st_shared_v4(a + r * 128, make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
  return found;
}

// Rows [from, to) of a page as bits, for positions relative to its first.
__device__ __forceinline__ uint32_t row_bits(int from, int to) {
  from = min(max(from, 0), kPage);
  to = min(max(to, from), kPage);
  return ((1u << to) - 1u) & ~((1u << from) - 1u);
}

// The schedule: this block's list, the running sums over it, its run.  Warp 0 works it out, 32 sequences a round, and
// the block waits for it once.  (Rounds are loops, not unrolled: what runs once a call is bound by fetching its
// instructions.)  Returns false when the call is refused.
template <typename C, typename S>
__device__ __forceinline__ bool make_schedule(const TreeParams& p, S& s) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    bool refused = false, backwards = false;
    int total = 0;  // lane r: the pages of list r (the same for every KV head)
    // (weight, lists) of sequence b
    const auto weigh = [&](int b, bool& bad) {
      const Sequence q = make_sequence(p, s.cu_q[b], s.cu_q[b + 1], s.len[b], bad);
      constexpr int kNodes = C::kQueries * C::kCluster;
      return q.pages > 0 ? make_int2(q.pages + kSegWeight, (q.n + kNodes - 1) / kNodes) : make_int2(0, 0);
    };
#pragma unroll 1
    for (int b0 = 0; b0 <= p.batch; b0 += 32) {
      const int b = b0 + lane;
      if (b <= p.batch) s.cu_q[b] = p.cu_q[b];
      if (b < p.batch) s.len[b] = p.seq_lens[b];
    }
    __syncwarp();
#pragma unroll 1
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      int2 w = make_int2(0, 0);
      if (b < p.batch) {
        bool bad;
        w = weigh(b, bad);
        refused |= bad;
        backwards |= s.cu_q[b + 1] < s.cu_q[b];
      }
#pragma unroll 1
      for (int r = 0; r < p.lists; ++r) {
        const int sum = __reduce_add_sync(0xffffffffu, w.y > r ? w.x : 0);
        if (lane == r) total += sum;
      }
    }
    refused = __any_sync(0xffffffffu, refused);
    backwards = __any_sync(0xffffffffu, backwards);  // sequences overlap
    if (refused && blockIdx.x == 0 && lane == 0) report(p.status, ATTN_DEV_BAD_SEQ_LEN);
    const int g = static_cast<int>(blockIdx.x / C::kCluster);
    int list, kv, per, run;
    if (p.whole) {
      const int per_seq = p.lists * C::kHkv;
      list = g % per_seq / C::kHkv;
      kv = g % C::kHkv;
      per = 1;
      run = g / per_seq;
    } else {
      const int grid = static_cast<int>(gridDim.x / C::kCluster);
      const int sum = __reduce_add_sync(0xffffffffu, total);
      int lo = max(kMinPer, (sum * C::kHkv + grid - 1) / grid);  // (at most 256 * 16388 pages * 8 heads a list)
      // (every list's last run may be short: with that many runs less there is room for all)
      const int lists = p.lists * C::kHkv;
      int hi = __reduce_max_sync(0xffffffffu, total);
      if (grid > lists) hi = min(hi, (sum * C::kHkv + grid - lists - 1) / (grid - lists));
      hi = max(lo, hi);
      const auto runs = [&](int n) { return __reduce_add_sync(0xffffffffu, (total + n - 1) / n) * C::kHkv; };
      if (runs(lo) <= grid) {
        hi = lo;
      } else {
        while (lo + 1 < hi) {  // runs(lo) > grid >= runs(hi)
          const int mid = (lo + hi) >> 1;
          if (runs(mid) <= grid) hi = mid; else lo = mid;
        }
      }
      per = hi;
      const int mine = (total + per - 1) / per * C::kHkv;  // this list's clusters
      int before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += u;
      }
      before -= mine;
      const unsigned here = __ballot_sync(0xffffffffu, mine > 0 && before <= g && g < before + mine);
      const int owner = here ? __ffs(here) - 1 : 0;
      before = __shfl_sync(0xffffffffu, before, owner);
      list = owner;
      kv = here ? (g - before) % C::kHkv : 0;
      run = here ? (g - before) / C::kHkv : -1;  // -1: the block has nothing to do
    }
    // the running sums of this block's list
    int carry = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      bool bad;
      const int2 w = b < p.batch ? weigh(b, bad) : make_int2(0, 0);
      int sum = w.y > list ? w.x : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (b < p.batch) s.pre[b + 1] = carry + sum;
      carry += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
      s.pre[0] = 0;
      s.sched[0] = list;
      s.sched[1] = kv;
      s.sched[2] = per;
      s.sched[3] = run;
      s.refused = backwards;
    }
  }
  __syncthreads();
  return s.refused == 0;
}

// Tells the merge which sequence is cut first in this block; run by one thread.
template <typename C, typename S>
__device__ __forceinline__ void note_cut(const TreeParams& p, const S& s) {
  Walk<C> walk;
  walk.start(p, s);
  Segment g;
  int4 cut = make_int4(0, 0, 0, 0);
  while (walk.next(p, s, g)) {
    if (g.p0 == 0 && !g.whole) {
      const int last = (s.pre[g.b] + kSegWeight + g.q.pages - 1) / s.sched[2];  // the run that holds its last page
      cut = make_int4(g.row0, g.nodes | (walk.kv << 8), g.slot, last - s.sched[3] + 1);
    }
  }
  p.cuts[blockIdx.x] = cut;
}

// Multicast copy of a 3-D tile into the same place of every CTA of the cluster in `mask`, completing on the same
// barrier of each.
__device__ __forceinline__ void tma_load_3d_multicast(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                                      uint64_t* bar, uint16_t mask) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.multicast::cluster"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)), "h"(mask)
      : "memory");
}

template <int kCluster>
__device__ __forceinline__ void load_page(void* dst, const CUtensorMap* map, int32_t y, int32_t z, uint64_t* bar) {
  if constexpr (kCluster == 1)
    prefill_tc::tma_load_3d(dst, map, 0, y, z, bar);
  else
    tma_load_3d_multicast(dst, map, 0, y, z, bar, static_cast<uint16_t>((1 << kCluster) - 1));
}

// Arrives on `bar` of every CTA of the cluster once the products this thread issued before are done.
template <int kCluster>
__device__ __forceinline__ void commit_all(uint64_t* bar) {
  if constexpr (kCluster == 1) {
    umma_commit_warp(bar);
  } else {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>((1 << kCluster) - 1))
        : "memory");
  }
}

template <int kCluster>
__device__ __forceinline__ bool wait_stage(uint64_t* bar, uint32_t parity) {  // a barrier that the whole cluster arrives on
  if constexpr (kCluster == 1) return mbar_wait_fast(bar, parity);
  return mbar_wait_cluster(bar, parity);
}

template <typename C>
__device__ __forceinline__ void tree_body(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                          const TreeParams& p) {
  using prefill_tc::kHeadroom;
  using prefill_tc::kSlack;
  using prefill_tc::tma_load_4d;
  constexpr int kD = C::kD, kG = C::kG, kN = C::kN, kHalf = C::kHalf, kTiles = C::kTiles, kBlock = C::kBlock;
  constexpr int kCluster = C::kCluster, kPBufs = C::kPBufs;
  extern __shared__ uint8_t smem_raw[];
  typename C::Smem& s =
      *reinterpret_cast<typename C::Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x % kCluster);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_empty[i], kCluster);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&s.v_full[i], 1);
      mbar_init(&s.v_empty[i], kCluster);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.s_free[i], 8);
    }
    for (int i = 0; i < kPBufs; ++i) {
      mbar_init(&s.p_full[i], 8);
      mbar_init(&s.p_empty[i], 1);
    }
    mbar_init(&s.q_ready, 1);
    mbar_init(&s.q_empty, 1);
    mbar_init(&s.o_full, 2);  // the last product's commit, and the issuer (poison)
    mbar_init(&s.o_free, 8);
    mbar_init(&s.mma_done, 2);
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tensor_map(&tm_q);
    prefetch_tensor_map(&tm_k);
    prefetch_tensor_map(&tm_v);
  }
  if (warp == 10) tmem_alloc(&s.tmem_base, C::kTmemCols);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s.tmem_base;

  // q, the cache and the tables may be written by the previous kernel in the stream.
  wait_for_primary_grid();
  allow_dependent_launch();
  const bool run = make_schedule<C>(p, s);
  if constexpr (kCluster > 1) cluster_sync_all();  // the other CTA's barriers are there
  if (!run) {
    if (threadIdx.x == 0 && !p.whole) p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
  } else if (warp == 8) {
    // ---------------- Q and K producer: lane i < 8 copies page i of a step, chunk by chunk ----------------
    bool ok = true;
    int gt = 0, gk = 0, st = 0, st_ph = 1;  // segments, K chunks; stage and its phase
    Walk<C> walk;
    walk.start(p, s);
    Segment g;
    while (ok && walk.next(p, s, g)) {
      if (gt >= 1) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.q_empty, (gt - 1) & 1));
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&s.q_ready, C::kChunks * p.q_box * kG * 128);
      __syncwarp();
      if (lane < C::kChunks) tma_load_4d(s.q[lane], &tm_q, 0, lane, walk.kv * kG, g.row0, &s.q_ready);
      ++gt;
      const int32_t* table = p.block_table + static_cast<int64_t>(g.b) * p.max_blocks + g.q.page0;
      const auto entry = [&](int pg) { return lane < kStepPages && pg + lane < g.p1 ? table[pg + lane] : 0; };
      int next_id = entry(g.p0);
      for (int pg = g.p0; pg < g.p1 && ok; pg += kStepPages) {
        const int id = next_id;
        next_id = entry(pg + kStepPages);
        const int np = min(kStepPages, g.p1 - pg);
        int32_t y = id * kPage;
        if (lane < np && (id < 0 || static_cast<int64_t>(id) >= p.num_pages)) {
          report(p.status, ATTN_DEV_BAD_PAGE);
          y = -kPage;
        }
        for (int ch = 0; ch < C::kChunks; ++ch) {
          if (gk >= C::kKStages) ok = __all_sync(0xffffffffu, wait_stage<kCluster>(&s.k_empty[st], st_ph));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&s.k_full[st], np * kPage * 128);
          __syncwarp();
          if (lane < np && lane % kCluster == rank)
            load_page<kCluster>(s.k[st] + lane * (kPage * 128), &tm_k, y, walk.kv * C::kChunks + ch, &s.k_full[st]);
          ++gk;
          if (++st == C::kKStages) st = 0, st_ph ^= 1;
          __syncwarp();
        }
      }
    }
    if (!ok && lane == 0) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
    if (lane == 0) {  // no copy may still be landing, nor a commit arriving, when the CTA retires
      if (gt >= 1) {
        if (!mbar_wait(&s.q_ready, (gt - 1) & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
        if (ok && !mbar_wait(&s.q_empty, (gt - 1) & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
      }
      for (int i = 0; i < C::kKStages && i < gk; ++i) {
        const int uses = (gk - 1 - i) / C::kKStages;
        if (!mbar_wait(&s.k_full[i], uses & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
        if (ok && !wait_stage<kCluster>(&s.k_empty[i], uses & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
      }
    }
  } else if (warp == 9) {
    // ---------------- V producer: a page per stage ----------------
    bool ok = true;
    int gv = 0, st = 0, st_ph = 1;
    Walk<C> walk;
    walk.start(p, s);
    Segment g;
    while (ok && walk.next(p, s, g)) {
      const int32_t* table = p.block_table + static_cast<int64_t>(g.b) * p.max_blocks + g.q.page0;
      const auto entry = [&](int pg) { return pg < g.p1 ? table[pg] : 0; };
      int cur = 0, nxt = entry(g.p0 + lane);
      for (int pg = g.p0; pg < g.p1 && ok; ++pg) {
        const int u = (pg - g.p0) & 31;
        if (u == 0) {
          cur = nxt;
          nxt = entry(pg + 32 + lane);
        }
        const int id = __shfl_sync(0xffffffffu, cur, u);
        if (gv >= C::kVStages) ok = __all_sync(0xffffffffu, wait_stage<kCluster>(&s.v_empty[st], st_ph));
        if (!ok) break;
        if (lane == 0) {
          const bool there = id >= 0 && static_cast<int64_t>(id) < p.num_pages;  // (the K producer reports)
          mbar_arrive_expect_tx(&s.v_full[st], C::kVPage);
          if (u % kCluster == rank)
            load_page<kCluster>(s.v[st], &tm_v, there ? id * kPage : -kPage, walk.kv * C::kChunks, &s.v_full[st]);
        }
        ++gv;
        if (++st == C::kVStages) st = 0, st_ph ^= 1;
        __syncwarp();
      }
    }
    if (!ok && lane == 0) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
    if (lane == 0) {
      for (int i = 0; i < C::kVStages && i < gv; ++i) {
        const int uses = (gv - 1 - i) / C::kVStages;
        if (!mbar_wait(&s.v_full[i], uses & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
        if (ok && !wait_stage<kCluster>(&s.v_empty[i], uses & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
      }
    }
  } else if (warp == 10) {
    // ---------------- S^T issuer (whole warp; an elected lane issues) ----------------
    bool ok = true;
    int gt = 0, gs = 0, st = 0, st_ph = 0;
    const uint32_t q_base = smem_addr(s.q[0]);
    Walk<C> walk;
    walk.start(p, s);
    Segment g;
    while (walk.next(p, s, g)) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.q_ready, gt & 1));
      const uint32_t idesc = prefill_tc::warp_uniform_int(umma_idesc_bf16(128, g.N, 0, 0));
      const int steps = prefill_tc::warp_uniform_int(g.steps);
      for (int j = 0; j < steps; ++j) {
        const int sb = gs & 1;
        if (ok && gs >= 2) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.s_free[sb], ((gs >> 1) - 1) & 1));
        const uint32_t d = tmem + C::kSCol + sb * kN;
        for (int ch = 0; ch < C::kChunks; ++ch) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.k_full[st], st_ph));
          tc_fence_after_sync();
          const uint32_t k_base = smem_addr(s.k[st]);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_warp(d, umma_desc(k_base + kk * 32, 16, 1024, 2),
                           umma_desc(q_base + ch * (kN * 128) + kk * 32, 16, 1024, 2), idesc, (ch | kk) > 0 ? 1u : 0u);
          commit_all<kCluster>(&s.k_empty[st]);
          if (++st == C::kKStages) st = 0, st_ph ^= 1;
        }
        umma_commit_warp(&s.s_full[sb]);
        ++gs;
      }
      umma_commit_warp(&s.q_empty);
      ++gt;
    }
    // the softmax warps' last arrivals on s_free (not waited for above)
    for (int k = gs >= 2 ? gs - 2 : 0; k < gs; ++k)
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.s_free[k & 1], (k >> 1) & 1));
    umma_commit_warp(&s.mma_done);
    if (!__all_sync(0xffffffffu, mbar_wait_fast(&s.mma_done, 0))) ok = false;  // every product done before the memory is freed
    if (!ok && lane == 0) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
  } else if (warp == 11) {
    // ---------------- O^T issuer; it also cleans the rows of V that not every node sees ----------------
    if (lane == 0 && !p.whole) note_cut<C>(p, s);
    __syncwarp();
    bool ok = true;
    int gt = 0, gs = 0, st = 0, st_ph = 0;
    Walk<C> walk;
    walk.start(p, s);
    Segment g;
    while (walk.next(p, s, g)) {
      if (ok && gt >= 1) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.o_free, (gt - 1) & 1));
      const uint32_t idesc = prefill_tc::warp_uniform_int(umma_idesc_bf16(128, g.N, 1, 1));
      bool poison = false;
      const int all0 = all_from(g.q, p.window);
      for (int pg0 = g.p0; pg0 < g.p1; pg0 += kStepPages) {
        const int pb = gs % kPBufs;
        const int np = prefill_tc::warp_uniform_int(min(kStepPages, g.p1 - pg0));
        const uint32_t p_base = smem_addr(s.p[pb]);
        for (int kk = 0; kk < np; ++kk) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.v_full[st], st_ph));
          const uint32_t v_base = smem_addr(s.v[st]);
          const int pos0 = (g.q.page0 + pg0 + kk) * kPage;
          if (ok && (pos0 < all0 || pos0 + kPage > g.q.ctx)) {  // (lo <= all0)
            const uint32_t none = row_bits(0, g.q.lo - pos0) | row_bits(g.q.L - pos0, kPage);
            const uint32_t some = (row_bits(0, all0 - pos0) | row_bits(g.q.ctx - pos0, kPage)) & ~none;
            poison |= clean_page<C>(v_base + (lane >> 3) * (kPage * 128) + (lane & 7) * 16, none, some);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (kk == 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.p_full[pb], (gs / kPBufs) & 1));
          tc_fence_after_sync();
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
            umma_bf16_warp(tmem + t * kN, umma_desc(v_base + t * (2 * kPage * 128), kPage * 128, 1024, 2),
                           umma_desc(p_base + kk * (kPage * 128), C::kPChunk, 1024, 2), idesc,
                           (pg0 > g.p0 || kk > 0) ? 1u : 0u);
          commit_all<kCluster>(&s.v_empty[st]);
          if (++st == C::kVStages) st = 0, st_ph ^= 1;
        }
        umma_commit_warp(&s.p_empty[pb]);
        ++gs;
      }
      umma_commit_warp(&s.o_full);
      poison = __any_sync(0xffffffffu, poison);
      if (lane == 0) {
        s.poison = poison;
        mbar_arrive(&s.o_full);
      }
      __syncwarp();
      ++gt;
    }
    if (ok && gt >= 1) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.o_free, (gt - 1) & 1));
    umma_commit_warp(&s.mma_done);
    if (!__all_sync(0xffffffffu, mbar_wait_fast(&s.mma_done, 0))) ok = false;
    if (!ok && lane == 0) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
  } else {
    // ---------------- softmax and epilogue: thread = key of the step, then dim of a tile ----------------
    const int h = warp >> 2;             // half of the columns
    const int key = threadIdx.x & 127;   // tensor-memory lane, thread of the warpgroup
    const uint32_t bar = 2 + h;
    const uint32_t t_row = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const auto fmax2 = [](float a, float b) { return fmaxf(a, b); };
    const auto add2 = [](float a, float b) { return a + b; };
    const float2 log2e2 = make_float2(kLog2e, kLog2e);
    bool ok = true;
    int gt = 0, gs = 0;
    Walk<C> walk;
    walk.start(p, s);
    Segment g, ahead;
    int parent[2], ahead_parent[2] = {-1, -1};  // the next segment and its parents are read before this one's end
    bool more = walk.next(p, s, ahead);
    if (more) read_parents(p.parents + ahead.q.q0, ahead.q.n, ahead_parent);
    while (more) {
      g = ahead;
      parent[0] = ahead_parent[0];
      parent[1] = ahead_parent[1];
      const int half = g.N >> 1;
      const int c0 = h * half;  // this warpgroup's first column
      const int all0 = all_from(g.q, p.window);
      const int node0 = walk.group * C::kQueries;
      const int seg0 = (g.q.page0 + g.p0) * kPage, seg1 = (g.q.page0 + g.p1) * kPage;
      named_barrier_sync(1, kSoftmaxThreads);  // all are done with the last segment's shared state
      if (seg0 < all0 || seg1 > g.q.ctx) {
        // the sequence's tree: every warp works it out and writes its share of the masks
        int depth[2];
        unsigned long long mask[2];
        if (check_parents(g.q.n, parent) && threadIdx.x == 0) report(p.status, ATTN_DEV_BAD_TREE);
        depths(parent, depth);
        ancestors(parent, mask);
        if (warp == 0) {
          s.depth[lane] = depth[0];
          s.depth[lane + 32] = depth[1];
        }
        const uint32_t m0 = static_cast<uint32_t>(warp < 4 ? mask[0] : mask[0] >> 32);  // ancestors 8 warp .. 8 warp + 7
        const uint32_t m1 = static_cast<uint32_t>(warp < 4 ? mask[1] : mask[1] >> 32);
#pragma unroll 4
        for (int j = 8 * warp; j < 8 * warp + 8; ++j) {
          const uint32_t b0 = __ballot_sync(0xffffffffu, lane < g.q.n && (m0 >> (j & 31) & 1));
          const uint32_t b1 = __ballot_sync(0xffffffffu, lane + 32 < g.q.n && (m1 >> (j & 31) & 1));
          const uint32_t d0 = __ballot_sync(0xffffffffu, depth[0] <= j);
          const uint32_t d1 = __ballot_sync(0xffffffffu, depth[1] <= j);
          if (lane == 0) {
            s.below[j] = b0 | static_cast<unsigned long long>(b1) << 32;
            s.shallow[j] = d0 | static_cast<unsigned long long>(d1) << 32;
          }
        }
      }
      if (key < half) {
        s.neg_m[c0 + key] = 0.f;
        s.bound[c0 + key] = -INFINITY;
      }
      named_barrier_sync(1, kSoftmaxThreads);
      float l[kHalf];
#pragma unroll
      for (int c = 0; c < kHalf; ++c) l[c] = 0.f;

      for (int j = 0; j < g.steps; ++j) {
        const int sb = gs & 1, pb = gs % kPBufs;
        const int step0 = seg0 + j * kKeys;
        const bool masked = step0 < all0 || step0 + kKeys > min(g.q.ctx, seg1);
        unsigned long long vis = 0;
        if (masked && step0 + key < seg1) vis = seen_by(g.q, p.window, s, step0 + key) >> node0;
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.s_full[sb], (gs >> 1) & 1));
        tc_fence_after_sync();
#pragma unroll
        for (int blk = 0; blk < kHalf; blk += kBlock) {
          if (blk >= half) continue;
          const int cb = c0 + blk;  // first column of the block
          float sv[kBlock];
#pragma unroll
          for (int b8 = 0; b8 < kBlock / 8; ++b8) {
            if (blk + 8 * b8 < half) {
              tmem_ld8(t_row + C::kSCol + sb * kN + cb + 8 * b8, *reinterpret_cast<float(*)[8]>(&sv[8 * b8]));
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) sv[8 * b8 + e] = -INFINITY;
            }
          }
          tmem_wait_ld();
          if (blk + kBlock >= half) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.s_free[sb]);
          }
          if (masked) {
#pragma unroll
            for (int b8 = 0; b8 < kBlock / 8; ++b8) {
              const uint32_t bits = static_cast<uint32_t>(vis >> ((cb + 8 * b8) / kG & 63));
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (!((bits >> (kG >= 8 ? 0 : e / kG)) & 1)) sv[8 * b8 + e] = -INFINITY;
            }
          }
          if (j == 0) {
            // first references: the scores of a key that every node sees, if there is one
            if (step0 + key == max(step0, all0) && step0 + key < min(g.q.ctx, seg1)) {
#pragma unroll
              for (int c = 0; c < kBlock; ++c)
                if (blk + c < half && sv[c] > -INFINITY && sv[c] < INFINITY) {
                  const float m = fmaf(sv[c], kLog2e, kHeadroom);
                  s.neg_m[cb + c] = -m;
                  s.bound[cb + c] = (m + kSlack) * (1.f / kLog2e);
                }
            }
            named_barrier_sync(bar, 128);
          }
          bool moves = false;
#pragma unroll
          for (int c4 = 0; c4 < kBlock / 4; ++c4) {
            if (blk + 4 * c4 < half) {
              const float4 t = *reinterpret_cast<const float4*>(&s.bound[cb + 4 * c4]);
              moves |= (sv[4 * c4] > t.x) | (sv[4 * c4 + 1] > t.y) | (sv[4 * c4 + 2] > t.z) | (sv[4 * c4 + 3] > t.w);
            }
          }
          if (barrier_or(bar, 128, moves)) {
            float* const red = s.red[warp] + blk;
            reduce_into<kBlock>(sv, red, fmax2);
            named_barrier_sync(bar, 128);
            if (key < kBlock && blk + key < half) {
              const int w0 = h * 4, c = blk + key, col = c0 + c;
              const float mx = fmaxf(fmaxf(s.red[w0][c], s.red[w0 + 1][c]), fmaxf(s.red[w0 + 2][c], s.red[w0 + 3][c]));
              float f = 1.f;
              if (mx > s.bound[col]) {
                const float m = fmaf(mx, kLog2e, kHeadroom);
                if (s.bound[col] != -INFINITY) f = ex2_approx(-s.neg_m[col] - m);
                s.neg_m[col] = -m;
                s.bound[col] = (m + kSlack) * (1.f / kLog2e);
              }
              s.f[col] = f;
            }
            named_barrier_sync(bar, 128);
#pragma unroll
            for (int c = 0; c < kBlock; ++c)
              if (blk + c < half) l[blk + c] *= s.f[cb + c];
            if (j > 0) {
              // O^T holds the products up to step j - 1: wait for the last, then scale in place
              if (ok) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.p_empty[(gs - 1) % kPBufs], ((gs - 1) / kPBufs) & 1));
              tc_fence_after_sync();
#pragma unroll 1
              for (int c = 0; c < kBlock && blk + c < half; c += 8) {
#pragma unroll 1
                for (int t = 0; t < kTiles; ++t) {
                  float ov[8];
                  uint32_t w[8];
                  tmem_ld8(t_row + t * kN + cb + c, ov);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(ov[e] * s.f[cb + c + e]);
                  tmem_st8(t_row + t * kN + cb + c, w);
                }
              }
              tmem_wait_st();
            }
          }
          // weights; the buffer's last reader was the product of step j - kPBufs
          if (blk == 0 && ok && gs >= kPBufs)
            ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.p_empty[pb], (gs / kPBufs - 1) & 1));
#pragma unroll
          for (int b8 = 0; b8 < kBlock / 8; ++b8) {
            if (blk + 8 * b8 < half) {
              float2 w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 m = *reinterpret_cast<const float2*>(&s.neg_m[cb + 8 * b8 + 2 * e]);
                const float2 x = __ffma2_rn(make_float2(sv[8 * b8 + 2 * e], sv[8 * b8 + 2 * e + 1]), log2e2, m);
                w[e] = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                const int c = blk + 8 * b8 + 2 * e;
                const float2 sum = __fadd2_rn(make_float2(l[c], l[c + 1]), w[e]);
                l[c] = sum.x;
                l[c + 1] = sum.y;
              }
              const int col = cb + 8 * b8;
              st_shared_v4(
                  smem_addr(s.p[pb]) + (col >> 6) * C::kPChunk + key * 128 + ((((col & 63) >> 3) ^ (key & 7)) << 4),
                  make_uint4(pack_bf16x2(w[0].x, w[0].y), pack_bf16x2(w[1].x, w[1].y), pack_bf16x2(w[2].x, w[2].y),
                             pack_bf16x2(w[3].x, w[3].y)));
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[pb]);
        ++gs;
      }

      more = walk.next(p, s, ahead);
      if (more) read_parents(p.parents + ahead.q.q0, ahead.q.n, ahead_parent);
      // ---- end of the segment: sums, then this thread's dim of every row ----
      reduce_into<kHalf>(l, s.red[warp], add2);
      named_barrier_sync(bar, 128);
      if (key < half) {
        const int w0 = h * 4, col = c0 + key;
        const float sum = (s.red[w0][key] + s.red[w0 + 1][key]) + (s.red[w0 + 2][key] + s.red[w0 + 3][key]);
        if (g.whole)
          s.f[col] = sum > 0.f ? 1.f / sum : sum;  // 0: a row that sees nothing; NaN stays
        else if (col < g.cols)
          p.part_ml[static_cast<size_t>(g.slot) * kN + col] = partial_stats(-s.neg_m[col], sum);
      }
      named_barrier_sync(bar, 128);
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.o_full, gt & 1));
      tc_fence_after_sync();
      const bool poison = s.poison != 0;
      // column col's row of the output: node col / kG, head col % kG
      const size_t row0 = static_cast<size_t>(g.row0) * C::kHq + walk.kv * kG;
#pragma unroll 1
      for (int c = 0; c < half; c += 8) {
        const int col = c0 + c;
        if (col >= g.cols) break;  // (uniform: whole blocks of 8 columns)
        float ov[kTiles][8];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) tmem_ld8(t_row + t * kN + col, ov[t]);
        tmem_wait_ld();
        if (poison) {
          // the elements that were zeroed, for the rows that see them
#pragma unroll 1
          for (int pos = max(g.q.lo, seg0); pos < min(g.q.L, seg1); ++pos) {
            if (pos >= all0 && pos < g.q.ctx) {
              pos = g.q.ctx - 1;
              continue;
            }
            const int id = p.block_table[static_cast<int64_t>(g.b) * p.max_blocks + pos / kPage];
            if (id < 0 || static_cast<int64_t>(id) >= p.num_pages) continue;
            const __nv_bfloat16* v = p.v_pool + ((static_cast<size_t>(id) * kPage + pos % kPage) * C::kHkv + walk.kv) * kD;
            const unsigned long long vis = seen_by(g.q, p.window, s, pos) >> node0;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              const float x = __bfloat162float(v[t * 128 + key]);
              if (fabsf(x) < INFINITY) continue;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if ((vis >> ((col + e) / kG & 63)) & 1) ov[t][e] += x;
            }
          }
        }
        if (g.whole) {
          const size_t at = (row0 + static_cast<size_t>(col / kG) * C::kHq + col % kG) * kD;
          const auto row_of = [](int e) { return (kG >= 8 ? e : (e / kG) * C::kHq + e % kG) * kD; };
          if (p.out_f32) {
            float* const out = static_cast<float*>(p.o) + at + key;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float f = s.f[col + e];
              if (kG < 8 && col + e >= g.cols) continue;
#pragma unroll
              for (int t = 0; t < kTiles; ++t) out[row_of(e) + t * 128] = ov[t][e] * f;
            }
          } else {
            // two columns at a time: even lanes store dims (d, d + 1) of the first, odd lanes (d - 1, d) of the second
            const int odd = lane & 1;
            __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(p.o) + at + (key & ~1);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float f = s.f[col + e + odd];
#pragma unroll
              for (int t = 0; t < kTiles; ++t) {
                const float mine = odd ? ov[t][e + 1] : ov[t][e];
                const float other = __shfl_xor_sync(0xffffffffu, odd ? ov[t][e] : ov[t][e + 1], 1);
                const uint32_t w = odd ? pack_bf16x2(other * f, mine * f) : pack_bf16x2(mine * f, other * f);
                if (kG >= 8 || col + e + odd < g.cols)
                  *reinterpret_cast<uint32_t*>(out + (odd ? row_of(e + 1) : row_of(e)) + t * 128) = w;
              }
            }
          }
        } else {
          float* const out = p.part_o + (static_cast<size_t>(g.slot) * kN + col) * kD + key;
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int t = 0; t < kTiles; ++t) out[e * kD + t * 128] = ov[t][e];
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.o_free);  // the next segment's first product may overwrite O^T
      ++gt;
    }
    // the last products' commits (not all waited for above)
    for (int k = gs >= kPBufs ? gs - kPBufs : 0; k < gs; ++k)
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.p_empty[k % kPBufs], (k / kPBufs) & 1));
    if (!ok && lane == 0) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
  }

  // ---------------- teardown: free the tensor memory ----------------
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if constexpr (kCluster > 1) cluster_sync_all();  // nothing of the other CTA may arrive in one that has left
}

template <typename C>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeParams p) {
  tree_body<C>(tm_q, tm_k, tm_v, p);
}

template <typename C>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    tree_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeParams p) {
  tree_body<C>(tm_q, tm_k, tm_v, p);
}

// ---------------------------------------------------------------------------
// The cut sequences' rows, joined from their partials: o = sum 2^(m_i - M) O_i /
// sum 2^(m_i - M) l_i.  Every block reads the cuts that the blocks of the first kernel
// noted.  Many rows: a warp takes one whole, four dims of every 128 a lane.  Few: a block
// takes 128 dims of one, its warps the partials in turn, and they meet in shared memory.
// Bound by latency: kMergeInFlight loads of 16 bytes are in flight a lane.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 4;
constexpr int kMergeBlocksPerSm = 6;
constexpr int kMergeInFlight = 8;

struct MergeParams {
  TreeParams t;
  int32_t grid;    // blocks of the first kernel
  int32_t stride;  // distance of consecutive blocks of a list: KV heads, times the cluster
};

template <int kT>
struct MergeItem {
  int row0, kv, col;  // first node of the group, KV head, row of the group
  float m, l;
  float4 o[kT];
};

// Partials member, member + team, .. of a row, kT * 128 dims from tile0 * 128 on, four a lane.
template <typename C, int kT>
__device__ __forceinline__ MergeItem<kT> merge_partials(const MergeParams& mp, const int32_t* rows, int row, int tile0,
                                                        int member, int team) {
  constexpr int kFly = kMergeInFlight / kT;
  const TreeParams& p = mp.t;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = mp.grid - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (rows[mid] <= row) lo = mid; else hi = mid - 1;
  }
  const int4 cut = p.cuts[lo];
  MergeItem<kT> it;
  it.row0 = cut.x;
  it.kv = cut.y >> 8;
  it.col = row - rows[lo];
  it.m = -INFINITY;
  it.l = 0.f;
#pragma unroll
  for (int t = 0; t < kT; ++t) it.o[t] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = member; i0 < cut.w; i0 += team * kFly) {
    float2 e[kFly];
    float4 a[kFly][kT];
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      const int i = i0 + u * team;
      const size_t at = static_cast<size_t>(i == 0 ? cut.z : 2 * (lo + i * mp.stride)) * C::kN + it.col;
      e[u] = i < cut.w ? p.part_ml[at] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int t = 0; t < kT; ++t)
        a[u][t] = i < cut.w ? __ldcs(reinterpret_cast<const float4*>(p.part_o + at * C::kD + (tile0 + t) * 128 + 4 * lane))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m = it.m;
#pragma unroll
    for (int u = 0; u < kFly; ++u)
      if (e[u].y > 0.f) m = fmaxf(m, e[u].x);
    if (m == -INFINITY) continue;
    const float f = it.m == -INFINITY ? 0.f : exp2f(it.m - m);
    it.m = m;
    it.l *= f;
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      it.o[t].x *= f; it.o[t].y *= f; it.o[t].z *= f; it.o[t].w *= f;
    }
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      if (!(e[u].y > 0.f)) continue;
      const float w = exp2f(e[u].x - m);
      it.l += w * e[u].y;
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        it.o[t].x += w * a[u][t].x; it.o[t].y += w * a[u][t].y; it.o[t].z += w * a[u][t].z; it.o[t].w += w * a[u][t].w;
      }
    }
  }
  return it;
}

template <typename C, int kT>
__device__ __forceinline__ void store_merged(const TreeParams& p, const MergeItem<kT>& it, int tile0) {
  const int lane = threadIdx.x & 31;
  const float inv = it.l > 0.f ? 1.f / it.l : it.l;
  const size_t at = (static_cast<size_t>(it.row0 + it.col / C::kG) * C::kHq + it.kv * C::kG + it.col % C::kG) * C::kD +
                    tile0 * 128 + 4 * lane;
#pragma unroll
  for (int t = 0; t < kT; ++t) {
    const float4 v = make_float4(it.o[t].x * inv, it.o[t].y * inv, it.o[t].z * inv, it.o[t].w * inv);
    if (p.out_f32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at + t * 128) = v;
    } else {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at + t * 128) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
  }
}

template <typename C>
__global__ void __launch_bounds__(kMergeWarps * 32, kMergeBlocksPerSm) merge_kernel(const __grid_constant__ MergeParams mp) {
  const TreeParams& p = mp.t;
  constexpr int kD = C::kD, kThreadsHere = kMergeWarps * 32;
  __shared__ int32_t s_rows[kMaxGrid + 1];
  __shared__ int32_t s_warp[kMergeWarps];
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
  __shared__ float4 s_o[kMergeWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_primary_grid();
  allow_dependent_launch();
  // running sum of the cut rows
  int carry = 0;
  if (threadIdx.x == 0) s_rows[0] = 0;
  for (int g0 = 0; g0 < mp.grid; g0 += kThreadsHere) {
    const int g = g0 + threadIdx.x;
    int n = 0;
    if (g < mp.grid) {
      const int4 cut = p.cuts[g];
      n = cut.w > 0 ? (cut.y & 255) * C::kG : 0;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += u;
    }
    if (lane == 31) s_warp[warp] = n;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      if (w < warp) n += s_warp[w];
      total += s_warp[w];
    }
    if (g < mp.grid) s_rows[g + 1] = carry + n;
    carry += total;
    __syncthreads();
  }
  // few rows: an item is 128 dims of a row, a block's; many: a row, a warp's
  if (carry * C::kTiles * 2 < static_cast<int>(gridDim.x) * kMergeWarps) {
    for (int item = blockIdx.x; item < carry * C::kTiles; item += gridDim.x) {
      const MergeItem<1> it = merge_partials<C, 1>(mp, s_rows, item / C::kTiles, item % C::kTiles, warp, kMergeWarps);
      if (lane == 0) {
        s_m[warp] = it.m;
        s_l[warp] = it.l;
      }
      s_o[warp][lane] = it.o[0];
      __syncthreads();
      if (warp == 0) {
        MergeItem<1> all = it;
#pragma unroll
        for (int w = 1; w < kMergeWarps; ++w) all.m = fmaxf(all.m, s_m[w]);
        all.l = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
          const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - all.m);
          const float4 v = s_o[w][lane];
          all.l += f * s_l[w];
          O.x += f * v.x; O.y += f * v.y; O.z += f * v.z; O.w += f * v.w;
        }
        all.o[0] = O;
        store_merged<C, 1>(p, all, item % C::kTiles);
      }
      __syncthreads();  // the shared partials were read
    }
  } else {
    for (int row = blockIdx.x * kMergeWarps + warp; row < carry; row += gridDim.x * kMergeWarps)
      store_merged<C, C::kTiles>(p, merge_partials<C, C::kTiles>(mp, s_rows, row, 0, 0, 1), 0);
  }
}

// D = 512: 64 rows, four nodes, alone or in pairs; D = 256: 128 rows, 64 nodes, or fewer with longer rings.
using GlobalConfig = Config<ATTN_GLOBAL_D, ATTN_GLOBAL_HQ / ATTN_GLOBAL_HKV, ATTN_GLOBAL_HKV, 64, 1, 4, 4>;
using GlobalPairConfig = Config<ATTN_GLOBAL_D, ATTN_GLOBAL_HQ / ATTN_GLOBAL_HKV, ATTN_GLOBAL_HKV, 64, 1, 4, 4, 2>;
using SlidingWideConfig = Config<ATTN_SLIDING_D, ATTN_SLIDING_HQ / ATTN_SLIDING_HKV, ATTN_SLIDING_HKV, 128, 2, 3, 5>;
using SlidingConfig = Config<ATTN_SLIDING_D, ATTN_SLIDING_HQ / ATTN_SLIDING_HKV, ATTN_SLIDING_HKV, 32, 2, 6, 8>;

}  // namespace tree
}  // namespace pda
