// tree_common.cuh -- around the products of tree_decode.cuh: the schedule of a call over
// trees of drafted tokens, its masks, the cleaning of V rows that not every node sees,
// and the merge of cut sequences.
//
// Schedule.  Rows come in groups of kQueries nodes; group r of KV head c of all
// sequences that have one is a list of pages, with seg_weight virtual pages in front of
// every sequence (its Q, its end).  All lists are cut into runs of `per` pages, the fewest
// that give no more runs than blocks: every block has the same work whatever the
// lengths, and those of neighbouring lists walk the same keys at the same time.  A
// sequence inside one run is finished there; of a cut one every block leaves a partial
// (O, m, sum), and merge_kernel joins them.
//
// What a node does not see.  Scores are masked, and rows of V that no node sees are
// zeroed in shared memory.  A row that some nodes see and others do not (a node of the
// tree, the window's edge) may hold an infinity or NaN, and 0 * inf would reach the
// others: such elements are zeroed too, and the epilogue writes them into the rows that
// do see them.
#pragma once

#include "attn_tree.h"
#include "common.cuh"
#include "prefill_tc.cuh"
#include "tcgen05.cuh"
#include "tree_nodes.cuh"

namespace pda {
namespace tree {

constexpr int kMaxGroups = 16;              // of rows, per KV head; the smallest grid
// Pages of the smallest run: fewer mean more partials to merge, more leave blocks without work.  us a call with 2, 4 and 8:
// one global tree of 4 nodes behind 900 positions 12.8, 13.6, 15.1; 8 of them behind 800 22.8, 20.0, 19.7; one of 8 behind
// 2000 19.4, 15.7, 16.5.
constexpr int kMinPer = 4;
constexpr int kSoftmaxThreads = 256;
constexpr int kThreads = 384;
constexpr int kMaxGrid = kMaxSplits;

struct TreeParams {
  const __nv_bfloat16* v_pool;  // (for cleaned elements; read through the tensor maps)
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
  int32_t lists;    // per KV head: ceil(max_q / kQueries), or more
  int32_t q_box;    // nodes that a copy of Q brings
  int32_t out_f32;
  int32_t seg_weight;  // virtual pages charged per sequence
  int32_t whole;    // a block per (sequence, group, KV head) instead of runs
};

// A sequence's tree in shared memory.
struct Masks {
  alignas(8) unsigned long long below[ATTN_MAX_TREE];    // nodes that see node j by ancestry
  alignas(8) unsigned long long shallow[ATTN_MAX_TREE];  // nodes of depth <= x
  int32_t depth[ATTN_MAX_TREE];
};

// What the schedule leaves in shared memory.
struct Shared {
  int32_t pre[kMaxBatch + 1];  // pages (virtual ones included) before sequence b in this block's list
  int32_t cu_q[kMaxBatch + 1], len[kMaxBatch];
  int32_t sched[4];            // list, KV head, per, run
  int32_t refused;             // the call as a whole
  int32_t misfit;              // a sequence's numbers do not fit together
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

// A call without nodes: its lengths may deny that.  A thread per sequence.
__global__ void __launch_bounds__(kMaxBatch) check_kernel(const __grid_constant__ TreeParams p) {
  wait_for_primary_grid();
  allow_dependent_launch();
  const int b = static_cast<int>(threadIdx.x);
  bool refused = false;
  if (b < p.batch) make_sequence(p, p.cu_q[b], p.cu_q[b + 1], p.seq_lens[b], refused);
  if (refused) report(p.status, ATTN_DEV_BAD_SEQ_LEN);
}

// Positions below are not seen by every node.
__device__ __forceinline__ int all_from(const Sequence& q, int window) {
  return window > 0 ? q.ctx + (q.n - 1) - window + 1 : 0;  // (a depth is at most n - 1)
}

// A part of one sequence's pages for one group of rows.
struct Segment {
  Sequence q;
  int b, row0, nodes, cols, N;  // first node of the group (packed), its nodes, rows, columns of the products
  int p0, p1, steps;            // pages, and steps of C::kStepPages
  bool whole;
  int slot;                     // of its partial
};

// Walks a block's segments; every role does it for itself, with the same result.
template <typename C>
struct Walk {
  int b, w0, w1, group, kv, index;
  __device__ __forceinline__ void start(const TreeParams& p, const Shared& s) {
    group = s.sched[0];
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
#pragma unroll 1
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.pre[mid] <= w0) lo = mid; else hi = mid - 1;
    }
    b = lo;
  }
  __device__ __forceinline__ bool next(const TreeParams& p, const Shared& s, Segment& g) {
#pragma unroll 1
    for (; b < p.batch && s.pre[b] < w1; ++b) {
      const int pages = s.pre[b + 1] - s.pre[b] - p.seg_weight;
      if (pages <= 0) continue;
      const int first = s.pre[b] + p.seg_weight;
      g.p0 = w0 > first ? w0 - first : 0;
      g.p1 = w1 - first < pages ? w1 - first : pages;
      if (g.p1 <= g.p0) continue;
      bool refused;
      g.q = make_sequence(p, s.cu_q[b], s.cu_q[b + 1], s.len[b], refused);
      g.b = b;
      g.row0 = g.q.q0 + group * C::kQueries;
      g.nodes = min(C::kQueries, g.q.n - group * C::kQueries);
      g.cols = g.nodes * C::kG;
      g.N = max(16, (g.cols + 15) & ~15);
      g.steps = (g.p1 - g.p0 + C::kStepPages - 1) / C::kStepPages;
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
__device__ __forceinline__ void reduce_into(const float (&v)[kHalf], int n, float* red, Op op) {  // the first n columns
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
      if (c0 >= n) break;
      float t[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) t[i] = v[c0 + i];
      red[c0 + lane] = reduce_columns<32>(t, op);
    }
  }
}

// Column maxima over the warp's 32 keys: lane c of `red` (a row of the warp's) gets column c.  Only in steps that move a
// reference.  (-0 counts as below +0: the comparison with the bounds does not tell them apart.)
template <int kW>
__device__ __forceinline__ void max_into(const float (&v)[kW], float* red) {
  const int lane = threadIdx.x & 31;
  int mine = 0;
#pragma unroll
  for (int c = 0; c < kW; ++c) {
    const int bits = __float_as_int(v[c] == v[c] ? v[c] : -INFINITY);  // a NaN moves nothing
    const int m = __reduce_max_sync(0xffffffffu, bits ^ (bits >> 31 & 0x7fffffff));  // ordered as integers
    mine = lane == c ? m : mine;
  }
  if (lane < kW) red[lane] = __int_as_float(mine ^ (mine >> 31 & 0x7fffffff));
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
__device__ __forceinline__ unsigned long long seen_by(const Sequence& q, int window, const Masks& s, int pos) {
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

// The masks of a sequence's tree, by all softmax warps: every warp works the tree out and writes its share.
__device__ __forceinline__ void make_masks(Masks& s, int32_t* status, int n, int parent0, int parent1) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int parent[2] = {parent0, parent1};
  uint32_t m0, m1 = 0;  // nodes lane and lane + 32: their ancestors among 32 (warp / 4) .. + 31
  int depth0, depth1 = ATTN_MAX_TREE;
  if (check_parents(n, parent) && threadIdx.x == 0) report(status, ATTN_DEV_BAD_TREE);
  if (n <= 32) {
    m0 = ancestors32(parent[0]);
    depth0 = __popc(m0) - 1;
    if (warp >= 4) m0 = 0;
  } else {
    unsigned long long mask[2];
    ancestors(parent, mask);
    depth0 = __popcll(mask[0]) - 1;
    depth1 = __popcll(mask[1]) - 1;
    m0 = static_cast<uint32_t>(warp < 4 ? mask[0] : mask[0] >> 32);
    m1 = static_cast<uint32_t>(warp < 4 ? mask[1] : mask[1] >> 32);
  }
  if (lane >= n) m0 = 0;
  if (lane + 32 >= n) m1 = 0;
  if (warp == 0) {
    s.depth[lane] = depth0;
    s.depth[lane + 32] = depth1;
  }
#pragma unroll 2
  for (int j = 8 * warp; j < 8 * warp + 8; ++j) {
    const uint32_t b0 = __ballot_sync(0xffffffffu, m0 >> (j & 31) & 1), b1 = __ballot_sync(0xffffffffu, m1 >> (j & 31) & 1);
    const uint32_t d0 = __ballot_sync(0xffffffffu, depth0 <= j), d1 = __ballot_sync(0xffffffffu, depth1 <= j);
    if (lane == 0) {
      s.below[j] = b0 | static_cast<unsigned long long>(b1) << 32;
      s.shallow[j] = d0 | static_cast<unsigned long long>(d1) << 32;
    }
  }
}

// The lengths, read into shared memory by warp 0; with `kAgain`, whether any differs from what is there.
template <bool kAgain>
__device__ __forceinline__ bool read_lengths(const TreeParams& p, Shared& s) {
  bool differ = false;
#pragma unroll 1
  for (int b0 = 0; b0 <= p.batch; b0 += 32) {
    const int b = b0 + (threadIdx.x & 31);
    const int q = b <= p.batch ? __ldcg(p.cu_q + b) : 0, L = b < p.batch ? __ldcg(p.seq_lens + b) : 0;
    if (kAgain) differ |= (b <= p.batch && s.cu_q[b] != q) || (b < p.batch && s.len[b] != L);
    if (b <= p.batch) s.cu_q[b] = q;
    if (b < p.batch) s.len[b] = L;
  }
  __syncwarp();
  return __any_sync(0xffffffffu, differ);
}

// The schedule: this block's list, the running sums over it, its run; by warp 0, 32 sequences a round.  (Rounds are
// loops, not unrolled: what runs once a call is bound by fetching its instructions.)  It is made before the block waits
// for the previous kernel, whose last writes may still change the lengths, and again where they did change; what is
// reported is reported by the second reading.
template <typename C>
__device__ __noinline__ void make_schedule(const TreeParams& p, Shared& s, bool final) {
  const int lane = threadIdx.x & 31;
  {
    bool refused = false, backwards = false;
    int total = 0;  // lane r: the pages of list r (the same for every KV head)
    // (weight, lists) of sequence b
    const auto weigh = [&](int b, bool& bad) {
      const Sequence q = make_sequence(p, s.cu_q[b], s.cu_q[b + 1], s.len[b], bad);
      return q.pages > 0 ? make_int2(q.pages + p.seg_weight, (q.n + C::kQueries - 1) / C::kQueries) : make_int2(0, 0);
    };
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
    if (refused && final && blockIdx.x == 0 && lane == 0) report(p.status, ATTN_DEV_BAD_SEQ_LEN);
    const int g = static_cast<int>(blockIdx.x);
    int list, kv, per, run;
    if (p.whole) {
      const int per_seq = p.lists * C::kHkv;
      list = g % per_seq / C::kHkv;
      kv = g % C::kHkv;
      per = 1;
      run = g / per_seq;
    } else {
      const int grid = static_cast<int>(gridDim.x);
      const int sum = __reduce_add_sync(0xffffffffu, total);
      // (sum * kHkv <= 256 sequences * (16384 pages + seg_weight) * 16, lists times KV heads at most: 2^27)
      int lo = max(kMinPer, (sum * C::kHkv + grid - 1) / grid);
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
      const int mine = (total + per - 1) / per * C::kHkv;  // this list's blocks
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
      s.misfit = refused;
    }
  }
  __syncwarp();
}

// The elements of V that were zeroed, for the rows that see them: an infinity or NaN among a sum's terms adds itself,
// whatever its weight, to what the products gave, which may be one too (of a key, or of a value that all nodes see).  By a
// softmax thread, for dims key + 128 i of columns [from, to), after it (or its warp) stored them.
template <typename C>
__device__ __noinline__ void add_back(const TreeParams& p, const Masks& s, const Segment& g, int kv, int node0, int from,
                                      int to) {
  const int all0 = all_from(g.q, p.window);
  const int pos0 = max(g.q.lo, (g.q.page0 + g.p0) * kPage), pos1 = min(g.q.L, (g.q.page0 + g.p1) * kPage);
#pragma unroll 1
  for (int d = threadIdx.x & 127; d < C::kD; d += 128) {
#pragma unroll 1
    for (int col = from; col < to; ++col) {
      float sum = 0.f;
#pragma unroll 1
      for (int pos = pos0; pos < pos1; ++pos) {
        if (pos >= all0 && pos < g.q.ctx) {
          pos = g.q.ctx - 1;
          continue;
        }
        if (!(seen_by(g.q, p.window, s, pos) >> (node0 + col / C::kG) & 1)) continue;
        const int id = p.block_table[static_cast<int64_t>(g.b) * p.max_blocks + pos / kPage];
        if (id < 0 || static_cast<int64_t>(id) >= p.num_pages) continue;
        const float x = __bfloat162float(p.v_pool[((static_cast<size_t>(id) * kPage + pos % kPage) * C::kHkv + kv) * C::kD + d]);
        if (!(fabsf(x) < INFINITY)) sum += x;
      }
      if (sum == 0.f) continue;  // (anything else is an infinity or NaN)
      if (!g.whole) {
        p.part_o[(static_cast<size_t>(g.slot) * C::kN + col) * C::kD + d] += sum;
        continue;
      }
      const size_t at = (static_cast<size_t>(g.row0 + col / C::kG) * C::kHq + kv * C::kG + col % C::kG) * C::kD + d;
      if (p.out_f32) {
        static_cast<float*>(p.o)[at] += sum;
      } else {
        __nv_bfloat16* const o = static_cast<__nv_bfloat16*>(p.o) + at;
        *o = __float2bfloat16_rn(__bfloat162float(*o) + sum);
      }
    }
  }
}

// Tells the merge which sequence is cut first in this block; run by one thread.
template <typename C>
__device__ __forceinline__ void note_cut(const TreeParams& p, const Shared& s) {
  Walk<C> walk;
  walk.start(p, s);
  Segment g;
  int4 cut = make_int4(0, 0, 0, 0);
  while (walk.next(p, s, g)) {
    if (g.p0 == 0 && !g.whole) {
      const int last = (s.pre[g.b] + p.seg_weight + g.q.pages - 1) / s.sched[2];  // the run that holds its last page
      cut = make_int4(g.row0, g.nodes | (walk.kv << 8), g.slot, last - s.sched[3] + 1);
    }
  }
  p.cuts[blockIdx.x] = cut;
}

// mbar_wait_fast in few instructions: with some forty waits of the kernel inlined, its code outgrew the instruction
// cache (159 KB; a sliding call of 64 sequences took 140 us).  False once kWaitLimitNs have passed.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_addr(bar);
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 0;; ++n) {
    uint32_t done;
    if (n == 0) {
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(done)
          : "r"(a), "r"(parity)
          : "memory");
    } else {
      done = mbar_try_wait(a, parity);
    }
    if (done) return true;
    if ((n & 63) == 63) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) return false;
    }
  }
}

// The rows of a segment's output from tensor memory, by the 128 threads of a warpgroup: columns [from, to), of each a
// thread's dim of every tile, tile t's columns from t_row + t * kN on; factor f per column.
template <typename C>
__device__ __forceinline__ void store_columns(const TreeParams& p, const Segment& g, int kv, int from, int to, uint32_t t_row,
                                              const float* f) {
  constexpr int kG = C::kG, kD = C::kD, kT = C::kTiles;
  const int key = threadIdx.x & 127, lane = threadIdx.x & 31;
  // column col's row: of a whole sequence node col / kG, head col % kG of the output, else row col of the partial
  const bool to_f32 = !g.whole || p.out_f32;
  const size_t base =
      (g.whole ? static_cast<size_t>(g.row0) * C::kHq + kv * kG : static_cast<size_t>(g.slot) * C::kN) * kD;
  const int node_pitch = (g.whole ? C::kHq : kG) * kD;
  float* const out = (g.whole ? static_cast<float*>(p.o) : p.part_o) + base + key;
  __nv_bfloat16* const out16 = static_cast<__nv_bfloat16*>(p.o) + base + (key & ~1);
#pragma unroll 1
  for (int col = from; col < to; col += 8) {
    float ov[kT][8];
#pragma unroll
    for (int t = 0; t < kT; ++t) tmem_ld8(t_row + t * C::kN + col, ov[t]);
    tmem_wait_ld();
    const int node = col / kG, head = col % kG;
    if (to_f32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float fe = f[col + e];
        float* const row = out + (node + (kG >= 8 ? 0 : e / kG)) * node_pitch + (head + (kG >= 8 ? e : e % kG)) * kD;
        if (kG < 8 && col + e >= to) continue;
#pragma unroll
        for (int t = 0; t < kT; ++t) row[t * 128] = ov[t][e] * fe;
      }
    } else {
      // two columns at a time: even lanes store dims (d, d + 1) of the first, odd lanes (d - 1, d) of the second
      const int odd = lane & 1;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float fe = f[col + e + odd];
        __nv_bfloat16* const row =
            out16 + (node + (kG >= 8 ? 0 : e / kG)) * node_pitch + (head + (kG >= 8 ? e : e % kG) + odd) * kD;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          const float mine = odd ? ov[t][e + 1] : ov[t][e];
          const float other = __shfl_xor_sync(0xffffffffu, odd ? ov[t][e] : ov[t][e + 1], 1);
          const uint32_t w = odd ? pack_bf16x2(other * fe, mine * fe) : pack_bf16x2(mine * fe, other * fe);
          if (kG >= 8 || col + e + odd < to) *reinterpret_cast<uint32_t*>(row + t * 128) = w;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The cut sequences' rows, joined from their partials: o = sum 2^(m_i - M) O_i /
// sum 2^(m_i - M) l_i.  Every block reads the cuts that those of the first kernel
// noted.  A warp takes a row whole, four dims of every 128 a lane, or a block 128 dims of
// one, its warps the partials in turn, and they meet in shared memory (merge_kernel has
// the rule).  A part whose weight is below fp32's range adds nothing but its infinities and NaN, which a whole sequence
// would show, too (0 * inf would be NaN).  Bound by latency: kMergeInFlight loads of 16 bytes are in flight a lane; 2 us
// behind a small call, 12 us alone for the 29 MB of 32 trees of 64 nodes.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 4;
constexpr int kMergeBlocksPerSm = 6;  // (2: 64 global trees of 8 nodes 85.3 us, not 77.9; 32 of 64 nodes 601.9, not 595.7)
constexpr int kMergeInFlight = 8;

struct MergeParams {
  TreeParams t;
  int32_t grid;    // blocks of the first kernel
};

// The cut rows of all blocks, numbered: every warp for itself, lane l the blocks l * each .. (l + 1) * each - 1.  No
// shared memory and no barrier, so that the next call's blocks, which take nearly all of an SM's, can start beside it.
template <typename C>
struct CutRows {
  int each, before, total;  // (before: rows of the lanes below)
  int most;                 // partials of a row
  __device__ __forceinline__ static int of(const int4& c) { return c.w > 0 ? (c.y & 255) * C::kG : 0; }
  __device__ __forceinline__ CutRows(const TreeParams& p, int grid) : each((grid + 31) / 32) {
    const int lane = threadIdx.x & 31;
    int n = 0, w = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < each; i0 += 5) {  // (152 blocks: one round, all loads in flight)
      int4 c[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        const int g = lane * each + i0 + i;
        c[i] = i0 + i < each && g < grid ? p.cuts[g] : make_int4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        n += of(c[i]);
        w = max(w, c[i].w);
      }
    }
    most = __reduce_max_sync(0xffffffffu, w);
    before = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += u;
    }
    total = __shfl_sync(0xffffffffu, before, 31);
    before -= n;
  }
  // The block whose rows hold `row` < total (the same in every lane), and its first one.
  __device__ __forceinline__ int find(const TreeParams& p, int row, int& first) const {
    const int owner = 31 - __clz(__ballot_sync(0xffffffffu, before <= row));
    first = __shfl_sync(0xffffffffu, before, owner);
    int g = owner * each;
#pragma unroll 1
    for (;; ++g) {
      const int n = of(p.cuts[g]);
      if (row < first + n) return g;
      first += n;
    }
  }
};

template <int kT>
struct MergeItem {
  int row0, kv, col;  // first node of the group, KV head, row of the group
  float m, l;
  float4 o[kT];
};

// acc + w * v, where w is 0 only what of v is not finite.
__device__ __forceinline__ float4 add_weighed(float4 acc, float w, float4 v) {
  if (w == 0.f) {
    const auto kept = [](float x) { return fabsf(x) < INFINITY ? 0.f : x; };
    return make_float4(acc.x + kept(v.x), acc.y + kept(v.y), acc.z + kept(v.z), acc.w + kept(v.w));
  }
  return make_float4(acc.x + w * v.x, acc.y + w * v.y, acc.z + w * v.z, acc.w + w * v.w);
}

// Partials member, member + team, .. of a row, kT * 128 dims from tile0 * 128 on, four a lane.
template <typename C, int kT>
__device__ __forceinline__ MergeItem<kT> merge_partials(const MergeParams& mp, const CutRows<C>& rows, int row, int tile0,
                                                        int member, int team) {
  constexpr int kFly = kMergeInFlight / kT;
  const TreeParams& p = mp.t;
  const int lane = threadIdx.x & 31;
  int first;
  const int lo = rows.find(p, row, first);
  const int4 cut = p.cuts[lo];
  MergeItem<kT> it;
  it.row0 = cut.x;
  it.kv = cut.y >> 8;
  it.col = row - first;
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
      const size_t at = static_cast<size_t>(i == 0 ? cut.z : 2 * (lo + i * C::kHkv)) * C::kN + it.col;
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
    for (int t = 0; t < kT; ++t) it.o[t] = add_weighed(make_float4(0.f, 0.f, 0.f, 0.f), f, it.o[t]);
#pragma unroll
    for (int u = 0; u < kFly; ++u) {
      if (!(e[u].y > 0.f)) continue;
      const float w = exp2f(e[u].x - m);
      it.l += w * e[u].y;
#pragma unroll
      for (int t = 0; t < kT; ++t) it.o[t] = add_weighed(it.o[t], w, a[u][t]);
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
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
  __shared__ float4 s_o[kMergeWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_primary_grid();
  allow_dependent_launch();
  const CutRows<C> rows(p, mp.grid);
  const int carry = rows.total;
  // An item is 128 dims of a row, a block's, or a row, a warp's: whichever waits less, in units of a load's latency.  A
  // block's first takes some six and a load for every 32 partials (they meet in shared memory), a warp's one and a bit
  // more for every kMergeInFlight / kTiles.  us a call, by blocks and by warps: 4 short sliding trees (8 partials a row)
  // 15.3 and 13.7, a global tree of 4 nodes (15) 13.8 and 16.2, of 8 behind 30000 positions (76) 31 and 70, four of these
  // (19, three items a block) 66 and 73, 8 of 4 nodes (13, three) 20.8 and 20.9, 32 of 64 nodes 643 and 596.
  constexpr int kFly = kMergeInFlight / C::kTiles;
  const float blocks = static_cast<float>(gridDim.x), most = static_cast<float>(rows.most);
  const float by_block = 4.f + ceilf(__fdividef(carry * C::kTiles, blocks)) * (2.f + most * (1.f / (8 * kMergeWarps)));
  const float by_warp = ceilf(__fdividef(carry, kMergeWarps * blocks)) * (1.f + 1.2f * ceilf(most * (1.f / kFly)));
  if (by_block < by_warp) {
    for (int item = blockIdx.x; item < carry * C::kTiles; item += gridDim.x) {
      const MergeItem<1> it = merge_partials<C, 1>(mp, rows, item / C::kTiles, item % C::kTiles, warp, kMergeWarps);
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
          all.l += f * s_l[w];
          O = add_weighed(O, f, s_o[w][lane]);
        }
        all.o[0] = O;
        store_merged<C, 1>(p, all, item % C::kTiles);
      }
      __syncthreads();  // the shared partials were read
    }
  } else {
    for (int row = blockIdx.x * kMergeWarps + warp; row < carry; row += gridDim.x * kMergeWarps)
      store_merged<C, C::kTiles>(p, merge_partials<C, C::kTiles>(mp, rows, row, 0, 0, 1), 0);
  }
}

}  // namespace tree
}  // namespace pda
