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
// Weights are rounded to bf16 (half a step, 2^-8 of each) because P^T is an operand of the tensor cores, as in the bf16
// decode and prefill: outputs are 0.0024 off the 64-bit result (relative, root mean square) where bf16 outputs of exact
// weights are 0.0017.  The sums add them unrounded: summed as rounded, single outputs were off by up to 1.25 times the
// bound that the tests derive.
//
// What bounds it (GB300, 2070 MHz; copy rate 6784 GB/s).  Long contexts HBM where a tree has one group: 16 trees of 4
// nodes behind 131072 positions 632 us, the copy rate; with two groups all keys go to both: 16 of 8 nodes 765 to 781, 0.82
// of it, 73 KB a us into every SM with 128 KB in flight.  Many nodes on global layers shared memory: per 128 keys and four nodes 256 KB of K and V are
// written and read as A, 128 KB read as B, 5120 clocks at 128 bytes each: 32 trees of 64 nodes behind 4000 to 8192 take
// 596 us, 7200 clocks a step, 675 TFLOP/s.  (Pairs of CTAs on one product, cta_group::2 with 128 rows and rings of 120
// KB, read A once for both and took 790 us: too little in flight.  Pages brought into L2 ahead of the copies: 600 -> 656,
// 771 -> 863.)  Sliding windows the softmax's chain of a step and the ends of segments: 64 trees of 17 to 45 nodes 120
// us, 0.72 of the copy rate; 200 of 5 nodes 269, 0.95.  One short call latency: 4 nodes behind 900 positions 13.7.
//
// Roles: warps 0-7 softmax and epilogue, 8 copies Q and K, 9 copies V, 10 issues S^T,
// 11 issues O^T.  Every wait is bounded.
#pragma once

#include "tree_common.cuh"

namespace pda {
namespace tree {

template <int kD_, int kG_, int kHkv_, int kN_, int kPBufs_, int kKStages_, int kVStages_>
struct Config {
  static constexpr int kD = kD_, kG = kG_, kHkv = kHkv_, kHq = kG * kHkv;
  static constexpr int kN = kN_;               // rows per group, at most
  static constexpr int kHalf = kN / 2;         // columns per softmax warpgroup
  static constexpr int kBlock = kHalf < 32 ? kHalf : 32;  // columns at a time
  static constexpr int kQueries = kN / kG;     // nodes of a group
  static constexpr int kKeys = 128;             // per step
  static constexpr int kStepPages = kKeys / kPage;
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

  struct Smem {
    alignas(1024) uint8_t q[kChunks][kN * 128];
    alignas(1024) uint8_t p[kPBufs][kPBytes];
    alignas(1024) uint8_t k[kKStages][kKChunk];
    alignas(1024) uint8_t v[kVStages][kVPage];
    alignas(16) float neg_m[kN];      // minus the reference max (log2 units), 0 before there is one
    alignas(16) float bound[kN];      // a score above this moves it; -inf before there is one
    alignas(16) float f[kN];          // first scores; factor of a moved reference; 1 / sum at the end
    alignas(16) float red[8][kN / 2]; // per softmax warp and column: max, sum
    Shared sh;
    Masks masks[2];                   // of the segment at hand, and of the next
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

template <typename C>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TreeParams p) {
  using prefill_tc::kHeadroom;
  using prefill_tc::kSlack;
  using prefill_tc::tma_load_4d;
  constexpr int kG = C::kG, kN = C::kN, kHalf = C::kHalf, kTiles = C::kTiles, kBlock = C::kBlock;
  constexpr int kPBufs = C::kPBufs, kKeys = C::kKeys, kStepPages = C::kStepPages;
  extern __shared__ uint8_t smem_raw[];
  typename C::Smem& s =
      *reinterpret_cast<typename C::Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_empty[i], 1);
    }
#pragma unroll 1
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&s.v_full[i], 1);
      mbar_init(&s.v_empty[i], 1);
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
  if (warp == 0) {
    read_lengths<false>(p, s.sh);
    make_schedule<C>(p, s.sh, false);
  }
  // q, the cache and the tables may be written by the previous kernel in the stream.
  wait_for_primary_grid();
  allow_dependent_launch();
  if (warp == 0) {
    if (read_lengths<true>(p, s.sh))
      make_schedule<C>(p, s.sh, true);
    else if (s.sh.misfit && blockIdx.x == 0 && lane == 0)
      report(p.status, ATTN_DEV_BAD_SEQ_LEN);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s.tmem_base;
  const bool run = s.sh.refused == 0;
  if (!run) {
    if (threadIdx.x == 0 && !p.whole) p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
  } else if (warp == 8) {
    // ---------------- Q and K producer: lane i < 8 copies page i of a step, chunk by chunk ----------------
    bool ok = true;
    int gt = 0, gk = 0, st = 0, st_ph = 1;  // segments, K chunks; stage and its phase
    Walk<C> walk;
    walk.start(p, s.sh);
    Segment g;
#pragma unroll 1
    while (ok && walk.next(p, s.sh, g)) {
      if (gt >= 1) ok = __all_sync(0xffffffffu, wait_for(&s.q_empty, (gt - 1) & 1));
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&s.q_ready, C::kChunks * p.q_box * kG * 128);
      __syncwarp();
      if (lane < C::kChunks) tma_load_4d(s.q[lane], &tm_q, 0, lane, walk.kv * kG, g.row0, &s.q_ready);
      ++gt;
      const int32_t* table = p.block_table + static_cast<int64_t>(g.b) * p.max_blocks + g.q.page0;
      const auto entry = [&](int pg) { return lane < kStepPages && pg + lane < g.p1 ? table[pg + lane] : 0; };
      int next_id = entry(g.p0);
#pragma unroll 1
      for (int pg = g.p0; pg < g.p1 && ok; pg += kStepPages) {
        const int id = next_id;
        next_id = entry(pg + kStepPages);
        const int np = min(kStepPages, g.p1 - pg);
        int32_t y = id * kPage;
        if (lane < np && (id < 0 || static_cast<int64_t>(id) >= p.num_pages)) {
          report(p.status, ATTN_DEV_BAD_PAGE);
          y = -kPage;
        }
#pragma unroll 1
        for (int ch = 0; ch < C::kChunks; ++ch) {
          if (gk >= C::kKStages) ok = __all_sync(0xffffffffu, wait_for(&s.k_empty[st], st_ph));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&s.k_full[st], np * kPage * 128);
          __syncwarp();
          if (lane < np)
            prefill_tc::tma_load_3d(s.k[st] + lane * (kPage * 128), &tm_k, 0, y, walk.kv * C::kChunks + ch, &s.k_full[st]);
          ++gk;
          if (++st == C::kKStages) st = 0, st_ph ^= 1;
          __syncwarp();
        }
      }
    }
    if (!ok && lane == 0) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
    if (lane == 0) {  // no copy may still be landing, nor a commit arriving, when the CTA retires
      if (gt >= 1) {
        if (!wait_for(&s.q_ready, (gt - 1) & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
        if (ok && !wait_for(&s.q_empty, (gt - 1) & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
      }
#pragma unroll 1
      for (int i = 0; i < C::kKStages && i < gk; ++i) {
        const int uses = (gk - 1 - i) / C::kKStages;
        if (!wait_for(&s.k_full[i], uses & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
        if (ok && !wait_for(&s.k_empty[i], uses & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
      }
    }
  } else if (warp == 9) {
    // ---------------- V producer: a page per stage ----------------
    bool ok = true;
    int gv = 0, st = 0, st_ph = 1;
    Walk<C> walk;
    walk.start(p, s.sh);
    Segment g;
#pragma unroll 1
    while (ok && walk.next(p, s.sh, g)) {
      const int32_t* table = p.block_table + static_cast<int64_t>(g.b) * p.max_blocks + g.q.page0;
      const auto entry = [&](int pg) { return pg < g.p1 ? table[pg] : 0; };
      int cur = 0, nxt = entry(g.p0 + lane);
#pragma unroll 1
      for (int pg = g.p0; pg < g.p1 && ok; ++pg) {
        const int u = (pg - g.p0) & 31;
        if (u == 0) {
          cur = nxt;
          nxt = entry(pg + 32 + lane);
        }
        const int id = __shfl_sync(0xffffffffu, cur, u);
        if (gv >= C::kVStages) ok = __all_sync(0xffffffffu, wait_for(&s.v_empty[st], st_ph));
        if (!ok) break;
        if (lane == 0) {
          const bool there = id >= 0 && static_cast<int64_t>(id) < p.num_pages;  // (the K producer reports)
          mbar_arrive_expect_tx(&s.v_full[st], C::kVPage);
          prefill_tc::tma_load_3d(s.v[st], &tm_v, 0, there ? id * kPage : -kPage, walk.kv * C::kChunks, &s.v_full[st]);
        }
        ++gv;
        if (++st == C::kVStages) st = 0, st_ph ^= 1;
        __syncwarp();
      }
    }
    if (!ok && lane == 0) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
    if (lane == 0) {
#pragma unroll 1
      for (int i = 0; i < C::kVStages && i < gv; ++i) {
        const int uses = (gv - 1 - i) / C::kVStages;
        if (!wait_for(&s.v_full[i], uses & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
        if (ok && !wait_for(&s.v_empty[i], uses & 1)) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
      }
    }
  } else if (warp == 10) {
    // ---------------- S^T issuer (whole warp; an elected lane issues) ----------------
    bool ok = true;
    int gt = 0, gs = 0, st = 0, st_ph = 0;
    const uint32_t q_base = smem_addr(s.q[0]);
    Walk<C> walk;
    walk.start(p, s.sh);
    Segment g;
#pragma unroll 1
    while (walk.next(p, s.sh, g)) {
      if (ok) ok = __all_sync(0xffffffffu, wait_for(&s.q_ready, gt & 1));
      const uint32_t idesc = prefill_tc::warp_uniform_int(umma_idesc_bf16(128, g.N, 0, 0));
      const int steps = prefill_tc::warp_uniform_int(g.steps);
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        const int sb = gs & 1;
        if (ok && gs >= 2) ok = __all_sync(0xffffffffu, wait_for(&s.s_free[sb], ((gs >> 1) - 1) & 1));
        const uint32_t d = tmem + C::kSCol + sb * kN;
#pragma unroll 1
        for (int ch = 0; ch < C::kChunks; ++ch) {
          if (ok) ok = __all_sync(0xffffffffu, wait_for(&s.k_full[st], st_ph));
          tc_fence_after_sync();
          const uint32_t k_base = smem_addr(s.k[st]);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_warp(d, umma_desc(k_base + kk * 32, 16, 1024, 2),
                           umma_desc(q_base + ch * (kN * 128) + kk * 32, 16, 1024, 2), idesc, (ch | kk) > 0 ? 1u : 0u);
          umma_commit_warp(&s.k_empty[st]);
          if (++st == C::kKStages) st = 0, st_ph ^= 1;
        }
        umma_commit_warp(&s.s_full[sb]);
        ++gs;
      }
      umma_commit_warp(&s.q_empty);
      ++gt;
    }
    // the softmax warps' last arrivals on s_free (not waited for above)
#pragma unroll 1
    for (int k = gs >= 2 ? gs - 2 : 0; k < gs; ++k)
      if (ok) ok = __all_sync(0xffffffffu, wait_for(&s.s_free[k & 1], (k >> 1) & 1));
    umma_commit_warp(&s.mma_done);
    if (!__all_sync(0xffffffffu, wait_for(&s.mma_done, 0))) ok = false;  // every product done before the memory is freed
    if (!ok && lane == 0) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
  } else if (warp == 11) {
    // ---------------- O^T issuer; it also cleans the rows of V that not every node sees ----------------
    if (lane == 0 && !p.whole) note_cut<C>(p, s.sh);
    __syncwarp();
    bool ok = true;
    int gt = 0, gs = 0, st = 0, st_ph = 0;
    Walk<C> walk;
    walk.start(p, s.sh);
    Segment g;
#pragma unroll 1
    while (walk.next(p, s.sh, g)) {
      if (ok && gt >= 1) ok = __all_sync(0xffffffffu, wait_for(&s.o_free, (gt - 1) & 1));
      const uint32_t idesc = prefill_tc::warp_uniform_int(umma_idesc_bf16(128, g.N, 1, 1));
      bool poison = false;
      const int all0 = all_from(g.q, p.window);
#pragma unroll 1
      for (int pg0 = g.p0; pg0 < g.p1; pg0 += kStepPages) {
        const int pb = gs % kPBufs;
        const int np = prefill_tc::warp_uniform_int(min(kStepPages, g.p1 - pg0));
        const uint32_t p_base = smem_addr(s.p[pb]);
#pragma unroll 1
        for (int kk = 0; kk < np; ++kk) {
          if (ok) ok = __all_sync(0xffffffffu, wait_for(&s.v_full[st], st_ph));
          const uint32_t v_base = smem_addr(s.v[st]);
          const int pos0 = (g.q.page0 + pg0 + kk) * kPage;
          if (ok && (pos0 < all0 || pos0 + kPage > g.q.ctx)) {  // (lo <= all0)
            const uint32_t none = row_bits(0, g.q.lo - pos0) | row_bits(g.q.L - pos0, kPage);
            const uint32_t some = (row_bits(0, all0 - pos0) | row_bits(g.q.ctx - pos0, kPage)) & ~none;
            poison |= clean_page<C>(v_base + (lane >> 3) * (kPage * 128) + (lane & 7) * 16, none, some);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (kk == 0 && ok) ok = __all_sync(0xffffffffu, wait_for(&s.p_full[pb], (gs / kPBufs) & 1));
          tc_fence_after_sync();
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
            umma_bf16_warp(tmem + t * kN, umma_desc(v_base + t * (2 * kPage * 128), kPage * 128, 1024, 2),
                           umma_desc(p_base + kk * (kPage * 128), C::kPChunk, 1024, 2), idesc,
                           (pg0 > g.p0 || kk > 0) ? 1u : 0u);
          umma_commit_warp(&s.v_empty[st]);
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
    if (ok && gt >= 1) ok = __all_sync(0xffffffffu, wait_for(&s.o_free, (gt - 1) & 1));
    umma_commit_warp(&s.mma_done);
    if (!__all_sync(0xffffffffu, wait_for(&s.mma_done, 0))) ok = false;
    if (!ok && lane == 0) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
  } else {
    // ---------------- softmax and epilogue: thread = key of the step, then dim of a tile ----------------
    const int h = warp >> 2;             // half of the columns
    const int hb = h * kHalf;            // their first place in neg_m, bound and f, whatever the segment
    const int key = threadIdx.x & 127;   // tensor-memory lane, thread of the warpgroup
    const uint32_t bar = 2 + h;
    const uint32_t t_row = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float2 log2e2 = make_float2(kLog2e, kLog2e);
    bool ok = true;
    int gt = 0, gs = 0;
    Walk<C> walk;
    walk.start(p, s.sh);
    Segment g, ahead{};
    int parent[2] = {-1, -1};  // of the next segment, which is read and whose masks are made before this one's end
    // (the masks are there where a segment holds positions that not all nodes see)
    const auto prepare_masks = [&](int buf) {
      if ((ahead.q.page0 + ahead.p0) * kPage < all_from(ahead.q, p.window) ||
          (ahead.q.page0 + ahead.p1) * kPage > ahead.q.ctx)
        make_masks(s.masks[buf], p.status, ahead.q.n, parent[0], parent[1]);
    };
    // the references of this warpgroup's columns, by the threads that have one each
    const auto reset_references = [&] {
      const int half = ahead.N >> 1;
      if (key < half) {
        s.neg_m[hb + key] = 0.f;
        s.bound[hb + key] = -INFINITY;
      }
    };
    bool more = walk.next(p, s.sh, ahead);
    if (more) {
      read_parents(p.parents + ahead.q.q0, ahead.q.n, parent);
      prepare_masks(0);
      reset_references();
    }
#pragma unroll 1
    while (more) {
      g = ahead;
      const int half = g.N >> 1;
      const int c0 = h * half;  // this warpgroup's first column
      const int all0 = all_from(g.q, p.window);
      const int node0 = walk.group * C::kQueries;
      const int seg0 = (g.q.page0 + g.p0) * kPage, seg1 = (g.q.page0 + g.p1) * kPage;
      const Masks& masks = s.masks[gt & 1];
      named_barrier_sync(1, kSoftmaxThreads);  // the masks and references are there
      float l[kHalf];
#pragma unroll
      for (int c = 0; c < kHalf; ++c) l[c] = 0.f;

#pragma unroll 1
      for (int j = 0; j < g.steps; ++j) {
        const int sb = gs & 1, pb = gs % kPBufs;
        const int step0 = seg0 + j * kKeys;
        const bool masked = step0 < all0 || step0 + kKeys > min(g.q.ctx, seg1);
        unsigned long long vis = 0;
        if (masked && step0 + key < seg1) vis = seen_by(g.q, p.window, masks, step0 + key) >> node0;
        if (ok) ok = __all_sync(0xffffffffu, wait_for(&s.s_full[sb], (gs >> 1) & 1));
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
          if (j == 0 && max(step0, all0) < min(min(g.q.ctx, seg1), step0 + kKeys)) {
            // first references: the scores of a key that every node sees
            if (step0 + key == max(step0, all0)) {
#pragma unroll
              for (int c4 = 0; c4 < kBlock / 4; ++c4)
                if (blk + 4 * c4 < half)
                  *reinterpret_cast<float4*>(&s.f[hb + blk + 4 * c4]) =
                      make_float4(sv[4 * c4], sv[4 * c4 + 1], sv[4 * c4 + 2], sv[4 * c4 + 3]);
            }
            named_barrier_sync(bar, 128);
            if (key < kBlock && blk + key < half) {
              const float x = s.f[hb + blk + key];
              if (fabsf(x) < INFINITY) {
                const float m = fmaf(x, kLog2e, kHeadroom);
                s.neg_m[hb + blk + key] = -m;
                s.bound[hb + blk + key] = (m + kSlack) * (1.f / kLog2e);
              }
            }
            named_barrier_sync(bar, 128);
          }
          bool moves = false;
#pragma unroll
          for (int c4 = 0; c4 < kBlock / 4; ++c4) {
            if (blk + 4 * c4 < half) {
              const float4 t = *reinterpret_cast<const float4*>(&s.bound[hb + blk + 4 * c4]);
              moves |= (sv[4 * c4] > t.x) | (sv[4 * c4 + 1] > t.y) | (sv[4 * c4 + 2] > t.z) | (sv[4 * c4 + 3] > t.w);
            }
          }
          if (barrier_or(bar, 128, moves)) {
            float* const red = s.red[warp] + blk;
            max_into<kBlock>(sv, red);
            named_barrier_sync(bar, 128);
            if (key < kBlock && blk + key < half) {
              const int w0 = h * 4, c = blk + key, col = hb + c;
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
              if (blk + c < half) l[blk + c] *= s.f[hb + blk + c];
            if (j > 0) {
              // O^T holds the products up to step j - 1: wait for the last, then scale in place
              if (ok) ok = __all_sync(0xffffffffu, wait_for(&s.p_empty[(gs - 1) % kPBufs], ((gs - 1) / kPBufs) & 1));
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
                  for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(ov[e] * s.f[hb + blk + c + e]);
                  tmem_st8(t_row + t * kN + cb + c, w);
                }
              }
              tmem_wait_st();
            }
          }
          // weights; the buffer's last reader was the product of step j - kPBufs
          if (blk == 0 && ok && gs >= kPBufs)
            ok = __all_sync(0xffffffffu, wait_for(&s.p_empty[pb], (gs / kPBufs - 1) & 1));
#pragma unroll
          for (int b8 = 0; b8 < kBlock / 8; ++b8) {
            if (blk + 8 * b8 < half) {
              float2 w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 m = *reinterpret_cast<const float2*>(&s.neg_m[hb + blk + 8 * b8 + 2 * e]);
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

      more = walk.next(p, s.sh, ahead);
      if (more) read_parents(p.parents + ahead.q.q0, ahead.q.n, parent);
      // ---- end of the segment: sums, then this thread's dim of every row ----
      reduce_into<kHalf>(l, half, s.red[warp], [](float a, float b) { return a + b; });
      named_barrier_sync(bar, 128);
      if (key < half) {
        const int w0 = h * 4, col = c0 + key;
        const float sum = (s.red[w0][key] + s.red[w0 + 1][key]) + (s.red[w0 + 2][key] + s.red[w0 + 3][key]);
        s.f[hb + key] = !g.whole ? 1.f : sum > 0.f ? 1.f / sum : sum;  // 0: a row that sees nothing; NaN stays
        if (!g.whole && col < g.cols)
          p.part_ml[static_cast<size_t>(g.slot) * kN + col] = partial_stats(-s.neg_m[hb + key], sum);
      }
      named_barrier_sync(bar, 128);
      if (more) prepare_masks((gt + 1) & 1);  // (while the last products run)
      if (ok) ok = __all_sync(0xffffffffu, wait_for(&s.o_full, gt & 1));
      tc_fence_after_sync();
      const int to = min(c0 + half, g.cols);
      store_columns<C>(p, g, walk.kv, c0, to, t_row, s.f + hb - c0);
      if (s.poison != 0) {
        __syncwarp();  // (a lane's elements were stored by its neighbour)
        const Segment same = g;  // (g itself stays in registers: no address of it is taken)
        add_back<C>(p, masks, same, walk.kv, node0, c0, to);
      }
      tc_fence_before_sync();
      __syncwarp();
      if (more) reset_references();  // (read by no other thread since the sums)
      if (lane == 0) mbar_arrive(&s.o_free);  // the next segment's first product may overwrite O^T
      ++gt;
    }
    // the last products' commits (not all waited for above)
#pragma unroll 1
    for (int k = gs >= kPBufs ? gs - kPBufs : 0; k < gs; ++k)
      if (ok) ok = __all_sync(0xffffffffu, wait_for(&s.p_empty[k % kPBufs], (k / kPBufs) & 1));
    if (!ok && lane == 0) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
  }

  // ---------------- teardown: free the tensor memory ----------------
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// D = 512: 64 rows, four nodes; D = 256: 128, 64 or 32 rows, the fewer the longer the rings.  Buffers
// share 227 KB.  P^T twice where a step's products on V are short of its softmax; us for 64 sliding trees of 17 to 45 nodes
// (128 rows), P^T buffers / K stages / V stages: 2/3/5 120.6, 2/2/7 128.6, 1/3/9 122.3, 1/4/7 123.8, 1/5/5 131.7; for 64
// of 26 nodes (64 rows): 2/5/8 109.0, 2/4/10 107.9, 1/5/10 107.8, 2/6/6 111.4.
using GlobalConfig = Config<ATTN_GLOBAL_D, ATTN_GLOBAL_HQ / ATTN_GLOBAL_HKV, ATTN_GLOBAL_HKV, 64, 1, 4, 4>;
template <int kN, int kKStages, int kVStages>
using SlidingConfig =
    Config<ATTN_SLIDING_D, ATTN_SLIDING_HQ / ATTN_SLIDING_HKV, ATTN_SLIDING_HKV, kN, 2, kKStages, kVStages>;
using SlidingWide = SlidingConfig<128, 3, 5>;
using SlidingMid = SlidingConfig<64, 5, 8>;
using SlidingNarrow = SlidingConfig<32, 6, 8>;

}  // namespace tree
}  // namespace pda
