// pages.cuh -- the block tables of a step from its requests' lengths
// (attn_pages_assign).
//
// Request b holds logical pages [hf, he) and needs [f, e) (f from the window,
// e from its length): it gives back what lies in the first range only, a part in
// front and a part behind, and takes what lies in the second only.  The running
// sums of both counts over the requests say which entry of the free ring each page
// is: the i-th page given back goes to entry head + count + i, the i-th page taken
// comes from entry head + i.  Both parts of the ring are disjoint, and so are the table entries read
// (given back) and written (taken), so the pages move in any order.
//
// One cluster of kBlocks blocks: every block reads the state and works the sums
// out for itself (at most 256 requests, a thread each), the pages are dealt out
// over all threads, and the cluster's barrier stands between the last read of the
// old state and the first write of the new one, which may lie in its place.  Bound
// by latency: lengths, sums, one entry, one store; 64 requests of a step 4.6 us (7 from
// Python), 200 of which many come and go, 131072 pages, 10.4 (16.2 with 4 blocks, 48.5 with
// one).
#pragma once

#include "attn_tree.h"
#include "common.cuh"
#include "tcgen05.cuh"

namespace pda {
namespace pages {

constexpr int kBlocks = 8;     // a portable cluster
constexpr int kThreads = 1024;  // the first kMaxBatch take a request each
constexpr int kInFlight = 4;    // pages of a thread on their way
static_assert(kThreads >= kMaxBatch, "a thread per request");

struct PagesParams {
  const int32_t* cached;
  const int32_t* fresh;
  int32_t* block_table;
  const int2* held;
  int32_t* free_list;
  const int2* free_state;
  int2* held_out;
  int2* free_state_out;
  int32_t* seq_lens;
  int32_t* cu_q;
  int32_t* status;
  int32_t num_pages;
  int32_t batch;
  int32_t max_blocks;
  int32_t window;
};

struct Smem {
  int32_t give[kMaxBatch + 1], take[kMaxBatch + 1];  // running sums
  int3 give_part[kMaxBatch], take_part[kMaxBatch];   // first page in front, how many there, first page behind
  int32_t warp_sum[3][kMaxBatch / 32];
};

// Moves `total` pages, numbered by the running sum over the requests' parts: move(i, entry) gets the i-th one's place in
// the block table and returns where to read it and where it goes.  A warp takes kInFlight * 32 consecutive ones at a
// time, looks the first one's request up and walks on from there, and reads all before it writes any.
template <typename Move>
__device__ __forceinline__ void move_pages(const int32_t* sum, const int3* parts, const PagesParams& p, int total, int warp,
                                           Move move) {
  constexpr int kRun = kInFlight * 32;
  const int lane = threadIdx.x & 31;
  for (int base = warp * kRun; base < total; base += kBlocks * (kThreads / 32) * kRun) {
    int lo = 0, hi = p.batch - 1;  // the request whose part of the sum holds base (sum[batch] > base)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sum[mid] <= base) lo = mid; else hi = mid - 1;
    }
    int32_t page[kInFlight];
    int32_t* to[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int i = base + 32 * u + lane;
      to[u] = nullptr;
      if (i < total) {
        while (sum[lo + 1] <= i) ++lo;
        const int k = i - sum[lo];
        const int3 part = parts[lo];
        const int32_t* from;
        move(i, static_cast<int64_t>(lo) * p.max_blocks + (k < part.y ? part.x + k : part.z + (k - part.y)), from, to[u]);
        page[u] = *from;
      }
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (to[u] != nullptr) *to[u] = page[u];
  }
}

__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kThreads) assign_kernel(const __grid_constant__ PagesParams p) {
  __shared__ Smem s;
  const int tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  wait_for_primary_grid();
  allow_dependent_launch();

  const int cap = p.max_blocks < ATTN_MAX_SEQ_LEN / kPage ? p.max_blocks * kPage : ATTN_MAX_SEQ_LEN;
  const int2 ring = *p.free_state;  // head, count
  int cached = 0, fresh = 0, f = 0, e = 0, give = 0, take = 0;
  int2 old = make_int2(0, 0);
  bool bad = ring.x < 0 || ring.x >= p.num_pages || ring.y < 0 || ring.y > p.num_pages;
  if (tid < p.batch) {
    cached = p.cached[tid];
    fresh = p.fresh[tid];
    old = p.held[tid];
    if (cached < 0 || fresh < 0 || cached > cap || fresh > cap - cached || old.x < 0 || old.y < old.x ||
        old.y > cap / kPage) {
      bad = true;
      fresh = 0;
    } else {
      f = p.window > 0 && cached >= p.window ? (cached - p.window + 1) / kPage : 0;
      e = max(f, (cached + fresh + kPage - 1) / kPage);
      const int hf = old.x < old.y ? old.x : f, he = old.x < old.y ? old.y : f;
      bad |= f < hf && cached > 0;  // it needs what it gave back
      const int give_low = max(0, min(f, he) - hf), give_hi = max(hf, min(e, he));
      const int take_low = max(0, min(hf, e) - f), take_hi = max(he, f);
      s.give_part[tid] = make_int3(hf, give_low, give_hi);
      s.take_part[tid] = make_int3(f, take_low, take_hi);
      give = give_low + he - give_hi;
      take = take_low + max(0, e - take_hi);
    }
  }
  // running sums over the requests
  int give_sum = give, take_sum = take, fresh_sum = fresh;
  if (tid < kMaxBatch) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, give_sum, o), b = __shfl_up_sync(0xffffffffu, take_sum, o),
                c = __shfl_up_sync(0xffffffffu, fresh_sum, o);
      if (lane >= o) {
        give_sum += a;
        take_sum += b;
        fresh_sum += c;
      }
    }
    if (lane == 31) {
      s.warp_sum[0][warp] = give_sum;
      s.warp_sum[1][warp] = take_sum;
      s.warp_sum[2][warp] = fresh_sum;
    }
  }
  const bool misfit = __syncthreads_or(bad);
  int total_give = 0, total_take = 0;
#pragma unroll
  for (int w = 0; w < kMaxBatch / 32; ++w) {
    if (w < warp) {
      give_sum += s.warp_sum[0][w];
      take_sum += s.warp_sum[1][w];
      fresh_sum += s.warp_sum[2][w];
    }
    total_give += s.warp_sum[0][w];
    total_take += s.warp_sum[1][w];
  }
  if (tid < p.batch) {
    s.give[tid + 1] = give_sum;
    s.take[tid + 1] = take_sum;
  }
  if (tid == 0) s.give[0] = s.take[0] = 0;
  // (given back more than the ring has room for: held says what the free list denies)
  const bool overfull = total_give > p.num_pages - ring.y;
  const bool no_pages = !misfit && !overfull && total_take > ring.y;
  const bool refused = misfit || overfull || no_pages;
  __syncthreads();
  const uint32_t rank = cluster_ctarank();

  if (!refused) {
    const int mine = static_cast<int>(rank) * (kThreads / 32) + warp;
    move_pages(s.take, s.take_part, p, total_take, mine, [&](int i, int64_t entry, const int32_t*& from, int32_t*& to) {
      from = p.free_list + (ring.x + i < p.num_pages ? ring.x + i : ring.x + i - p.num_pages);  // i < count <= num_pages
      to = p.block_table + entry;
    });
    move_pages(s.give, s.give_part, p, total_give, mine, [&](int i, int64_t entry, const int32_t*& from, int32_t*& to) {
      // head < num_pages, count + i < num_pages: at most once round
      const int room = p.num_pages - (ring.y + i);
      from = p.block_table + entry;
      to = p.free_list + (ring.x < room ? ring.x + ring.y + i : ring.x - room);
    });
  }
  // every block has read the old state before any of it is written
  cluster_sync_all();
  if (rank != 0) return;
  if (tid < p.batch) {
    p.held_out[tid] = refused ? old : make_int2(f, e);
    p.seq_lens[tid] = refused ? max(0, min(cached, cap)) : cached + fresh;
    p.cu_q[tid + 1] = refused ? 0 : fresh_sum;
  }
  if (tid == 0) {
    p.cu_q[0] = 0;
    *p.free_state_out = refused ? ring : make_int2(static_cast<int>((static_cast<int64_t>(ring.x) + total_take) % p.num_pages),
                                                   ring.y - total_take + total_give);
    if (refused) report(p.status, no_pages ? ATTN_DEV_NO_PAGES : ATTN_DEV_BAD_SEQ_LEN);
  }
}

}  // namespace pages
}  // namespace pda
