// prefix.cuh -- decodeGQA for a batch that shares a prefix: sequence b sees
// the prefix's positions (one page list for all) and then its own.
//
//   o[b,h] = sum over prefix and own positions l of softmax_l(<q[b,h], k_l>) v_l
//
// The softmax over the union is regrouped exactly from partial results (O, m,
// sum) as in combine.cuh; sums, maxima and partial outputs are fp32.  The weights
// are rounded to bf16 for their product with the values, here and in joined.cuh,
// because the tensor cores take two operands of one type and the values are bf16
// (in f16 one outside 2^-14 .. 2^16 would lose bits); a second product for the
// rest of the weights would double the time of P V.  64 sequences behind 32768
// positions: 0.0023 off the 64-bit result (2-norm, bf16 outputs), where unrounded
// weights leave 0.0017, the rounding of the outputs alone.
//
// Three kernels (short prefixes and small batches take joined.cuh's way):
//   * the prefix as a multi-query attention whose queries are the batch's
//     sequences (prefill_pair.cuh with PrefixParams): its pages are read once
//     for 16 sequences x 16 heads instead of once per sequence, and the
//     products run on tcgen05, 2048 flops x batch per byte pair;
//   * the sequences' own positions with the decode kernel (global.cuh), every
//     segment left as a partial;
//   * this merge, which also serves the 8-bit global decode (no prefix, and the
//     rows that one block finished whole are left alone).
//
// A block takes kDims dims of row b*Hq + h, a row's partials being its prefix
// spans followed by its blocks of the balanced schedule: groups of kDims / 4
// threads, four dims a thread, group i takes partials i, i + kMergeGroups, ..
// with kInFlight loads in flight, and the groups meet in shared memory.  Bound
// by latency: the schedule is worked out before the block waits for the kernels
// ahead of it.  With a prefix one block takes a row, in four groups where the
// rows' blocks are resident at once (16 sequences, 16384 positions: a call takes
// 35.4 us; with four blocks of four groups 39.5), in two where they come in
// waves (64 sequences, 15 partials: 127.5 us, with four groups 131.4; 119 since the
// own positions' kernel no longer waits for the prefix kernel).
#pragma once

#include "combine.cuh"
#include "prefill_pair.cuh"

namespace pda {
namespace prefix {

// The own positions' call.  Weight of a sequence's start 1 and 4, us: 32 sequences
// of up to 2000 behind 16384 56.2 and 53.8, 64 of up to 1000 behind 500 36.8 and 35.1.
struct OwnParams : DecodeParams {
  static constexpr int kSeqWeight = 4;
};

template <typename Params>
struct MergeParams {
  Params d;                  // the own positions' call: schedule, partials, output
  const float* part_o;       // prefix partials (PrefixParams)
  const float2* part_ml;
  const int32_t* prefix_len;
  int32_t prefix_blocks;
  int32_t splits;
};

// kPrefixSlices: slices of the output dims the prefix partials' (max, sum) come
// in; 0 for no prefix.
template <int kD, int kPrefixSlices, int kStepPages, int kDims, int kMergeGroups, typename Params>
__global__ void __launch_bounds__(kMergeGroups* kDims / 4) merge_kernel(const __grid_constant__ MergeParams<Params> mp) {
  const Params& p = mp.d;
  constexpr int kGroupThreads = kDims / 4;  // four dims per thread
  constexpr int kBlocks = kD / kDims;       // per row
  constexpr int kInFlight = kBlocks > 1 ? 8 : 4;  // partials in flight per thread
  constexpr int kSched = 128;  // threads that work out the schedule
  static_assert(kMergeGroups * kGroupThreads >= kSched, "they must exist");
  __shared__ int s_sched[kSched / 32][3];
  __shared__ float s_m[kMergeGroups][kGroupThreads];  // per thread: the two dim slices differ
  __shared__ float s_l[kMergeGroups][kGroupThreads];
  __shared__ float4 s_o[kMergeGroups][kGroupThreads];

  const int h = blockIdx.x / kBlocks;
  const int Hq = gridDim.x / kBlocks;
  const int b = blockIdx.y;
  const int tid = threadIdx.x % kGroupThreads;
  const int group = threadIdx.x / kGroupThreads;
  const int d0 = blockIdx.x % kBlocks * kDims + 4 * tid;
  const size_t row = static_cast<size_t>(b) * Hq + h;

  // The schedule: weighted pages before sequence b, its own pages, the weighted
  // total (common.cuh).  The lengths are final and visible already: the kernel
  // ahead lets this one launch only after its own wait, or, where it is the own
  // positions' and does not wait, was itself let launch by the prefix kernel after
  // that one's wait.
  if (threadIdx.x < kSched) {
    int before = 0, mine = 0, total = 0;
    for (int j = threadIdx.x; j < p.batch; j += kSched) {
      const int n = visible_pages(schedule_len(p, p.seq_lens[j], false), p.window);
      const int wn = n > 0 ? n + Params::kSeqWeight : 0;
      total += wn;
      before += j < b ? wn : 0;
      mine += j == b ? n : 0;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    mine = __reduce_add_sync(0xffffffffu, mine);
    total = __reduce_add_sync(0xffffffffu, total);
    if ((threadIdx.x & 31) == 0) {
      s_sched[threadIdx.x >> 5][0] = before;
      s_sched[threadIdx.x >> 5][1] = mine;
      s_sched[threadIdx.x >> 5][2] = total;
    }
  }
  int used = 0;  // prefix spans
  if constexpr (kPrefixSlices > 0)
    used = prefill_pair::PrefixSpans(*mp.prefix_len, mp.prefix_blocks, mp.splits, kStepPages).used;
  __syncthreads();
  int before = 0, mine = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kSched / 32; ++w) {
    before += s_sched[w][0];
    mine += s_sched[w][1];
    total += s_sched[w][2];
  }
  const int per = span_pages(total, p.grid_x, p.min_pages);
  const int g0 = mine > 0 ? (before + Params::kSeqWeight) / per : 0;
  const int g1 = mine > 0 ? (before + Params::kSeqWeight + mine - 1) / per : -1;
  int own = g1 - g0 + 1;
  if (own > kMaxSplits || (own > 0 && (static_cast<int64_t>(g1) + b + 1) * Hq > p.part_rows)) {
    if (threadIdx.x == 0) report(p.status, ATTN_DEV_INTERNAL);  // cannot happen: partials beyond the workspace
    own = 0;
  }
  const int ns = used + own;
  if (kPrefixSlices == 0 && own == 1) {  // one block held the whole sequence and wrote o
    // (the grid must not complete before the decode grid: see combine.cuh)
    if (blockIdx.x == 0 && blockIdx.y == 0) wait_for_primary_grid();
    return;
  }

  // partial i: prefix span i, or block g0 + i - used of the own positions
  const size_t rows = static_cast<size_t>(p.batch) * Hq;
  const float* pre_o = mp.part_o + row * kD + d0;
  const int slice = d0 * kPrefixSlices / kD;
  const float2* pre_ml = mp.part_ml + slice * rows + row;  // (not read without a prefix)
  const float* own_o = p.part_o + ((static_cast<size_t>(g0) + b) * Hq + h) * kD + d0;
  const float2* own_ml = p.part_ml + (static_cast<size_t>(g0) + b) * Hq + h;

  wait_for_primary_grid();
  allow_dependent_launch();
  float M = -INFINITY, L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r0 = group; r0 < ns; r0 += kMergeGroups * kInFlight) {
    float2 e[kInFlight];
    float4 a[kInFlight];
#pragma unroll
    for (int j = 0; j < kInFlight; ++j) {
      const int i = r0 + j * kMergeGroups;
      e[j] = make_float2(-INFINITY, 0.f);
      a[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < used) {
        e[j] = pre_ml[static_cast<size_t>(i) * kPrefixSlices * rows];
        a[j] = __ldcs(reinterpret_cast<const float4*>(pre_o + static_cast<size_t>(i) * rows * kD));
      } else if (i < ns) {
        e[j] = own_ml[static_cast<size_t>(i - used) * Hq];
        a[j] = __ldcs(reinterpret_cast<const float4*>(own_o + static_cast<size_t>(i - used) * Hq * kD));
      }
      if (e[j].y != e[j].y) e[j] = make_float2(INFINITY, 1.f);  // a NaN sum has to show: inf - inf below
    }
    float m = M;
#pragma unroll
    for (int j = 0; j < kInFlight; ++j)
      if (e[j].y > 0.f) m = fmaxf(m, e[j].x);
    if (m == -INFINITY) continue;
    const float f = M == -INFINITY ? 0.f : exp2f(M - m);
    L *= f;
    O.x *= f; O.y *= f; O.z *= f; O.w *= f;
#pragma unroll
    for (int j = 0; j < kInFlight; ++j) {
      if (e[j].y > 0.f) {
        const float w = exp2f(e[j].x - m);
        L += w * e[j].y;
        O.x += w * a[j].x; O.y += w * a[j].y; O.z += w * a[j].z; O.w += w * a[j].w;
      }
    }
    M = m;
  }
  s_m[group][tid] = M;
  s_l[group][tid] = L;
  s_o[group][tid] = O;
  __syncthreads();
  if (group != 0) return;
  float m = M;
#pragma unroll
  for (int w = 1; w < kMergeGroups; ++w) m = fmaxf(m, s_m[w][tid]);
  L = 0.f;
  O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kMergeGroups; ++w) {
    const float f = s_m[w][tid] == -INFINITY ? 0.f : exp2f(s_m[w][tid] - m);
    const float4 v = s_o[w][tid];
    L += f * s_l[w][tid];
    O.x += f * v.x; O.y += f * v.y; O.z += f * v.z; O.w += f * v.w;
  }
  const float inv = L > 0.f ? 1.f / L : L;  // 0: no visible position at all
  store_out4(p, row * kD + d0, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
}

}  // namespace prefix
}  // namespace pda
