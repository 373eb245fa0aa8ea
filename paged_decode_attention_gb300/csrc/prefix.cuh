// prefix.cuh -- decodeGQA for a batch that shares a prefix: sequence b sees
// the prefix's positions (one page list for all) and then its own.
//
//   o[b,h] = sum over prefix and own positions l of softmax_l(<q[b,h], k_l>) v_l
//
// The softmax over the union is regrouped exactly from partial results (O, m,
// sum) as in combine.cuh.  Three kernels:
//   * the prefix as a multi-query attention whose queries are the batch's
//     sequences (prefill_pair.cuh with PrefixParams): its pages are read once
//     for 16 sequences x 16 heads instead of once per sequence, and the
//     products run on tcgen05, 2048 flops x batch per byte pair;
//   * the sequences' own positions with the decode kernel (global.cuh), every
//     segment left as a partial;
//   * this merge.
//
// One 4-warp block per (row b*Hq + h, slice of 128 dims), as combine.cuh; a
// row's partials are its prefix spans followed by its blocks of the balanced
// schedule.
#pragma once

#include "combine.cuh"
#include "prefill_pair.cuh"

namespace pda {
namespace prefix {

struct MergeParams {
  DecodeParams d;            // the own positions' call: schedule, partials, output
  const float* part_o;       // prefix partials (PrefixParams)
  const float2* part_ml;
  const int32_t* prefix_len;
  int32_t prefix_blocks;
  int32_t splits;
};

template <int kD, int kPrefixSlices, int kStepPages>
__global__ void __launch_bounds__(kCombineWarps * 32) merge_kernel(const __grid_constant__ MergeParams mp) {
  const DecodeParams& p = mp.d;
  constexpr int kSlices = kD / kCombineCols;
  __shared__ float s_max[kCombineWarps];
  __shared__ float s_l[kCombineWarps];
  __shared__ float4 s_o[kCombineWarps][32];
  __shared__ int s_sched[3];

  const int h = blockIdx.x / kSlices;
  const int slice = blockIdx.x % kSlices;
  const int b = blockIdx.y;
  const int Hq = gridDim.x / kSlices;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const size_t row = static_cast<size_t>(b) * Hq + h;
  const int d0 = slice * kCombineCols + lane * 4;

  wait_for_primary_grid();
  allow_dependent_launch();
  // weighted pages before sequence b, its own pages, the weighted total (common.cuh)
  if (warp == 0) {
    int before = 0, mine = 0, total = 0;
    for (int j = lane; j < p.batch; j += 32) {
      const int n = visible_pages(clamp_len(p, p.seq_lens[j], false), p.window);
      const int wn = n > 0 ? n + kSeqWeight : 0;
      total += wn;
      before += j < b ? wn : 0;
      mine += j == b ? n : 0;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    mine = __reduce_add_sync(0xffffffffu, mine);
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) {
      s_sched[0] = before;
      s_sched[1] = mine;
      s_sched[2] = total;
    }
  }
  __syncthreads();
  const int before = s_sched[0], mine = s_sched[1], total = s_sched[2];
  const int per = span_pages(total, p.grid_x, p.min_pages);
  const int g0 = mine > 0 ? (before + kSeqWeight) / per : 0;
  const int g1 = mine > 0 ? (before + kSeqWeight + mine - 1) / per : -1;
  int own = g1 - g0 + 1;
  if (own > kMaxSplits || (own > 0 && (static_cast<int64_t>(g1) + b + 1) * Hq > p.part_rows)) {
    if (threadIdx.x == 0) report(p.status, ATTN_DEV_INTERNAL);  // cannot happen: partials beyond the workspace
    own = 0;
  }
  const prefill_pair::PrefixSpans ps(*mp.prefix_len, mp.prefix_blocks, mp.splits, kStepPages);
  const int ns = ps.used + own;

  // partial i: prefix span i, or block g0 + i - used of the own positions
  const size_t rows = static_cast<size_t>(p.batch) * Hq;
  const float* pre_o = mp.part_o + row * kD + d0;
  const float2* pre_ml = mp.part_ml + (slice / (kSlices / kPrefixSlices)) * rows + row;
  const float* own_o = p.part_o + ((static_cast<size_t>(g0) + b) * Hq + h) * kD + d0;
  const float2* own_ml = p.part_ml + (static_cast<size_t>(g0) + b) * Hq + h;
  float wm = -INFINITY, wl = 0.f;
  float4 wo = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r0 = warp; r0 < ns; r0 += kCombineWarps * kPerWarp) {
    float2 e[kPerWarp];
    float4 a[kPerWarp];
#pragma unroll
    for (int j = 0; j < kPerWarp; ++j) {
      const int i = r0 + j * kCombineWarps;
      e[j] = make_float2(-INFINITY, 0.f);
      a[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < ps.used) {
        e[j] = pre_ml[static_cast<size_t>(i) * kPrefixSlices * rows];
        a[j] = *reinterpret_cast<const float4*>(pre_o + static_cast<size_t>(i) * rows * kD);
      } else if (i < ns) {
        e[j] = own_ml[static_cast<size_t>(i - ps.used) * Hq];
        a[j] = *reinterpret_cast<const float4*>(own_o + static_cast<size_t>(i - ps.used) * Hq * kD);
      }
    }
    float rm = wm;
#pragma unroll
    for (int j = 0; j < kPerWarp; ++j)
      if (e[j].y != e[j].y) e[j] = make_float2(INFINITY, 1.f);  // a NaN sum has to show: inf - inf below
#pragma unroll
    for (int j = 0; j < kPerWarp; ++j)
      if (e[j].y > 0.f) rm = fmaxf(rm, e[j].x);
    if (rm == -INFINITY) continue;
    const float cw = wm == -INFINITY ? 0.f : exp2f(wm - rm);
    wl *= cw;
    wo.x *= cw; wo.y *= cw; wo.z *= cw; wo.w *= cw;
#pragma unroll
    for (int j = 0; j < kPerWarp; ++j) {
      if (e[j].y > 0.f) {
        const float w = exp2f(e[j].x - rm);
        wl += w * e[j].y;
        wo.x += w * a[j].x; wo.y += w * a[j].y; wo.z += w * a[j].z; wo.w += w * a[j].w;
      }
    }
    wm = rm;
  }

  if (lane == 0) s_max[warp] = wm;
  __syncthreads();
  float M = s_max[0];
#pragma unroll
  for (int w = 1; w < kCombineWarps; ++w) M = fmaxf(M, s_max[w]);
  const float f = (M == -INFINITY || wm == -INFINITY) ? 0.f : exp2f(wm - M);
  if (lane == 0) s_l[warp] = f * wl;
  s_o[warp][lane] = make_float4(f * wo.x, f * wo.y, f * wo.z, f * wo.w);
  __syncthreads();
  if (warp == 0) {
    float L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kCombineWarps; ++w) {
      L += s_l[w];
      const float4 v = s_o[w][lane];
      O.x += v.x; O.y += v.y; O.z += v.z; O.w += v.w;
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;  // 0: no visible position at all
    store_out4(p, row * kD + d0, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
  }
}

}  // namespace prefix
}  // namespace pda
