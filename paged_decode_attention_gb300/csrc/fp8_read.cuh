// fp8_read.cuh -- cached positions of an 8-bit cache (fp8.cuh) read back into
// bf16 pages, for the calls that take a bf16 cache (multi-query attention).
//
// For every sequence the last min(L, span) positions (all for span <= 0) are
// copied row by row from page block_table[b, l/16] to page out_table[b, l/16]
// of the bf16 pools as e4m3(c) * 2^(s - 127).  The product is exact in fp32
// and, in bf16's range, in bf16.  Rows outside are not written.
//
// Bound by memory: D + 1 bytes in and 2 D out per row.  The concatenated
// pages of all sequences are cut into equal spans (the balanced schedule of
// common.cuh), one per block; blockIdx.y takes the keys or the values.  A thread
// converts 8 values at a time (8 bytes in, 16 out, both coalesced) and keeps up
// to 8 such loads in flight.  Eight sliding contexts of 2047 positions: 34 us,
// 0.87 of the measured rate of a copy, which writes one byte per byte read and
// not two.
#pragma once

#include "fp8.cuh"

namespace pda {
namespace fp8_read {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 4;
// Blocks launched per SM and pool: two waves of short spans balance better than
// one of long ones (eight sliding contexts of 2047 positions 38.6 -> 34.0 us, one
// global context of 32768 20.0 -> 19.0 us; 16 per SM: 34.0 and 20.5).
constexpr int kGridPerSm = 8;

struct ReadParams {
  DecodeParams d;               // batch, seq_lens, block_table, max_blocks, window (= span), schedule, status
  const uint8_t* src[2];        // e4m3 [num_pages, 16, Hkv, D]: keys, values
  const uint8_t* scale[2];      // [num_pages, Hkv, 16]
  __nv_bfloat16* dst[2];        // [out_pages, 16, Hkv, D]
  const int32_t* out_table;     // [batch, max_blocks]
  int64_t out_pages;
};

template <int kHkv, int kD>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kRowUnits = kHkv * kD / 8;                // 8-value units of a token row
  constexpr int kUnits = kPage * kRowUnits / kThreads;    // units per thread and page
  constexpr int kBatch = kUnits < 8 ? kUnits : 8;         // loads in flight together
  static_assert(kUnits * kThreads == kPage * kRowUnits && kUnits % kBatch == 0, "whole units per thread");
  __shared__ SeqTable t;
  wait_for_primary_grid();
  allow_dependent_launch();
  if (threadIdx.x < 32) scan_seq_lens<false>(p.d, t, blockIdx.x);
  __syncthreads();
  const Span sp = t.span;
  if (sp.end <= sp.begin) return;
  const uint8_t* src = p.src[blockIdx.y];
  const uint8_t* scale = p.scale[blockIdx.y];
  __nv_bfloat16* dst = p.dst[blockIdx.y];
  PageCursor cur;
  cur.start(p.d, t, sp);
  for (int f = sp.begin; f < sp.end; ++f) {
    cur.advance(p.d, t, sp, f);
    const int pos0 = cur.pos0(t, f);
    const int64_t entry = static_cast<int64_t>(cur.b) * p.d.max_blocks + pos0 / kPage;
    const int32_t from = p.d.block_table[entry], to = p.out_table[entry];
    if (from < 0 || static_cast<int64_t>(from) >= p.d.num_pages || to < 0 || static_cast<int64_t>(to) >= p.out_pages) {
      if (threadIdx.x == 0) report(p.d.status, ATTN_DEV_BAD_PAGE);
      continue;
    }
    const uint8_t* page = src + static_cast<size_t>(from) * (kPage * kHkv * kD);
    const uint8_t* page_scale = scale + static_cast<size_t>(from) * (kHkv * kPage);
    __nv_bfloat16* out = dst + static_cast<size_t>(to) * (kPage * kHkv * kD);
#pragma unroll
    for (int k0 = 0; k0 < kUnits; k0 += kBatch) {
      uint2 w[kBatch];
      uint32_t sc[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int u = threadIdx.x + (k0 + k) * kThreads;
        const int row = u / kRowUnits, head = u % kRowUnits / (kD / 8);
        const bool in = pos0 + row >= cur.lo && pos0 + row < cur.L;
        w[k] = in ? __ldcs(reinterpret_cast<const uint2*>(page) + u) : make_uint2(0, 0);
        sc[k] = in ? page_scale[head * kPage + row] : 0;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int u = threadIdx.x + (k0 + k) * kThreads;
        const int row = u / kRowUnits;
        if (pos0 + row < cur.lo || pos0 + row >= cur.L) continue;
        const float f2 = fp8::scale_value(sc[k]);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t word = j < 2 ? w[k].x : w[k].y;
          const uint32_t h = (j & 1) ? fp8::hi_f16x2(word) : fp8::lo_f16x2(word);
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
          o[j] = pack_bf16x2(v.x * f2, v.y * f2);
        }
        reinterpret_cast<uint4*>(out)[u] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

}  // namespace fp8_read
}  // namespace pda
