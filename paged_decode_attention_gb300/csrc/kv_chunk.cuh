// kv_chunk.cuh -- per-head norms, RoPE and the cache append of a ragged chunk
// of new tokens per sequence (the steps of kv_append.cuh, for any number of
// tokens), into a bf16 cache or an 8-bit one (fp8.cuh).
//
// Token t of the packed chunk belongs to the sequence b with
// cu_q[b] <= t < cu_q[b+1] and sits at position
//   pos = seq_lens[b] - (cu_q[b+1] - cu_q[b]) + (t - cu_q[b]),
// the convention of the multi-query attention (prefill_tc.cuh).  Per head row
// x of the token:
//   q and k:  rope(x / sqrt(sum_j x[j]^2 / D + eps) * w, pos)
//   v:        x / sqrt(sum_j x[j]^2 / D + eps)
//
// Bound by memory: a sliding token moves 32 KB (28 KB with an 8-bit cache), a
// global one 35 KB (34 KB).  So every byte is read once and written once, and
// the arithmetic that several rows share is done once: a block of 8 warps
// takes one token at a time, each thread below kPairs turns one pair's angle
// into (cos, sin) for all of the token's heads, and each warp holds the norm
// weights of its lanes in registers for as long as the block lives.  The pair
// frequencies theta^(-2i/D) are products of at most 7 host-computed factors
// (one per set bit of i, in float pairs: 2^-43 relative), formed before the
// block waits for the previous kernel; the angles are rope.cuh's.
//
// Warp w of a sliding token takes q heads 2w and 2w+1, key head w and value
// head w; of a global one q heads 2w and 2w+1, and the warp that t mod 8
// names also the key/value head.  Lane l holds dims [V l, V l + V) and their
// rotation partners, V = D / 64, as in kv_append.cuh.
#pragma once

#include "fp8.cuh"
#include "kv_append.cuh"

namespace pda {
namespace chunk {

using append::Row;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlocksPerSm = 4;
constexpr int kPairBits = 7;  // pairs 0..127

struct ChunkParams {
  const __nv_bfloat16* qkv;    // [total_q, row_len]
  const __nv_bfloat16* w_q;    // [D]
  const __nv_bfloat16* w_k;    // [D]
  const int32_t* block_table;  // [batch, max_blocks]
  const int32_t* seq_lens;     // [batch], new tokens included
  const int32_t* cu_q;         // [batch + 1]
  __nv_bfloat16* q_out;        // [total_q, Hq, D]
  void* k_pool;                // [num_pages, 16, Hkv, D] bf16 or e4m3; null: values-only global cache (bf16)
  void* v_pool;
  uint8_t* k_scale;            // [num_pages, Hkv, 16], 8-bit cache only
  uint8_t* v_scale;
  int32_t* status;             // optional ATTN_DEV_* word
  int64_t num_pages;
  int32_t batch;
  int32_t total_q;
  int32_t max_blocks;
  float eps;
  TwoPi two_pi;
  FloatPair bit_factor[kPairBits];  // theta^(-2 * 2^k / D)
};

struct Smem {
  int32_t cu_q[kMaxBatch + 1];
  alignas(16) float2 turn[2][1 << kPairBits];  // (cos, sin) of the token's pairs, double-buffered
};

// One row as raw bf16 words: dims [V l, +V) and [D/2 + V l, +V).
template <int kD>
struct RawRow {
  static constexpr int kWords = kD / 64 / 2;  // per half
  uint32_t lo[kWords], hi[kWords];
};

template <int kD>
__device__ __forceinline__ void load_raw(const __nv_bfloat16* src, RawRow<kD>& r) {
  const int lane = threadIdx.x & 31;
  constexpr int kV = kD / 64;
  if constexpr (kV == 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(src + kV * lane);
    const uint4 b = *reinterpret_cast<const uint4*>(src + kD / 2 + kV * lane);
    r.lo[0] = a.x; r.lo[1] = a.y; r.lo[2] = a.z; r.lo[3] = a.w;
    r.hi[0] = b.x; r.hi[1] = b.y; r.hi[2] = b.z; r.hi[3] = b.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(src + kV * lane);
    const uint2 b = *reinterpret_cast<const uint2*>(src + kD / 2 + kV * lane);
    r.lo[0] = a.x; r.lo[1] = a.y;
    r.hi[0] = b.x; r.hi[1] = b.y;
  }
}

template <int kD>
__device__ __forceinline__ void widen(const RawRow<kD>& r, Row<kD>& x) {
#pragma unroll
  for (int j = 0; j < RawRow<kD>::kWords; ++j) {
    const float2 a = bf16x2_to_float2(r.lo[j]), b = bf16x2_to_float2(r.hi[j]);
    x.lo[2 * j] = a.x; x.lo[2 * j + 1] = a.y;
    x.hi[2 * j] = b.x; x.hi[2 * j + 1] = b.y;
  }
}

// Rotation by the token's shared (cos, sin) table; kPairs is a multiple of V.
template <int kD, int kPairs>
__device__ __forceinline__ void rotate(const float2* turn, Row<kD>& r) {
  constexpr int kV = kD / 64;
  const int lane = threadIdx.x & 31;
  if (kV * lane >= kPairs) return;
  const float4* t4 = reinterpret_cast<const float4*>(turn + kV * lane);
#pragma unroll
  for (int j = 0; j < kV; j += 2) {
    const float4 t = t4[j / 2];  // cos, sin of pairs j, j + 1
    const float a0 = r.lo[j], b0 = r.hi[j], a1 = r.lo[j + 1], b1 = r.hi[j + 1];
    r.lo[j] = a0 * t.x - b0 * t.y;
    r.hi[j] = b0 * t.x + a0 * t.y;
    r.lo[j + 1] = a1 * t.z - b1 * t.w;
    r.hi[j + 1] = b1 * t.z + a1 * t.w;
  }
}

// The row as e4m3 with its scale byte (fp8.cuh).
template <int kD>
__device__ __forceinline__ void store_fp8(uint8_t* dst, uint8_t* scale, const Row<kD>& r) {
  constexpr int kV = kD / 64;
  const int lane = threadIdx.x & 31;
  uint32_t amax = 0;  // non-negative floats order like their bits; a NaN lies above everything
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const uint32_t a = __float_as_uint(r.lo[j]) & 0x7fffffffu, b = __float_as_uint(r.hi[j]) & 0x7fffffffu;
    amax = max(amax, max(a, b));
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  float inv;
  const uint32_t s = fp8::scale_byte(amax, inv);
  uint32_t lo[kV / 4], hi[kV / 4];
#pragma unroll
  for (int j = 0; j < kV / 4; ++j) {
    lo[j] = fp8::pack_e4m3x4(r.lo[4 * j] * inv, r.lo[4 * j + 1] * inv, r.lo[4 * j + 2] * inv, r.lo[4 * j + 3] * inv);
    hi[j] = fp8::pack_e4m3x4(r.hi[4 * j] * inv, r.hi[4 * j + 1] * inv, r.hi[4 * j + 2] * inv, r.hi[4 * j + 3] * inv);
  }
  if constexpr (kV == 8) {
    *reinterpret_cast<uint2*>(dst + kV * lane) = make_uint2(lo[0], lo[1]);
    *reinterpret_cast<uint2*>(dst + kD / 2 + kV * lane) = make_uint2(hi[0], hi[1]);
  } else {
    *reinterpret_cast<uint32_t*>(dst + kV * lane) = lo[0];
    *reinterpret_cast<uint32_t*>(dst + kD / 2 + kV * lane) = hi[0];
  }
  if (lane == 0) *scale = static_cast<uint8_t>(s);
}

template <int kD, int kHq, int kHkv, int kPairs, bool kShared, bool kFp8>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) chunk_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int kRowLen = kHq * kD + (kShared ? kD : 2 * kHkv * kD);
  static_assert(kHq == 2 * kWarps && (kShared ? kHkv == 1 : kHkv == kWarps), "rows of a token by warp");
  static_assert(kPairs <= kThreads && kPairs <= (1 << kPairBits) && kPairs % (kD / 64) == 0, "pairs by thread");
  __shared__ Smem s;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // this thread's pair frequency, while the previous kernel finishes
  FloatPair freq{1.f, 0.f};
  if (threadIdx.x < kPairs) {
#pragma unroll
    for (int k = 0; k < kPairBits; ++k)
      if ((threadIdx.x >> k) & 1) freq = df_mul(freq, p.bit_factor[k]);
  }
  // The previous kernel in the stream may still be writing qkv, the lengths
  // or the tables, or reading the cache.
  wait_for_primary_grid();
  allow_dependent_launch();
  for (int i = threadIdx.x; i <= p.batch; i += kThreads) s.cu_q[i] = p.cu_q[i];
  RawRow<kD> wq_raw, wk_raw;
  load_raw<kD>(p.w_q, wq_raw);
  load_raw<kD>(p.w_k, wk_raw);
  __syncthreads();

  int buf = 0;
  for (int t = blockIdx.x; t < p.total_q; t += gridDim.x) {
    // the token's sequence: the number of sequences that end at or before t
    // (the same in every warp of the block)
    int b = 0;
    for (int j0 = 0; j0 < p.batch; j0 += 32) {
      const int j = j0 + lane;
      b += __popc(__ballot_sync(0xffffffffu, j < p.batch && s.cu_q[j + 1] <= t));
    }
    if (b >= p.batch) continue;  // rows behind the last sequence are left alone
    const int q0 = s.cu_q[b], q1 = s.cu_q[b + 1];
    const int L = p.seq_lens[b];
    const int n = q1 - q0;
    const int cap = p.max_blocks < ATTN_MAX_SEQ_LEN / kPage ? p.max_blocks * kPage : ATTN_MAX_SEQ_LEN;
    // a sequence whose numbers do not fit together is left alone as a whole
    if (q0 < 0 || t < q0 || q1 > p.total_q || n > L || L > cap) {
      if (threadIdx.x == 0) report(p.status, ATTN_DEV_BAD_SEQ_LEN);
      continue;
    }
    const int pos = L - n + (t - q0);
    const __nv_bfloat16* row = p.qkv + static_cast<size_t>(t) * kRowLen;

    // this warp's rows, all in flight together
    const bool has_kv = !kShared || warp == (t & (kWarps - 1));
    RawRow<kD> rq[2], rk, rv;
    load_raw<kD>(row + (2 * warp) * kD, rq[0]);
    load_raw<kD>(row + (2 * warp + 1) * kD, rq[1]);
    if (has_kv) load_raw<kD>(row + (kHq + (kShared ? 0 : warp)) * kD, rk);
    if constexpr (!kShared) load_raw<kD>(row + (kHq + kHkv + warp) * kD, rv);
    const int32_t phys = has_kv ? p.block_table[static_cast<int64_t>(b) * p.max_blocks + pos / kPage] : 0;

    if (threadIdx.x < kPairs) {
      float c, sn;
      rope_angle(p.two_pi, freq, pos, c, sn);
      s.turn[buf][threadIdx.x] = make_float2(c, sn);
    }
    __syncthreads();  // one per token: the buffer written next was read before this barrier
    const float2* turn = s.turn[buf];
    buf ^= 1;

    Row<kD> x, w;
    widen<kD>(wq_raw, w);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      widen<kD>(rq[i], x);
      append::normalise<kD>(x, p.eps);
      append::scale<kD>(x, w);
      rotate<kD, kPairs>(turn, x);
      append::store_row<kD>(p.q_out + (static_cast<size_t>(t) * kHq + 2 * warp + i) * kD, x);
    }
    if (!has_kv) continue;
    if (phys < 0 || static_cast<int64_t>(phys) >= p.num_pages) {
      if (lane == 0) report(p.status, ATTN_DEV_BAD_PAGE);
      continue;
    }
    const int c = kShared ? 0 : warp;
    const size_t off = ((static_cast<size_t>(phys) * kPage + pos % kPage) * kHkv + c) * kD;
    const size_t soff = (static_cast<size_t>(phys) * kHkv + c) * kPage + pos % kPage;
    const auto store = [&](void* pool, uint8_t* scales, const Row<kD>& y) {
      if constexpr (kFp8)
        store_fp8<kD>(static_cast<uint8_t*>(pool) + off, scales + soff, y);
      else
        append::store_row<kD>(static_cast<__nv_bfloat16*>(pool) + off, y);
    };
    if constexpr (!kShared) {
      widen<kD>(rv, x);
      append::normalise<kD>(x, p.eps);
      store(p.v_pool, p.v_scale, x);
    }
    widen<kD>(rk, x);
    append::normalise<kD>(x, p.eps);
    if constexpr (kShared) {
      store(p.v_pool, p.v_scale, x);
      if (p.k_pool == nullptr) continue;  // a values-only cache
    }
    widen<kD>(wk_raw, w);
    append::scale<kD>(x, w);
    rotate<kD, kPairs>(turn, x);
    store(p.k_pool, p.k_scale, x);
  }
}

}  // namespace chunk
}  // namespace pda
