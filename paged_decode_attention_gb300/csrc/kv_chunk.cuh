// kv_chunk.cuh -- per-head norms, RoPE and the cache append of a ragged chunk
// of new tokens per sequence (the steps of kv_append.cuh, for any number of
// tokens), into a bf16 cache or an 8-bit one (fp8.cuh).
//
// Token t of the packed chunk belongs to the sequence b with
// cu_q[b] <= t < cu_q[b+1] and sits at position
//   pos = seq_lens[b] - (cu_q[b+1] - cu_q[b]) + (t - cu_q[b]),
// the convention of the multi-query attention (prefill_tc.cuh).  Behind a shared
// prefix (prefix.cuh) a sequence's own positions are numbered from 0, which is
// where the cache row goes, and turned by prefix_len + pos.  Per head row x of the
// token:
//   q and k:  rope(x / sqrt(sum_j x[j]^2 / D + eps) * w, pos)
//   v:        x / sqrt(sum_j x[j]^2 / D + eps)
//
// Bound by memory: a sliding token moves 32 KB (28 KB with an 8-bit cache), a
// global one 35 KB (34 KB).  So every byte is read once and written once, and
// the arithmetic that several rows share is done once: a block takes a token at
// a time, each thread below kPairs turns one pair's angle into (cos, sin) for all
// heads of the token, one barrier a token.  The pair frequencies theta^(-2i/D)
// are products of at most 7 host-computed factors (one per set bit of i, in float
// pairs: 2^-43 relative), formed before the block waits for the previous kernel.
// The row arithmetic runs on pairs of dims (packed fp32 instructions).
//
// Warp w of the first eight takes q heads 2w and 2w+1, on sliding layers also key
// head w and value head w; on global layers a ninth warp takes the head that is
// key and value.  8192 sliding tokens: 43.7 us, 0.90 of the measured copy rate;
// 4096 global tokens into an 8-bit cache 24.3 us, 0.86 (8192: 45.3, 0.93); 8192
// sliding tokens into an 8-bit cache 44.2 us, 0.78: 14 % fewer bytes than into a
// bf16 one, but two more reductions and the conversions in a token's chain.
// Slower, on 4096 global tokens at 23.6 us (before the tests for rows beyond range):
// the shared head as a second job of one of eight warps, for which the others
// wait at the barrier (27.0 us with two tokens a round, 31.5 with one), two tokens
// a round of the nine warps (25.2; 608 tokens 4.1 us against 5.1, more than three
// blocks per SM holding one each), two blocks per SM instead of three (26.8), tasks
// that each warp takes on its own, without barrier or shared angles (34.8).
// Lane l holds dims [V l, V l + V) and their rotation partners, V = D / 64, as in
// kv_append.cuh.
#pragma once

#include <type_traits>

#include "fp8.cuh"
#include "kv_append.cuh"
#include "tree_nodes.cuh"

namespace pda {
namespace chunk {

constexpr int kQWarps = 8;  // two query heads each
template <bool kShared>
constexpr int kThreads = (kShared ? kQWarps + 1 : kQWarps) * 32;
constexpr int kBlocksPerSm = 3;
constexpr int kPairBits = 7;  // pairs 0..127

struct ChunkParams {
  const __nv_bfloat16* qkv;    // [total_q, row_len]
  const __nv_bfloat16* w_q;    // [D]
  const __nv_bfloat16* w_k;    // [D]
  const int32_t* block_table;  // [batch, max_blocks]
  const int32_t* seq_lens;     // [batch], new tokens included
  const int32_t* cu_q;         // [batch + 1]
  const int32_t* prefix_len;   // one int32 on the device, added to every angle's position; null: 0
  const int32_t* parents;      // [total_q], nodes of trees only
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
  FloatPair inv_pi;
  FloatPair bit_factor[kPairBits];  // theta^(-2 * 2^k / D)
};

// A node of a tree: its slot's position (-1: it is left alone), where it is rotated, the slot's page.
struct Node {
  int32_t pos, turned, phys;
};
constexpr int kAhead = kQWarps;  // nodes looked up together

template <bool kTree>
struct Smem {
  int32_t cu_q[kMaxBatch + 1];
  int32_t len[kMaxBatch];
  Node node[kTree ? kAhead : 1];
  // cos and sin of the token's pairs, double-buffered
  alignas(16) float cos[2][1 << kPairBits];
  alignas(16) float sin[2][1 << kPairBits];
};

// Node t, by one warp.  A chain of lookups (sequence, parents, page) and the tree's depth, some 2000 cycles: in front of
// every token's angles they cost 2032 sliding nodes 16.7 us, looked up ahead 13.4 (inputs in L2; 15.0 from HBM, where
// their bytes take 9.8).
__device__ __forceinline__ Node look_up_node(const ChunkParams& p, const int32_t* cu_q, const int32_t* len, int t) {
  const int lane = threadIdx.x & 31;
  int b = 0;
  for (int j0 = 0; j0 < p.batch; j0 += 32) {
    const int j = j0 + lane;
    b += __popc(__ballot_sync(0xffffffffu, j < p.batch && cu_q[j + 1] <= t));
  }
  if (b >= p.batch) return {-1, 0, 0};  // rows behind the last sequence are left alone
  const int q0 = cu_q[b], q1 = cu_q[b + 1], L = len[b];
  const int cap = p.max_blocks < ATTN_MAX_SEQ_LEN / kPage ? p.max_blocks * kPage : ATTN_MAX_SEQ_LEN;
  // a sequence whose numbers do not fit together is left alone as a whole
  if (q0 < 0 || t < q0 || q1 > p.total_q || q1 - q0 > L || L > cap || q1 - q0 > ATTN_MAX_TREE) {
    if (lane == 0) report(p.status, ATTN_DEV_BAD_SEQ_LEN);
    return {-1, 0, 0};
  }
  int parent[2];
  tree::read_parents(p.parents + q0, q1 - q0, parent);
  const int pos = L - (q1 - q0) + (t - q0);
  const int32_t phys = p.block_table[static_cast<int64_t>(b) * p.max_blocks + pos / kPage];
  if (tree::check_parents(q1 - q0, parent) && lane == 0) report(p.status, ATTN_DEV_BAD_TREE);
  return {pos, L - (q1 - q0) + tree::depth_of(q1 - q0, parent, t - q0), phys};
}

// cos and sin of pos * (f.hi + f.lo), a frequency in half turns.  For an integer
// 0 <= pos < 2^24 the float product and its fma remainder hold pos * f.hi
// exactly, and subtracting whole turns, an even integer, is exact.  What the
// last sum rounds away, up to 2^-25 half turns, turns the result by a first-order
// step, so that the units in the last place of sincospif are all that is left:
// an angle off by more moves values across the borders of e4m3.
__device__ __forceinline__ void sincos_at(FloatPair f, int pos, float* sn, float* cs) {
  const float fp = static_cast<float>(pos);  // exact
  const float hi = fp * f.hi;
  const float rest = fmaf(fp, f.lo, fmaf(fp, f.hi, -hi));
  const float turn = fmaf(-2.f, rintf(0.5f * hi), hi);
  const float x = turn + rest;
  const float d = 3.14159265f * (rest - (x - turn));
  float s0, c0;
  sincospif(x, &s0, &c0);
  *sn = fmaf(d, c0, s0);
  *cs = fmaf(-d, s0, c0);
}

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

// The row in fp32, pairs of dims.
template <int kD>
struct Row {
  static constexpr int kWords = kD / 64 / 2;  // per half
  float2 lo[kWords], hi[kWords];
};

template <int kD>
__device__ __forceinline__ void widen(const RawRow<kD>& r, Row<kD>& x) {
#pragma unroll
  for (int j = 0; j < RawRow<kD>::kWords; ++j) {
    x.lo[j] = bf16x2_to_float2(r.lo[j]);
    x.hi[j] = bf16x2_to_float2(r.hi[j]);
  }
}

template <int kD>
__device__ __forceinline__ void times(Row<kD>& r, float f) {
  const float2 f2 = make_float2(f, f);
#pragma unroll
  for (int j = 0; j < Row<kD>::kWords; ++j) {
    r.lo[j] = __fmul2_rn(r.lo[j], f2);
    r.hi[j] = __fmul2_rn(r.hi[j], f2);
  }
}

// sum(x^2), the same in every lane
template <int kD>
__device__ __forceinline__ float sum_squares(const Row<kD>& r) {
  float2 ss = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < Row<kD>::kWords; ++j) ss = __ffma2_rn(r.lo[j], r.lo[j], __ffma2_rn(r.hi[j], r.hi[j], ss));
  float sum = ss.x + ss.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// 1 / sqrt(mean(x^2) + eps).  The squares of a finite row can add up beyond
// fp32's range (a mean square above 2^119).  Without kWide the factor is NaN then
// and `beyond` is set; with it such a row is first brought down by 2^70: 512
// squares of at most 2^116 stay below 2^126, and eps no longer counts.  (Exact but
// for elements below 2^-56, of which less than 2^-115 is left.)  An infinity gives
// NaN either way, through the Newton step.
template <int kD, bool kWide>
__device__ __forceinline__ float norm_factor(Row<kD>& r, float eps, bool& beyond) {
  float sum = sum_squares<kD>(r);
  if constexpr (kWide) {
    if (sum == INFINITY) {
      times<kD>(r, 0x1p-70f);
      sum = sum_squares<kD>(r);
      eps = 0.f;
    }
  } else {
    beyond |= sum == INFINITY;
  }
  const float mean = sum / static_cast<float>(kD) + eps;
  const float inv = rsqrtf(mean);
  return fmaf(0.5f * inv, fmaf(-mean * inv, inv, 1.f), inv);  // one Newton step: the root to its last bit
}

// The norm's weights come first where they can: the product of two bf16 values
// is exact in fp32, so a weighted row is rounded once, by its norm factor.
template <int kD>
__device__ __forceinline__ void scale(Row<kD>& r, const Row<kD>& w) {
#pragma unroll
  for (int j = 0; j < Row<kD>::kWords; ++j) {
    r.lo[j] = __fmul2_rn(r.lo[j], w.lo[j]);
    r.hi[j] = __fmul2_rn(r.hi[j], w.hi[j]);
  }
}

// Rotation by the token's shared tables; kPairs is a multiple of V.
template <int kD, int kPairs>
__device__ __forceinline__ void rotate(const float* cs, const float* sn, Row<kD>& r) {
  constexpr int kV = kD / 64;
  const int lane = threadIdx.x & 31;
  if (kV * lane >= kPairs) return;
#pragma unroll
  for (int j = 0; j < kV / 2; ++j) {
    const float2 c = *reinterpret_cast<const float2*>(cs + kV * lane + 2 * j);
    const float2 t = *reinterpret_cast<const float2*>(sn + kV * lane + 2 * j);
    const float2 a = r.lo[j], b = r.hi[j];
    r.lo[j] = __ffma2_rn(make_float2(-b.x, -b.y), t, __fmul2_rn(a, c));
    r.hi[j] = __ffma2_rn(a, t, __fmul2_rn(b, c));
  }
}

template <int kD>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* dst, const Row<kD>& r) {
  constexpr int kV = kD / 64;
  const int lane = threadIdx.x & 31;
  uint32_t lo[kV / 2], hi[kV / 2];
#pragma unroll
  for (int j = 0; j < kV / 2; ++j) {
    lo[j] = pack_bf16x2(r.lo[j].x, r.lo[j].y);
    hi[j] = pack_bf16x2(r.hi[j].x, r.hi[j].y);
  }
  if constexpr (kV == 8) {
    *reinterpret_cast<uint4*>(dst + kV * lane) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(dst + kD / 2 + kV * lane) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  } else {
    *reinterpret_cast<uint2*>(dst + kV * lane) = make_uint2(lo[0], lo[1]);
    *reinterpret_cast<uint2*>(dst + kD / 2 + kV * lane) = make_uint2(hi[0], hi[1]);
  }
}

// The row as e4m3 with its scale byte (fp8.cuh).
template <int kD>
__device__ __forceinline__ void store_fp8(uint8_t* dst, uint8_t* scale, Row<kD>& r) {
  constexpr int kV = kD / 64;
  const int lane = threadIdx.x & 31;
  uint32_t amax = 0;  // non-negative floats order like their bits; a NaN lies above everything
#pragma unroll
  for (int j = 0; j < kV / 2; ++j) {
    const uint32_t a = max(__float_as_uint(r.lo[j].x) & 0x7fffffffu, __float_as_uint(r.lo[j].y) & 0x7fffffffu);
    const uint32_t b = max(__float_as_uint(r.hi[j].x) & 0x7fffffffu, __float_as_uint(r.hi[j].y) & 0x7fffffffu);
    amax = max(amax, max(a, b));
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  float inv;
  const uint32_t s = fp8::scale_byte(amax, inv);
  const float2 inv2 = make_float2(inv, inv);
  uint32_t lo[kV / 4], hi[kV / 4];
#pragma unroll
  for (int j = 0; j < kV / 4; ++j) {
    const float2 a = __fmul2_rn(r.lo[2 * j], inv2), b = __fmul2_rn(r.lo[2 * j + 1], inv2);
    const float2 c = __fmul2_rn(r.hi[2 * j], inv2), d = __fmul2_rn(r.hi[2 * j + 1], inv2);
    lo[j] = fp8::pack_e4m3x4(a.x, a.y, b.x, b.y);
    hi[j] = fp8::pack_e4m3x4(c.x, c.y, d.x, d.y);
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

template <int kD, int kHq, int kHkv, int kPairs, bool kShared, bool kFp8, bool kTree = false>
__global__ void __launch_bounds__(kThreads<kShared>, kBlocksPerSm) chunk_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int kRowLen = kHq * kD + (kShared ? kD : 2 * kHkv * kD);
  static_assert(kHq == 2 * kQWarps && (kShared ? kHkv == 1 : kHkv == kQWarps), "rows of a token by warp");
  static_assert(kPairs <= kThreads<kShared> && kPairs <= (1 << kPairBits) && kPairs % (kD / 64) == 0 && kPairs % 32 == 0,
                "pairs by thread");
  __shared__ Smem<kTree> s;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // this thread's pair frequency, while the previous kernel finishes
  FloatPair freq = p.inv_pi;
#pragma unroll
  for (int k = 0; k < kPairBits; ++k)
    if ((threadIdx.x % kPairs >> k) & 1) freq = df_mul(freq, p.bit_factor[k]);
  // The previous kernel in the stream may still be writing qkv, the lengths
  // or the tables, or reading the cache.
  wait_for_primary_grid();
  allow_dependent_launch();
  const int base = p.prefix_len != nullptr ? *p.prefix_len : 0;
  bool refused = base < 0 || base > ATTN_MAX_SEQ_LEN;
  for (int i = threadIdx.x; i <= p.batch; i += kThreads<kShared>) {
    const int q0 = p.cu_q[i];
    s.cu_q[i] = q0;
    if (i < p.batch) {
      s.len[i] = p.seq_lens[i];
      refused |= p.cu_q[i + 1] < q0;
    }
  }
  const bool has_kv = !kShared || warp == kQWarps;
  RawRow<kD> w_raw, wk_raw;  // the warp's weights; of a warp with both, the keys'
  load_raw<kD>(kShared && has_kv ? p.w_k : p.w_q, w_raw);
  if constexpr (!kShared) load_raw<kD>(p.w_k, wk_raw);
  // Where cu_q decreases, sequences overlap or run backwards: a token found by
  // counting ends may lie behind its sequence, at a position beyond the table.
  // The call is left alone as a whole, as for a prefix of no length.
  if (__syncthreads_or(refused)) {
    if (threadIdx.x == 0) report(p.status, ATTN_DEV_BAD_SEQ_LEN);
    return;
  }

  int buf = 0;
  [[maybe_unused]] int round = 0;
  bool beyond = false;
  const auto tokens = [&](auto wide_c) {
    constexpr bool kWide = decltype(wide_c)::value;
    round = 0;
    for (int t = blockIdx.x; t < p.total_q; t += gridDim.x) {
      // this warp's rows, all in flight together
      const __nv_bfloat16* src = p.qkv + static_cast<size_t>(t) * kRowLen;
      RawRow<kD> rq[2];  // (global layers: the shared head, head kHq, in the ninth warp's rq[0])
      [[maybe_unused]] RawRow<kD> rk, rv;
      load_raw<kD>(src + (2 * warp) * kD, rq[0]);
      if (!kShared || warp < kQWarps) load_raw<kD>(src + (2 * warp + 1) * kD, rq[1]);
      if constexpr (!kShared) {
        load_raw<kD>(src + (kHq + warp) * kD, rk);
        load_raw<kD>(src + (kHq + kHkv + warp) * kD, rv);
      }
      int pos = -1;  // the token is left alone
      int turned = 0;  // where it is rotated
      int32_t phys = 0;
      if constexpr (kTree) {
        // nodes are looked up a warp each, as many as there are warps, ahead of the rounds that take them
        const int k = round++ % kAhead;
        if (k == 0) {
          __syncthreads();  // the last ones were read
          if (warp < kAhead) {
            const int64_t at = t + static_cast<int64_t>(warp) * gridDim.x;
            const Node node = at < p.total_q ? look_up_node(p, s.cu_q, s.len, static_cast<int>(at)) : Node{-1, 0, 0};
            if (lane == 0) s.node[warp] = node;
          }
          __syncthreads();
        }
        pos = s.node[k].pos;
        turned = s.node[k].turned;
        phys = s.node[k].phys;
      } else {
        // the token's sequence: the number of sequences that end at or before t
        // (the same in every warp of the block)
        int b = 0;
        for (int j0 = 0; j0 < p.batch; j0 += 32) {
          const int j = j0 + lane;
          b += __popc(__ballot_sync(0xffffffffu, j < p.batch && s.cu_q[j + 1] <= t));
        }
        if (b < p.batch) {  // rows behind the last sequence are left alone
          const int q0 = s.cu_q[b], q1 = s.cu_q[b + 1];
          const int L = s.len[b];
          const int cap = p.max_blocks < ATTN_MAX_SEQ_LEN / kPage ? p.max_blocks * kPage : ATTN_MAX_SEQ_LEN;
          // a sequence whose numbers do not fit together is left alone as a whole
          if (q0 < 0 || t < q0 || q1 > p.total_q || q1 - q0 > L || L > cap) {
            if (threadIdx.x == 0) report(p.status, ATTN_DEV_BAD_SEQ_LEN);
          } else {
            pos = L - (q1 - q0) + (t - q0);
            if (has_kv) phys = p.block_table[static_cast<int64_t>(b) * p.max_blocks + pos / kPage];
          }
        }
        turned = base + pos;
      }
      if (threadIdx.x < kPairs)
        sincos_at(freq, pos < 0 ? 0 : turned, &s.sin[buf][threadIdx.x], &s.cos[buf][threadIdx.x]);
      __syncthreads();  // one per token: the buffer written next was read before this barrier
      const float* cs = s.cos[buf];
      const float* sn = s.sin[buf];
      buf ^= 1;
      if (pos < 0) continue;

      Row<kD> x, w;
      if (!kShared || warp < kQWarps) {
        widen<kD>(w_raw, w);
  #pragma unroll
        for (int i = 0; i < 2; ++i) {
          widen<kD>(rq[i], x);
          const float f = norm_factor<kD, kWide>(x, p.eps, beyond);
          scale<kD>(x, w);
          times<kD>(x, f);
          rotate<kD, kPairs>(cs, sn, x);
          store_bf16<kD>(p.q_out + (static_cast<size_t>(t) * kHq + 2 * warp + i) * kD, x);
        }
        if (kShared) continue;
      }
      if (phys < 0 || static_cast<int64_t>(phys) >= p.num_pages) {
        if (lane == 0) report(p.status, ATTN_DEV_BAD_PAGE);
        continue;
      }
      const int c = kShared ? 0 : warp;
      const int row = pos % kPage;
      const size_t off = ((static_cast<size_t>(phys) * kPage + row) * kHkv + c) * kD;
      [[maybe_unused]] const size_t soff = (static_cast<size_t>(phys) * kHkv + c) * kPage + row;
      const auto store = [&](void* pool, uint8_t* scales, Row<kD>& y) {
        if constexpr (kFp8)
          store_fp8<kD>(static_cast<uint8_t*>(pool) + off, scales + soff, y);
        else
          store_bf16<kD>(static_cast<__nv_bfloat16*>(pool) + off, y);
      };
      if constexpr (!kShared) {
        widen<kD>(rv, x);
        times<kD>(x, norm_factor<kD, kWide>(x, p.eps, beyond));
        store(p.v_pool, p.v_scale, x);
      }
      widen<kD>(kShared ? rq[0] : rk, x);
      const float f = norm_factor<kD, kWide>(x, p.eps, beyond);
      if constexpr (kShared) {  // (the keys are rounded after each of the two products: the raw row once
        times<kD>(x, f);        // more, for one rounding, costs 8 % of a call in registers)
        store(p.v_pool, p.v_scale, x);
        if (p.k_pool == nullptr) continue;  // a values-only cache
      }
      widen<kD>(kShared ? w_raw : wk_raw, w);
      scale<kD>(x, w);
      if constexpr (!kShared) times<kD>(x, f);
      rotate<kD, kPairs>(cs, sn, x);
      store(p.k_pool, p.k_scale, x);
    }
  };
  tokens(std::false_type{});
  // Rows whose squares left fp32's range (no model's): the block's tokens once more,
  // with a test in front of every factor.  In the first pass those tests would cost
  // (8192 sliding tokens 45.8 us; as a call behind the stores 44.2, this way 43.7,
  // without them 43.4).
  if (__syncthreads_or(beyond)) tokens(std::true_type{});
}

}  // namespace chunk
}  // namespace pda
