// fp8.cuh -- the 8-bit cache format: e4m3 values with one power-of-two scale
// (E8M0) per cached position and KV head.
//
// A row y[0..D) (the key or the value of one head at one position) is stored
// as bytes c_i and one scale byte s with
//   y_i ~ e4m3(c_i) * 2^(s - 127);
// s = 255 reads as NaN, s = 0 (no append writes it: a cleared page) as zero.
// The writer takes the smallest k with max|y| <= 448 * 2^k (448 is the
// largest e4m3 value) and s = k + 127, clamped to [1, 254], and rounds
// y_i * 2^-k to e4m3 once, to nearest even.  Multiplying by a power of two is
// exact, so that rounding is the only one: half an e4m3 step, 2^-4 of the
// value down to 2^-6 * 2^k (at most 2^-13.8 of the row's largest), and
// 2^-10 * 2^k below.  The largest lands in (224, 448].  A row of zeros has
// s = 1.  A row with a NaN or an infinity has s = 255, E8M0's NaN, and reads
// back as NaN throughout.  Every e4m3(c) * 2^k is a bf16 value where it lies
// in bf16's normal range (4 significant bits of 8).
//
// Scales lie as [num_pages, Hkv, 16], so the 16 rows of a page and head are
// one 16-byte unit.
#pragma once

#include <cuda_fp8.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "common.cuh"

namespace pda {

// The decode calls over this cache: a sequence's start (scaling q, the first
// pages' latency, closing the segment) costs a block as much as a few pages.
// Global layers, weight 1 and 4, us: 8 sequences of 4700 19.0 and 17.2, 16 of 5000
// 27.8 and 25.8, 32 of 1000 18.1 and 16.5.  Sliding layers, 4 and 12 (their pages
// are half as long and four warps take them side by side): 8 of 1000 15.3 and
// 13.0, 16 of 5000 21.5 and 18.6, 32 of 200 15.2 and 12.0, 4 of 800 8.8 and 9.3, 256
// of 500 101.5 and 102.8.
struct Fp8GlobalParams : DecodeParams {
  static constexpr int kSeqWeight = 4;
};
struct Fp8SlidingParams : DecodeParams {
  static constexpr int kSeqWeight = 12;
};

// Block g takes sequence g: no partials, no merge.  (A type of its own: as a
// field it cost the kernel in spans registers, 347 us instead of 340 for 16
// global sequences of 131072.)
struct Fp8WholeParams : DecodeParams {};
__device__ __forceinline__ bool by_sequence(const Fp8WholeParams&) { return true; }

namespace fp8 {

constexpr uint32_t kNanScale = 255;

// The scale byte of a row whose largest |y| has the bit pattern `amax`
// (sign cleared), and the exact factor 2^-k; NaN or infinity: 255 and NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, float& inv) {
  if (amax >= 0x7f800000u) {
    inv = __uint_as_float(0x7fc00000u);
    return kNanScale;
  }
  // amax = 1.f * 2^E: 448 = 1.75 * 2^8, so k = E - 8, one more above 1.75
  int k = static_cast<int>(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (k < -126) k = -126;
  inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  return static_cast<uint32_t>(k + 127);
}

// 2^(s - 127); 255 gives NaN, 0 gives 0.
__device__ __forceinline__ float scale_value(uint32_t s) {
  return s == kNanScale ? __uint_as_float(0x7fc00000u) : __uint_as_float(s << 23);
}

// Four fp32 -> four e4m3 bytes, first value lowest (nearest even, saturating).
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Two e4m3 bytes (the low or the high half of w) -> f16x2; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}
__device__ __forceinline__ uint32_t lo_f16x2(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w)); }
__device__ __forceinline__ uint32_t hi_f16x2(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16)); }

// ---------------------------------------------------------------------------
// What the two decode kernels over this cache share.
//
// e4m3 values widen to f16 exactly, so both contractions run as
// mma.m16n8k16 f16 -> fp32 on unscaled values, with the power-of-two scales
// applied exactly in fp32 outside the products: a key's to its logits, a
// value's to its weight.  (mma.m16n8k32 on the bytes themselves is no way
// around the conversion: with q and the weights split into e4m3 terms it is
// right, but it executed 1049 instructions per page and head against 845, and
// the f16 tensor pipe was active four times as long as 24 such MMAs would
// need at the rate of their constant-operand loop: 5.2 -> 3.8 TB/s.)
//
// q is bf16, whose range f16 has not: each q row is multiplied by 2^-k with
// 2^14 <= max|q| 2^-k < 2^15 (exact), rounded to f16 and the 2^k goes to the
// row's logits.  Elements of at least 2^-28 of the row's largest stay exact
// (8 of 11 significant bits); below, the error is at most 2^-39 of it.
//
// Value scales differ from row to row, so the weight of row l that meets v8_l
// is p_l 2^{kv_l} with p_l = 2^{x_l - m} (x the logits in log2 units, m their
// running max).  Two references are kept per query row: m for the sum of the
// p_l, and T = max_l (x_l + kv_l) for the output; R = ceil(T - m).  The f16
// weight is
//     w_l = 2^{(x_l - m) + kv_l - R + 15}  <=  2^15,
// so the largest lies in (2^14, 2^15], and in the usual case that the largest
// p has the largest scale it is a power of two, exact in f16.  A weight is
// rounded by 2^-11 at most, down to 2^-28 of the largest, and below never by
// more than 2^-39 of it: 262,144 weights rounded to nothing lose 2^-21.  With
// one reference per page for the scales alone, a large scale on a row of no
// weight would take the bits of the others.  Accumulators hold 2^{15 - R}
// times the output sum relative to m and follow both references.
//
// Fragments.  A cache row's bytes are read 16 at a time: lane (g, t) = (lane/4,
// lane%4) takes unit 2t + j of a 128-byte chunk (even and odd units make the
// 128-byte swizzle conflict free), 16 dims that it contracts with the same
// dims of q, so their order does not matter.  The positions of a page are
// dealt to the N (or M) index of the first product so that position 4t + i is
// where a transposing byte load (ldmatrix .b8) of the value page puts it in
// the second: index n of the first half is row 4 (n/2) + n%2, of the second
// half two rows below.
// ---------------------------------------------------------------------------
constexpr int kWeightBias = 15;  // weights are at most 2^15 in f16 (largest finite 65504)

// Page row of index n (0..7) of the first half; the second half's is 2 below.
__device__ __forceinline__ int dealt_row(int n) { return 4 * (n >> 1) + (n & 1); }

// log2 of a scale: s - 127, NaN for 255, -inf for 0.
__device__ __forceinline__ float scale_log2(uint32_t s) {
  const float f = s == 0 ? -INFINITY : static_cast<float>(static_cast<int>(s) - 127);
  return s == kNanScale ? __uint_as_float(0x7fc00000u) : f;
}

// The references of one query row, moved by the maxima mx of x and mt of
// x + kv over new positions: the factors of the sum and of the accumulators.
struct Reference {
  float m, T, R;  // R is a whole number
  __device__ __forceinline__ void reset() {
    m = T = -INFINITY;
    R = 0.f;
  }
  __device__ __forceinline__ void move(float mx, float mt, float& sum_scale, float& acc_scale) {
    const float m_new = fmaxf(m, mx);
    T = fmaxf(T, mt);
    const float R_new = T == -INFINITY || m_new == -INFINITY ? R : ceilf(T - m_new);
    const float dm = m_new == m ? 0.f : m - m_new;  // -inf on the first visible position
    sum_scale = dm == 0.f ? 1.f : ex2_approx(dm);
    const float da = dm + (R - R_new);  // in one exponent: either part alone may leave fp32's range
    acc_scale = da == 0.f ? 1.f : ex2_approx(da);
    m = m_new;
    R = R_new;
  }
  __device__ __forceinline__ float m_use() const { return m == -INFINITY ? 0.f : m; }
  __device__ __forceinline__ float weight_bias() const { return static_cast<float>(kWeightBias) - R; }
};

// Accumulator -> output sum: x * 2^(R - 15) = x * f0 * f1, in two exact steps
// where 2^(R - 15) is below the normal range.
__device__ __forceinline__ void unscale_factors(float R, float& f0, float& f1) {
  const int e = max(static_cast<int>(R) - kWeightBias, -190);
  const bool low = e < -126;
  f0 = __uint_as_float(static_cast<uint32_t>((low ? e + 64 : min(e, 127)) + 127) << 23);
  f1 = low ? 0x1p-64f : 1.f;
}

// A q row's exponent k from the bits of its largest |q| (bf16 in the upper
// half, sign cleared), and the factor 2^-k.
__device__ __forceinline__ int q_exponent(uint32_t amax, float& inv) {
  int e = static_cast<int>(amax >> 23) - 127 - 14;
  if (e < -126) e = -126;
  if (e > 113) e = 113;
  inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  return e;
}

// Two bf16 of q times 2^-k, as f16x2.
__device__ __forceinline__ uint32_t q_f16x2(uint32_t w, float inv) {
  const float2 v = bf16x2_to_float2(w);
  const __half2 h = __floats2half2_rn(v.x * inv, v.y * inv);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// D = A(16x16, row) * B(16x8, col) + D, f16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8x8 matrix of 16-bit elements held as one word per lane
// (row lane / 4, columns 2 (lane % 4), +1).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t r) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(r));
  return d;
}

// Two 16x16 byte matrices (row addresses from lanes 0..15 and 16..31),
// transposed: lane (g = lane/4, t = lane%4) gets, of each, rows 4t .. 4t + 3 of
// column g and of column g + 8, one byte each.
__device__ __forceinline__ void ldmatrix_b8_x2_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// The dynamic shared memory rounded up to 1024 bytes.  By adding an offset to
// the array itself, so that accesses compile to shared-memory instructions: a
// pointer rounded as an integer is generic (with this, and the MMAs free to be
// scheduled, 16 global contexts of 131072 went from 443 to 410 us).
template <typename S>
__device__ __forceinline__ S& aligned_smem(uint8_t* raw) {
  return *reinterpret_cast<S*>(raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u));
}

// byte offset of 16-byte unit `unit` of row `row` in a 128B-swizzled [16][128 B] tile
__device__ __forceinline__ uint32_t swz(int row, int unit) { return row * 128 + ((unit ^ (row & 7)) << 4); }

constexpr int kChunkBytes = kPage * 128;  // 128 dims of a page's 16 rows

}  // namespace fp8
}  // namespace pda
