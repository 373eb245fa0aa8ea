// sliding_fp8.cuh -- slidingDecodeGQA over an 8-bit cache (fp8.cuh): 16 query
// heads over 8 KV heads, D = 256, G = 2, scale 1.
//
//   o[h] = sum_l 2^{kv_l} w_l v8_l / sum_l w_l,
//   w_l = exp(2^{kk_l} <q[h], k8_l> - max),  v8, k8 e4m3, kk, kv their scales.
//
// A page's head is 8 KB here, half of the bf16 cache's, so at the rate of
// memory a page has half the time.  On the CUDA cores every value would cost
// a conversion more than in the bf16 kernel; so both products run on
// mma.m16n8k16 with the cache as the A operand (16 positions, or 16 dims, by
// 16) and the two query heads in B's eight columns, each four times over, so
// that every lane has both heads' logits of its positions.
//
// The balanced spans as in sliding.cuh, grid (8, grid_x): the eight heads of a
// span run at the same time, so that a row is read whole (256 windows 182 us,
// 184.5 with the spans along x).  Warp 4 copies pages; each of the warps 0..3
// takes every fourth page whole and keeps its own running max, sum and output,
// so no barrier is met between a segment's first page and its end, where the
// four are merged two by two through shared memory.  256 windows of 1024: 182 us,
// 0.875 of the measured copy rate; the page copies alone, with nothing computed,
// take 171 to 174 us (a head's share of a row is 256 bytes, a page 16 such pieces).
//
// S^T[pos, h] = K q^T, then O^T[d, h] = V^T P^T: the weights of a lane's two
// positions, packed, become B fragments by one transposition in registers
// (movmatrix), and V^T comes as A fragments from the transposing byte load.
#pragma once

#include "fp8.cuh"
#include "sliding.cuh"
#include "tcgen05.cuh"

namespace pda {
namespace sliding_fp8 {

using sliding::kD;
using sliding::kG;
using sliding::kHkv;
using sliding::kHq;

constexpr int kConsumerWarps = 4;
constexpr int kThreads = (kConsumerWarps + 1) * 32;
constexpr int kChunks = kD / 128;                      // 2
constexpr int kTileBytes = kPage * kD;                 // 4 KB per K (or V) page-head
constexpr int kStages = 8;  // two per consumer warp: page i of the span is warp i % 4's, in stage i % 8
constexpr int kStageTx = 2 * kTileBytes + 2 * kPage;   // K, V and their scales
constexpr int kBlocksPerSm = sliding::kBlocksPerSm;    // the plan of the bf16 kernel
constexpr int kWarmPages = 8;

struct Smem {
  alignas(1024) uint8_t k[kStages][kTileBytes];  // kChunks tiles of [16 rows][128 dims], swizzled
  alignas(1024) uint8_t v[kStages][kTileBytes];
  alignas(128) uint8_t k_scale[kStages][128];  // 16 bytes used: a copy lands on a 128-byte boundary
  alignas(128) uint8_t v_scale[kStages][128];
  alignas(16) uint4 qfrag[kChunks * 4][4 * kG];  // q B fragments
  alignas(16) float merge_o[kConsumerWarps / 2][kG][kD];
  uint32_t q_max[kConsumerWarps][kG];
  float merge_m[kConsumerWarps / 2][kG];
  float merge_l[kConsumerWarps / 2][kG];
  int32_t merge_last;
  int32_t merge_cnt[kConsumerWarps];
  SeqTable table;
  alignas(8) uint64_t full[kStages];
  alignas(8) uint64_t empty[kStages];
};

constexpr size_t kSmemBytes = sizeof(Smem) + 1024;  // + alignment slack
static_assert(kConsumerWarps == 2 * kChunks, "a (chunk, j) of q per warp");
static_assert(kStages % kConsumerWarps == 0, "a stage belongs to one warp, which sees each of its phases");
static_assert(kBlocksPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of the resident blocks");

template <typename Params>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                  const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& s = fp8::aligned_smem<Smem>(smem_raw);

  const int gb = blockIdx.y;
  const int c = blockIdx.x;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(&s.full[st], 1);
      mbar_init(&s.empty[st], 1);  // the one warp that takes the page
    }
    fence_mbar_init();
  }
  if (warp == kConsumerWarps && lane == 0) {
    prefetch_tensor_map(&tm_k);
    prefetch_tensor_map(&tm_v);
    prefetch_tensor_map(&tm_ks);
    prefetch_tensor_map(&tm_vs);
  }
  // The prologue overlaps the previous kernel; see sliding.cuh.
  build_seq_table_hint(p, s.table, gb);  // ends with __syncthreads
  if (warp == kConsumerWarps) {
    warm_first_pages(p, s.table, kWarmPages, [&](int32_t y) {
      tma_prefetch_3d(&tm_k, 0, y, c * kChunks);
      tma_prefetch_3d(&tm_v, 0, y, c * kChunks);
    });
  } else {
    warm_q(p, s.table, kHq * kD, c * kG * kD, kG * kD * 2, kConsumerWarps * 32);
  }
  wait_for_primary_grid();
  int first = warp == kConsumerWarps ? page_entry(p, s.table, s.table.span, lane, false) : 0;
  confirm_seq_table(p, s.table, gb);  // ends with __syncthreads
  const SeqTable& t = s.table;
  const Span sp = t.span;
  const int n_pages = sp.end - sp.begin;
  if (p.merge_in_grid && gb == 0 && warp < kConsumerWarps) {
    // no combine kernel: block 0 of each column writes the empty sums (L = 0)
    for (int b = 0; b < p.batch; ++b) {
      if (t.prefix[b + 1] != t.prefix[b]) continue;
      const size_t row = static_cast<size_t>(b) * kHq + c * kG + (threadIdx.x >> 6);
      store_out4(p, row * kD + (threadIdx.x & 63) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
    }
  }
  if (n_pages <= 0) return;

  if (warp == kConsumerWarps) {
    // ---------------- producer ----------------
    const uint64_t policy = l2_policy_evict_first();
    if (t.rebuilt) first = page_entry(p, t, sp, lane, true);
    produce_pages<kStages, kStageTx>(p, t, sp, s.full, s.empty, first, [&](int stage, int32_t y) {
      tma_load_3d_hint(s.k[stage], &tm_k, 0, y, c * kChunks, &s.full[stage], policy);
      tma_load_3d_hint(s.v[stage], &tm_v, 0, y, c * kChunks, &s.full[stage], policy);
      // the scales of this head: 16 bytes in row (page * Hkv + c) of the scale pools
      const int32_t ys = y < 0 ? -1 : y / kPage * kHkv + c;
      tma_load_2d(s.k_scale[stage], &tm_ks, 0, ys, &s.full[stage]);
      tma_load_2d(s.v_scale[stage], &tm_vs, 0, ys, &s.full[stage]);
    });
    allow_dependent_launch();
    return;
  }

  // ---------------- consumers ----------------
  const int hq0 = c * kG;
  const int g = lane >> 2;
  const int tq = lane & 3;
  const int r0 = fp8::dealt_row(g);  // this lane's rows of a page: r0 and r0 + 2

  PageCursor cur;
  cur.start(p, t, sp);

  // q as B fragments in shared memory (32 registers would spill): column n = g
  // holds head g % 2 (the products' columns beyond the two heads repeat them),
  // k-step (chunk, j, word): dims 128 chunk + 16 (2 tq + j) + 4 word .. + 3.  Two
  // k-steps per 16 bytes.  Each warp prepares one (chunk, j): it loads its dims
  // of the next sequence while it works on this one, leaves their largest for
  // the other warps, and writes the fragments once all have.
  const int qlane = (g & 1) * 4 + tq;
  float qs[2];  // logit factor 2^k log2(e) of heads 0 and 1
  uint4 qn[2];  // the next sequence's q: 16 dims of head g % 2
  auto fetch_q = [&](int b) {
    const __nv_bfloat16* src = p.q + (static_cast<size_t>(b) * kHq + hq0 + (g & 1)) * kD + 128 * (warp >> 1) +
                               16 * (2 * tq + (warp & 1));
    qn[0] = ld_global_nc_v4(src);
    qn[1] = ld_global_nc_v4(src + 8);
  };
  auto publish_q = [&]() {  // a barrier of the consumers follows
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w[4] = {qn[k].x, qn[k].y, qn[k].z, qn[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) amax = max(amax, max(w[e] << 16 & 0x7fff0000u, w[e] & 0x7fff0000u));
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));  // over the row's four lanes
    if (g < kG && tq == 0) s.q_max[warp][g] = amax;
  };
  auto take_q = [&]() {
    float inv[kG];
#pragma unroll
    for (int h = 0; h < kG; ++h) {
      uint32_t amax = s.q_max[0][h];
#pragma unroll
      for (int w = 1; w < kConsumerWarps; ++w) amax = max(amax, s.q_max[w][h]);
      const int e = fp8::q_exponent(amax, inv[h]);
      qs[h] = __uint_as_float(static_cast<uint32_t>(e + 127) << 23) * kLog2e;
    }
    const float f = g & 1 ? inv[1] : inv[0];
    if (g < kG) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        s.qfrag[2 * warp + k][qlane] = make_uint4(fp8::q_f16x2(qn[k].x, f), fp8::q_f16x2(qn[k].y, f),
                                                  fp8::q_f16x2(qn[k].z, f), fp8::q_f16x2(qn[k].w, f));
    }
    const int nb = next_seq_in_span(p, t, sp, cur.b);
    if (nb >= 0) fetch_q(nb);
    named_barrier_sync(1, kConsumerWarps * 32);
  };
  fetch_q(cur.b);
  publish_q();
  named_barrier_sync(1, kConsumerWarps * 32);
  take_q();

  fp8::Reference ref[2];  // heads 0 and 1
  float l[2];             // this lane's share of the sums
  float acc[16][4];    // 16-dim blocks: (dim g; heads 0, 1), (dim g + 8; heads 0, 1)
  auto reset = [&]() {
    ref[0].reset();
    ref[1].reset();
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  };
  reset();
  bool ok = true;

  for (int f0 = sp.begin; f0 < sp.end;) {
    const int seg_end = cur.seg_end;
    // this warp's pages of the segment: i % 4 == warp, i counted from the span's start
    for (int i = f0 - sp.begin + ((warp - (f0 - sp.begin)) & (kConsumerWarps - 1)); i < seg_end - sp.begin;
         i += kConsumerWarps) {
      const int f = sp.begin + i;
      const int st = i % kStages;
      if (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait_fast(&s.full[st], (i / kStages) & 1));
        if (!ok && lane == 0) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
      }
      const int pos0 = cur.pos0(t, f);
      const uint8_t* kst = s.k[st];
      const uint32_t vst = smem_addr(s.v[st]);
      const bool edge = pos0 < cur.lo || pos0 + kPage > cur.L;
      const bool in0 = pos0 + r0 >= cur.lo && pos0 + r0 < cur.L;          // row r0 is visible
      const bool in1 = pos0 + r0 + 2 >= cur.lo && pos0 + r0 + 2 < cur.L;  // row r0 + 2

      // ---- S^T = K q^T: four chains of MMAs ----
      float sc[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[k][e] = 0.f;
#pragma unroll
      for (int k = 0; k < kChunks * 2; ++k) {  // chunk, j
        const uint8_t* base = kst + (k >> 1) * fp8::kChunkBytes;
        const uint4 a = *reinterpret_cast<const uint4*>(base + fp8::swz(r0, 2 * tq + (k & 1)));
        const uint4 b = *reinterpret_cast<const uint4*>(base + fp8::swz(r0 + 2, 2 * tq + (k & 1)));
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int w = 0; w < 4; w += 2) {
          const uint4 q = s.qfrag[2 * k + w / 2][qlane];
          fp8::mma_f16_16816(sc[w], fp8::lo_f16x2(aw[w]), fp8::lo_f16x2(bw[w]), fp8::hi_f16x2(aw[w]),
                             fp8::hi_f16x2(bw[w]), q.x, q.y);
          fp8::mma_f16_16816(sc[w + 1], fp8::lo_f16x2(aw[w + 1]), fp8::lo_f16x2(bw[w + 1]), fp8::hi_f16x2(aw[w + 1]),
                             fp8::hi_f16x2(bw[w + 1]), q.z, q.w);
        }
      }
      const float kf0 = fp8::scale_value(s.k_scale[st][r0]), kf1 = fp8::scale_value(s.k_scale[st][r0 + 2]);
      float kv0 = fp8::scale_log2(s.v_scale[st][r0]), kv1 = fp8::scale_log2(s.v_scale[st][r0 + 2]);
      // x[0..3]: (row r0; heads 0, 1), (row r0 + 2; heads 0, 1), in log2 units
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = ((sc[0][e] + sc[1][e]) + (sc[2][e] + sc[3][e])) * (e < 2 ? kf0 : kf1) * qs[e & 1];
      if (edge) {
        if (!in0) { x[0] = x[1] = -INFINITY; kv0 = 0.f; }
        if (!in1) { x[2] = x[3] = -INFINITY; kv1 = 0.f; }
        // zero V rows outside [lo, L): weight 0 times NaN would be NaN
#pragma unroll 1
        for (int rr = 0; rr < kPage; ++rr) {
          const int pos = pos0 + rr;
          if ((pos < cur.lo || pos >= cur.L) && lane < 16)
            st_shared_v4(vst + (lane >> 3) * fp8::kChunkBytes + rr * 128 + (lane & 7) * 16, make_uint4(0, 0, 0, 0));
        }
        fence_proxy_async_smem();  // before TMA rewrites this stage
        __syncwarp();
      }

      // ---- online softmax, in log2 units ----
      float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
      float mt[2] = {fmaxf(x[0] + kv0, x[2] + kv1), fmaxf(x[1] + kv0, x[3] + kv1)};
      if (__any_sync(0xffffffffu, mx[0] > ref[0].m || mx[1] > ref[1].m || mt[0] > ref[0].T || mt[1] > ref[1].T)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], o));
            mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], o));
          }
          float ls, as;
          ref[h].move(mx[h], mt[h], ls, as);
          l[h] *= ls;
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            acc[n][h] *= as;
            acc[n][2 + h] *= as;
          }
        }
      }
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const fp8::Reference& r = ref[e & 1];
        const float d = x[e] - r.m_use();
        l[e & 1] += ex2_approx(d);
        w[e] = ex2_approx(d + (r.weight_bias() + (e < 2 ? kv0 : kv1)));
      }
      const uint32_t pb0 = fp8::transpose_8x8(fp8::pack_f16x2(w[0], w[1]));  // positions 4 t, 4 t + 1
      const uint32_t pb1 = fp8::transpose_8x8(fp8::pack_f16x2(w[2], w[3]));  // 4 t + 2, 4 t + 3

      // ---- O^T += V^T P^T ----
      const uint32_t vrow = vst + (lane & 15) * 128;
#pragma unroll
      for (int np = 0; np < 8; ++np) {  // 32 dims each: lanes 0..15 address the first 16, lanes 16..31 the others
        uint32_t r[4];
        fp8::ldmatrix_b8_x2_trans(
            vrow + (np >> 2) * fp8::kChunkBytes + (((2 * (np & 3) + (lane >> 4)) ^ (lane & 7)) << 4), r);
#pragma unroll
        for (int u = 0; u < 2; ++u)
          fp8::mma_f16_16816(acc[2 * np + u], fp8::lo_f16x2(r[2 * u]), fp8::lo_f16x2(r[2 * u + 1]),
                             fp8::hi_f16x2(r[2 * u]), fp8::hi_f16x2(r[2 * u + 1]), pb0, pb1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.empty[st]);
    }

    {
      // ---------------- finish this sequence's segment ----------------
      // The four warps' results are merged two by two: warps 2 and 3 hand
      // theirs to warps 0 and 1 through shared memory, and all threads join
      // what those leave there.  Lane t of the four that hold the same values
      // takes every fourth 16-dim block.
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
      // (one copy of the code for both turns: it runs rarely, and what it costs is
      // mostly fetching its instructions)
#pragma unroll 1
      for (int turn = 0; turn < 2; ++turn) {
        const bool join = turn == 1;
        if ((warp < kConsumerWarps / 2) == join) {
          const int slot = warp & 1;
          float fm[2], fo[2];  // factors of this warp's values and of the slot's
#pragma unroll
          for (int h = 0; h < kG; ++h) {
            const float mo = join ? s.merge_m[slot][h] : -INFINITY, lo = join ? s.merge_l[slot][h] : 0.f;
            const float M = fmaxf(ref[h].m, mo), M_use = M == -INFINITY ? 0.f : M;
            fm[h] = exp2f(ref[h].m - M_use);
            fo[h] = exp2f(mo - M_use);
            // (a sum under m = -inf is 0, or a NaN that has to show)
            l[h] = (ref[h].m == -INFINITY ? l[h] : fm[h] * l[h]) + (mo == -INFINITY ? lo : fo[h] * lo);
            if (!join) fm[h] = 1.f;
            __syncwarp();
            if (lane == 0) {
              s.merge_m[slot][h] = M;
              s.merge_l[slot][h] = l[h];
            }
          }
          // 2^(R - 15) in two exact steps (it may lie below the normal range)
          float u0[kG], u1[kG];
#pragma unroll
          for (int h = 0; h < kG; ++h) fp8::unscale_factors(ref[h].R, u0[h], u1[h]);
          float* dst = &s.merge_o[slot][0][16 * tq + g];
          float old[4][4];
          if (join) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) old[j][e] = dst[(e & 1) * kD + 64 * j + 8 * (e >> 1)];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a01 = tq & 1 ? acc[4 * j + 1][e] : acc[4 * j][e];
              const float a23 = tq & 1 ? acc[4 * j + 3][e] : acc[4 * j + 2][e];
              const float mine = (tq & 2 ? a23 : a01) * u0[e & 1] * u1[e & 1] * fm[e & 1];
              dst[(e & 1) * kD + 64 * j + 8 * (e >> 1)] = join ? fmaf(old[j][e], fo[e & 1], mine) : mine;
            }
        }
        named_barrier_sync(1, kConsumerWarps * 32);
      }
      const int tt = threadIdx.x;  // 0..127: 2 heads x 64 groups of 4 dims
      const int h = tt >> 6;
      const int d0 = (tt & 63) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kConsumerWarps / 2; ++w) M = fmaxf(M, s.merge_m[w][h]);
      float Lsum = 0.f;
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
      // (with M = -inf every weight was 0 or NaN; a NaN has to show)
      const float M_use = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < kConsumerWarps / 2; ++w) {
        const float fw = exp2f(s.merge_m[w][h] - M_use);
        Lsum += (s.merge_m[w][h] == -INFINITY ? 1.f : fw) * s.merge_l[w][h];
        const float4 a = *reinterpret_cast<const float4*>(&s.merge_o[w][h][d0]);
        O.x += fw * a.x;
        O.y += fw * a.y;
        O.z += fw * a.z;
        O.w += fw * a.w;
      }
      if (cur.whole(t, sp)) {
        const float inv = Lsum > 0.f ? 1.f / Lsum : Lsum;
        const size_t row = static_cast<size_t>(cur.b) * kHq + hq0 + h;
        store_out4(p, row * kD + d0, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
      } else if ((static_cast<int64_t>(gb) + cur.b + 1) * kHq > p.part_rows) {
        if (tt == 0) report(p.status, ATTN_DEV_INTERNAL);  // cannot happen: slot beyond the workspace
      } else {
        const float2 ml = partial_stats(M, Lsum);
        const size_t slot = (static_cast<size_t>(gb) + cur.b) * kHq + hq0 + h;
        *reinterpret_cast<float4*>(p.part_o + slot * kD + d0) = O;
        if (d0 == 0) p.part_ml[slot] = ml;
        if (p.merge_in_grid) sliding::merge_partials(p, t, s, cur.b, gb, c, h, d0, ml.x, ml.y, O);
      }
      if (seg_end < sp.end) publish_q();
      named_barrier_sync(1, kConsumerWarps * 32);  // merge buffers and q free again
      reset();
    }
    f0 = seg_end;
    if (f0 < sp.end) {
      cur.advance(p, t, sp, f0);  // lands on the sequence whose q is in qn
      take_q();
    }
  }
  allow_dependent_launch();
}

}  // namespace sliding_fp8
}  // namespace pda
