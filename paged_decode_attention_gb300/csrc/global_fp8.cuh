// global_fp8.cuh -- decodeGQA over an 8-bit cache (fp8.cuh): 16 query heads
// over 1 KV head, D = 512, scale 1.  The formulas are sliding_fp8.cuh's.
//
// A page is 16 KB here (K and V) against 32 KB in bf16, so at the rate of
// memory the bf16 kernel's work per page, four copies of the softmax and an
// exchange of partial logits for every page, would take twice the share of
// the time.  Instead the four consumer warps take two consecutive pages of a
// segment together, with two barriers to a group:
//   * every warp multiplies its own 128 of the 512 dims of both pages' keys (q
//     fragments in registers) and leaves the partial logits in shared memory;
//   * each warp adds up those of eight of the 32 positions, scales and masks
//     them, and leaves their weights as A fragments of the second product;
//   * every warp multiplies both pages' weights with its own 128 output dims,
//     so that no output is merged between warps.
// So each byte is widened once and the softmax runs once per position.
// On 16 contexts of 131072 positions: 335 us, 0.95 of the measured copy rate;
// with groups of four pages, which hold more of the ring (five stages beside
// their partial logits), 381 us; with page w's logits by warp w alone and q read
// from shared memory 410 us.
#pragma once

#include "fp8.cuh"
#include "global.cuh"
#include "tcgen05.cuh"

namespace pda {
namespace global_fp8 {

using global::kD;
using global::kHq;

constexpr int kGroup = 2;          // pages taken together
constexpr int kConsumerWarps = 4;  // a chunk of 128 dims each in the products, a (page, n-tile) in the softmax
constexpr int kThreads = (kConsumerWarps + 1) * 32;
constexpr int kChunks = kD / 128;                     // 4: one per consumer warp in the second product
constexpr int kPageBytes = kPage * kD;                // 8 KB
constexpr int kStages = 6;
constexpr int kStageTx = 2 * kPageBytes + 2 * kPage;  // K, V and their scales
constexpr int kBlocksPerSm = global::kBlocksPerSm;    // the plan of the bf16 kernel
constexpr int kWarmPages = 4;
constexpr int kKSteps = kD / 16 / kConsumerWarps;     // 8 of the first product, per warp

static_assert(kChunks == kConsumerWarps, "128 output dims per warp");
static_assert(2 * kGroup == kConsumerWarps, "two warps per page of a group");

struct Smem {
  alignas(1024) uint8_t k[kStages][kPageBytes];  // kChunks tiles of [16 rows][128 dims], swizzled
  alignas(1024) uint8_t v[kStages][kPageBytes];
  alignas(128) uint8_t k_scale[kStages][128];  // 16 bytes used: a copy lands on a 128-byte boundary
  alignas(128) uint8_t v_scale[kStages][128];
  alignas(16) float4 xs[kGroup][kConsumerWarps][2][32];  // partial logits: page, chunk, n-tile
  alignas(16) uint2 pfrag[kGroup][2][32];        // weights of the group's pages, as A fragments by n-tile
  float2 row_max[kConsumerWarps][kHq];           // the warps' row maxima of x and of x + kv (fp8.cuh)
  alignas(16) int32_t moves[kConsumerWarps];     // a warp's positions move a reference
  uint32_t q_max[kConsumerWarps][kHq];
  float row_sum[kConsumerWarps][kHq];
  SeqTable table;
  alignas(8) uint64_t full[kStages];
  alignas(8) uint64_t empty[kStages];
};

constexpr size_t kSmemBytes = sizeof(Smem) + 1024;  // + alignment slack
static_assert(kBlocksPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of the resident blocks");

template <typename Params>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                  const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& s = fp8::aligned_smem<Smem>(smem_raw);

  const int gb = blockIdx.x;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(&s.full[st], 1);
      mbar_init(&s.empty[st], kConsumerWarps);
    }
    fence_mbar_init();
  }
  if (warp == kConsumerWarps && lane == 0) {
    prefetch_tensor_map(&tm_k);
    prefetch_tensor_map(&tm_v);
    prefetch_tensor_map(&tm_ks);
    prefetch_tensor_map(&tm_vs);
  }
  // The prologue overlaps the previous kernel; see global.cuh.
  build_seq_table_hint(p, s.table, gb);  // ends with __syncthreads
  if (warp == kConsumerWarps) {
    warm_first_pages(p, s.table, kWarmPages, [&](int32_t y) {
      // (pools of bytes, so the typed pointers of the parameters are cast)
      bulk_prefetch_l2(reinterpret_cast<const uint8_t*>(p.k_pool) + static_cast<size_t>(y) * kD, kPageBytes);
      bulk_prefetch_l2(reinterpret_cast<const uint8_t*>(p.v_pool) + static_cast<size_t>(y) * kD, kPageBytes);
    });
  } else {
    warm_q(p, s.table, kHq * kD, 0, kHq * kD * 2, kConsumerWarps * 32);
  }
  wait_for_primary_grid();
  allow_dependent_launch();
  int first = warp == kConsumerWarps ? page_entry(p, s.table, s.table.span, lane, false) : 0;
  confirm_seq_table(p, s.table, gb);  // ends with __syncthreads
  const SeqTable& t = s.table;
  const Span sp = t.span;
  const int n_pages = sp.end - sp.begin;
  if (n_pages <= 0) {
    if (by_sequence(p) && gb < p.batch)  // there is no merge to write the empty sums
      for (int i = threadIdx.x; i < kHq * kD / 4; i += kThreads)
        store_out4(p, static_cast<size_t>(gb) * kHq * kD + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }

  if (warp == kConsumerWarps) {
    // ---------------- producer ----------------
    const uint64_t policy = l2_policy_evict_first();
    if (t.rebuilt) first = page_entry(p, t, sp, lane, true);
    produce_pages<kStages, kStageTx>(p, t, sp, s.full, s.empty, first, [&](int stage, int32_t y) {
      tma_load_3d_hint(s.k[stage], &tm_k, 0, y, 0, &s.full[stage], policy);
      tma_load_3d_hint(s.v[stage], &tm_v, 0, y, 0, &s.full[stage], policy);
      const int32_t ys = y < 0 ? -1 : y / kPage;  // 16 bytes per page in the scale pools
      tma_load_2d(s.k_scale[stage], &tm_ks, 0, ys, &s.full[stage]);
      tma_load_2d(s.v_scale[stage], &tm_vs, 0, ys, &s.full[stage]);
    });
    return;
  }

  // ---------------- consumers ----------------
  const int g = lane >> 2;  // fragment row: query heads g and g + 8
  const int tq = lane & 3;
  constexpr int kConsumers = kConsumerWarps * 32;
  const int page = warp >> 1;  // of the group, and its n-tile, in the softmax
  const int tile = warp & 1;

  PageCursor cur;
  cur.start(p, t, sp);

  // q as A fragments over this warp's 128 dims: k-step (j, word): dims 128 w +
  // 16 (2 tq + j) + 4 word .. + 3 of rows g and g + 8, scaled by each row's
  // power of two.
  uint32_t qf[kKSteps][4];
  float qs[2];  // logit factor 2^k log2(e) of rows g and g + 8
  auto load_q = [&]() {
    uint32_t amax[2] = {0, 0};
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const __nv_bfloat16* src = p.q + (static_cast<size_t>(cur.b) * kHq + g + 8 * r) * kD + 128 * warp +
                                   16 * (2 * tq + j);
        const uint4 a = ld_global_nc_v4(src), b = ld_global_nc_v4(src + 8);
        qf[4 * j][r] = a.x; qf[4 * j][2 + r] = a.y; qf[4 * j + 1][r] = a.z; qf[4 * j + 1][2 + r] = a.w;
        qf[4 * j + 2][r] = b.x; qf[4 * j + 2][2 + r] = b.y; qf[4 * j + 3][r] = b.z; qf[4 * j + 3][2 + r] = b.w;
#pragma unroll
        for (int k = 4 * j; k < 4 * j + 4; ++k)
#pragma unroll
          for (int e = r; e < 4; e += 2)
            amax[r] = max(amax[r], max(qf[k][e] << 16 & 0x7fff0000u, qf[k][e] & 0x7fff0000u));
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      amax[r] = max(amax[r], __shfl_xor_sync(0xffffffffu, amax[r], 1));
      amax[r] = max(amax[r], __shfl_xor_sync(0xffffffffu, amax[r], 2));
      if (tq == 0) s.q_max[warp][g + 8 * r] = amax[r];
    }
    named_barrier_sync(1, kConsumers);  // the other warps' maxima
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t a = 0;
#pragma unroll
      for (int k = 0; k < kConsumerWarps; ++k) a = max(a, s.q_max[k][g + 8 * r]);
      float inv;
      const int e = fp8::q_exponent(a, inv);
      qs[r] = __uint_as_float(static_cast<uint32_t>(e + 127) << 23) * kLog2e;
#pragma unroll
      for (int k = 0; k < kKSteps; ++k) {
        qf[k][r] = fp8::q_f16x2(qf[k][r], inv);
        qf[k][2 + r] = fp8::q_f16x2(qf[k][2 + r], inv);
      }
    }
  };
  auto prefetch_next_q = [&]() {
    const int nb = next_seq_in_span(p, t, sp, cur.b);
    if (nb >= 0)
      prefetch_l2(reinterpret_cast<const uint8_t*>(p.q + static_cast<size_t>(nb) * kHq * kD) + threadIdx.x * 128);
  };
  load_q();
  prefetch_next_q();

  fp8::Reference ref[2];  // rows g, g + 8 (the same in every warp)
  float l[2];             // this lane's share of the sums
  float acc[16][4];  // 16 n-tiles of 8 dims
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
  // NP (1 or 2) pages from page i of the span, page f of the list
  auto page_group = [&](auto np_c, int i, int f) {
    constexpr int NP = decltype(np_c)::value;
    const int gpos0 = cur.pos0(t, f);  // position of the group's first row
    const bool edge = gpos0 < cur.lo || gpos0 + NP * kPage > cur.L;
    int st[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) st[j] = (i + j) % kStages;
    // lane j waits for page j (one wait's latency for both), and the barrier of the
    // warp hands on what it sees: a vote would order no memory.  (ok is a lane's own:
    // a wait that runs out is reported by its lane and ends that lane's waits.)
    if (ok && lane < NP) {
      ok = mbar_wait_fast(&s.full[(i + lane) % kStages], ((i + lane) / kStages) & 1);
      if (!ok) report(p.status, ATTN_DEV_WAIT_TIMEOUT);
    }
    __syncwarp();

    // ---- every page's logits over this warp's dims ----
    float sc[NP][2][2][4];  // page, n-tile, even / odd k-steps
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[j][a][b][e] = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const uint8_t* kst = s.k[st[j]] + warp * fp8::kChunkBytes;
        const uint4 a = *reinterpret_cast<const uint4*>(kst + fp8::swz(fp8::dealt_row(g), 2 * tq + k));
        const uint4 b = *reinterpret_cast<const uint4*>(kst + fp8::swz(fp8::dealt_row(g) + 2, 2 * tq + k));
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t (&q)[4] = qf[4 * k + w];
          fp8::mma_f16_16816(sc[j][0][w & 1], q[0], q[1], q[2], q[3], fp8::lo_f16x2(aw[w]), fp8::hi_f16x2(aw[w]));
          fp8::mma_f16_16816(sc[j][1][w & 1], q[0], q[1], q[2], q[3], fp8::lo_f16x2(bw[w]), fp8::hi_f16x2(bw[w]));
        }
      }
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        s.xs[j][warp][nt][lane] =
            make_float4(sc[j][nt][0][0] + sc[j][nt][1][0], sc[j][nt][0][1] + sc[j][nt][1][1],
                        sc[j][nt][0][2] + sc[j][nt][1][2], sc[j][nt][0][3] + sc[j][nt][1][3]);
    named_barrier_sync(1, kConsumers);

    // ---- this warp's eight positions: x[e]: head g + 8 (e >> 1), position pos0 + 4 tq + 2 tile + (e & 1) ----
    float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    float kv[2] = {0.f, 0.f};  // log2 of those positions' value scales
    if (page < NP) {
      const int sp_ = NP == 2 && page ? st[NP - 1] : st[0];
      const int pos = gpos0 + page * kPage + 4 * tq + 2 * tile;
      float4 v = s.xs[page][0][tile][lane];
#pragma unroll
      for (int w = 1; w < kConsumerWarps; ++w) {
        const float4 o = s.xs[page][w][tile][lane];
        v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
      }
      const uint32_t kb = *reinterpret_cast<const uint16_t*>(&s.k_scale[sp_][4 * tq + 2 * tile]);
      const uint32_t vb = *reinterpret_cast<const uint16_t*>(&s.v_scale[sp_][4 * tq + 2 * tile]);
      const float k0 = fp8::scale_value(kb & 255u), k1 = fp8::scale_value(kb >> 8);
      if (!edge || (pos >= cur.lo && pos < cur.L)) {
        kv[0] = fp8::scale_log2(vb & 255u);
        x[0] = v.x * k0 * qs[0];
        x[2] = v.z * k0 * qs[1];
      }
      if (!edge || (pos + 1 >= cur.lo && pos + 1 < cur.L)) {
        kv[1] = fp8::scale_log2(vb >> 8);
        x[1] = v.y * k1 * qs[0];
        x[3] = v.w * k1 * qs[1];
      }
    }
    // ---- weights ----
    // The references move only when some position exceeds them, which after a
    // sequence's first pages is rare.  So the weights are formed with the
    // references as they are, and with them goes a note whether this warp's
    // positions exceed one; if any warp's do, all maxima are exchanged and the
    // weights formed anew.
    float ps[2];  // this group's share of the sums
    auto weights = [&]() {
      float pr[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mu = ref[r].m_use(), bias = ref[r].weight_bias();
        const float d0 = x[2 * r] - mu, d1 = x[2 * r + 1] - mu;
        ps[r] = ex2_approx(d0) + ex2_approx(d1);
        pr[2 * r] = ex2_approx(d0 + (bias + kv[0]));
        pr[2 * r + 1] = ex2_approx(d1 + (bias + kv[1]));
      }
      if (page < NP)
        s.pfrag[page][tile][lane] = make_uint2(fp8::pack_f16x2(pr[0], pr[1]), fp8::pack_f16x2(pr[2], pr[3]));
    };
    float mx[2], mt[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(x[2 * r], x[2 * r + 1]);
      mt[r] = fmaxf(x[2 * r] + kv[0], x[2 * r + 1] + kv[1]);
    }
    const bool moves = __any_sync(0xffffffffu, mx[0] > ref[0].m || mx[1] > ref[1].m || mt[0] > ref[0].T ||
                                                   mt[1] > ref[1].T);
    weights();
    if (lane == 0) s.moves[warp] = moves;
    named_barrier_sync(1, kConsumers);
    const int4 mv = *reinterpret_cast<const int4*>(s.moves);
    if (mv.x | mv.y | mv.z | mv.w) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mt[r] = fmaxf(mt[r], __shfl_xor_sync(0xffffffffu, mt[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        mt[r] = fmaxf(mt[r], __shfl_xor_sync(0xffffffffu, mt[r], 2));
        if (tq == 0) s.row_max[warp][g + 8 * r] = make_float2(mx[r], mt[r]);
      }
      named_barrier_sync(1, kConsumers);
      float scale[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float2 m2 = s.row_max[0][g + 8 * r];
#pragma unroll
        for (int w = 1; w < kConsumerWarps; ++w) {
          const float2 o = s.row_max[w][g + 8 * r];
          m2 = make_float2(fmaxf(m2.x, o.x), fmaxf(m2.y, o.y));
        }
        float ls;
        ref[r].move(m2.x, m2.y, ls, scale[r]);
        l[r] *= ls;
      }
#pragma unroll
      for (int b = 0; b < 16; ++b) {
        acc[b][0] *= scale[0];
        acc[b][1] *= scale[0];
        acc[b][2] *= scale[1];
        acc[b][3] *= scale[1];
      }
      weights();
      named_barrier_sync(1, kConsumers);
    }
    l[0] += ps[0];
    l[1] += ps[1];

    // ---- O += P V over this warp's 128 dims ----
    const uint32_t vst = smem_addr(s.v[0]) + warp * fp8::kChunkBytes;
    if (edge) {
      // zero this warp's V rows outside [lo, L): weight 0 times NaN would be NaN
#pragma unroll 1
      for (int rr = 0; rr < NP * kPage; ++rr) {
        const int pos = gpos0 + rr;
        if ((pos < cur.lo || pos >= cur.L) && lane < 8)
          st_shared_v4(vst + (NP == 2 && rr >= kPage ? st[NP - 1] : st[0]) * kPageBytes + (rr & (kPage - 1)) * 128 +
                           lane * 16,
                       make_uint4(0, 0, 0, 0));
      }
      fence_proxy_async_smem();  // before TMA rewrites these stages
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const uint2 p0 = s.pfrag[j][0][lane], p1 = s.pfrag[j][1][lane];
      const uint32_t vrow = vst + st[j] * kPageBytes + (lane & 15) * 128;
      uint32_t r[4][4];
#pragma unroll
      for (int np = 0; np < 4; ++np)  // 32 dims each: lanes 0..15 address the first 16, lanes 16..31 the others
        fp8::ldmatrix_b8_x2_trans(vrow + (((2 * np + (lane >> 4)) ^ (lane & 7)) << 4), r[np]);
#pragma unroll
      for (int np = 0; np < 4; ++np)
#pragma unroll
        for (int u = 0; u < 4; ++u)  // 8 dims each
          fp8::mma_f16_16816(acc[4 * np + u], p0.x, p0.y, p1.x, p1.y, fp8::lo_f16x2(r[np][u]), fp8::hi_f16x2(r[np][u]));
    }
    __syncwarp();
    if (lane < NP) mbar_arrive(&s.empty[(i + lane) % kStages]);
  };

  for (int i = 0; i < n_pages;) {
    const int f = sp.begin + i;
    if (f >= t.prefix[cur.b + 1]) {
      cur.advance(p, t, sp, f);
      load_q();
      prefetch_next_q();
    }
    const int n = min(kGroup, cur.seg_end - f);  // pages of this group
    if (n == 2)
      page_group(std::integral_constant<int, 2>{}, i, f);
    else
      page_group(std::integral_constant<int, 1>{}, i, f);
    i += n;

    if (f + n == cur.seg_end) {
      // ---------------- finish this sequence's segment ----------------
      float lt[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        lt[r] = l[r] + __shfl_xor_sync(0xffffffffu, l[r], 1);
        lt[r] += __shfl_xor_sync(0xffffffffu, lt[r], 2);
        if (tq == 0) s.row_sum[warp][g + 8 * r] = lt[r];
      }
      named_barrier_sync(1, kConsumers);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        lt[r] = s.row_sum[0][g + 8 * r];
#pragma unroll
        for (int w = 1; w < kConsumerWarps; ++w) lt[r] += s.row_sum[w][g + 8 * r];
      }
      const bool whole = cur.whole(t, sp);
      if (!whole && (static_cast<int64_t>(gb) + cur.b + 1) * kHq > p.part_rows) {
        if (lane == 0) report(p.status, ATTN_DEV_INTERNAL);  // cannot happen: slot beyond the workspace
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const size_t row = static_cast<size_t>(whole ? cur.b : gb + cur.b) * kHq + g + 8 * r;
          const float inv = lt[r] > 0.f ? 1.f / lt[r] : lt[r];  // 0, or a NaN that has to show
          float u0, u1;
          fp8::unscale_factors(ref[r].R, u0, u1);
#pragma unroll
          for (int b = 0; b < 16; ++b) {
            const float v0 = acc[b][2 * r] * u0 * u1, v1 = acc[b][2 * r + 1] * u0 * u1;
            const size_t at = row * kD + 128 * warp + 8 * b + 2 * tq;
            if (whole)
              store_out2(p, at, v0 * inv, v1 * inv);
            else
              *reinterpret_cast<float2*>(p.part_o + at) = make_float2(v0, v1);
          }
          if (!whole && warp == 0 && tq == 0) p.part_ml[row] = partial_stats(ref[r].m, lt[r]);
        }
      }
      named_barrier_sync(1, kConsumers);  // row_sum read
      reset();
    }
  }
}

}  // namespace global_fp8
}  // namespace pda
