// joined.cuh -- decodeGQA behind a shared prefix as one list of pages per
// sequence: the prefix's pages, then its own.  The decode and combine kernels
// (global.cuh, combine.cuh) run on it unchanged but for three questions that
// their code asks of the parameters: a sequence's length, where a page is
// listed, and which positions are none.
//
// Positions are counted over whole pages: the prefix's are 0 .. prefix_len - 1,
// the sequence's own start at the next page, 16 * ceil(prefix_len / 16), and what
// lies between is a hole.  (Decode attention does not depend on the numbers.)
//
// Every sequence reads the prefix's pages for itself, from L2 after the first,
// but there is no kernel for the prefix, and where the lists are short, with a
// block for each, no merge either: the better way where the prefix is short or
// the batch small (attn_decode_global_prefix chooses).
#pragma once

#include "combine.cuh"
#include "global.cuh"

namespace pda {

struct JoinedParams : DecodeParams {
  // A sequence's start in pages; 1 and 4, us: 8 sequences behind 5003 19.4 and
  // 18.7, 26 of up to 1413 behind 6 20.0 and 17.9, 32 of 300 behind 100 17.9 and 18.1.
  static constexpr int kSeqWeight = 4;
  const int32_t* prefix_table;  // [prefix_blocks]
  const int32_t* prefix_len;    // one int32 on the device
  int32_t prefix_blocks;
  int32_t whole_sequences;      // block g takes sequence g: no partials, no merge
};
__device__ __forceinline__ bool by_sequence(const JoinedParams& p) { return p.whole_sequences; }

// (Read past L1: asked before the previous kernel is done, too.)
__device__ __forceinline__ int joined_prefix(const JoinedParams& p, bool report_it) {
  const int raw = __ldcg(p.prefix_len);
  const int cap = p.prefix_blocks < ATTN_MAX_SEQ_LEN / kPage ? p.prefix_blocks * kPage : ATTN_MAX_SEQ_LEN;
  if (raw < 0 || raw > cap) {
    if (report_it) report(p.status, ATTN_DEV_BAD_SEQ_LEN);
    return raw < 0 ? 0 : cap;
  }
  return raw;
}

__device__ __forceinline__ int schedule_len(const JoinedParams& p, int L, bool report_it) {
  const int own = clamp_len(p, L, report_it);
  const int n = joined_prefix(p, report_it);
  return own > 0 ? (n + kPage - 1) / kPage * kPage + own : n;
}

__device__ __forceinline__ const int32_t* table_entry(const JoinedParams& p, int b, int lp) {
  const int n = (joined_prefix(p, false) + kPage - 1) / kPage;
  if (lp < n) return lp < 0 || lp >= p.prefix_blocks ? nullptr : p.prefix_table + lp;
  return table_entry(static_cast<const DecodeParams&>(p), b, lp - n);
}

struct PrefixHole {
  int begin, end;
  __device__ __forceinline__ bool covers(int pos, int n) const { return pos + n > begin && pos < end; }
};
__device__ __forceinline__ PrefixHole hole_of(const JoinedParams& p) {
  const int len = joined_prefix(p, false);
  return {len, (len + kPage - 1) / kPage * kPage};
}

}  // namespace pda
