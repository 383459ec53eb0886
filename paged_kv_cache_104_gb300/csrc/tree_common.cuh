// What the kernels for drafted tokens share: a sequence's lengths with their
// checks, and which stored keys a drafted token sees.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace pkv {

struct TreeSeq {
  int len;      // stored tokens, the drafted ones among them
  int drafted;  // 0: nothing to do (no drafted tokens, or an invalid sequence)
  int row0;     // first row of q
};

// Sequence b's lengths; what is out of range is recorded (report) and skipped.
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, bool report) {
  TreeSeq s;
  s.row0 = __ldg(a.draft_offsets + b);
  const int end = __ldg(a.draft_offsets + b + 1);
  s.len = __ldg(a.seq_lens + b);
  const bool rows_ok = s.row0 >= 0 && end >= s.row0 && end <= a.num_rows && end - s.row0 <= a.max_draft;
  s.drafted = rows_ok ? end - s.row0 : 0;
  if (!rows_ok) {
    if (report) record_error(a.err, DEVERR_DRAFT_RANGE);
  } else if (s.drafted > 0) {
    const bool len_ok = s.len >= s.drafted && s.len <= a.max_seq_len &&
                        (int64_t)s.len <= (int64_t)a.max_blocks_per_seq * kBlockSize;
    if (!len_ok) {
      if (report) record_error(a.err, DEVERR_SEQLEN_RANGE);
      s.drafted = 0;
    }
  }
  return s;
}

// The drafted tokens that drafted token i of the sequence sees, as bits: its
// mask's word, or in a chain itself and the ones before it.
__device__ __forceinline__ uint64_t tree_bits(const TreeArgs& a, const TreeSeq& s, int i) {
  const uint64_t all = s.drafted >= 64 ? ~0ull : (1ull << s.drafted) - 1;
  const uint64_t word =
      a.tree_mask ? (uint64_t)__ldg(reinterpret_cast<const unsigned long long*>(a.tree_mask) + s.row0 + i)
                  : (2ull << i) - 1;   // i = 63: 2 << 63 wraps to 0, all bits
  return word & all;
}

}  // namespace pkv
