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

// ---- the balanced plan of the tensor-core kernels
//
// A stream is one (sequence, KV head), or with row tiles one (sequence, KV
// head, 256 rows); a stage is one of its 128-key tiles.  The stages of the
// batch, in order, are cut into one equal share per CTA; what a CTA gets of a
// stream is an item.  One warp of every CTA works the plan out from the
// lengths, 32 sequences at a time, so no shared memory grows with the batch.
constexpr int kTreeTile = 128;      // keys of a stage
constexpr int kTreeRows = 256;      // rows of a stream
constexpr int kTreeMaxCtas = 160;

struct TreeItem {
  int n;          // stages; 0: no more items
  int t0;         // first key tile
  int b, g;
  int row0;       // first row (drafted token * group + query head) of the stream
  int rows;       // rows of the stream, 1 .. 256 (without row tiles: of the sequence)
  int q_tok;      // q's row of the sequence's first drafted token
  int len, ctx;   // stored tokens, and those before the drafted ones
  int slot;       // -1: the whole stream; else which of the CTA's two partials this is
  int pieces;     // of the stream, where this is the first of several (else 0)
};

template <bool ROW_TILES>
struct TreePlan {
  const TreeArgs& a;
  const int lane, group;
  int windows, w = -1;                 // windows of 32 sequences, the loaded one
  int total = 0, ctas = 0;             // stages; CTAs that share them
  int pos = 0, end = 0;                // this CTA's next stage and end
  int start = 0, sum = 0;              // the window's first stage, its stages
  TreeSeq seq;                         // lane: its sequence
  int tiles = 0, stages = 0, first = 0;

  __device__ TreePlan(const TreeArgs& args)
      : a(args), lane(threadIdx.x & 31), group(args.num_q_heads / args.num_kv_heads),
        windows((args.num_seqs + 31) / 32) {
    const bool report = blockIdx.x == 0;
    int mine = 0;
    for (int i = 0; i < windows; ++i) {
      load(i, report);
      mine += stages;
    }
    total = __reduce_add_sync(0xffffffffu, mine);
    ctas = min((int)gridDim.x, total);
    if ((int)blockIdx.x >= ctas) return;
    pos = (int)((int64_t)blockIdx.x * total / ctas);
    end = (int)((int64_t)(blockIdx.x + 1) * total / ctas);
    open(0);
  }
  __device__ void load(int i, bool report = false) {
    if (w == i) return;
    w = i;
    const int b = 32 * i + lane;
    seq.len = seq.drafted = seq.row0 = 0;
    if (b < a.num_seqs) seq = tree_seq(a, b, report);
    tiles = seq.drafted > 0 ? (seq.len + kTreeTile - 1) / kTreeTile : 0;
    const int parts = ROW_TILES ? (seq.drafted * group + kTreeRows - 1) / kTreeRows : 1;
    stages = tiles * parts * a.num_kv_heads;
  }
  // window i, whose first stage is `start`
  __device__ void open(int i) {
    load(i);
    int x = stages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    first = start + x - stages;
    sum = __shfl_sync(0xffffffffu, x, 31);
  }
  __device__ int cta_of(int stage) const { return (int)(((int64_t)(stage + 1) * ctas - 1) / total); }
  // The CTA's next item (n = 0: none).  Every lane gets it.
  __device__ TreeItem next() {
    TreeItem it;
    it.n = it.slot = it.pieces = 0;
    if (pos >= end) return it;
    while (pos >= start + sum) {
      start += sum;
      open(w + 1);
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, first <= pos && pos < first + stages)) - 1;
    const int at = __shfl_sync(0xffffffffu, first, l), nt = __shfl_sync(0xffffffffu, tiles, l);
    const int drafted = __shfl_sync(0xffffffffu, seq.drafted, l);
    const int stream = (pos - at) / nt, s0 = at + stream * nt, s1 = s0 + nt;
    const int parts = ROW_TILES ? (drafted * group + kTreeRows - 1) / kTreeRows : 1;
    it.b = 32 * w + l;
    it.g = stream / parts;
    it.row0 = stream % parts * kTreeRows;
    it.rows = ROW_TILES ? min(drafted * group - it.row0, kTreeRows) : drafted * group;
    it.t0 = pos - s0;
    it.n = min(s1, end) - pos;
    it.q_tok = __shfl_sync(0xffffffffu, seq.row0, l);
    it.len = __shfl_sync(0xffffffffu, seq.len, l);
    it.ctx = it.len - drafted;
    if (it.n == nt) {
      it.slot = -1;
    } else {
      it.slot = it.t0 == 0 ? 1 : 0;
      if (it.t0 == 0) it.pieces = cta_of(s1 - 1) - (int)blockIdx.x + 1;
    }
    pos += it.n;
    return it;
  }
};

}  // namespace pkv
