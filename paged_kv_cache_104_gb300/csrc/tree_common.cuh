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

// Sequence b's lengths as they are given (drafted: q's rows end there).
__device__ __forceinline__ TreeSeq tree_seq_fetch(const TreeArgs& a, int b) {
  TreeSeq s;
  s.row0 = __ldg(a.draft_offsets + b);
  s.drafted = __ldg(a.draft_offsets + b + 1);
  s.len = __ldg(a.seq_lens + b);
  return s;
}

// ... with their checks: what is out of range is recorded (report) and skipped.
__device__ __forceinline__ TreeSeq tree_seq_check(const TreeArgs& a, TreeSeq s, bool report) {
  const int end = s.drafted;
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
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, bool report) {
  return tree_seq_check(a, tree_seq_fetch(a, b), report);
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
// head, 256 rows), or a pair of KV heads of up to 128 rows each, cut into tiles of
// 128 keys.  The tiles of the batch, in
// order, are shared out to one persistent CTA per SM, and what a CTA gets of a
// stream is an item.  Where a CTA gets many tiles, shares are of equal weight:
// 3 units for a tile of more than 128 rows, 2 for one of fewer, a tile with the
// CTA in whose units it starts; a stream's last tile is followed by 10 or 6
// units for its start and end (13,000 and 7,000 cycles).  For 32 ragged
// sequences of 1 to 64 drafted tokens that took 60 us off the 231 of equal
// numbers of tiles (6 and 5 units, nearer to a tile's 3,300 and 2,700 cycles
// alone: 1.5% slower).  Where a CTA gets a few tiles, every tile counts alike.
// Pairs save starts and ends and cut the batch more coarsely, so sequences of up
// to eight tiles go in pairs where there is work for all CTAs: 126 of 27 to 609
// tokens 65.4 -> 55.3 us (57.0 with pairs up to four tiles only), 112 of 1 to 5
// 33.3 -> 22.6; pairs of any length made 64 of 2,301 5% slower, 105.7 -> 111.2, and
// these leave 32 ragged ones, few of them paired, at 154 instead of 150.
// One warp of every CTA works the plan out from the lengths, 32 sequences at a
// time, so no shared memory grows with the batch.
constexpr int kTreeTile = 128;      // keys of a tile
constexpr int kTreeRows = 256;      // rows of a stream
constexpr int kTreeMaxCtas = 160;
constexpr int kTreeManyTiles = 8;   // a CTA, from where on tiles are weighted
constexpr int kTreePairTiles = 2;   // ... and from where on KV heads go in pairs
constexpr int kTwinTiles = 8;       // ... of sequences of at most so many tiles
constexpr int kTwinEnds = 8;        // units for the start and end of a pair (4 or 12: up to 3% slower)

struct TreeItem {
  int n;          // tiles; 0: no more items
  int t0;         // first tile
  int b, g;       // sequence, (first) KV head
  int heads;      // 2: a pair of KV heads, of `rows` rows each
  int row0;       // first row (drafted token * group + query head) of the stream
  int rows;       // rows of the stream, 1 .. 256 (without row tiles: of the sequence)
  int q_tok;      // q's row of the sequence's first drafted token
  int len, ctx;   // stored tokens, and those before the drafted ones
  int slot;       // -1: the whole stream; else which of the CTA's two partials this is
  int pieces;     // of the stream, where this is the first of several (else 0)
};

template <bool ROW_TILES, bool PAIRS = false>
struct TreePlan {
  const TreeArgs& a;
  const int lane, group;
  const bool whole;                    // streams are not cut
  int windows, w = -1;                 // windows of 32 sequences, the loaded one
  bool weighted = false, paired = false;
  int share = 0, longer = 0;           // units of a CTA; the first `longer` CTAs have one more
  int pos = 0, end = 0;                // this CTA's next unit and end
  int start = 0, sum = 0;              // the window's first unit, its units
  TreeSeq seq;                         // lane: its sequence
  int tiles = 0, units = 0, first = 0;

  // Units of a tile of so many rows.
  __device__ int weight(int rows, bool heavy) const {
    if (!heavy || rows == 0) return rows > 0;
    return (rows > 128 ? 3 : 2) * (ROW_TILES ? 1 : (rows + kTreeRows - 1) / kTreeRows);
  }
  // Units of a stream of nt tiles, and of all the streams of a KV head.
  __device__ int stream_units(int nt, int rows, bool heavy) const {
    if (rows <= 0) return 0;
    const int each = weight(rows, heavy);
    return nt * each + (heavy ? 4 * each - 2 : 0);
  }
  __device__ int head_units(int nt, int rows, bool heavy) const {
    if (!ROW_TILES) return stream_units(nt, rows, heavy);
    return rows / kTreeRows * stream_units(nt, kTreeRows, heavy) + stream_units(nt, rows % kTreeRows, heavy);
  }
  // Two KV heads of a sequence of nt tiles are one stream?
  __device__ bool twin(int nt, int rows, bool pairs) const {
    return PAIRS && pairs && rows <= kTreeRows / 2 && nt <= kTwinTiles;
  }
  __device__ int twin_units(int nt, bool heavy) const { return heavy ? 4 * nt + kTwinEnds : nt; }
  // ... and of all of a sequence's streams.
  __device__ int seq_units(int nt, int rows, bool heavy, bool pairs) const {
    if (twin(nt, rows, pairs)) return rows > 0 ? twin_units(nt, heavy) * (a.num_kv_heads >> 1) : 0;
    return head_units(nt, rows, heavy) * a.num_kv_heads;
  }
  // For one warp (active), while the others still set the CTA up.
  __device__ TreePlan(const TreeArgs& args, bool active, bool uncut = false)
      : a(args), lane(threadIdx.x & 31), group(args.num_q_heads / args.num_kv_heads), whole(uncut),
        windows((args.num_seqs + 31) / 32) {
    if (!active) return;
    const bool report = blockIdx.x == 0;
    int plain = 0, twins = 0, heavy = 0;
    // four windows' lengths are asked for before the first is looked at, the
    // first window last, as the walk often starts there
    for (int i = (windows - 1) / 4; i >= 0; --i) {
      TreeSeq s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = fetch(4 * i + j);
#pragma unroll
      for (int j = 3; j >= 0; --j) {
        const int b = 32 * (4 * i + j) + lane;
        seq = tree_seq_check(a, s[j], report && b < a.num_seqs);
        tiles = seq.drafted > 0 ? (seq.len + kTreeTile - 1) / kTreeTile : 0;
        plain += seq_units(tiles, seq.drafted * group, false, false);
        if (PAIRS) twins += seq_units(tiles, seq.drafted * group, false, true);
        heavy += seq_units(tiles, seq.drafted * group, true, PAIRS);
      }
    }
    w = 0;
    int total = __reduce_add_sync(0xffffffffu, plain);
    weighted = total >= kTreeManyTiles * (int)gridDim.x;
    paired = PAIRS && total >= kTreePairTiles * (int)gridDim.x;
    if (weighted || paired) total = __reduce_add_sync(0xffffffffu, weighted ? heavy : twins);
    // (a kernel starts with none of its code in the SM: every few instructions
    // before the first item cost a fetch, so there is one division here)
    share = total / gridDim.x;
    longer = total - share * gridDim.x;
    pos = begin_of(blockIdx.x);
    end = begin_of(blockIdx.x + 1);
    if (pos == end) return;
    open(0);
  }
  __device__ TreeSeq fetch(int i) const {
    const int b = 32 * i + lane;
    TreeSeq s;
    s.len = s.drafted = s.row0 = 0;
    if (b < a.num_seqs) s = tree_seq_fetch(a, b);
    return s;
  }
  // window i, whose first unit is `start`
  __device__ void open(int i) {
    if (w != i) {
      w = i;
      seq = tree_seq_check(a, fetch(i), false);
      tiles = seq.drafted > 0 ? (seq.len + kTreeTile - 1) / kTreeTile : 0;
    }
    units = seq_units(tiles, seq.drafted * group, weighted, paired);
    int x = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    first = start + x - units;
    sum = __shfl_sync(0xffffffffu, x, 31);
  }
  __device__ int begin_of(int cta) const { return cta * share + min(cta, longer); }
  __device__ int cta_of(int unit) const {
    const int rest = unit - longer * (share + 1);
    return rest < 0 ? unit / (share + 1) : longer + rest / share;
  }
  // Tiles that start in so many units of a stream.
  __device__ int tiles_before(int n, int each) const {
    return each == 1 ? n : each == 2 ? (n + 1) >> 1 : each == 4 ? (n + 3) >> 2 : (n + each - 1) / each;
  }
  // The CTA's next item (n = 0: none).  Every lane gets it.
  __device__ TreeItem next() {
    TreeItem it;
    it.n = it.slot = it.pieces = 0;
    while (pos < end) {
      while (pos >= start + sum) {
        if (w + 1 >= windows) {        // lengths that changed meanwhile: end here
          pos = end;
          return it;
        }
        start += sum;
        open(w + 1);
      }
      const int l = __ffs(__ballot_sync(0xffffffffu, first <= pos && pos < first + units)) - 1;
      const int at = __shfl_sync(0xffffffffu, first, l), nt = __shfl_sync(0xffffffffu, tiles, l);
      const int drafted = __shfl_sync(0xffffffffu, seq.drafted, l), rows = drafted * group;
      const bool two = twin(nt, rows, paired);
      const int per_head = two ? twin_units(nt, weighted) : head_units(nt, rows, weighted);
      int s0 = at;                                         // the stream's first unit
      it.heads = two ? 2 : 1;
      for (it.g = 0; pos - s0 >= per_head; it.g += it.heads) s0 += per_head;
      it.row0 = 0;
      it.rows = rows;
      if (ROW_TILES) {
        const int full = stream_units(nt, kTreeRows, weighted);
        while (it.rows > kTreeRows && pos - s0 >= full) {
          s0 += full;
          it.row0 += kTreeRows;
          it.rows -= kTreeRows;
        }
        it.rows = min(it.rows, kTreeRows);
      }
      const int each = two ? (weighted ? 4 : 1) : weight(it.rows, weighted);
      const int s1 = s0 + (two ? per_head : stream_units(nt, it.rows, weighted));
      if (whole && pos > s0) {                             // started in an earlier CTA
        pos = s1;
        continue;
      }
      // tiles that start in this CTA's units
      it.t0 = tiles_before(pos - s0, each);
      it.n = whole ? nt : min(tiles_before(min(s1, end) - s0, each), nt) - it.t0;
      pos = whole ? s1 : min(s1, end);
      if (it.n <= 0) {
        it.n = 0;
        continue;
      }
      it.b = 32 * w + l;
      it.q_tok = __shfl_sync(0xffffffffu, seq.row0, l);
      it.len = __shfl_sync(0xffffffffu, seq.len, l);
      it.ctx = it.len - drafted;
      if (it.n == nt) {
        it.slot = -1;
      } else {
        it.slot = it.t0 == 0 ? 1 : 0;
        // a CTA has more units than any tile, so the pieces are in CTAs one after another
        if (it.t0 == 0) it.pieces = cta_of(s0 + (nt - 1) * each) - (int)blockIdx.x + 1;
      }
      return it;
    }
    return it;
  }
};

}  // namespace pkv
