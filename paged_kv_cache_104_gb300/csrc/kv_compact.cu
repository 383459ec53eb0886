// Rows that stay move up, in place.
//
// For each sequence b and KV head g, row first + i of the sequence becomes
// what row kept[b][g][i] was (i < kept_lens[b]; keys, values and running
// weights), and the running weights behind them, up to seq_lens[b], become 0.
//
// Every kept row lies at or behind its place (kept[i] >= first + i, checked),
// so a row is overwritten by entry j only if the entry that wants it is i <= j:
// reading the entries in order, any number ahead of those that are written,
// never loses a row.
//
// What bounds it: every moved row is read and written once.  K and V of a
// (sequence, KV head) are streams of their own, a stream a cluster of up to
// eight CTAs.  A round is 16 KiB of rows (at most 128) of each CTA, in the
// entries' order; once all CTAs hold their rows of a round in shared memory
// (one cluster barrier), all write them, with the next rounds' rows on their
// way (cp.async).  Where rows lie takes a chain of loads (entry, block ids,
// weight): every thread follows it for one entry of a batch of rounds, a batch
// ahead at each link (a round ahead, the chain was the bound: 102 us against 50
// for 8 sequences of 32,001 cut to 4,096 in each of 8 heads, 5.5 TB/s).
//
// A few short rows (an accepted path) are one warp's: it reads all of them into
// registers, then writes them.
#include <climits>

#include <cooperative_groups.h>

#include "common.cuh"
#include "host_cache.h"
#include "launch.h"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kCpThreads = 256;
constexpr int kRoundBytes = 16384, kRoundRows = 128;
constexpr int kAhead = 1, kSlots = kAhead + 1;   // rounds on their way
static_assert(kAhead < kCpThreads / kRoundRows, "a batch's addresses are written a round before its first copies");

struct CompactSeq {
  int len, first, n;   // n: entries; < 0: nothing to do
};

// Sequence b's numbers; what is out of range is recorded (report) and skipped.
__device__ __forceinline__ CompactSeq compact_seq(const CompactArgs& a, int b, bool report) {
  CompactSeq s;
  s.len = __ldg(a.seq_lens + b);
  s.first = a.first ? __ldg(a.first + b) : 0;
  s.n = __ldg(a.kept_lens + b);
  if (s.len < 0 || (int64_t)s.len > (int64_t)a.max_blocks_per_seq * kBlockSize ||
      (a.weights && (int64_t)s.len > a.weights_len)) {
    if (report) record_error(a.err, DEVERR_SEQLEN_RANGE);
    s.n = -1;
  } else if (s.n < 0 || s.n > a.kept_len || s.first < 0 || s.first > s.len || s.n > s.len - s.first) {
    if (report) record_error(a.err, DEVERR_KEPT_RANGE);
    s.n = -1;
  }
  return s;
}

__global__ void __launch_bounds__(kCpThreads) compact_kernel(const CompactArgs a, int log_round, int shift) {
  extern __shared__ __align__(16) unsigned char smem[];   // [kSlots][round rows]
  __shared__ int64_t src[2][kCpThreads], dst[2][kCpThreads];   // of two batches: [round of the batch][row]
  __shared__ float sums[2][kCpThreads];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks(), tid = threadIdx.x;
  const int item = blockIdx.x / ranks;                    // (sequence, KV head, K or V)
  const bool is_v = item & 1;
  const int b = (item >> 1) / a.num_kv_heads, g = (item >> 1) % a.num_kv_heads;
  const CompactSeq s = compact_seq(a, b, rank == 0 && tid == 0);
  if (s.n < 0) return;                                    // the same for the whole cluster
  const int32_t* kept = a.kept + ((int64_t)b * a.kept_heads + (a.kept_heads > 1 ? g : 0)) * a.kept_len;
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks_per_seq;
  float* w = a.weights && !is_v ? a.weights + ((int64_t)b * a.num_kv_heads + g) * a.weights_len : nullptr;
  char* pool = static_cast<char*>(is_v ? a.v_cache : a.k_cache);
  // 16-byte chunks of a row: 2^shift, or with shift < 0 another number
  const int round = 1 << log_round, chunks = a.row_bytes / 16, all = round * chunks;
  auto row_of = [&](int i) { return shift >= 0 ? i >> shift : i / chunks; };
  auto byte_of = [&](int i) { return (shift >= 0 ? i & (chunks - 1) : i % chunks) * 16; };
  const uint32_t sbase = smem_u32(smem);
  const int rounds = (s.n + round * ranks - 1) / (round * ranks);
  const int log_batch = 8 - log_round, batch = 1 << log_batch;   // rounds of a batch
  static_assert(kCpThreads == 256, "a batch has an entry a thread");

  // this thread's entry of batch q, where it belongs, and whether there is one
  auto entry = [&](int q) { return ((q * batch + (tid >> log_round)) * ranks + rank) * round + (tid & (round - 1)); };
  int from_next = 0, from = 0, from_block = 0, to_block = 0;
  float sum = 0.f;
  auto ask_kept = [&](int q) {
    if (entry(q) < s.n) from_next = __ldg(kept + entry(q));
  };
  auto ask_blocks = [&](int q) {
    from = -1;
    if (entry(q) < s.n) {
      const int to = s.first + entry(q);
      if (from_next < to || from_next >= s.len) {
        record_error(a.err, DEVERR_KEPT_RANGE);
      } else if (from_next > to) {
        from = from_next;
        from_block = __ldg(table + from / kBlockSize);
        to_block = __ldg(table + to / kBlockSize);
        if (w) sum = w[from];
      }
    }
  };
  auto address = [&](int q) {
    int64_t x = -1, y = -1;
    if (from >= 0) {
      if (from_block < 0 || (int64_t)from_block >= a.num_blocks || to_block < 0 || (int64_t)to_block >= a.num_blocks) {
        record_error(a.err, DEVERR_BLOCK_RANGE);
      } else {
        const int to = s.first + entry(q);
        x = (((int64_t)from_block * a.num_kv_heads + g) * kBlockSize + from % kBlockSize) * a.row_bytes;
        y = (((int64_t)to_block * a.num_kv_heads + g) * kBlockSize + to % kBlockSize) * a.row_bytes;
        sums[q & 1][tid] = sum;
      }
    }
    src[q & 1][tid] = x;
    dst[q & 1][tid] = y;
  };
  // the addresses of round k's rows
  auto in_batch = [&](int k) { return (k >> log_batch & 1) * kCpThreads + ((k & (batch - 1)) << log_round); };
  auto load = [&](int k) {
    const uint32_t to = sbase + (k % kSlots) * all * 16;
    if (k < rounds)
      for (int i = tid; i < all; i += kCpThreads) {
        const int64_t x = (&src[0][0])[in_batch(k) + row_of(i)];
        if (x >= 0)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 16), "l"(pool + x + byte_of(i))
                       : "memory");
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  ask_kept(0);
  ask_blocks(0);
  ask_kept(1);
  address(0);
  ask_blocks(1);
  ask_kept(2);
  __syncthreads();
  for (int k = 0; k < kAhead; ++k) load(k);
  for (int k = 0; k < rounds; ++k) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");   // round k's rows are here
    __syncthreads();                                      // ... of every thread, and round k - 1 is written
    // The cluster's barrier orders nothing by itself (relaxed: a release would
    // wait for the stores of the round before).  It need not: what the others
    // overwrite behind it this CTA has read, and those reads are complete, not
    // only issued: the round's rows by cp.async.wait_group and the barrier
    // above, its weights, asked for a batch ahead, as `sums` was written before
    // an earlier such barrier.  No read of rows or weights that a round needs
    // may be in flight here.
    if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    if ((k & (batch - 1)) == 0) {                         // the batch before is done with
      const int q = (k >> log_batch) + 1;
      address(q);
      ask_blocks(q + 1);
      ask_kept(q + 2);
    }
    load(k + kAhead);
    if (ranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    for (int i = tid; i < all; i += kCpThreads) {
      const int64_t y = (&dst[0][0])[in_batch(k) + row_of(i)];
      if (y >= 0)
        *reinterpret_cast<uint4*>(pool + y + byte_of(i)) =
            *reinterpret_cast<const uint4*>(smem + (k % kSlots) * all * 16 + i * 16);
    }
    if (w && tid < round && (&dst[0][0])[in_batch(k) + tid] >= 0)
      w[s.first + (k * ranks + rank) * round + tid] = (&sums[0][0])[in_batch(k) + tid];
  }
  if (w)                                                  // every read is done
    for (int t = s.first + s.n + rank * kCpThreads + tid; t < s.len; t += ranks * kCpThreads) w[t] = 0.f;
}

constexpr int kFewChunks = 8;     // 16-byte chunks a lane holds

// kept_len <= 32 and kept_len * 2^shift chunks <= 256: a warp per (sequence,
// KV head, K or V), lane i following entry i.
__global__ void __launch_bounds__(128) compact_few_kernel(const CompactArgs a, int shift) {
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (item >= 2ll * a.num_seqs * a.num_kv_heads) return;
  const bool is_v = item & 1;
  const int b = (int)(item >> 1) / a.num_kv_heads, g = (int)(item >> 1) % a.num_kv_heads;
  const CompactSeq s = compact_seq(a, b, lane == 0);
  if (s.n < 0) return;
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks_per_seq;
  float* w = a.weights && !is_v ? a.weights + ((int64_t)b * a.num_kv_heads + g) * a.weights_len : nullptr;
  char* pool = static_cast<char*>(is_v ? a.v_cache : a.k_cache);
  int64_t src = -1, dst = -1;
  float sum = 0.f;
  if (lane < s.n) {
    const int from = __ldg(a.kept + ((int64_t)b * a.kept_heads + (a.kept_heads > 1 ? g : 0)) * a.kept_len + lane);
    const int to = s.first + lane;
    if (from < to || from >= s.len) {
      record_error(a.err, DEVERR_KEPT_RANGE);
    } else if (from > to) {
      const int x = __ldg(table + from / kBlockSize), y = __ldg(table + to / kBlockSize);
      if (w) sum = w[from];
      if (x < 0 || (int64_t)x >= a.num_blocks || y < 0 || (int64_t)y >= a.num_blocks) {
        record_error(a.err, DEVERR_BLOCK_RANGE);
      } else {
        src = (((int64_t)x * a.num_kv_heads + g) * kBlockSize + from % kBlockSize) * a.row_bytes;
        dst = (((int64_t)y * a.num_kv_heads + g) * kBlockSize + to % kBlockSize) * a.row_bytes;
      }
    }
  }
  const int chunks = s.n << shift, mask = (1 << shift) - 1;
  uint4 x[kFewChunks];
#pragma unroll
  for (int m = 0; m < kFewChunks; ++m) {
    const int i = lane + 32 * m;
    const int64_t at = __shfl_sync(0xffffffffu, src, i >> shift & 31);
    if (i < chunks && at >= 0) x[m] = *reinterpret_cast<const uint4*>(pool + at + (i & mask) * 16);
  }
  __syncwarp();                                           // every row and weight is read
#pragma unroll
  for (int m = 0; m < kFewChunks; ++m) {
    const int i = lane + 32 * m;
    const int64_t at = __shfl_sync(0xffffffffu, dst, i >> shift & 31);
    if (i < chunks && at >= 0) *reinterpret_cast<uint4*>(pool + at + (i & mask) * 16) = x[m];
  }
  if (w) {
    if (dst >= 0) w[s.first + lane] = sum;
    for (int t = s.first + s.n + lane; t < s.len; t += 32) w[t] = 0.f;
  }
}

}  // namespace

cudaError_t launch_kv_compact(const CompactArgs& a, int num_sms, cudaStream_t stream) {
  const int64_t streams = 2ll * a.num_seqs * a.num_kv_heads;
  int log_round = 7, shift = -1;
  while (a.row_bytes << log_round > kRoundBytes) --log_round;
  for (int i = 0; i <= 6; ++i)
    if (a.row_bytes == 16 << i) shift = i;
  // a warp's worth of rows (64 accepted paths of up to 6: 3.2 us, against
  // 8.9 in clusters)
  if (a.kept_len <= 32 && shift >= 0 && a.kept_len << shift <= 32 * kFewChunks) {
    compact_few_kernel<<<(unsigned)((streams + 3) / 4), 128, 0, stream>>>(a, shift);
    return cudaGetLastError();
  }
  const int round = 1 << log_round, smem = kSlots * round * a.row_bytes;
  cudaError_t e = allow_dynamic_smem(compact_kernel, smem);
  if (e != cudaSuccess) return e;
  // CTAs of a stream, no more than its rounds: enough for four on every SM
  // (128 streams: 100, 65, 50 and 52 us with 1, 2, 4 and 8), and two where the
  // streams alone are that many, as they are rarely of one length (768 ragged
  // ones: 45, 41, 42 and 50 us)
  int ranks = 1;
  while (ranks < 8 && 2 * ranks * round <= a.kept_len &&
         streams * 2 * ranks <= (ranks == 1 ? 12 : 4) * (int64_t)num_sms)
    ranks *= 2;
  if (streams * ranks > INT_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(streams * ranks));
  cfg.blockDim = dim3(kCpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, compact_kernel, a, log_round, shift);
}

}  // namespace pkv
