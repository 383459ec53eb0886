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
// eight CTAs.  A CTA takes every ranks-th 64 entries (fewer of long rows, 16 KiB
// of them); a round is so many of each: once all CTAs hold their rows of a round in shared memory (one cluster
// barrier), all write them.  The rows of the next rounds are on their way
// meanwhile (cp.async, kAhead rounds).
#include <climits>

#include <cooperative_groups.h>

#include "common.cuh"
#include "host_cache.h"
#include "launch.h"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kCpThreads = 256, kRound = 64, kAhead = 3;
// Rows of round k + kAhead are asked for once all have written round k - 1;
// its addresses are written before that, when only round k - 2 is sure to be.
constexpr int kSlots = kAhead + 1, kAddrs = kAhead + 2;
constexpr int kRoundBytes = 16384;

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

// Byte offset of token t's row in a pool; -1 for a bad block id, which is
// recorded.
__device__ __forceinline__ int64_t row_at(const CompactArgs& a, const int32_t* table, int g, int t) {
  const int blk = __ldg(table + t / kBlockSize);
  if (blk < 0 || (int64_t)blk >= a.num_blocks) {
    record_error(a.err, DEVERR_BLOCK_RANGE);
    return -1;
  }
  return (((int64_t)blk * a.num_kv_heads + g) * kBlockSize + t % kBlockSize) * a.row_bytes;
}

// Where entry i's row is and goes (both -1: it stays, or is skipped).
__device__ __forceinline__ void entry(const CompactArgs& a, const CompactSeq& s, const int32_t* table, int g, int i,
                                      int from, int64_t* src, int64_t* dst) {
  const int to = s.first + i;
  *src = *dst = -1;
  if (from < to || from >= s.len) {
    record_error(a.err, DEVERR_KEPT_RANGE);
  } else if (from > to) {
    const int64_t x = row_at(a, table, g, from), y = row_at(a, table, g, to);
    if (x >= 0 && y >= 0) {
      *src = x;
      *dst = y;
    }
  }
}

__global__ void __launch_bounds__(kCpThreads) compact_kernel(const CompactArgs a, int round, int shift) {
  extern __shared__ __align__(16) unsigned char smem[];   // [kSlots][round rows]
  __shared__ int64_t src[kAddrs][kRound], dst[kAddrs][kRound];
  __shared__ float sums[kAddrs][kRound];
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
  const int chunks = a.row_bytes / 16, all = round * chunks;
  auto row_of = [&](int i) { return shift >= 0 ? i >> shift : i / chunks; };
  auto byte_of = [&](int i) { return (shift >= 0 ? i & (chunks - 1) : i % chunks) * 16; };
  const uint32_t sbase = smem_u32(smem);
  const int rounds = (s.n + round * ranks - 1) / (round * ranks);

  // this thread's entry of round k (the first threads)
  auto index = [&](int k) { return (k * ranks + rank) * round + tid; };
  int ahead = 0;                                          // kept[] of the next round to be addressed
  auto fetch = [&](int k) {
    if (tid < round && k < rounds && index(k) < s.n) ahead = __ldg(kept + index(k));
  };
  auto address = [&](int k) {
    if (tid < round) {
      int64_t x = -1, y = -1;
      if (k < rounds && index(k) < s.n) {
        entry(a, s, table, g, index(k), ahead, &x, &y);
        if (w && x >= 0) sums[k % kAddrs][tid] = w[ahead];
      }
      src[k % kAddrs][tid] = x;
      dst[k % kAddrs][tid] = y;
    }
    fetch(k + 1);
  };
  auto load = [&](int k) {
    const uint32_t to = sbase + (k % kSlots) * all * 16;
    if (k < rounds)
      for (int i = tid; i < all; i += kCpThreads) {
        const int64_t from = src[k % kAddrs][row_of(i)];
        if (from >= 0)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 16), "l"(pool + from + byte_of(i))
                       : "memory");
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(0);
  for (int k = 0; k < kAhead; ++k) address(k);
  __syncthreads();
  for (int k = 0; k < kAhead; ++k) load(k);
  for (int k = 0; k < rounds; ++k) {
    address(k + kAhead);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");   // round k's rows are here
    if (ranks > 1) cluster.sync();                        // ... in every CTA, and the addresses are written
    else __syncthreads();
    for (int i = tid; i < all; i += kCpThreads) {
      const int64_t to = dst[k % kAddrs][row_of(i)];
      if (to >= 0)
        *reinterpret_cast<uint4*>(pool + to + byte_of(i)) =
            *reinterpret_cast<const uint4*>(smem + (k % kSlots) * all * 16 + i * 16);
    }
    if (w && tid < round && dst[k % kAddrs][tid] >= 0) w[s.first + index(k)] = sums[k % kAddrs][tid];
    load(k + kAhead);
  }
  if (w)                                                  // every read is done
    for (int t = s.first + s.n + rank * kCpThreads + tid; t < s.len; t += ranks * kCpThreads) w[t] = 0.f;
}

}  // namespace

cudaError_t launch_kv_compact(const CompactArgs& a, int num_sms, cudaStream_t stream) {
  int round = kRound, shift = -1;
  while (round * a.row_bytes > kRoundBytes) round /= 2;
  for (int i = 0; i <= 6; ++i)
    if (a.row_bytes == 16 << i) shift = i;
  const int smem = kSlots * round * a.row_bytes;
  cudaError_t e = allow_dynamic_smem(compact_kernel, smem);
  if (e != cudaSuccess) return e;
  const int64_t streams = 2ll * a.num_seqs * a.num_kv_heads;
  // CTAs of a stream: no more than its rounds, nor than fill the SMs twice
  int ranks = 1;
  while (ranks < 8 && 2 * ranks * round <= a.kept_len && streams * 2 * ranks <= 4 * num_sms) ranks *= 2;
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
  return cudaLaunchKernelEx(&cfg, compact_kernel, a, round, shift);
}

}  // namespace pkv
