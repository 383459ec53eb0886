// Rows that stay move up, in place.
//
// For each sequence b and KV head g, row first + i of the sequence becomes
// what row kept[b][g][i] was (i < kept_lens[b]; keys, values and running
// weights), and the running weights behind them, up to seq_lens[b], become 0.
//
// Every kept row lies at or behind its place (kept[i] >= first + i, checked),
// so a row is overwritten by entry j only if the entry that wants it is i <= j:
// reading the entries in order, some ahead of those that are written, never
// loses a row.  A CTA takes one (sequence, KV head) and moves 64 entries a
// round: all are read, a barrier, all are written.
#include "common.cuh"
#include "host_cache.h"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kCpThreads = 256, kRound = 64;

__global__ void __launch_bounds__(kCpThreads) compact_kernel(const CompactArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  uint4* rows = reinterpret_cast<uint4*>(smem);        // [kRound][chunks] of K, then of V
  __shared__ int64_t src[kRound], dst[kRound];
  __shared__ float sums[kRound];
  const int b = blockIdx.x / a.num_kv_heads, g = blockIdx.x % a.num_kv_heads, tid = threadIdx.x;
  const int len = a.seq_lens[b], first = a.first ? a.first[b] : 0, n = a.kept_lens[b];
  if (len < 0 || (int64_t)len > (int64_t)a.max_blocks_per_seq * kBlockSize ||
      (a.weights && (int64_t)len > a.weights_len)) {
    if (tid == 0) record_error(a.err, DEVERR_SEQLEN_RANGE);
    return;
  }
  if (n < 0 || n > a.kept_len || first < 0 || first > len || n > len - first) {
    if (tid == 0) record_error(a.err, DEVERR_KEPT_RANGE);
    return;
  }
  const int32_t* kept = a.kept + ((int64_t)b * a.kept_heads + (a.kept_heads > 1 ? g : 0)) * a.kept_len;
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks_per_seq;
  float* w = a.weights ? a.weights + ((int64_t)b * a.num_kv_heads + g) * a.weights_len : nullptr;
  const int chunks = a.row_bytes / 16;
  // byte offset of token t's row in a pool; -1 for a bad block id, which is recorded
  auto at = [&](int t) -> int64_t {
    const int blk = __ldg(table + t / kBlockSize);
    if (blk < 0 || (int64_t)blk >= a.num_blocks) {
      record_error(a.err, DEVERR_BLOCK_RANGE);
      return -1;
    }
    return (((int64_t)blk * a.num_kv_heads + g) * kBlockSize + t % kBlockSize) * a.row_bytes;
  };
  for (int base = 0; base < n; base += kRound) {
    if (tid < kRound) {
      const int i = base + tid;
      src[tid] = dst[tid] = -1;
      if (i < n) {
        const int from = kept[i], to = first + i;
        if (from < to || from >= len) {
          record_error(a.err, DEVERR_KEPT_RANGE);
        } else if (from > to) {
          src[tid] = at(from);
          dst[tid] = at(to);
          if (src[tid] < 0) dst[tid] = -1;
          if (dst[tid] < 0) src[tid] = -1;
          if (w) sums[tid] = w[from];
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < kRound * chunks; i += kCpThreads) {
      const int64_t from = src[i / chunks];
      if (from >= 0) {
        rows[i] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.k_cache) + from + i % chunks * 16);
        rows[i + kRound * chunks] =
            *reinterpret_cast<const uint4*>(static_cast<const char*>(a.v_cache) + from + i % chunks * 16);
      }
    }
    __syncthreads();
    for (int i = tid; i < kRound * chunks; i += kCpThreads) {
      const int64_t to = dst[i / chunks];
      if (to >= 0) {
        *reinterpret_cast<uint4*>(static_cast<char*>(a.k_cache) + to + i % chunks * 16) = rows[i];
        *reinterpret_cast<uint4*>(static_cast<char*>(a.v_cache) + to + i % chunks * 16) = rows[i + kRound * chunks];
      }
    }
    if (w && tid < kRound && dst[tid] >= 0) w[first + base + tid] = sums[tid];
    __syncthreads();
  }
  if (w)
    for (int t = first + n + tid; t < len; t += kCpThreads) w[t] = 0.f;
}

}  // namespace

cudaError_t launch_kv_compact(const CompactArgs& a, int num_sms, cudaStream_t stream) {
  const int smem = 2 * kRound * a.row_bytes;
  cudaError_t e = allow_dynamic_smem(compact_kernel, smem);
  if (e != cudaSuccess) return e;
  compact_kernel<<<a.num_seqs * a.num_kv_heads, kCpThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
