// Which tokens of a sequence stay, by the attention they got so far.
//
// Of sequence b's n = seq_lens[b] tokens, KV head g keeps min(n, budget): the
// first `sinks`, the last `recent`, and of the rest those with the largest
// weights[b][g][t]; among equal weights the earlier token, a NaN below every
// number.  Their positions go to kept[b][g] in ascending order.
//
// A radix selection over the weights' order-preserving 32-bit keys: histograms
// of their digits, from the highest, narrow the key of the last token that
// stays; then every token's place is a prefix sum.
//
// The bytes are few (4 a token); what bounds it is the chain of barriers, and the
// code itself, which every launch fetches anew.  Cycles of a cold launch (clock64 in
// one CTA) for 64 sequences of 2,301: 4,900 until its weights are there, 1,600 for
// the histogram, 1,000 for the digit, 2,300 to collect and 1,500 to rank the
// candidates, 3,900 to place what stays: 16,500 in all.  For 8 of 32,001, seven
// barriers of clusters of four: 5,500 for the weights, 5,800 until the last CTA has
// its own, 5,200 and 5,800 for two passes, 4,100 for the candidates, 5,100 to place:
// 33,000.  So a (sequence, KV head) is read once, 16 tokens a thread, and its keys
// stay in shared memory (in registers every loop over them was unrolled: 17.3 us for
// 64 sequences of 2,301, against 11.9) through up to three passes of 11, 11 and 10
// bits.  As soon as at most 256 tokens share the digits of the last one that stays,
// those are ranked by comparing each with all, which for 2,301 tokens is mostly after
// the first pass.  Beyond 8,192 tokens a cluster of up to eight CTAs shares a
// (sequence, KV head), adding its histograms up in the first one's shared memory
// (16.4 us for 8 sequences of 32,001).  Where the bound passes the shared memory of
// eight, at 65,536 tokens, a cluster of eight reads its weights anew for every pass:
// 62 us at 65,537 for 64 (sequence, KV head)s, against 33 at 65,536, and 81 at
// 131,072, where one CTA took 438.
#include <climits>

#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kSelThreads = 1024;

// Keys order as the weights do: -0 with +0, NaN first of all.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// The head of either kernel: the sequence's length, kept_lens, and the trivial
// cases (false: done, for every thread of the cluster alike).
__device__ __forceinline__ bool select_begin(const SelectArgs& a, int item, int index, int threads, int* length) {
  const int b = item / a.num_kv_heads, g = item % a.num_kv_heads;
  const int n = __ldg(a.seq_lens + b);
  const bool bad = n < 0 || n > a.max_seq_len;
  if (index == 0 && bad) record_error(a.err, DEVERR_SEQLEN_RANGE);
  if (index == 0 && g == 0) a.kept_lens[b] = bad ? 0 : min(n, a.budget);
  *length = n;
  if (bad) return false;
  if (n <= a.budget) {
    for (int i = index; i < n; i += threads) a.kept[(int64_t)item * a.budget + i] = i;
    return false;
  }
  return true;
}

constexpr int kPerThread = 16;     // tokens
constexpr int kBins = 2048;
// Tokens that are ranked by comparing each with all.  With 64 or 128 instead 64
// sequences of 2,301 and 8 of 32,001 take the same (11.5, 16.6 us), 64 of 8,000 24.6, not
// 25.8, 64 of 4,000 14.3, not 16.1; twice as many do not fit the static
// shared memory of 512 threads.
constexpr int kFew = 256;

// Sums of all threads before this one, and of all (one barrier; warp_sums is
// free again after the next).
template <int THREADS>
__device__ __forceinline__ uint32_t scan_before(uint32_t own, uint32_t* warp_sums, uint32_t& total) {
  constexpr int WARPS = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  uint32_t v = lane < WARPS ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < WARPS; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  total = __shfl_sync(0xffffffffu, v, WARPS - 1);
  const uint32_t before = __shfl_sync(0xffffffffu, v, (warp + 31) & 31);
  return x - own + (warp > 0 ? before : 0);
}

// THREADS * 16 tokens a CTA, a cluster per (sequence, KV head), or one CTA alone
// (without the code of clusters 11.9 -> 11.5 us for 64 sequences of 2,301).
template <int THREADS, bool ALONE>
__global__ void __launch_bounds__(THREADS, 1536 / THREADS) select_smem_kernel(const SelectArgs a) {
  constexpr int TOKENS = THREADS * kPerThread;
  __shared__ uint32_t keys[TOKENS + TOKENS / kPerThread];   // token t at t + t / 16: free of bank conflicts
  __shared__ __align__(16) uint32_t bins[kBins];
  __shared__ uint32_t stays[TOKENS / 32];                // ranked tokens that stay
  __shared__ uint32_t warp_sums[2][32];
  __shared__ uint32_t found[3];                          // digit, how many of it stay, how many have it
  __shared__ uint32_t counts[8][2];                      // per CTA: tokens that stay for sure, ties
  __shared__ unsigned long long few[kFew], mine[kFew];   // key, then the earlier token first: all, this CTA's
  __shared__ uint32_t few_n, mine_n, few_base;           // (few_n: the first CTA's)
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = ALONE ? 0 : cluster.block_rank(), ranks = ALONE ? 1 : cluster.num_blocks(), tid = threadIdx.x;
  const int item = blockIdx.x / ranks;
  const float* w = a.weights + (int64_t)item * a.weights_len;
  const int base = rank * TOKENS;
  auto at = [](int t) { return t + t / kPerThread; };
  // the weights up to the bound on the length, asked for with the length
  const int here = min(TOKENS, a.max_seq_len - base);
#pragma unroll 8
  for (int t = tid; t < here; t += THREADS) keys[at(t)] = order_key(__ldg(w + base + t));
  int n;
  if (!select_begin(a, item, rank * THREADS + tid, ranks * THREADS, &n)) return;
  auto sync = [&] {
    if (ranks > 1) cluster.sync();
    else __syncthreads();
  };
  // the tokens to choose from are lo .. hi - 1 (of this CTA: lo0 .. hi0 - 1),
  // and `want` of them, which are fewer
  const int lo = a.sinks, hi = n - a.recent;
  const int lo0 = max(lo - base, 0), hi0 = min(hi - base, TOKENS);
  uint32_t want = a.budget - a.sinks - a.recent;
  const bool any = want > 0;
  auto clear = [&] {
    for (int i = tid; i < kBins / 4; i += THREADS) reinterpret_cast<uint4*>(bins)[i] = make_uint4(0, 0, 0, 0);
  };
  clear();
  for (int i = tid; i < TOKENS / 32; i += THREADS) stays[i] = 0;
  if (tid == 0) few_n = mine_n = 0;
  sync();
  uint32_t prefix = 0, above = 0;                        // the digits so far, and their bits
  bool ranked = false;
#pragma unroll 1
  for (int pass = 0; pass < 3 && any; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 2 ? 1023 : 2047;
#pragma unroll 4
    for (int t = lo0 + tid; t < hi0; t += THREADS) {
      const uint32_t key = keys[at(t)];
      if (((key ^ prefix) & above) == 0) atomicAdd(&bins[key >> shift & mask], 1u);
    }
    __syncthreads();
    if (ranks > 1) {
      if (rank > 0) {
        uint32_t* sum = cluster.map_shared_rank(bins, 0);
        for (int i = tid; i < kBins; i += THREADS)
          if (bins[i]) atomicAdd(sum + i, bins[i]);
      }
      cluster.sync();
    }
    if (rank == 0) {
      // bins from the highest down, kBins / THREADS a thread: whose do the
      // wanted tokens end in?
      constexpr int W = kBins / THREADS;
      const int bottom = kBins - (tid + 1) * W;
      uint32_t own = 0, total;
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(bins + bottom + i);
        own += x.x + x.y + x.z + x.w;
      }
      const uint32_t before = scan_before<THREADS>(own, warp_sums[pass & 1], total);
      if (before < want && before + own >= want) {
        uint32_t left = want - before;
        int bin = bottom + W - 1;
        while (bins[bin] < left) left -= bins[bin--];
        for (int k = 0; k < ranks; ++k) {
          uint32_t* f = ALONE ? found : cluster.map_shared_rank(found, k);
          f[0] = bin;
          f[1] = left;
          f[2] = bins[bin];
        }
      }
      __syncthreads();
    }
    clear();
    sync();
    prefix |= found[0] << shift;
    above |= mask << shift;
    want = found[1];
    if (pass < 2 && found[2] <= kFew) {
      ranked = true;
      break;
    }
  }
  // Keys above `prefix` stay, and of those that have it the first `want` in
  // the order of the weights (ranked), or of the tokens where they are equal.
  if (ranked) {
#pragma unroll 4
    for (int t = lo0 + tid; t < hi0; t += THREADS) {
      const uint32_t key = keys[at(t)];
      if ((key & above) == prefix)
        mine[atomicAdd(&mine_n, 1u)] = (unsigned long long)key << 32 | (0xffffffffu - (uint32_t)(base + t));
    }
    __syncthreads();
    const unsigned long long* all = mine;
    if (ranks > 1) {
      if (tid == 0) few_base = atomicAdd(cluster.map_shared_rank(&few_n, 0), mine_n);
      __syncthreads();
      for (int i = tid; i < (int)mine_n * ranks; i += THREADS)
        cluster.map_shared_rank(few, i % ranks)[few_base + i / ranks] = mine[i / ranks];
      cluster.sync();
      all = few;
    }
    // this CTA's, each with all, by 1 .. 8 neighbouring threads
    const int have = found[2], own = mine_n;
    int log_parts = 0;
    while (log_parts < 3 && own << (log_parts + 1) <= THREADS) ++log_parts;
    const int parts = 1 << log_parts;
    for (int j = tid >> log_parts; j < ((own + 31) & ~31); j += THREADS >> log_parts) {
      const unsigned long long x = j < own ? mine[j] : 0;
      uint32_t ahead = 0;
#pragma unroll 4
      for (int k = tid & (parts - 1); k < have; k += parts) ahead += all[k] > x;
      for (int o = 1; o < parts; o <<= 1) ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
      if (j < own && ahead < want && (tid & (parts - 1)) == 0) {
        const int t = (int)(0xffffffffu - (uint32_t)x) - base;
        atomicOr(&stays[t >> 5], 1u << (t & 31));
      }
    }
    want = 0;
    __syncthreads();
  }
  // a thread's 16 tokens: which stay, and which are equal to the last that does
  const int t0 = tid * kPerThread;
  uint32_t sure = ranked ? stays[t0 >> 5] >> (t0 & 31) & 0xffff : 0, ties = 0;
#pragma unroll 4
  for (int i = 0; i < kPerThread; ++i) {
    const int t = t0 + i;
    const bool mid = t >= lo0 && t < hi0;
    const uint32_t key = keys[at(t)] & above;
    sure |= (uint32_t)(base + t < n && (!mid || (any && key > prefix))) << i;
    ties |= (uint32_t)(!ranked && mid && any && key == prefix) << i;
  }
  // both counts in one scan: at most 8,192 of each in a CTA
  uint32_t total;
  const uint32_t before = scan_before<THREADS>(__popc(sure) | __popc(ties) << 16, warp_sums[1], total);
  uint32_t sure_at = before & 0xffff, ties_at = before >> 16;
  if (ranks > 1) {
    if (tid < ranks) {
      uint32_t* c = cluster.map_shared_rank(&counts[0][0], tid);
      c[2 * rank] = total & 0xffff;
      c[2 * rank + 1] = total >> 16;
    }
    cluster.sync();                                      // the last access to another's shared memory
    for (int k = 0; k < rank; ++k) {
      sure_at += counts[k][0];
      ties_at += counts[k][1];
    }
  }
  int32_t* kept = a.kept + (int64_t)item * a.budget;
  for (uint32_t left = sure | ties; left; left &= left - 1) {
    const int i = __ffs(left) - 1;
    const bool tie = ties >> i & 1;
    if (!tie || ties_at < want) kept[sure_at + min(ties_at, want)] = base + t0 + i;
    sure_at += !tie;
    ties_at += tie;
  }
}

// Any length: a cluster per (sequence, KV head), whose CTAs read their share of
// the weights once a pass, mostly from the L2, and twice more.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
  __shared__ __align__(16) uint32_t bins[kBins];
  __shared__ uint32_t warp_sums[2][32];
  __shared__ uint32_t found[2];                          // digit, how many of it stay
  __shared__ uint32_t counts[8][2];                      // per CTA: tokens that stay for sure, ties
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks(), tid = threadIdx.x;
  const int item = blockIdx.x / ranks;
  const float* w = a.weights + (int64_t)item * a.weights_len;
  int n;
  if (!select_begin(a, item, rank * kSelThreads + tid, ranks * kSelThreads, &n)) return;
  const int span = (n + ranks - 1) / ranks, begin = min(rank * span, n), end = min(begin + span, n);
  const int lo = a.sinks, hi = n - a.recent;             // the tokens to choose from
  const int lo0 = max(lo, begin), hi0 = min(hi, end);
  uint32_t want = a.budget - a.sinks - a.recent;         // and how many, which are fewer
  const bool any = want > 0;
  auto clear = [&] {
    for (int i = tid; i < kBins; i += kSelThreads) bins[i] = 0;
  };
  clear();
  cluster.sync();
  uint32_t prefix = 0, above = 0;                        // the digits so far, and their bits
#pragma unroll 1
  for (int pass = 0; pass < 3 && any; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 2 ? 1023 : 2047;
#pragma unroll 8
    for (int t = lo0 + tid; t < hi0; t += kSelThreads) {
      const uint32_t key = order_key(__ldg(w + t));
      if (((key ^ prefix) & above) == 0) atomicAdd(&bins[key >> shift & mask], 1u);
    }
    __syncthreads();
    if (rank > 0) {
      uint32_t* sum = cluster.map_shared_rank(bins, 0);
      for (int i = tid; i < kBins; i += kSelThreads)
        if (bins[i]) atomicAdd(sum + i, bins[i]);
    }
    cluster.sync();
    if (rank == 0) {
      uint32_t total;
      const int top = kBins - 1 - 2 * tid;               // two bins a thread, from the highest down
      const uint32_t x = bins[top], y = bins[top - 1];
      const uint32_t before = scan_before<kSelThreads>(x + y, warp_sums[0], total);
      if (before < want && before + x + y >= want) {
        const bool second = before + x < want;
        for (int k = 0; k < ranks; ++k) {
          uint32_t* f = cluster.map_shared_rank(found, k);
          f[0] = top - second;
          f[1] = want - before - (second ? x : 0);
        }
      }
      __syncthreads();
    }
    clear();
    cluster.sync();
    prefix |= found[0] << shift;
    above |= mask << shift;
    want = found[1];
  }
  // Keys above `prefix` stay, and the first `want` tokens that have it.
  auto look = [&](int t, uint32_t& sure, uint32_t& tie) {
    const bool mid = any && t >= lo && t < hi;
    const uint32_t key = mid ? order_key(__ldg(w + t)) : 0;
    sure = t < lo || t >= hi || (mid && key > prefix);
    tie = mid && key == prefix;
  };
  uint32_t sure_at = 0, ties_at = 0, total;
#pragma unroll 8
  for (int t = begin + tid; t < end; t += kSelThreads) {
    uint32_t sure, tie;
    look(t, sure, tie);
    sure_at += sure;
    ties_at += tie;
  }
  scan_before<kSelThreads>(sure_at, warp_sums[0], total);
  if (tid < ranks) cluster.map_shared_rank(&counts[0][0], tid)[2 * rank] = total;
  scan_before<kSelThreads>(ties_at, warp_sums[1], total);
  if (tid < ranks) cluster.map_shared_rank(&counts[0][0], tid)[2 * rank + 1] = total;
  cluster.sync();                                        // the last access to another's shared memory
  sure_at = ties_at = 0;                                 // of the tokens before
  for (int k = 0; k < rank; ++k) {
    sure_at += counts[k][0];
    ties_at += counts[k][1];
  }
  int32_t* kept = a.kept + (int64_t)item * a.budget;
  int turn = 0;
  for (int t0 = begin; t0 < end; t0 += 8 * kSelThreads, turn ^= 1) {
    uint32_t sure = 0, ties = 0;                         // of this thread's eight tokens
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = t0 + 8 * tid + i;
      uint32_t x = 0, y = 0;
      if (t < end) look(t, x, y);
      sure |= x << i;
      ties |= y << i;
    }
    const uint32_t before =
        scan_before<kSelThreads>(__popc(sure) | __popc(ties) << 16, warp_sums[turn], total);
    uint32_t to = sure_at + (before & 0xffff), tie = ties_at + (before >> 16);
    for (uint32_t left = sure | ties; left; left &= left - 1) {
      const int i = __ffs(left) - 1;
      const bool is_tie = ties >> i & 1;
      if (!is_tie || tie < want) kept[to + min(tie, want)] = t0 + 8 * tid + i;
      to += !is_tie;
      tie += is_tie;
    }
    sure_at += total & 0xffff;
    ties_at += total >> 16;
  }
}

cudaError_t launch_clusters(void (*kernel)(SelectArgs), int threads, const SelectArgs& a, int ranks,
                            cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_seqs * a.num_kv_heads * ranks));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_kv_select(const SelectArgs& a, cudaStream_t stream) {
  // The fewest threads that hold the bound's tokens, 16 each, 64, 256 or 512: a
  // large batch then has more CTAs on an SM (256 sequences of 1,000 in 8 heads 17.2,
  // 26.4 and 41.1 us with 64, 256 and 512 threads, 64 of 4,000 16.2 and 21.0 with 256
  // and 512); one sequence alone would take more (1,000 tokens 9.2, 6.5, 6.2 us, 4,000
  // 10.1 and 9.1).
  const int tokens = a.max_seq_len;
  if (tokens <= 64 * kPerThread) return launch_clusters(select_smem_kernel<64, true>, 64, a, 1, stream);
  if (tokens <= 256 * kPerThread) return launch_clusters(select_smem_kernel<256, true>, 256, a, 1, stream);
  if (tokens <= 512 * kPerThread) return launch_clusters(select_smem_kernel<512, true>, 512, a, 1, stream);
  for (int ranks = 2; ranks <= 8; ranks *= 2)
    if (tokens <= 512 * kPerThread * ranks)
      return launch_clusters(select_smem_kernel<512, false>, 512, a, ranks, stream);
  return launch_clusters(select_kernel, kSelThreads, a, 8, stream);
}

}  // namespace pkv
