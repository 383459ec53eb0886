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
// The bytes are few (4 a token); what bounds it is the chain of barriers.  So a
// (sequence, KV head) is read once, eight tokens a thread, and its keys stay in
// registers through three passes of 11, 11 and 10 bits (against 4 of 8 with
// re-reads: 88 -> 19 us for 64 sequences of 2,301); beyond 8,192 tokens a
// cluster of up to eight CTAs shares it, adding its histograms up in the first
// one's shared memory (122 -> 30 us for 8 sequences of 32,001).  Longer
// bounds than 65,536 take one CTA that reads the weights once a pass.
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

// Inclusive prefix sums over the CTA's threads, and the total.
template <int THREADS>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* warp_sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  return before + x;
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

constexpr int kPerThread = 8;      // tokens
constexpr int kBins = 2048;

// THREADS * 8 tokens a CTA, a cluster per (sequence, KV head).
template <int THREADS>
__global__ void __launch_bounds__(THREADS) select_reg_kernel(const SelectArgs a) {
  __shared__ uint32_t bins[kBins];
  __shared__ uint32_t warp_sums[THREADS / 32];
  __shared__ uint32_t found[2];                          // digit, how many of it
  __shared__ uint32_t counts[8][2];                      // per CTA: tokens that stay for sure, ties
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks(), tid = threadIdx.x;
  const int item = blockIdx.x / ranks;
  int n;
  if (!select_begin(a, item, rank * THREADS + tid, ranks * THREADS, &n)) return;
  auto sync = [&] {
    if (ranks > 1) cluster.sync();
    else __syncthreads();
  };
  const float* w = a.weights + (int64_t)item * a.weights_len;
  const int lo = a.sinks, hi = n - a.recent;             // the tokens to choose from
  uint32_t want = a.budget - a.sinks - a.recent;         // and how many; < hi - lo
  const bool any = want > 0;
  const int t0 = (rank * THREADS + tid) * kPerThread;
  uint32_t key[kPerThread], mid = 0;                     // mid: which tokens are to be chosen from
  if (t0 + kPerThread <= n && (reinterpret_cast<uintptr_t>(w + t0) & 15) == 0) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(w + t0)), y = __ldg(reinterpret_cast<const float4*>(w + t0) + 1);
    const float v[kPerThread] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) key[i] = order_key(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) key[i] = t0 + i < n ? order_key(__ldg(w + t0 + i)) : 0;
  }
#pragma unroll
  for (int i = 0; i < kPerThread; ++i)
    if (t0 + i >= lo && t0 + i < hi) mid |= 1u << i;
  for (int i = tid; i < kBins; i += THREADS) bins[i] = 0;
  sync();
  uint32_t prefix = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3 && any; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t above = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u, mask = pass == 2 ? 1023 : 2047;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      if ((mid >> i & 1) && ((key[i] ^ prefix) & above) == 0) atomicAdd(&bins[key[i] >> shift & mask], 1u);
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
      const int top = kBins - 1 - tid * W;
      uint32_t own = 0, total;
#pragma unroll
      for (int i = 0; i < W; ++i) own += bins[top - i];
      const uint32_t through = block_scan<THREADS>(own, warp_sums, total);
      if (through >= want && through - own < want) {
        uint32_t left = want - (through - own);
        int bin = top;
        while (bins[bin] < left) left -= bins[bin--];
        for (int k = 0; k < ranks; ++k) {
          uint32_t* f = ranks > 1 ? cluster.map_shared_rank(found, k) : found;
          f[0] = bin;
          f[1] = left;
        }
      }
      __syncthreads();
    }
    for (int i = tid; i < kBins; i += THREADS) bins[i] = 0;
    sync();
    prefix |= found[0] << shift;
    want = found[1];
  }
  // keys above `prefix` stay, and the first `want` tokens that have it
  uint32_t sure = 0, ties = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const bool m = mid >> i & 1;
    sure |= (uint32_t)(t0 + i < n && (!m || (any && key[i] > prefix))) << i;
    ties |= (uint32_t)(m && any && key[i] == prefix) << i;
  }
  // both counts in one scan: at most 8,192 of each in a CTA
  uint32_t total;
  uint32_t at = block_scan<THREADS>(__popc(sure) | __popc(ties) << 16, warp_sums, total);
  uint32_t sure_at = (at & 0xffff) - __popc(sure), ties_at = (at >> 16) - __popc(ties);
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
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const bool tie = ties >> i & 1;
    if ((sure >> i & 1) || (tie && ties_at < want)) kept[sure_at + min(ties_at, want)] = t0 + i;
    sure_at += sure >> i & 1;
    ties_at += tie;
  }
}

// Any length: the weights are read once a pass, and once more.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
  __shared__ uint32_t bins[256];
  __shared__ uint32_t warp_sums[kSelThreads / 32];
  __shared__ uint32_t found[2];
  const int tid = threadIdx.x;
  int n;
  if (!select_begin(a, blockIdx.x, tid, kSelThreads, &n)) return;
  int32_t* kept = a.kept + (int64_t)blockIdx.x * a.budget;
  const float* w = a.weights + (int64_t)blockIdx.x * a.weights_len;
  const int lo = a.sinks, hi = n - a.recent;             // the tokens to choose from
  uint32_t want = a.budget - a.sinks - a.recent;         // and how many; < hi - lo
  uint32_t prefix = 0;
  for (int shift = 24; want > 0 && shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) bins[i] = 0;
    __syncthreads();
    for (int t = lo + tid; t < hi; t += kSelThreads) {
      const uint32_t key = order_key(w[t]);
      if (shift == 24 || key >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&bins[key >> shift & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t left = want;
      int bin = 255;
      while (bin > 0 && bins[bin] < left) left -= bins[bin--];
      found[0] = bin;
      found[1] = left;
    }
    __syncthreads();
    prefix |= found[0] << shift;
    want = found[1];
    __syncthreads();
  }
  // keys above `prefix` stay, and the first `want` tokens that have it
  const bool any = a.budget > a.sinks + a.recent;
  uint32_t equal_before = 0, kept_before = 0, total;
  for (int base = 0; base < n; base += kSelThreads) {
    const int t = base + tid;
    const bool mid = t >= lo && t < hi;
    const uint32_t key = mid ? order_key(w[t]) : 0;
    const bool equal = any && mid && key == prefix;
    const uint32_t rank = equal_before + block_scan<kSelThreads>(equal, warp_sums, total);
    equal_before += total;
    const bool stays = t < n && (!mid || (any && key > prefix) || (equal && rank <= want));
    const uint32_t at = kept_before + block_scan<kSelThreads>(stays, warp_sums, total);
    kept_before += total;
    if (stays) kept[at - 1] = t;
  }
}

template <int THREADS>
cudaError_t launch_reg(const SelectArgs& a, int ranks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_seqs * a.num_kv_heads * ranks));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_reg_kernel<THREADS>, a);
}

}  // namespace

cudaError_t launch_kv_select(const SelectArgs& a, cudaStream_t stream) {
  const int tokens = a.max_seq_len;
  if (tokens <= 128 * kPerThread) return launch_reg<128>(a, 1, stream);
  if (tokens <= 512 * kPerThread) return launch_reg<512>(a, 1, stream);
  for (int ranks = 1; ranks <= 8; ranks *= 2)
    if (tokens <= 1024 * kPerThread * ranks) return launch_reg<1024>(a, ranks, stream);
  select_kernel<<<a.num_seqs * a.num_kv_heads, kSelThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
