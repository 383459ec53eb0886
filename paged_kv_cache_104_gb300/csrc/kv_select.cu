// Which tokens of a sequence stay, by the attention they got so far.
//
// Of sequence b's n = seq_lens[b] tokens, KV head g keeps min(n, budget): the
// first `sinks`, the last `recent`, and of the rest those with the largest
// weights[b][g][t]; among equal weights the earlier token, a NaN below every
// number.  Their positions go to kept[b][g] in ascending order.
//
// A radix selection over the weights' order-preserving 32-bit keys: four
// passes of a 256-bin histogram narrow the key of the last token that stays;
// one more pass writes the positions, ranked by prefix sums.  One CTA per
// (sequence, KV head).
#include <climits>

#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kSelThreads = 1024;

// Keys order as the weights do: -0 with +0, NaN first of all.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// Inclusive prefix sums over the CTA's threads (values below 2^16 in each
// half: two counts at once), and the total.
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
  for (int w = 0; w < kSelThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  return before + x;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
  __shared__ uint32_t bins[256];
  __shared__ uint32_t warp_sums[kSelThreads / 32];
  __shared__ uint32_t found[2];
  const int b = blockIdx.x / a.num_kv_heads, g = blockIdx.x % a.num_kv_heads, tid = threadIdx.x;
  const int n = a.seq_lens[b];
  if (n < 0 || n > a.max_seq_len) {
    if (tid == 0) record_error(a.err, DEVERR_SEQLEN_RANGE);
    if (tid == 0 && g == 0) a.kept_lens[b] = 0;
    return;
  }
  if (tid == 0 && g == 0) a.kept_lens[b] = min(n, a.budget);
  int32_t* kept = a.kept + (int64_t)blockIdx.x * a.budget;
  if (n <= a.budget) {
    for (int i = tid; i < n; i += kSelThreads) kept[i] = i;
    return;
  }
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
    const uint32_t rank = equal_before + block_scan(equal, warp_sums, total);
    equal_before += total;
    const bool stays = t < n && (!mid || (any && key > prefix) || (equal && rank <= want));
    const uint32_t at = kept_before + block_scan(stays, warp_sums, total);
    kept_before += total;
    if (stays) kept[at - 1] = t;
  }
}

}  // namespace

cudaError_t launch_kv_select(const SelectArgs& a, cudaStream_t stream) {
  select_kernel<<<a.num_seqs * a.num_kv_heads, kSelThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
