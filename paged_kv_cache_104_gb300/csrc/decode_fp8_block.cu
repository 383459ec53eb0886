// Decode attention over the block-scaled fp8 cache: the kernel of
// decode_fp8_kernel.cuh with the scales of every block and head, and the
// merge of its fp32 partials.
#include "decode_fp8_kernel.cuh"

namespace pkv {
namespace {

constexpr int kMergeWarps = 8;

// Merge of a (sequence, query head) row's partials: o = sum w_s o_s / sum w_s,
// w_s = 2^(m_s - M) l_s, each o_s a result by itself.  A warp folds the partials
// first, first + step, ... under a running maximum, a lane four columns, and
// keeps the average of those it has met, which is within the values' range
// whatever that is; N rows are in flight, beside their (m, l).  The merges are programmatic dependents of the main kernel; lengths
// are the caller's and are read before it ends.
struct Folded {
  float m, l;
  float4 sum;
};
template <int N>
__device__ __forceinline__ Folded fold(const DecodeArgs& a, int row, int lane, int first, int step,
                                       int ns) {
  const int64_t base = (int64_t)row * a.max_splits;
  const float2* rml = reinterpret_cast<const float2*>(a.ws_ml) + base;
  const float4* acc = reinterpret_cast<const float4*>(a.ws_acc) + base * (kHD / 4) + lane;
  Folded r = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int s0 = first; s0 < ns; s0 += N * step) {
    float4 v[N];
    float2 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int s = s0 + i * step;
      x[i] = s < ns ? rml[s] : make_float2(-INFINITY, 0.f);
      v[i] = s < ns ? acc[(int64_t)s * (kHD / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = r.m;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, x[i].x);
    const float before = r.l * ex2(r.m - top);   // 0 at the first
    float w[N], l = before;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[i] = ex2(x[i].x - top) * x[i].y;
      l += w[i];
    }
    const float inv = 1.f / l, f = before * inv;
    r.m = top;
    r.l = l;
    r.sum.x *= f;
    r.sum.y *= f;
    r.sum.z *= f;
    r.sum.w *= f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (s0 + i * step >= ns) break;
      const float share = w[i] * inv;
      r.sum.x = fmaf(share, v[i].x, r.sum.x);
      r.sum.y = fmaf(share, v[i].y, r.sum.y);
      r.sum.z = fmaf(share, v[i].z, r.sum.z);
      r.sum.w = fmaf(share, v[i].w, r.sum.w);
    }
  }
  return r;
}

// Partials of a row of sequence b, whose length is n (0: it has none).
__device__ __forceinline__ int partials(const DecodeArgs& a, int row, int b, int n) {
  if (n < 1 || n > min(a.max_seq_len, a.max_blocks_per_seq * kBlockSize)) return 0;
  const int h = row - b * a.num_q_heads;
  return a.balanced ? a.ws_np[b * a.num_kv_heads + h / (a.num_q_heads / a.num_kv_heads)]
                    : (n + a.split_tokens - 1) / a.split_tokens;
}

// A CTA to a row, for the few rows of a small batch, which is cut into many
// short pieces (one sequence of 32,001 tokens: up to 228 a row).
__global__ void __launch_bounds__(kMergeWarps * 32)
merge_row_kernel(const DecodeArgs a) {
  __shared__ float4 part[kMergeWarps][32];
  __shared__ float2 ml[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x;
  const int b = row / a.num_q_heads;
  const int n = a.seq_lens[b];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int ns = partials(a, row, b, n);
  if (ns <= 1) return;              // none, or written directly by the main kernel
  const Folded r = fold<4>(a, row, lane, warp, kMergeWarps, ns);
  part[warp][lane] = r.sum;
  if (lane == 0) ml[warp] = make_float2(r.m, r.l);
  __syncthreads();
  if (threadIdx.x >= kHD) return;
  const int live = min(ns, kMergeWarps);   // the other warps had no partial
  float M = -INFINITY;
  for (int w = 0; w < live; ++w) M = fmaxf(M, ml[w].x);
  float L = 0.f, O = 0.f;
  for (int w = 0; w < live; ++w) L = fmaf(ex2(ml[w].x - M), ml[w].y, L);
  const float inv = 1.f / L;
  for (int w = 0; w < live; ++w)
    O = fmaf(ex2(ml[w].x - M) * ml[w].y * inv, reinterpret_cast<const float*>(part[w])[threadIdx.x], O);
  static_cast<__nv_bfloat16*>(a.out)[(int64_t)row * kHD + threadIdx.x] = __float2bfloat16_rn(O);
}

// A warp to a row, for many rows of few partials (64 sequences of 2,301 tokens,
// 2,048 rows: both kernels took 56.1 us of GPU time when this merge came, 60.3 with
// a CTA to a row, 56.3 with four partials in flight; now 55.8).
__global__ void __launch_bounds__(kMergeWarps * 32)
merge_warp_kernel(const DecodeArgs a) {
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  if (row >= a.num_seqs * a.num_q_heads) return;
  const int b = row / a.num_q_heads;
  const int n = a.seq_lens[b];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int ns = partials(a, row, b, n);
  if (ns <= 1) return;
  const Folded r = fold<8>(a, row, lane, 0, 1, ns);
  const __nv_bfloat162 lo = __floats2bfloat162_rn(r.sum.x, r.sum.y);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(r.sum.z, r.sum.w);
  reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (int64_t)row * kHD)[lane] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

}  // namespace

int fp8_block_split_tokens(int num_seqs, int num_kv_heads, int max_seq_len) {
  const int64_t streams = num_kv_heads % kBPS == 0 ? num_kv_heads / kBPS : num_kv_heads;
  const int64_t tokens = (int64_t)num_seqs * streams * max_seq_len;
  int s = kSplitTokens;
  while (s > kStageTok && tokens < 4ll * s * (3 * 152)) s /= 2;
  return s;
}

cudaError_t launch_paged_decode_fp8_block(const DecodeArgs& a, int num_sms, cudaStream_t stream) {
  if (a.chunk_prior >= 0 || a.split_tokens % kStageTok != 0 || !a.k_bscale || !a.v_bscale)
    return cudaErrorInvalidValue;
  DecodeArgs m = a;
  m.partials_f16 = 0;
  cudaError_t e = launch_fp8<true>(a, num_sms, stream, &m.balanced);
  if (e != cudaSuccess || a.max_splits <= 1) return e;
  // a warp a row fills the GPU once there are a thousand rows or more
  const int rows = a.num_seqs * a.num_q_heads;
  const bool by_warp = rows > 8 * 152;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(by_warp ? (rows + kMergeWarps - 1) / kMergeWarps : rows);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, by_warp ? merge_warp_kernel : merge_row_kernel, m);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pkv
