// Attention of drafted tokens over the paged cache, and the sums of what its
// softmax gave each key, on CUDA cores (fp32).
//
// Attention: for drafted token i of sequence b and query head h of KV head
// g = h / G, over the keys it sees (every token of the context, and the
// drafted tokens of its mask),
//   s_n = scale q_ih . k_n,  lse = ln sum_n e^{s_n},  out = sum_n e^{s_n - lse} v_n.
// A row that sees nothing gets out = 0 and lse = -inf.
//
// A row of this kernel is (drafted token, query head of the group), token
// first.  A CTA takes 32 rows of one (sequence, KV head) and walks key tiles
// of 32 tokens; the cluster's CTAs (up to 8) take turns on the tiles and join
// their running (m, l, O) through distributed shared memory at the end, so a
// short batch still fills the GPU and no workspace is needed.  Thread (r, c)
// of 32 x 8 forms the scores of row r with keys c, c + 8, c + 16, c + 24 and
// sums P V of row r for the dims 4 c + 32 i ...: K and V tiles are read from
// shared memory 16 bytes at a time.  It is bound by those reads (5 for 16
// multiply-adds); fp32 is the check's type, the bf16 cache has its own kernel.
#include <climits>

#include <cooperative_groups.h>

#include "common.cuh"
#include "host_cache.h"
#include "launch.h"
#include "tree_common.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kRows = 32, kKeys = 32, kThreadsCC = 256;
constexpr int kMaxCluster = 8;
constexpr int kWKeys = 128;            // keys of a CTA of the weights kernel
constexpr float kLog2e = 1.4426950408889634f;

template <typename T, int D>
struct TreeSmem {
  static constexpr int LD = D + 4;     // row stride in floats: 16 bytes off a multiple of 128
  float q[kRows][LD];
  float k[kKeys][LD];
  float v[kKeys][LD];
  float p[kRows][kKeys + 4];
  float o[kRows][LD];
  float m[kRows], l[kRows];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes of T as floats
template <typename T>
__device__ __forceinline__ void put16(float* dst, const uint4& x) {
  float f[Elem<T>::kPer16B];
  Elem<T>::unpack(x, f);
#pragma unroll
  for (int i = 0; i < Elem<T>::kPer16B; i += 4)
    *reinterpret_cast<float4*>(dst + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
}

// Pool row of token t of sequence b (block 0 for a block id out of range,
// which is recorded).
__device__ __forceinline__ int64_t pool_row(const TreeArgs& a, const int32_t* table, int t, int g) {
  int blk = __ldg(table + t / kBlockSize);
  if (blk < 0 || (int64_t)blk >= a.num_blocks) {
    record_error(a.err, DEVERR_BLOCK_RANGE);
    blk = 0;
  }
  return ((int64_t)blk * a.num_kv_heads + g) * kBlockSize + t % kBlockSize;
}

template <typename T, int D>
__device__ __forceinline__ void load_q(const TreeArgs& a, const TreeSeq& s, int g, int group, int row0, int rows,
                                       float (*q)[D + 4]) {
  constexpr int PER = Elem<T>::kPer16B, CH = D / PER;
  for (int i = threadIdx.x; i < kRows * CH; i += kThreadsCC) {
    const int r = i / CH, c = i % CH, row = row0 + r;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (row < rows) {
      const int64_t at = (int64_t)(s.row0 + row / group) * a.num_q_heads + g * group + row % group;
      x = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + at * D) + c);
    }
    put16<T>(&q[r][c * PER], x);
  }
}

// The scores of row r with keys c + 8 j (not scaled).
template <int D>
__device__ __forceinline__ void dots(const float* q, const float (*k)[D + 4], int c, float (&s)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j] = 0.f;
#pragma unroll 8
  for (int d = 0; d < D; d += 4) {
    const float4 x = *reinterpret_cast<const float4*>(q + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 y = *reinterpret_cast<const float4*>(&k[c + 8 * j][d]);
      s[j] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[j]))));
    }
  }
}

__device__ __forceinline__ bool seen(int t, int ctx, uint64_t bits) {
  return t < ctx || (t - ctx < 64 && ((bits >> (t - ctx)) & 1));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsCC) tree_cc_kernel(const TreeArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  TreeSmem<T, D>& sm = *reinterpret_cast<TreeSmem<T, D>*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
  const int group = a.num_q_heads / a.num_kv_heads;
  const int chunks = (a.max_draft * group + kRows - 1) / kRows;
  const int item = blockIdx.x / ranks;   // (sequence, KV head, 32 rows)
  const int b = item / chunks / a.num_kv_heads, g = item / chunks % a.num_kv_heads;
  const int row0 = item % chunks * kRows;
  const TreeSeq s = tree_seq(a, b, rank == 0 && threadIdx.x == 0);
  const int rows = s.drafted * group;
  if (row0 >= rows) return;              // the same for the whole cluster
  const int ctx = s.len - s.drafted;
  const int tid = threadIdx.x, r = tid >> 3, c = tid & 7;
  const int row = row0 + r;
  const uint64_t bits = row < rows ? tree_bits(a, s, row / group) : 0;
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks_per_seq;
  load_q<T, D>(a, s, g, group, row0, rows, sm.q);

  constexpr int PER = Elem<T>::kPer16B, CH = D / PER;
  constexpr int STEPS = (kKeys * CH + kThreadsCC - 1) / kThreadsCC;
  uint4 kr[STEPS], vr[STEPS];
  auto fetch = [&](int tile) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int at = tid + i * kThreadsCC, key = at / CH, t = tile * kKeys + key;
      kr[i] = vr[i] = make_uint4(0, 0, 0, 0);   // past the end: zeros, whatever the pool holds
      if (at < kKeys * CH && t < s.len) {
        const int64_t prow = pool_row(a, table, t, g) * D;
        kr[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_cache) + prow) + at % CH);
        vr[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.v_cache) + prow) + at % CH);
      }
    }
  };
  const int tiles = (s.len + kKeys - 1) / kKeys;
  const float sl2 = a.scale * kLog2e;
  float m = -INFINITY, l = 0.f, o[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i] = 0.f;
  if (rank < tiles) fetch(rank);
  for (int tile = rank; tile < tiles; tile += ranks) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int at = tid + i * kThreadsCC;
      if (at < kKeys * CH) {
        put16<T>(&sm.k[at / CH][at % CH * PER], kr[i]);
        put16<T>(&sm.v[at / CH][at % CH * PER], vr[i]);
      }
    }
    __syncthreads();
    if (tile + ranks < tiles) fetch(tile + ranks);
    float sc[4];
    dots<D>(sm.q[r], sm.k, c, sc);
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = tile * kKeys + c + 8 * j;
      sc[j] = t < s.len && seen(t, ctx, bits) ? sc[j] * sl2 : -INFINITY;
      mx = fmaxf(mx, sc[j]);
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const float m_new = fmaxf(m, mx), base = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = ex2(m - base);   // m = -inf: 0, of sums that are 0
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float p = ex2(sc[j] - base);
      sum += p;
      sm.p[r][c + 8 * j] = p;
    }
    l = l * alpha + sum;                 // this thread's share of the row's sum
    m = m_new;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i] *= alpha;
    __syncwarp();                        // a row's eight threads are in one warp
#pragma unroll 4
    for (int n = 0; n < kKeys; ++n) {
      const float p = sm.p[r][n];
      if (p == 0.f) continue;            // a masked key's value never counts, be it NaN
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(&sm.v[n][4 * c + 32 * i]);
        o[4 * i] = fmaf(p, v.x, o[4 * i]);
        o[4 * i + 1] = fmaf(p, v.y, o[4 * i + 1]);
        o[4 * i + 2] = fmaf(p, v.z, o[4 * i + 2]);
        o[4 * i + 3] = fmaf(p, v.w, o[4 * i + 3]);
      }
      if constexpr (D < 32) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i] = fmaf(p, sm.v[n][c * (D / 8) + i], o[i]);
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  // where this thread's o[i] belongs
  auto dim = [&](int i) { return D < 32 ? c * (D / 8) + i : 4 * c + 32 * (i / 4) + i % 4; };
#pragma unroll
  for (int i = 0; i < D / 8; ++i) sm.o[r][dim(i)] = o[i];
  if (c == 0) {
    sm.m[r] = m;
    sm.l[r] = l;
  }
  cluster.sync();
  // the ranks share the rows: rank k joins rows k, k + ranks, ...
  for (int rr = rank + ranks * r; rr < kRows; rr += ranks * kRows) {
    if (row0 + rr >= rows) break;
    float top = -INFINITY;
    for (int k = 0; k < ranks; ++k) top = fmaxf(top, cluster.map_shared_rank(sm.m, k)[rr]);
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f, acc[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) acc[i] = 0.f;
    for (int k = 0; k < ranks; ++k) {
      const float w = ex2(cluster.map_shared_rank(sm.m, k)[rr] - base);
      total = fmaf(w, cluster.map_shared_rank(sm.l, k)[rr], total);
      const float* line = cluster.map_shared_rank(&sm.o[0][0], k) + rr * TreeSmem<T, D>::LD;
      if (w != 0.f)
#pragma unroll
        for (int i = 0; i < D / 8; ++i) acc[i] = fmaf(w, line[dim(i)], acc[i]);
    }
    const bool none = total == 0.f;      // the row sees nothing (a NaN score makes total NaN)
    const float inv = 1.f / total;
    const int64_t at = (int64_t)(s.row0 + (row0 + rr) / group) * a.num_q_heads + g * group + (row0 + rr) % group;
    T* out = static_cast<T*>(a.out) + at * D;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) Elem<T>::store(out + dim(i), none ? 0.f : acc[i] * inv);
    if (a.lse && c == 0) a.lse[at] = none ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
  }
  cluster.sync();                        // nobody leaves while its shared memory is read
}

// weights[b][g][n] += sum over the rows that see key n of e^{s - lse}.  A CTA
// keeps 128 keys of one (sequence, KV head) in shared memory and walks the
// rows 32 at a time; thread (r, c) adds up rows r, r + 32, ... for its 16 keys
// and the 32 sums of a key are added in a fixed order, by one thread, into the
// running sum: no atomics, the same result every time.
template <int D>
struct WeightSmem {
  float q[kRows][D + 4];
  float k[kWKeys][D + 4];
  float part[kRows][kWKeys + 1];
  float lse[kRows];
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsCC) weights_cc_kernel(const TreeArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  WeightSmem<D>& sm = *reinterpret_cast<WeightSmem<D>*>(smem_raw);
  const int group = a.num_q_heads / a.num_kv_heads;
  const int tiles = (a.max_seq_len + kWKeys - 1) / kWKeys;
  const int item = blockIdx.x / tiles;   // (sequence, KV head)
  const int b = item / a.num_kv_heads, g = item % a.num_kv_heads;
  const TreeSeq s = tree_seq(a, b, blockIdx.x % tiles == 0 && threadIdx.x == 0);
  const int rows = s.drafted * group, key0 = (int)(blockIdx.x % tiles) * kWKeys;
  if (rows == 0 || key0 >= s.len) return;
  const int ctx = s.len - s.drafted;
  const int tid = threadIdx.x, r = tid >> 3, c = tid & 7;
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks_per_seq;
  constexpr int PER = Elem<T>::kPer16B, CH = D / PER;
  for (int i = tid; i < kWKeys * CH; i += kThreadsCC) {
    const int key = i / CH, t = key0 + key;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (t < s.len)
      x = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_cache) + pool_row(a, table, t, g) * D) +
                i % CH);
    put16<T>(&sm.k[key][i % CH * PER], x);
  }
  const float sl2 = a.scale * kLog2e;
  float acc[kWKeys / 8];
#pragma unroll
  for (int i = 0; i < kWKeys / 8; ++i) acc[i] = 0.f;
  for (int row0 = 0; row0 < rows; row0 += kRows) {
    __syncthreads();
    load_q<T, D>(a, s, g, group, row0, rows, sm.q);
    if (tid < kRows) {
      const int row = row0 + tid;
      // a row that sees nothing (lse = -inf) gives nothing: 2^(s - inf) = 0
      float x = INFINITY;
      if (row < rows) {
        x = a.lse[(int64_t)(s.row0 + row / group) * a.num_q_heads + g * group + row % group];
        x = x == -INFINITY ? INFINITY : x * kLog2e;
      }
      sm.lse[tid] = x;
    }
    __syncthreads();
    const int row = row0 + r;
    if (row < rows) {
      const uint64_t bits = tree_bits(a, s, row / group);
      const float lse = sm.lse[r];
#pragma unroll
      for (int part = 0; part < kWKeys / 32; ++part) {
        float sc[4];
        dots<D>(sm.q[r], sm.k + 32 * part, c, sc);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (seen(key0 + 32 * part + c + 8 * j, ctx, bits)) acc[4 * part + j] += ex2(fmaf(sc[j], sl2, -lse));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kWKeys / 8; ++i) sm.part[r][32 * (i / 4) + c + 8 * (i % 4)] = acc[i];
  __syncthreads();
  if (tid < kWKeys && key0 + tid < s.len) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) sum += sm.part[i][tid];
    a.weights[((int64_t)b * a.num_kv_heads + g) * a.weights_len + key0 + tid] += sum;
  }
}

template <typename T, int D>
cudaError_t launch_attention(const TreeArgs& a, cudaStream_t stream) {
  const int group = a.num_q_heads / a.num_kv_heads;
  const int chunks = (a.max_draft * group + kRows - 1) / kRows;
  const int tiles = (a.max_seq_len + kKeys - 1) / kKeys;
  int ranks = 1;
  while (ranks < kMaxCluster && 2 * ranks <= tiles) ranks *= 2;
  const int smem = (int)sizeof(TreeSmem<T, D>);
  cudaError_t e = allow_dynamic_smem(tree_cc_kernel<T, D>, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int64_t ctas = (int64_t)a.num_seqs * a.num_kv_heads * chunks * ranks;
  if (ctas > INT_MAX) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreadsCC);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tree_cc_kernel<T, D>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_weights(const TreeArgs& a, cudaStream_t stream) {
  const int smem = (int)sizeof(WeightSmem<D>);
  cudaError_t e = allow_dynamic_smem(weights_cc_kernel<T, D>, smem);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t)a.num_seqs * a.num_kv_heads * ((a.max_seq_len + kWKeys - 1) / kWKeys);
  if (ctas > INT_MAX) return cudaErrorInvalidValue;
  weights_cc_kernel<T, D><<<(unsigned)ctas, kThreadsCC, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_attention_cc(const TreeArgs& a, bool is_bf16, cudaStream_t stream) {
  if (is_bf16) return launch_attention<__nv_bfloat16, 128>(a, stream);
  return a.head_dim == 16 ? launch_attention<float, 16>(a, stream) : launch_attention<float, 128>(a, stream);
}

cudaError_t launch_kv_add_weights_cc(const TreeArgs& a, bool is_bf16, cudaStream_t stream) {
  if (is_bf16) return launch_weights<__nv_bfloat16, 128>(a, stream);
  return a.head_dim == 16 ? launch_weights<float, 16>(a, stream) : launch_weights<float, 128>(a, stream);
}

}  // namespace pkv
