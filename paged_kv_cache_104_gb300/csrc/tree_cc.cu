// Attention of drafted tokens over the paged fp32 cache, and the sums of what
// its softmax gave each key, on CUDA cores.
//
// Attention: for drafted token i of sequence b and query head h of KV head
// g = h / G, over the keys it sees (every token of the context, and the
// drafted tokens of its mask),
//   s_n = scale q_ih . k_n,  lse = ln sum_n e^{s_n},  out = sum_n e^{s_n - lse} v_n.
// A row that sees nothing gets out = 0 and lse = -inf.
//
// A row of this kernel is (drafted token, query head of the group), token
// first.  A CTA takes 32 rows of one (sequence, KV head), or 16 or 8 where no
// sequence has more, and walks key tiles of 32 tokens; the cluster's CTAs (up to
// 8) take turns on the tiles and join their running (m, l, O) through
// distributed shared memory at the end, so a short batch still fills the GPU and
// no workspace is needed.
//
// What bounds it is shared memory, its rate and, with 16 warps on an SM, its
// latency: for 4 sequences of 30,842 with 8 rows its data pipe is busy 58% of the
// time (DRAM 36%), and warps wait for it longer than for all else; a short
// batch (16%) is one chain of tiles.  Each query is read again for every tile.
// A warp has four rows of its own, so that a K or V value that it reads serves four: for the scores a
// lane has four keys and a quarter of the dims (8 reads of 16 bytes for 64
// multiply-adds; a row and four keys a thread took 5 for 16, and 52.8 us for
// four sequences of 500 to 1,500 against 21.4), for P V four dims of the four
// rows (2 reads for 16).  A warp without rows only helps to load; with up to 16 or
// 8 rows two or four warps split a tile's keys and join at the end (8 query heads
// to 4 KV heads and 5 drafted tokens over 500 to 1,500 21.4 -> 20.0 us; 4 sequences
// of 30,842 with 8 rows, 1 GB, 402 -> 354; 2 of 10,457 with 4 rows of 16 dims 58 ->
// 31; 16 of 2,000 with 12 rows 67 -> 66).
#include <climits>

#include <cooperative_groups.h>

#include "common.cuh"
#include "host_cache.h"
#include "launch.h"
#include "tree_common.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kRows = 32, kKeys = 32, kThreadsCC = 256, kWarps = kThreadsCC / 32;
constexpr int kMaxCluster = 8;
constexpr int kWKeys = 128;            // keys of a CTA of the weights kernel
constexpr float kLog2e = 1.4426950408889634f;
constexpr unsigned kAll = 0xffffffffu;
static_assert(kRows == 4 * kWarps, "four rows a warp");

template <int D>
struct TreeSmem {
  static constexpr int LD = D + 4;     // row stride in floats: 16 bytes off a multiple of 128
  float q[kRows][LD];
  float k[kKeys][LD];
  float v[kKeys][LD];
  float4 p[kWarps][kKeys];             // a key's weights of the warp's four rows
  float o[kRows][LD];
  float m[kRows], l[kRows];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

// Rows row0 .. row0 + ROWS - 1 of the queries (zeros behind the last).
template <int D, int ROWS = kRows>
__device__ __forceinline__ void load_q(const TreeArgs& a, const TreeSeq& s, int g, int group, int row0, int rows,
                                       float (*q)[D + 4]) {
  constexpr int CH = D / 4;
  for (int i = threadIdx.x; i < ROWS * CH; i += kThreadsCC) {
    const int r = i / CH, c = i % CH, row = row0 + r;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows) {
      const int64_t at = (int64_t)(s.row0 + row / group) * a.num_q_heads + g * group + row % group;
      x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at * D) + c);
    }
    *reinterpret_cast<float4*>(&q[r][c * 4]) = x;
  }
}

// Scores (not scaled) of a warp's four rows q with keys (lane & 7) + 8 j, j < J:
// a lane sums a quarter of the dims, then four lanes add theirs.
template <int D, int J>
__device__ __forceinline__ void scores(const float (*q)[D + 4], const float (*k)[D + 4], int lane, float (&s)[4][J]) {
  const int key = lane & 7, d0 = (lane >> 3) * (D / 4);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int d = d0; d < d0 + D / 4; d += 4) {
    float4 x[4], y[J];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(&q[i][d]);
#pragma unroll
    for (int j = 0; j < J; ++j) y[j] = *reinterpret_cast<const float4*>(&k[key + 8 * j][d]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
        s[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, s[i][j]))));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      s[i][j] += __shfl_xor_sync(kAll, s[i][j], 8);
      s[i][j] += __shfl_xor_sync(kAll, s[i][j], 16);
    }
}

__device__ __forceinline__ bool seen(int t, int ctx, uint64_t bits) {
  return t < ctx || (t - ctx < 64 && ((bits >> (t - ctx)) & 1));
}

// SPLIT: the keys of a tile are split between so many warps, of 32 / SPLIT rows.
template <int D, int SPLIT>
__global__ void __launch_bounds__(kThreadsCC, SPLIT > 1 ? 2 : 0) tree_cc_kernel(const TreeArgs a) {
  constexpr int ROWS = kRows / SPLIT, QUADS = ROWS / 4, J = 4 / SPLIT;
  static_assert(QUADS * SPLIT == kWarps, "a warp has four rows and 8 J keys");
  extern __shared__ __align__(16) unsigned char smem_raw[];
  TreeSmem<D>& sm = *reinterpret_cast<TreeSmem<D>*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
  const int group = a.num_q_heads / a.num_kv_heads;
  const int chunks = (a.max_draft * group + ROWS - 1) / ROWS;
  const int item = blockIdx.x / ranks;   // (sequence, KV head, ROWS rows)
  const int b = item / chunks / a.num_kv_heads, g = item / chunks % a.num_kv_heads;
  const int row0 = item % chunks * ROWS;
  const TreeSeq s = tree_seq(a, b, rank == 0 && threadIdx.x == 0);
  const int rows = s.drafted * group;
  if (row0 >= rows) return;              // the same for the whole cluster
  const int ctx = s.len - s.drafted;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks_per_seq;

  constexpr int CH = D / 4, STEPS = (kKeys * CH + kThreadsCC - 1) / kThreadsCC;
  constexpr int BLOCKS = kKeys / kBlockSize;
  static_assert(BLOCKS == 2, "two cache blocks a tile");
  float4 kr[STEPS], vr[STEPS];
  int blocks[BLOCKS];                    // of the tile to be fetched next
  auto ask_blocks = [&](int tile) {
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i) {
      blocks[i] = 0;
      if ((tile * BLOCKS + i) * kBlockSize < s.len) blocks[i] = __ldg(table + tile * BLOCKS + i);
    }
  };
  auto fetch = [&](int tile) {
#pragma unroll
    for (int i = 0; i < BLOCKS; ++i)
      if (blocks[i] < 0 || (int64_t)blocks[i] >= a.num_blocks) {
        record_error(a.err, DEVERR_BLOCK_RANGE);
        blocks[i] = 0;
      }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int at = tid + i * kThreadsCC, key = at / CH;
      kr[i] = vr[i] = make_float4(0.f, 0.f, 0.f, 0.f);   // past the end: zeros, whatever the pool holds
      if (at < kKeys * CH && tile * kKeys + key < s.len) {
        const int64_t prow =
            (((int64_t)(key < kBlockSize ? blocks[0] : blocks[1]) * a.num_kv_heads + g) * kBlockSize +
             key % kBlockSize) * D;
        kr[i] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.k_cache) + prow) + at % CH);
        vr[i] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.v_cache) + prow) + at % CH);
      }
    }
    ask_blocks(tile + ranks);
  };
  const int tiles = (s.len + kKeys - 1) / kKeys;
  ask_blocks(rank);
  if (rank < tiles) fetch(rank);
  load_q<D, ROWS>(a, s, g, group, row0, rows, sm.q);

  // this warp's rows r0 + i and keys k0 .., a lane's keys k0 + (lane & 7) + 8 j and dims 4 dg ..
  const int r0 = 4 * (SPLIT == 1 ? warp : warp % QUADS), part = SPLIT == 1 ? 0 : warp / QUADS, k0 = part * 8 * J;
  constexpr int DG = D / 4 < 32 ? D / 4 : 32, KS = 32 / DG;   // lanes over dims, and over keys
  static_assert(D == 4 * DG, "four dims a lane");
  const bool live = row0 + r0 < rows;
  const int dg = lane % DG;
  uint64_t bits[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + r0 + i;
    bits[i] = row < rows ? tree_bits(a, s, row / group) : 0;
  }
  const float sl2 = a.scale * kLog2e;
  float m[4], l[4], o[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  }
  for (int tile = rank; tile < tiles; tile += ranks) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int at = tid + i * kThreadsCC;
      if (at < kKeys * CH) {
        *reinterpret_cast<float4*>(&sm.k[at / CH][at % CH * 4]) = kr[i];
        *reinterpret_cast<float4*>(&sm.v[at / CH][at % CH * 4]) = vr[i];
      }
    }
    __syncthreads();
    if (tile + ranks < tiles) fetch(tile + ranks);
    if (!live) continue;
    float sc[4][J];
    scores<D, J>(sm.q + r0, sm.k + k0, lane, sc);
    const bool all = (tile + 1) * kKeys <= ctx;   // every row sees every key
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int t = tile * kKeys + k0 + (lane & 7) + 8 * j;
        sc[i][j] = all || (t < s.len && seen(t, ctx, bits[i])) ? sc[i][j] * sl2 : -INFINITY;
        mx = fmaxf(mx, sc[i][j]);
      }
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, d));
      const float m_new = fmaxf(m[i], mx), base = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = ex2(m[i] - base);   // m = -inf: 0, of sums that are 0
      l[i] *= alpha;                          // this lane's share of the row's sum
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < J) {
          sc[i][j % J] = ex2(sc[i][j % J] - base);
          l[i] += sc[i][j % J];
        }
        o[i][j] *= alpha;
      }
      m[i] = m_new;
    }
    // four lanes have the same weights: each writes one key's
    const int j = lane >> 3;
    auto pick = [&](int i) {
      if constexpr (J == 1) return sc[i][0];
      else if constexpr (J == 2) return j & 1 ? sc[i][1] : sc[i][0];
      else return j < 2 ? (j == 0 ? sc[i][0] : sc[i][1]) : (j == 2 ? sc[i][2] : sc[i][3]);
    };
    __syncwarp();
    if (j < J) sm.p[warp][lane] = make_float4(pick(0), pick(1), pick(2), pick(3));   // key (lane & 7) + 8 j
    __syncwarp();
#pragma unroll 4
    for (int n = lane / DG; n < 8 * J; n += KS) {
      const float4 p = sm.p[warp][n];
      const float4 v = *reinterpret_cast<const float4*>(&sm.v[k0 + n][4 * dg]);
      const float w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (w[i] != 0.f) {                    // a masked key's value never counts, be it NaN
          o[i][0] = fmaf(w[i], v.x, o[i][0]);
          o[i][1] = fmaf(w[i], v.y, o[i][1]);
          o[i][2] = fmaf(w[i], v.z, o[i][2]);
          o[i][3] = fmaf(w[i], v.w, o[i][3]);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) l[i] += __shfl_xor_sync(kAll, l[i], d);
#pragma unroll
    for (int d = DG; d < 32; d <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] += __shfl_xor_sync(kAll, o[i][j], d);
    const int at = part * ROWS + r0 + i;
    if (lane < DG) *reinterpret_cast<float4*>(&sm.o[at][4 * dg]) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
    if (lane == 0) {
      sm.m[at] = m[i];
      sm.l[at] = l[i];
    }
  }
  cluster.sync();
  // the ranks share the rows, a warp per row: rank k joins rows k, k + ranks, ...
  // piece e of a row: part e % SPLIT of rank e / SPLIT
  const int pieces = ranks * SPLIT;
  static_assert(kMaxCluster * SPLIT <= 32, "a lane per piece");
  for (int r = rank + ranks * warp; r < ROWS && row0 + r < rows; r += ranks * kWarps) {
    auto value = [&](int e) {
      return *reinterpret_cast<const float4*>(cluster.map_shared_rank(&sm.o[e % SPLIT * ROWS + r][4 * dg], e / SPLIT));
    };
    const int of = lane % SPLIT * ROWS + r;
    const float mine = lane < pieces ? cluster.map_shared_rank(sm.m, lane / SPLIT)[of] : -INFINITY;
    float total = lane < pieces ? cluster.map_shared_rank(sm.l, lane / SPLIT)[of] : 0.f;
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < pieces) x[k] = value(k);
    float top = mine;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
    const float w = ex2(mine - (top == -INFINITY ? 0.f : top));
    total *= w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(kAll, total, d);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int e = 0; e < (SPLIT == 1 ? 1 : pieces); e += 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float wk = __shfl_sync(kAll, w, (e + k) & 31);
        if (e + k < pieces && wk != 0.f) {
          acc.x = fmaf(wk, x[k].x, acc.x);
          acc.y = fmaf(wk, x[k].y, acc.y);
          acc.z = fmaf(wk, x[k].z, acc.z);
          acc.w = fmaf(wk, x[k].w, acc.w);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (SPLIT > 1 && e + 8 + k < pieces) x[k] = value(e + 8 + k);
    }
    const bool none = total == 0.f;      // the row sees nothing (a NaN score makes total NaN)
    const float inv = none ? 0.f : 1.f / total;
    const int64_t at = (int64_t)(s.row0 + (row0 + r) / group) * a.num_q_heads + g * group + (row0 + r) % group;
    if (lane < DG)
      reinterpret_cast<float4*>(static_cast<float*>(a.out) + at * D)[dg] =
          none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (a.lse && lane == 0) a.lse[at] = none ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
  }
  cluster.sync();                        // nobody leaves while its shared memory is read
}

// weights[b][g][n] += sum over the rows that see key n of e^{s - lse}.  A CTA
// keeps 128 keys of one (sequence, KV head) in shared memory and walks the
// rows 32 at a time; warp w takes 32 of the keys (w mod 4) with every other
// four rows, a lane four of those keys.  The sums of a key are added in a fixed
// order, by one thread, into the running sum: no atomics, the same result every
// time.
template <int D>
struct WeightSmem {
  float q[kRows][D + 4];
  float k[kWKeys][D + 4];
  float part[kWarps][kKeys];
  float lse[kRows];
};

template <int D>
__global__ void __launch_bounds__(kThreadsCC, 2) weights_cc_kernel(const TreeArgs a) {
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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks_per_seq;
  // block ids first, then eight keys' chunks on their way at a time
  constexpr int CH = D / 4, STEPS = kWKeys * CH / kThreadsCC, AT_ONCE = STEPS < 8 ? STEPS : 8;
  int64_t from[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int t = key0 + (tid + i * kThreadsCC) / CH;
    from[i] = t < s.len ? pool_row(a, table, t, g) : -1;
  }
#pragma unroll
  for (int i0 = 0; i0 < STEPS; i0 += AT_ONCE) {
    float4 x[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (from[i0 + i] >= 0)
        x[i] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.k_cache) + from[i0 + i] * D) + tid % CH);
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      *reinterpret_cast<float4*>(&sm.k[(tid + (i0 + i) * kThreadsCC) / CH][tid % CH * 4]) = x[i];
  }
  const float sl2 = a.scale * kLog2e;
  const int sub = kKeys * (warp & 3);    // this warp's keys
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int row0 = 0; row0 < rows; row0 += kRows) {
    __syncthreads();
    load_q<D>(a, s, g, group, row0, rows, sm.q);
    if (tid < kRows) {
      const int row = row0 + tid;
      float x = -INFINITY;
      if (row < rows) x = a.lse[(int64_t)(s.row0 + row / group) * a.num_q_heads + g * group + row % group] * kLog2e;
      sm.lse[tid] = x;
    }
    __syncthreads();
    for (int r = 4 * (warp >> 2); r < kRows && row0 + r < rows; r += 8) {
      float sc[4][4];
      scores<D, 4>(sm.q + r, sm.k + sub, lane, sc);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = row0 + r + i;
        if (row >= rows) break;
        if (sm.lse[r + i] == -INFINITY) continue;   // adds nothing, be its scores NaN
        const uint64_t bits = tree_bits(a, s, row / group);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (seen(key0 + sub + (lane & 7) + 8 * j, ctx, bits)) acc[j] += ex2(fmaf(sc[i][j], sl2, -sm.lse[r + i]));
      }
    }
  }
  if (lane < 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) sm.part[warp][lane + 8 * j] = acc[j];
  __syncthreads();
  if (tid < kWKeys && key0 + tid < s.len)
    a.weights[((int64_t)b * a.num_kv_heads + g) * a.weights_len + key0 + tid] +=
        sm.part[tid >> 5][tid & 31] + sm.part[(tid >> 5) + 4][tid & 31];
}

template <int D, int SPLIT>
cudaError_t launch_attention(const TreeArgs& a, cudaStream_t stream) {
  const int group = a.num_q_heads / a.num_kv_heads;
  const int chunks = (a.max_draft * group + kRows / SPLIT - 1) / (kRows / SPLIT);
  const int tiles = (a.max_seq_len + kKeys - 1) / kKeys;
  int ranks = 1;
  while (ranks < kMaxCluster && 2 * ranks <= tiles) ranks *= 2;
  const int smem = (int)sizeof(TreeSmem<D>);
  cudaError_t e = allow_dynamic_smem(tree_cc_kernel<D, SPLIT>, smem);
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
  e = cudaLaunchKernelEx(&cfg, tree_cc_kernel<D, SPLIT>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
cudaError_t launch_weights(const TreeArgs& a, cudaStream_t stream) {
  const int smem = (int)sizeof(WeightSmem<D>);
  cudaError_t e = allow_dynamic_smem(weights_cc_kernel<D>, smem);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t)a.num_seqs * a.num_kv_heads * ((a.max_seq_len + kWKeys - 1) / kWKeys);
  if (ctas > INT_MAX) return cudaErrorInvalidValue;
  weights_cc_kernel<D><<<(unsigned)ctas, kThreadsCC, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_attention_cc(const TreeArgs& a, cudaStream_t stream) {
  const int rows = a.max_draft * (a.num_q_heads / a.num_kv_heads);
  if (a.head_dim == 16)
    return rows <= 8 ? launch_attention<16, 4>(a, stream)
                     : rows <= 16 ? launch_attention<16, 2>(a, stream) : launch_attention<16, 1>(a, stream);
  return rows <= 8 ? launch_attention<128, 4>(a, stream)
                   : rows <= 16 ? launch_attention<128, 2>(a, stream) : launch_attention<128, 1>(a, stream);
}

cudaError_t launch_kv_add_weights_cc(const TreeArgs& a, cudaStream_t stream) {
  return a.head_dim == 16 ? launch_weights<16>(a, stream) : launch_weights<128>(a, stream);
}

}  // namespace pkv
