// Appends that rotate positions on the way into the paged pools, and the
// quantising append of the block-scaled 8-bit cache.
//
// Rotation: a head's first rot_dim elements form rot_dim / 2 pairs, (i, i +
// rot_dim/2) or, interleaved, (2i, 2i + 1); pair i of token t turns by the
// angle whose cosine and sin stand in the table row of positions[axis(i)][t]:
//   a' = a cos - b sin,  b' = b cos + a sin
// in fp32, rounded once to the storage type.  The other elements are copied.
// The axis of a pair is the caller's table, so one axis (text), sections of
// time, height and width, or axes taken in turn are one kernel.
#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kMinScaleExp = -126;   // block scale exponents an append writes:
constexpr int kMaxScaleExp = 119;    // 448 * 2^119 is the largest such value below 2^128

// The table row (rot_dim floats: cosines, then sines) of a pair's position,
// or null when the position is outside the table.
__device__ __forceinline__ const float* table_row(const RopeArgs& r, int axis, int64_t t,
                                                  int64_t num_tokens) {
  const int p = __ldg(r.positions + axis * num_tokens + t);
  return p < 0 || (int64_t)p >= r.num_positions ? nullptr : r.cos_sin + (int64_t)p * r.rot_dim;
}

// True if every axis' position of token t is inside the table.
__device__ __forceinline__ bool positions_ok(const RopeArgs& r, int64_t t, int64_t num_tokens) {
  bool ok = true;
  for (int ax = 0; ax < r.num_axes; ++ax) ok &= table_row(r, ax, t, num_tokens) != nullptr;
  return ok;
}

// Rows are moved in units of two 16-byte chunks that hold the two sides of V
// pairs (V elements a chunk): chunks (u, u + half/V) of a head rotated by
// halves, chunks (2u, 2u + 1) of one with adjacent pairs.  Where the pairs
// do not fill whole chunks a unit is a single pair.
template <typename T, bool VEC>
struct Unit2 {
  static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
  // elements of the unit's first and second run of V (interleaved single
  // pairs: the two neighbours)
  __device__ __forceinline__ static void place(const RopeArgs& r, int u, int& e0, int& e1) {
    const int half = r.rot_dim / 2;
    if (u * V >= half) {               // behind the rotated part
      e0 = r.rot_dim + (u * V - half) * 2;
      e1 = e0 + V;
    } else if (r.interleaved) {
      e0 = 2 * u * V;
      e1 = e0 + V;
    } else {
      e0 = u * V;
      e1 = half + e0;
    }
  }
};

template <typename T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen(float x) { return x; }
template <>
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

// V elements from / to memory (16-byte accesses when V > 1)
template <typename T, int V>
struct Run {
  uint4 raw;
  __device__ __forceinline__ void load(const T* p) {
    // plain loads: queries may be rotated in place
    if constexpr (V > 1) raw = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<T*>(&raw) = *p;
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (V > 1) *reinterpret_cast<uint4*>(p) = raw;
    else *p = *reinterpret_cast<const T*>(&raw);
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
    if constexpr (V > 1) Elem<T>::unpack(raw, f);
    else f[0] = widen(*reinterpret_cast<const T*>(&raw));
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
    T* t = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < V; ++i) Elem<T>::store(t + i, f[i]);
  }
};

// cosines and sines of a unit's V pairs
template <int V>
struct Turn {
  float c[V], s[V];
  __device__ __forceinline__ void load(const RopeArgs& r, int u, int64_t t, int64_t num_tokens) {
    const int half = r.rot_dim / 2, i0 = u * V;
    if (V > 1 && r.whole_axes) {   // the unit's pairs share an axis: whole 16-byte loads
      const float* row = table_row(r, r.pair_axis[i0], t, num_tokens);
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        if constexpr (V >= 4) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(row + i0 + i));
          const float4 y = __ldg(reinterpret_cast<const float4*>(row + half + i0 + i));
          c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
          s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float* row = table_row(r, r.pair_axis[i0 + i], t, num_tokens);
        c[i] = __ldg(row + i0 + i);
        s[i] = __ldg(row + half + i0 + i);
      }
    }
  }
};

// rotate the pairs of two runs in place
template <typename T, int V>
__device__ __forceinline__ void rotate(const RopeArgs& r, const Turn<V>& w, Run<T, V>& x,
                                       Run<T, V>& y) {
  float a[V], b[V];
  x.get(a);
  y.get(b);
  if (V > 1 && r.interleaved) {   // elements 2i, 2i + 1 of the two runs taken together
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      if constexpr (V > 1) {
        const float a0 = a[i], a1 = a[i + 1], b0 = b[i], b1 = b[i + 1];
        a[i] = a0 * w.c[i / 2] - a1 * w.s[i / 2];
        a[i + 1] = a1 * w.c[i / 2] + a0 * w.s[i / 2];
        b[i] = b0 * w.c[V / 2 + i / 2] - b1 * w.s[V / 2 + i / 2];
        b[i + 1] = b1 * w.c[V / 2 + i / 2] + b0 * w.s[V / 2 + i / 2];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float a0 = a[i], b0 = b[i];
      a[i] = a0 * w.c[i] - b0 * w.s[i];
      b[i] = b0 * w.c[i] + a0 * w.s[i];
    }
  }
  x.set(a);
  y.set(b);
}

// One thread takes one unit u of a token and every `slots`-th of its heads
// (query, key, then value heads), so the unit's cosines and sines are loaded
// once for all of them.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512)
kv_append_rope_kernel(const __grid_constant__ RopeAppendArgs a, int units, int slots) {
  constexpr int V = Unit2<T, VEC>::V;
  const int per_token = units * slots;
  const int tl = threadIdx.x / per_token;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / per_token) + tl;
  const int rem = threadIdx.x - tl * per_token;
  const int hs = rem / units, u = rem - hs * units;
  if (t >= a.num_tokens) return;
  const int64_t slot = __ldg(a.slot_mapping + t);
  if (slot < 0) return;
  if (slot >= a.num_blocks * kBlockSize) {
    record_error(a.err, DEVERR_SLOT_RANGE);
    return;
  }
  if (!positions_ok(a.rope, t, a.num_tokens)) {
    record_error(a.err, DEVERR_POSITION_RANGE);
    return;
  }
  const int64_t blk = slot / kBlockSize, row = slot - blk * kBlockSize;
  int e0, e1;
  Unit2<T, VEC>::place(a.rope, u, e0, e1);
  const bool turns = u * V < a.rope.rot_dim / 2;
  Turn<V> w;
  if (turns) w.load(a.rope, u, t, a.num_tokens);
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  for (int h = hs; h < heads; h += slots) {
    const T* src;
    T* dst;
    if (h < a.num_q_heads) {
      src = static_cast<const T*>(a.q) + t * a.q_stride + h * a.head_dim;
      dst = static_cast<T*>(a.q_out) + t * a.q_out_stride + h * a.head_dim;
    } else {
      const bool is_v = h >= a.num_q_heads + a.num_kv_heads;
      const int g = h - a.num_q_heads - (is_v ? a.num_kv_heads : 0);
      src = is_v ? static_cast<const T*>(a.v_new) + t * a.v_stride
                 : static_cast<const T*>(a.k_new) + t * a.k_stride;
      src += g * a.head_dim;
      dst = static_cast<T*>(is_v ? a.v_cache : a.k_cache) +
            ((blk * a.num_kv_heads + g) * kBlockSize + row) * a.head_dim;
    }
    Run<T, V> x, y;
    x.load(src + e0);
    y.load(src + e1);
    if (turns && h < a.num_q_heads + a.num_kv_heads) rotate<T, V>(a.rope, w, x, y);
    x.store(dst + e0);
    y.store(dst + e1);
  }
}

// ------------------------------------------------- block-scaled 8-bit cache

// 2^e as a float, e in [-126, 127]
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// Smallest exponent e with amax <= 448 * 2^e (448 = 1.75 * 2^8), amax >= 0 as
// the bits of a finite float.
__device__ __forceinline__ int scale_exp(uint32_t amax) {
  const int e = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(kMinScaleExp, min(kMaxScaleExp, e));
}

// One warp writes the N rows of a run of new tokens (t0 .. t0 + n - 1, n <=
// N) for one head of one pool: lane l owns pairs 2l and 2l + 1 of every row.
template <int N>
__device__ __forceinline__ void append_run(const RopeAppendArgs& a, const __nv_bfloat16* src,
                                           int64_t stride, uint8_t* pool, uint8_t* scale,
                                           bool rotated, int64_t t0, int n, int row0, int lane) {
  const RopeArgs& r = a.rope;
  const int half = r.rot_dim / 2;
  const int p0 = 2 * lane;                     // the lane's first pair
  const bool mine = 4 * lane < a.head_dim;
  const bool turns = rotated && p0 < half;
  // elements e0, e0 + 1 and e1, e1 + 1
  const bool adjacent = r.interleaved || p0 >= half;
  const int e0 = adjacent ? 4 * lane : p0, e1 = adjacent ? e0 + 2 : half + p0;
  uint32_t raw[N][2];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    raw[i][0] = raw[i][1] = 0u;
    if (mine && i < n) {
      const __nv_bfloat16* p = src + (t0 + i) * stride;
      raw[i][0] = __ldg(reinterpret_cast<const uint32_t*>(p + e0));
      raw[i][1] = __ldg(reinterpret_cast<const uint32_t*>(p + e1));
    }
  }
  float x[N][4];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i][0] = bf16lo(raw[i][0]);
    x[i][1] = bf16hi(raw[i][0]);
    x[i][2] = bf16lo(raw[i][1]);
    x[i][3] = bf16hi(raw[i][1]);
    if (turns && i < n) {
      float c[2], s[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float* trow = table_row(r, r.pair_axis[p0 + k], t0 + i, a.num_tokens);
        c[k] = __ldg(trow + p0 + k);
        s[k] = __ldg(trow + half + p0 + k);
      }
      if (r.interleaved) {   // pairs (x0, x1) and (x2, x3)
        const float x0 = x[i][0], x1 = x[i][1], x2 = x[i][2], x3 = x[i][3];
        x[i][0] = x0 * c[0] - x1 * s[0];
        x[i][1] = x1 * c[0] + x0 * s[0];
        x[i][2] = x2 * c[1] - x3 * s[1];
        x[i][3] = x3 * c[1] + x2 * s[1];
      } else {               // pairs (x0, x2) and (x1, x3)
        const float x0 = x[i][0], x1 = x[i][1], x2 = x[i][2], x3 = x[i][3];
        x[i][0] = x0 * c[0] - x2 * s[0];
        x[i][2] = x2 * c[0] + x0 * s[0];
        x[i][1] = x1 * c[1] - x3 * s[1];
        x[i][3] = x3 * c[1] + x1 * s[1];
      }
    }
    // the scale follows the finite elements only
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t m = __float_as_uint(x[i][k]) & 0x7fffffffu;
      if (m < 0x7f800000u) amax = max(amax, m);
    }
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  int e = scale_exp(amax);
  if (row0 > 0) {
    // the block's older rows: their codes are re-expressed where the scale grows
    const int b = *scale;
    const bool held = b >= 1 && b <= 253;      // otherwise they stand for nothing
    const int e_old = held ? b - 127 : e;
    if (!held || e > e_old) {
      const float f = held ? exp2i(max(e_old - e, -126)) : 0.f;
      if (mine) {
        for (int row = 0; row < row0; ++row) {
          uint32_t* p = reinterpret_cast<uint32_t*>(pool + row * a.head_dim + 4 * lane);
          const uint32_t c = *p;
          uint32_t out = 0;
          if (held) {
            const uint32_t lo = e4m3x2_to_f16x2((uint16_t)c), hi = e4m3x2_to_f16x2((uint16_t)(c >> 16));
            const float2 fl = __half22float2(*reinterpret_cast<const __half2*>(&lo));
            const float2 fh = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            out = f32x2_to_e4m3x2(fl.x * f, fl.y * f) |
                  ((uint32_t)f32x2_to_e4m3x2(fh.x * f, fh.y * f) << 16);
          }
          *p = out;
        }
      }
    }
    e = max(e, e_old);
  }
  const float inv = exp2i(-e);
  if (mine) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < n) {
        uint8_t* p = pool + (row0 + i) * a.head_dim;
        *reinterpret_cast<uint16_t*>(p + e0) = f32x2_to_e4m3x2(x[i][0] * inv, x[i][1] * inv);
        *reinterpret_cast<uint16_t*>(p + e1) = f32x2_to_e4m3x2(x[i][2] * inv, x[i][3] * inv);
      }
    }
  }
  __syncwarp();                                 // every lane has read the old scale
  if (lane == 0) *scale = (uint8_t)(e + 127);
}

constexpr int kAppendWarps = 8;

// CTA (t, y): y < head groups: if a run of new tokens starts at t, its rows
// for kAppendWarps / 2 heads, a warp for each head of each pool; the last y:
// token t's query.
__global__ void __launch_bounds__(kAppendWarps * 32)
kv_append_fp8_block_kernel(const __grid_constant__ RopeAppendArgs a, int groups, int units) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t slot = __ldg(a.slot_mapping + t);
  if (slot < 0) return;
  const int64_t pool_slots = a.num_blocks * kBlockSize;
  if (slot >= pool_slots) {
    record_error(a.err, DEVERR_SLOT_RANGE);
    return;
  }
  if ((int)blockIdx.y == groups) {              // the query
    if (!positions_ok(a.rope, t, a.num_tokens)) {
      record_error(a.err, DEVERR_POSITION_RANGE);
      return;
    }
    constexpr int V = 8;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_stride;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.q_out) + t * a.q_out_stride;
    for (int i = threadIdx.x; i < units * a.num_q_heads; i += blockDim.x) {
      const int h = i / units, u = i - h * units;
      int e0, e1;
      Run<__nv_bfloat16, V> x, y;
      Unit2<__nv_bfloat16, true>::place(a.rope, u, e0, e1);
      x.load(src + h * a.head_dim + e0);
      y.load(src + h * a.head_dim + e1);
      if (u * V < a.rope.rot_dim / 2) {
        Turn<V> w;
        w.load(a.rope, u, t, a.num_tokens);
        rotate<__nv_bfloat16, V>(a.rope, w, x, y);
      }
      x.store(dst + h * a.head_dim + e0);
      y.store(dst + h * a.head_dim + e1);
    }
    return;
  }
  const int64_t blk = slot / kBlockSize;
  const int row0 = (int)(slot - blk * kBlockSize);
  // a run starts at t unless the entry before holds the row before in this block
  if (row0 > 0 && t > 0 && __ldg(a.slot_mapping + t - 1) == slot - 1) return;
  // no nearby earlier entry may write this block: two runs would race on it
  const int64_t tb = t - 1 - lane;
  const int64_t before = tb >= 0 ? __ldg(a.slot_mapping + tb) : -1;
  if (__any_sync(0xffffffffu, before >= 0 && before / kBlockSize == blk)) {
    record_error(a.err, DEVERR_SLOT_ORDER);
    return;
  }
  // its length: following entries with following rows of the same block
  const int64_t ta = t + lane;
  const bool in = lane < kBlockSize - row0 && ta < a.num_tokens &&
                  __ldg(a.slot_mapping + min(ta, a.num_tokens - 1)) == slot + lane;
  const uint32_t run = __ballot_sync(0xffffffffu, in);
  int n = __ffs(~run) - 1;                      // >= 1: lane 0 is in
  // a bad position ends the run before its token
  if (a.rope.rot_dim > 0) {
    const uint32_t good =
        __ballot_sync(0xffffffffu, lane >= n || positions_ok(a.rope, ta, a.num_tokens));
    if (~good != 0u) {
      record_error(a.err, DEVERR_POSITION_RANGE);
      n = min(n, __ffs(~good) - 1);
      if (n == 0) return;
    }
  }
  const int unit = (int)blockIdx.y * kAppendWarps + warp;
  const bool is_v = unit & 1;
  const int g = unit >> 1;
  if (g >= a.num_kv_heads) return;
  const int64_t tile = blk * a.num_kv_heads + g;
  const __nv_bfloat16* src =
      static_cast<const __nv_bfloat16*>(is_v ? a.v_new : a.k_new) + g * a.head_dim;
  uint8_t* pool = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) +
                  tile * kBlockSize * a.head_dim;
  uint8_t* scale = (is_v ? a.v_scale : a.k_scale) + tile;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const bool rotated = !is_v && a.rope.rot_dim > 0;
  if (n == 1)
    append_run<1>(a, src, stride, pool, scale, rotated, t, n, row0, lane);
  else
    append_run<kBlockSize>(a, src, stride, pool, scale, rotated, t, n, row0, lane);
}

template <typename T, bool VEC>
cudaError_t launch_rope_typed(const RopeAppendArgs& a, cudaStream_t stream) {
  constexpr int V = Unit2<T, VEC>::V;
  const int units = a.head_dim / (2 * V);
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  int slots = heads;
  while (units * slots > 256 && slots > 1) slots = (slots + 1) / 2;
  const int per_token = units * slots;
  const int tokens = per_token >= 256 ? 1 : 256 / per_token;
  const int64_t grid = (a.num_tokens + tokens - 1) / tokens;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  kv_append_rope_kernel<T, VEC><<<(int)grid, per_token * tokens, 0, stream>>>(a, units, slots);
  return cudaGetLastError();
}

// True if the pairs fill whole 16-byte chunks of `size`-byte elements.
bool whole_chunks(const RopeAppendArgs& a, int size) {
  const int v = 16 / size;
  return (a.rope.rot_dim / 2) % v == 0 && (a.head_dim - a.rope.rot_dim) % (2 * v) == 0;
}

}  // namespace

cudaError_t launch_kv_append_rope(const RopeAppendArgs& args, bool is_bf16, cudaStream_t stream) {
  if (args.num_tokens == 0) return cudaSuccess;
  RopeAppendArgs a = args;
  const int v = is_bf16 ? 8 : 4;
  a.rope.whole_axes = 1;
  for (int i = 0; i < a.rope.rot_dim / 2; ++i)
    if (a.rope.pair_axis[i] != a.rope.pair_axis[i - i % v]) a.rope.whole_axes = 0;
  if (is_bf16)
    return whole_chunks(a, 2) ? launch_rope_typed<__nv_bfloat16, true>(a, stream)
                              : launch_rope_typed<__nv_bfloat16, false>(a, stream);
  return whole_chunks(a, 4) ? launch_rope_typed<float, true>(a, stream)
                            : launch_rope_typed<float, false>(a, stream);
}

bool append_fp8_block_supported(const RopeAppendArgs& a) {
  return a.head_dim % 16 == 0 && a.head_dim <= 128 && a.rope.rot_dim % 4 == 0 &&
         (!a.q || whole_chunks(a, 2));
}

cudaError_t launch_kv_append_fp8_block(const RopeAppendArgs& args, cudaStream_t stream) {
  if (args.num_tokens == 0) return cudaSuccess;
  if (args.num_tokens > 0x7fffffff) return cudaErrorInvalidValue;
  RopeAppendArgs a = args;
  a.rope.whole_axes = 1;
  for (int i = 0; i < a.rope.rot_dim / 2; ++i)
    if (a.rope.pair_axis[i] != a.rope.pair_axis[i - i % 8]) a.rope.whole_axes = 0;
  const int groups = (2 * a.num_kv_heads + kAppendWarps - 1) / kAppendWarps;
  const dim3 grid((unsigned)a.num_tokens, groups + (a.q ? 1 : 0));
  kv_append_fp8_block_kernel<<<grid, kAppendWarps * 32, 0, stream>>>(a, groups, a.head_dim / 16);
  return cudaGetLastError();
}

}  // namespace pkv
