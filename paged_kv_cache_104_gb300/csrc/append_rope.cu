// Appends that rotate positions on the way into the paged pools, and the
// quantising append of the block-scaled 8-bit cache.
//
// Rotation: a head's first rot_dim elements form rot_dim / 2 pairs, (i, i +
// rot_dim/2) or, interleaved, (2i, 2i + 1); pair i of token t turns by the
// angle whose cosine and sin stand in the table row of positions[axis(i)][t]:
//   a' = a cos - b sin,  b' = b cos + a sin
// in fp32, rounded once to the storage type (to E4M3 from the exact value).  The
// other elements are copied.
// The axis of a pair is the caller's table, so one axis (text), sections of
// time, height and width, or axes taken in turn are one kernel.
// Times in this file are GPU time, taken in CUDA graphs.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kMinScaleExp = -126;   // block scale exponents an append writes:
constexpr int kMaxScaleExp = 119;    // 448 * 2^119 is the largest such value below 2^128

// A token's positions, by axis.  Read together with the token's slot; one
// outside the table reads as 0, so that its row can be requested before the
// token is found bad.
struct Positions {
  int p[kRopeAxes];
  bool ok;
  __device__ __forceinline__ void load(const RopeArgs& r, int64_t t, int64_t num_tokens) {
    ok = true;
#pragma unroll
    for (int ax = 0; ax < kRopeAxes; ++ax) {
      p[ax] = ax < r.num_axes ? __ldg(r.positions + ax * num_tokens + t) : 0;
      const bool in = p[ax] >= 0 && (int64_t)p[ax] < r.num_positions;
      ok &= in;
      if (!in) p[ax] = 0;
    }
  }
  // the table row (rot_dim floats: cosines, then sines) of an axis' position
  __device__ __forceinline__ const float* row(const RopeArgs& r, int axis) const {
    int at = p[0];
#pragma unroll
    for (int ax = 1; ax < kRopeAxes; ++ax) at = axis == ax ? p[ax] : at;
    return r.cos_sin + (int64_t)at * r.rot_dim;
  }
};

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

// V elements from / to memory (16-byte accesses when V > 1).  STREAM: marked as
// used once.
template <typename T, int V>
struct Run {
  uint4 raw;
  template <bool STREAM>
  __device__ __forceinline__ void load(const T* p) {
    // not through the read-only path: queries may be rotated in place
    if constexpr (V > 1 && STREAM) raw = __ldcs(reinterpret_cast<const uint4*>(p));
    else if constexpr (V > 1) raw = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<T*>(&raw) = *p;
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (V > 1 && STREAM) __stcs(reinterpret_cast<uint4*>(p), raw);
    else if constexpr (V > 1) *reinterpret_cast<uint4*>(p) = raw;
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
  __device__ __forceinline__ void load(const RopeArgs& r, int u, const Positions& pos) {
    const int half = r.rot_dim / 2, i0 = u * V;
    if (V > 1 && r.whole_axes) {   // the unit's pairs share an axis: whole 16-byte loads
      const float* row = pos.row(r, r.pair_axis[i0]);
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
        const float* row = pos.row(r, r.pair_axis[i0 + i]);
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
// once for all of them.  HPT heads' rows are requested at once, beside the
// slot, the positions and, from those, the table: nothing is looked at before
// all is on its way (with the checks in between 50 us, so 38 us, for 8,192
// tokens of 32 + 8 heads; now 33.6 us).
template <typename T, bool VEC, int HPT, bool STREAM>
__device__ __forceinline__ void rope_token(const RopeAppendArgs& a, int64_t t, int u, int hs,
                                           int slots, int kv_heads) {
  constexpr int V = Unit2<T, VEC>::V;
  const int heads = a.num_q_heads + 2 * kv_heads;
  const int64_t slot = __ldg(a.slot_mapping + t);
  Positions pos;
  pos.load(a.rope, t, a.num_tokens);
  int e0, e1;
  Unit2<T, VEC>::place(a.rope, u, e0, e1);
  const bool turns = u * V < a.rope.rot_dim / 2;
  // source of head h: queries, then keys, then values
  auto source = [&](int h) {
    if (h < a.num_q_heads) return static_cast<const T*>(a.q) + t * a.q_stride + h * a.head_dim;
    h -= a.num_q_heads;
    return h < kv_heads ? static_cast<const T*>(a.k_new) + t * a.k_stride + h * a.head_dim
                        : static_cast<const T*>(a.v_new) + t * a.v_stride + (h - kv_heads) * a.head_dim;
  };
  Run<T, V> x[HPT], y[HPT];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
      const int h = h0 + i * slots;
      if (h < heads) {
        const T* src = source(h);
        x[i].template load<STREAM>(src + e0);
        y[i].template load<STREAM>(src + e1);
      }
    }
  };
  load(hs);
  Turn<V> w;
  if (turns) w.load(a.rope, u, pos);
  if (slot < 0) return;
  if (slot >= a.num_blocks * kBlockSize) {
    record_error(a.err, DEVERR_SLOT_RANGE);
    return;
  }
  if (!pos.ok) {
    record_error(a.err, DEVERR_POSITION_RANGE);
    return;
  }
  const int64_t blk = slot / kBlockSize, row = slot - blk * kBlockSize;
  for (int h0 = hs; h0 < heads; h0 += HPT * slots) {
    if (h0 != hs) load(h0);
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
      const int h = h0 + i * slots, k = h - a.num_q_heads;
      if (h >= heads) break;
      T* dst;
      if (k < 0) {
        dst = static_cast<T*>(a.q_out) + t * a.q_out_stride + h * a.head_dim;
      } else {
        const bool is_v = k >= kv_heads;
        dst = static_cast<T*>(is_v ? a.v_cache : a.k_cache) +
              ((blk * kv_heads + k - (is_v ? kv_heads : 0)) * kBlockSize + row) * a.head_dim;
      }
      if (turns && k < kv_heads) rotate<T, V>(a.rope, w, x[i], y[i]);
      x[i].template store<STREAM>(dst + e0);
      y[i].template store<STREAM>(dst + e1);
    }
  }
}

template <typename T, bool VEC, int HPT, bool STREAM>
__global__ void __launch_bounds__(256)
kv_append_rope_kernel(const __grid_constant__ RopeAppendArgs a, int units, int slots) {
  const int per_token = units * slots;
  const int tl = threadIdx.x / per_token;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / per_token) + tl;
  const int rem = threadIdx.x - tl * per_token;
  const int hs = rem / units, u = rem - hs * units;
  if (t < a.num_tokens) rope_token<T, VEC, HPT, STREAM>(a, t, u, hs, slots, a.num_kv_heads);
}

// Thread layout of a token's rows: `slots` threads share a unit's heads.
// While all threads fit the GPU at once each takes one head (latency counts);
// beyond that HPT heads a thread keep more bytes in flight.
template <int HPT>
int head_slots(int heads, int units, int most) {
  int slots = (heads + HPT - 1) / HPT;
  while (units * slots > most && slots > 1) slots = (slots + 1) / 2;
  return slots;
}
constexpr int64_t kThreadsAtOnce = 152 * 2048;
// From the L2's size on loads and stores are marked as used once: 8,192 tokens
// of 32 + 8 heads (206 MB) 33.6 us against 36.1, with the four prefills that read
// them 178.4 against 178.5 us; 4,096 tokens with theirs 91.4 against 90.6.
constexpr int64_t kStreamBytes = 128ll << 20;
constexpr int kHeadsPerThread = 6;   // 8,192 tokens of 32 + 8 heads (in CTAs of 256): 1 or 2 43 us, 4 39, 6 38
constexpr int kQueryHeads = 2;        // the same for the queries of the 8-bit append

// ------------------------------------------------- block-scaled 8-bit cache

// 2^e as a float, e in [-126, 127]
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// Smallest exponent e with amax <= 448 * 2^e (448 = 1.75 * 2^8), amax >= 0 as
// the bits of a finite float.
__device__ __forceinline__ int scale_exp(uint32_t amax) {
  const int e = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(kMinScaleExp, min(kMaxScaleExp, e));
}

constexpr int kWindow = 16;       // tokens of a CTA
constexpr int kRowLanes = 16;     // threads of a row, 8 elements (16 bytes) each
constexpr int kAppendThreads = kWindow * kRowLanes;

// x cos + y sin to within 2 ulps of the result, whatever cancels: where the
// sum loses 8 bits or more it is exact, and the product's own error is added.
__device__ __forceinline__ float turned(float x, float y, float c, float s) {
  const float p = y * s;
  return fmaf(x, c, p) - fmaf(-y, s, p);   // subtracted: a zero keeps its sign
}

// A thread's 8 elements of a row (chunk c) turned, or as they are.  Every lane
// of the warp calls it: the other side of a half's pairs comes by shuffle.
struct RowTurn {
  Turn<8> w;        // halves: the chunk's 8 pairs; adjacent pairs: the first 4
  __device__ __forceinline__ void load(const RopeArgs& r, const Positions& pos, int c) {
    const int half = r.rot_dim / 2, hc = half / 8;
    if (c >= r.rot_dim / 8) return;
    if (!r.interleaved) {
      w.load(r, c >= hc ? c - hc : c, pos);
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* row = pos.row(r, r.pair_axis[4 * c + i]);
      w.c[i] = __ldg(row + 4 * c + i);
      w.s[i] = __ldg(row + half + 4 * c + i);
    }
  }
  __device__ __forceinline__ void turn(const RopeArgs& r, uint4 raw, int c, float (&x)[8]) const {
    Elem<__nv_bfloat16>::unpack(raw, x);
    const int hc = r.rot_dim / 16;
    const bool turns = c < r.rot_dim / 8;
    if (r.interleaved) {          // pairs 4 c .. 4 c + 3, all here
      if (!turns) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = turned(a, -b, w.c[i], w.s[i]);
        x[2 * i + 1] = turned(b, a, w.c[i], w.s[i]);
      }
      return;
    }
    const bool second = c >= hc;  // the other side is hc chunks, that is threads, away
    const int from = (threadIdx.x & 16) + ((second ? c - hc : c + hc) & 15);
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, raw.x, from);
    o.y = __shfl_sync(0xffffffffu, raw.y, from);
    o.z = __shfl_sync(0xffffffffu, raw.z, from);
    o.w = __shfl_sync(0xffffffffu, raw.w, from);
    if (!turns) return;
    float y[8];
    Elem<__nv_bfloat16>::unpack(o, y);
#pragma unroll
    for (int i = 0; i < 8; ++i)   // a' = a cos - b sin, or b' = b cos + a sin
      x[i] = turned(x[i], second ? y[i] : -y[i], w.c[i], w.s[i]);
  }
};

// Keys turn in fp32, which can fall on the other side of the middle between
// two codes than the exact value does.  So the elements within kNear ulps of a
// middle (nine in a million) are turned again in fp64, and a key's code is the
// exact value's.  A middle has the 20 lowest of fp32's bits 0x80000, brought to
// the top here; below 2^-6, where codes are 2^-9 apart, so it has with 2^-6
// added.
// (GPU time of a chunk of 2,048 tokens: 13.0 us with the codes and scales of the
// fp32 values, 13.5 with the exact codes, 14.0 with the exact scales too;
// all in fp64, at 2 operations a clock and SM, would take 10 us more.)
constexpr uint32_t kNear = 4;
__device__ __forceinline__ uint32_t off_middle(float y) {
  return __float_as_uint(y) * 4096u - ((0x80000u - kNear) << 12);
}
constexpr uint32_t kAtMiddle = (2 * kNear + 1) << 12;   // off_middle of near ones is less

// Element el of token t's key row turned in fp64: the products are exact, so
// this is the exact rotation rounded once.
__device__ __forceinline__ double exact_turn(const RopeArgs& r, int64_t num_tokens,
                                             const __nv_bfloat16* row, int64_t t, int el) {
  const int half = r.rot_dim / 2;
  const int i = r.interleaved ? el >> 1 : el % half;
  const bool second = r.interleaved ? (el & 1) : el >= half;
  const int other = r.interleaved ? el ^ 1 : (second ? el - half : el + half);
  const float* turn =
      r.cos_sin + (int64_t)r.positions[r.pair_axis[i] * num_tokens + t] * r.rot_dim + i;
  const double x = (double)__bfloat162float(row[el]) * turn[0];
  const double y = (double)__bfloat162float(row[other]) * turn[half];
  return second ? x + y : x - y;
}

// The code of element el of token t's key row, turned in fp64, times inv.
__device__ __noinline__ uint32_t exact_code(const RopeArgs& r, int64_t num_tokens,
                                            const __nv_bfloat16* row, int64_t t, int el, float inv) {
  const double z = exact_turn(r, num_tokens, row, t, el) * inv;
  float f = __double2float_rz(z);
  if ((double)f != z) f = __uint_as_float(__float_as_uint(f) | 1u);   // not a middle
  return f32x2_to_e4m3x2(f, 0.f) & 0xffu;
}

// A scale's border, 448 * 2^e, has the mantissa 0x600000.  A maximum in fp32
// within kNear ulps of one can lie on its other side than the exact maximum.
__device__ __forceinline__ bool near_border(uint32_t amax) {
  return (amax << 9) - ((0x600000u - kNear) << 9) < (2 * kNear + 1) << 9;
}

// The largest finite magnitude among elements el0 .. el0 + 7 of token t's row,
// turned in fp64 (is_turned) or as they are, as the bits of a float that lies on
// the same side of every border (rounded up: a float at a border is met exactly).
// A turned element beyond fp32 counts as its largest number.
__device__ __noinline__ uint32_t exact_max(const RopeArgs& r, int64_t num_tokens,
                                           const __nv_bfloat16* row, int64_t t, int el0,
                                           bool is_turned) {
  uint32_t m = 0;
#pragma unroll 1
  for (int el = el0; el < el0 + 8; ++el) {
    const double z = fabs(is_turned ? exact_turn(r, num_tokens, row, t, el)
                                    : (double)__bfloat162float(row[el]));
    if (!isfinite(z)) continue;   // infinite or NaN: the scale follows the others
    m = max(m, min(__float_as_uint(__double2float_ru(z)), 0x7f7fffffu));
  }
  return m;
}

// Of a window: run_of[j], the run that token j belongs to (-1: none that starts
// here), and of the run that starts at token k its slot, old scale bytes and
// maxima by head.
template <int UPC>
struct WindowRuns {
  int8_t run_of[2 * kWindow];
  int first;        // the first such k (0: none)
  int64_t slot[kWindow];
  int old[UPC][kWindow];
  uint32_t top[UPC][kWindow];
  // whether the rows before run k (of head u) stand for something
  __device__ __forceinline__ bool held(int u, int k) const {
    return old[u][k] >= 1 && old[u][k] <= 253;
  }
  // the run's scale exponent
  __device__ __forceinline__ int exponent(int u, int k, int row0) const {
    const int e = scale_exp(top[u][k]);
    return row0 > 0 && held(u, k) ? max(e, old[u][k] - 127) : e;
  }
};

// Warp 0's part: lane l looks at entry w0 + l (slot) and w0 - 1 - l (back).
template <int UPC>
__device__ __forceinline__ void find_runs(const RopeAppendArgs& a, WindowRuns<UPC>& runs,
                                          int64_t slot, int64_t back, bool position_ok,
                                          const int (&old)[UPC]) {
  const int lane = threadIdx.x;
  const bool inside = slot >= 0 && slot < a.num_blocks * kBlockSize;
  const int64_t blk = inside ? slot / kBlockSize : -1;
  const int row = (int)(slot - blk * kBlockSize);
  const int64_t up = __shfl_up_sync(0xffffffffu, slot, 1);
  const int64_t prev = lane == 0 ? back : up;
  const int64_t back_blk = back >= 0 ? back / kBlockSize : -1;
  // an entry goes on with the run of the one before, or starts a run
  const bool goes_on = inside && row > 0 && prev == slot - 1;
  const bool here = lane < kWindow;
  const uint32_t starts = __ballot_sync(0xffffffffu, inside && !goes_on);
  const uint32_t broken = __ballot_sync(0xffffffffu, !inside || !position_ok);
  if (here && slot >= 0 && !inside) record_error(a.err, DEVERR_SLOT_RANGE);
  if (here && inside && !position_ok) record_error(a.err, DEVERR_POSITION_RANGE);
  // no nearby earlier entry may write a run's block: two runs would race on it
  uint32_t twice = 0;
  for (uint32_t left = starts & 0xffffu; left; left &= left - 1) {
    const int k = __ffs(left) - 1;
    const int64_t b = __shfl_sync(0xffffffffu, blk, k);
    if (__any_sync(0xffffffffu, (lane < k && blk == b) || (lane < 32 - k && back_blk == b)))
      twice |= 1u << k;
  }
  if (lane == 0 && twice) record_error(a.err, DEVERR_SLOT_ORDER);
  // the last start up to here; an entry with a bad position, and an invalid
  // one, ends the run before it, and what follows belongs to none
  const uint32_t upto = 0xffffffffu >> (31 - lane);
  const uint32_t before = starts & upto;
  const int k = before ? 31 - __clz(before) : -1;
  const bool member = k >= 0 && k < kWindow && inside && !(twice >> k & 1u) &&
                      (broken & upto & (0xffffffffu << k)) == 0;
  runs.run_of[lane] = (int8_t)(member ? k : -1);
  if (lane == 0) runs.first = starts & 0xffffu ? __ffs(starts & 0xffffu) - 1 : 0;
  if (here) {
    runs.slot[lane] = slot;
#pragma unroll
    for (int u = 0; u < UPC; ++u) {
      runs.top[u][lane] = 0;
      runs.old[u][lane] = old[u];
    }
  }
}

// The codes of token j (elements v of chunk c, pool and head `tile`) of run k,
// and the run's scale.  Returns the elements, one bit each, whose code
// exact_code has to say (is_turned: v was turned).
template <int UPC>
__device__ __forceinline__ uint32_t write_codes(const RopeAppendArgs& a,
                                                const WindowRuns<UPC>& runs, uint8_t* pools,
                                                uint8_t* scales, const float (&v)[8],
                                                int u, int g, int j, int k, int c, bool is_turned) {
  const int64_t slot = runs.slot[k], blk = slot / kBlockSize;
  const int row0 = (int)(slot - blk * kBlockSize), row = row0 + j - k;
  const int64_t tile = blk * a.num_kv_heads + g;
  uint8_t* pool = pools + tile * kBlockSize * a.head_dim + c * 8;
  const int e = runs.exponent(u, k, row0);
  if (row0 > 0 && j == k) {
    // where the scale grows, the block's older rows are re-expressed, by the
    // threads of the run's first token
    const bool held = runs.held(u, k);
    const int e_old = held ? runs.old[u][k] - 127 : e;
    if (!held || e > e_old) {
      const float f = held ? exp2i(max(e_old - e, -126)) : 0.f;
#pragma unroll 1
      for (int o = 0; o < row0; ++o) {
        uint2* p = reinterpret_cast<uint2*>(pool + o * a.head_dim);
        const uint2 w = *p;
        auto again = [&](uint32_t codes) {
          const uint32_t lo = e4m3x2_to_f16x2((uint16_t)codes);
          const uint32_t hi = e4m3x2_to_f16x2((uint16_t)(codes >> 16));
          const float2 fl = __half22float2(*reinterpret_cast<const __half2*>(&lo));
          const float2 fh = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          return f32x2_to_e4m3x2(fl.x * f, fl.y * f) |
                 ((uint32_t)f32x2_to_e4m3x2(fh.x * f, fh.y * f) << 16);
        };
        *p = held ? make_uint2(again(w.x), again(w.y)) : make_uint2(0u, 0u);
      }
    }
  }
  const float inv = exp2i(-e);
  uint32_t n[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) n[q] = f32x2_to_e4m3x2(v[2 * q] * inv, v[2 * q + 1] * inv);
  const uint2 codes = make_uint2(n[0] | n[1] << 16, n[2] | n[3] << 16);
  *reinterpret_cast<uint2*>(pool + row * a.head_dim) = codes;
  if (j == k && c == 0) scales[tile] = (uint8_t)(e + 127);
  if (!is_turned) return 0;
  constexpr float kSmall = 0.015625f;          // 2^-6
  uint32_t nearest = ~0u, least = ~0u;         // (a zero counts as large: it is exact)
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    nearest = min(nearest, off_middle(v[q] * inv));
    least = min(least, __float_as_uint(v[q] * inv) * 2u - 1u);
  }
  // (an infinite element, which turned() made a NaN, is one of them too)
  const uint32_t nan = (((codes.x & 0x7f7f7f7fu) + 0x01010101u) |
                        ((codes.y & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u;
  if (nearest >= kAtMiddle && least >= __float_as_uint(kSmall) * 2u && nan == 0) return 0;
  uint32_t again = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float y = fabsf(v[q] * inv);
    const bool near = off_middle(y < kSmall ? y + kSmall : y) < kAtMiddle;
    again |= (near || y != y ? 1u : 0u) << q;
  }
  return again;
}

// A run's maximum that is not the scale's yet: an element is infinite or NaN, or
// fp32 may have put the maximum on the other side of a border.
__device__ __forceinline__ bool unsettled(uint32_t top, bool rotated) {
  return top >= 0x7f800000u || (rotated && near_border(top));
}

// Such maxima taken again in fp64 (one run in a million), in the first `heads`
// heads: the caller's elements el0 .. el0 + 7 of tokens w0 + j, of run `of`, and
// w0 + j2, of run of2.  (Out of line: as a part of the kernel it took a chunk of
// 2,048 tokens from 14.0 to 14.3 us.)
template <int UPC>
__device__ __noinline__ void settle(const RopeAppendArgs& a, WindowRuns<UPC>& runs,
                                    const __nv_bfloat16* src, int64_t stride, int64_t w0, int heads,
                                    bool rotated, bool turned_here, int el0, int j, int of, int j2,
                                    int of2) {
  uint32_t todo = 0;
  for (int u = 0; u < UPC; ++u) {
    if (of >= 0 && unsettled(runs.top[u][of], rotated)) todo |= 1u << u;
    if (of2 >= 0 && unsettled(runs.top[u][of2], rotated)) todo |= 0x100u << u;
  }
  __syncthreads();
  if (threadIdx.x < kWindow) {
    for (int u = 0; u < UPC; ++u)
      if (unsettled(runs.top[u][threadIdx.x], rotated)) runs.top[u][threadIdx.x] = 0;
  }
  __syncthreads();
  todo &= ((1u << heads) - 1) * 0x101u;
#pragma unroll 1
  for (; todo; todo &= todo - 1) {
    const int bit = __ffs(todo) - 1, u = bit & 7;
    const int64_t t = w0 + (bit < 8 ? j : j2);
    atomicMax(&runs.top[u][bit < 8 ? of : of2],
              exact_max(a.rope, a.num_tokens, src + t * stride + u * a.head_dim, t, el0, turned_here));
  }
  __syncthreads();
}

// The first kv_ctas CTAs take the runs of new tokens that start in a window of
// 16 tokens, in up to UPC heads of one pool.  Thread (i, c) has chunk c of token
// i, and of token i + 16 where a run goes on beyond the window; the runs'
// maxima meet in shared memory, so all runs of a window, one of a prompt or 16
// of a decode step, are done at once.  Rows, positions and slots are requested
// together, then the table's rows and the old scales, before anything is
// decided.  With UPC > 1, where throughput counts, the rows wait for the slots
// instead and start at the window's first run, so that a prompt's runs, which
// lie anywhere to the windows, end within the threads' 16 tokens.  The other
// CTAs rotate queries.
// (A warp for each run and head, its rows in registers, took 20 to 36 us for a
// chunk of 2,048 tokens of 32 + 8 heads: 32 KiB of straight code that every
// warp ran once, waiting for it.)
template <int UPC>
__global__ void __launch_bounds__(kAppendThreads, 4)
kv_append_fp8_block_kernel(const __grid_constant__ RopeAppendArgs a, int kv_ctas, int q_units,
                           int q_slots) {
  if ((int)blockIdx.x >= kv_ctas) {
    const int per_token = q_units * q_slots;
    const int tl = threadIdx.x / per_token, tokens = blockDim.x / per_token;
    const int64_t t = (int64_t)((int)blockIdx.x - kv_ctas) * tokens + tl;
    const int rem = threadIdx.x - tl * per_token;
    const int hs = rem / q_units, u = rem - hs * q_units;
    if (tl < tokens && t < a.num_tokens)
      rope_token<__nv_bfloat16, true, kQueryHeads, false>(a, t, u, hs, q_slots, 0);
    return;
  }
  __shared__ WindowRuns<UPC> runs;
  const int i = threadIdx.x / kRowLanes, c = threadIdx.x % kRowLanes;
  const int groups = (a.num_kv_heads + UPC - 1) / UPC;    // of a pool
  const int group = (int)blockIdx.x % (2 * groups);
  const bool is_v = group >= groups;
  const int g0 = (is_v ? group - groups : group) * UPC, ng = min(UPC, a.num_kv_heads - g0);
  const int64_t w0 = (int64_t)((int)blockIdx.x / (2 * groups)) * kWindow;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const __nv_bfloat16* src =
      static_cast<const __nv_bfloat16*>(is_v ? a.v_new : a.k_new) + g0 * a.head_dim + c * 8;
  uint8_t* pools = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache);
  uint8_t* scales = is_v ? a.v_scale : a.k_scale;
  const bool mine = c * 8 < a.head_dim;
  const bool rotated = !is_v && a.rope.rot_dim > 0;
  int64_t slot = -1, back = -1;
  if (threadIdx.x < 32) {
    if (w0 + threadIdx.x < a.num_tokens) slot = __ldg(a.slot_mapping + w0 + threadIdx.x);
    if (w0 - 1 - (int)threadIdx.x >= 0) back = __ldg(a.slot_mapping + w0 - 1 - threadIdx.x);
  }
  uint4 raw[UPC];
  Positions pos;
  auto load_rows = [&](int64_t t) {
    const bool in = t < a.num_tokens;
#pragma unroll
    for (int u = 0; u < UPC; ++u)
      raw[u] = in && mine && u < ng
                   ? __ldg(reinterpret_cast<const uint4*>(src + t * stride + u * a.head_dim))
                   : make_uint4(0u, 0u, 0u, 0u);
    pos = Positions{};
    if (in && rotated) pos.load(a.rope, t, a.num_tokens);
  };
  RowTurn turn;
  int k0 = 0;                    // the threads' first token in the window
  if (UPC == 1) {
    load_rows(w0 + i);
    if (rotated) turn.load(a.rope, pos, c);
  }
  if (threadIdx.x < 32) {
    bool position_ok = true;
    if (a.rope.rot_dim > 0 && w0 + threadIdx.x < a.num_tokens) {
      Positions p;
      p.load(a.rope, w0 + threadIdx.x, a.num_tokens);
      position_ok = p.ok;
    }
    int old[UPC];
    const bool older = threadIdx.x < kWindow && slot >= 0 && slot < a.num_blocks * kBlockSize &&
                       slot % kBlockSize != 0;
#pragma unroll
    for (int u = 0; u < UPC; ++u)
      old[u] = older && u < ng ? scales[slot / kBlockSize * a.num_kv_heads + g0 + u] : 0;
    find_runs<UPC>(a, runs, slot, back, position_ok, old);
  }
  if (UPC > 1) {
    __syncthreads();
    k0 = runs.first;
    load_rows(w0 + k0 + i);
    if (rotated) turn.load(a.rope, pos, c);
  }
  // every lane takes part in the exchanges; what has no run is left out
  float x[UPC][8];
  auto turn_rows = [&] {
#pragma unroll
    for (int u = 0; u < UPC; ++u) {
      if (rotated) turn.turn(a.rope, raw[u], c, x[u]);
      else Elem<__nv_bfloat16>::unpack(raw[u], x[u]);
    }
  };
  const bool turned_here = rotated && c * 8 < a.rope.rot_dim;
  auto maxima = [&](int of) {
#pragma unroll
    for (int u = 0; u < UPC; ++u) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(x[u][k]) & 0x7fffffffu);
#pragma unroll
      for (int o = 1; o < kRowLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (c == 0 && of >= 0) atomicMax(&runs.top[u][of], m);
    }
  };
  auto write = [&](int j, int k) {
    if (k < 0 || !mine) return;
    uint32_t again = 0;
#pragma unroll
    for (int u = 0; u < UPC; ++u)
      if (u < ng)
        again |= write_codes<UPC>(a, runs, pools, scales, x[u], u, g0 + u, j, k, c, turned_here)
                 << 8 * u;
    for (; again; again &= again - 1) {
      const int u = (__ffs(again) - 1) >> 3, el = c * 8 + ((__ffs(again) - 1) & 7);
      const int64_t at = runs.slot[k], tile = at / kBlockSize * a.num_kv_heads + g0 + u;
      const int row0 = (int)(at % kBlockSize);
      pools[(tile * kBlockSize + row0 + j - k) * a.head_dim + el] = (uint8_t)exact_code(
          a.rope, a.num_tokens, src - c * 8 + (w0 + j) * stride + u * a.head_dim, w0 + j, el,
          exp2i(-runs.exponent(u, k, row0)));
    }
  };
  turn_rows();
  if (UPC == 1) __syncthreads();
  const int j = k0 + i, j2 = j + kWindow;
  const int run = j < 2 * kWindow ? runs.run_of[j] : -1;
  const int run2 = j2 < 2 * kWindow ? runs.run_of[j2] : -1;
  auto rows_of = [&](int of) {
    load_rows(w0 + of);
    if (rotated) turn.load(a.rope, pos, c);
    turn_rows();
  };
  maxima(run);
  // a run that goes on beyond the threads' tokens: its other rows, for the
  // maxima now and again for their codes
  const bool beyond = __syncthreads_or(run2 >= 0);
  if (beyond) {
    rows_of(j2);
    maxima(run2);
    __syncthreads();
  }
  bool some = false;
#pragma unroll
  for (int u = 0; u < UPC; ++u) some |= unsettled(runs.top[u][threadIdx.x % kWindow], rotated);
  if (__any_sync(0xffffffffu, some)) {     // the same in every warp
    settle<UPC>(a, runs, src - c * 8, stride, w0, mine ? ng : 0, rotated, turned_here, c * 8, j, run,
                j2, run2);
    rows_of(beyond ? j2 : j);              // read again, so that no registers wait for this
  }
  if (beyond) {
    write(j2, run2);
    rows_of(j);
  }
  write(j, run);
}

template <typename T, bool VEC, int HPT, bool STREAM>
cudaError_t launch_rope_heads(const RopeAppendArgs& a, cudaStream_t stream) {
  const int units = a.head_dim / (2 * Unit2<T, VEC>::V);
  const int slots = head_slots<HPT>(a.num_q_heads + 2 * a.num_kv_heads, units, 256);
  const int per_token = units * slots;
  // small CTAs give their registers back as soon as their rows are out: 8,192
  // tokens of 32 + 8 heads 37.8 us with 256 threads, 36.3 with 128, 35.6 with 64
  const int threads = HPT > 1 ? 64 : 256;
  const int tokens = per_token >= threads ? 1 : threads / per_token;
  const int64_t grid = (a.num_tokens + tokens - 1) / tokens;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  kv_append_rope_kernel<T, VEC, HPT, STREAM>
      <<<(int)grid, per_token * tokens, 0, stream>>>(a, units, slots);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t launch_rope_typed(const RopeAppendArgs& a, cudaStream_t stream) {
  const int64_t threads = a.num_tokens * (a.num_q_heads + 2 * a.num_kv_heads) *
                          (a.head_dim / (2 * Unit2<T, VEC>::V));
  if (threads <= kThreadsAtOnce) return launch_rope_heads<T, VEC, 1, false>(a, stream);
  const int64_t bytes = 2 * threads * 2 * Unit2<T, VEC>::V * (int)sizeof(T);   // read and written
  return bytes <= kStreamBytes ? launch_rope_heads<T, VEC, kHeadsPerThread, false>(a, stream)
                               : launch_rope_heads<T, VEC, kHeadsPerThread, true>(a, stream);
}

// 1 if every v pairs from a multiple of v on share an axis.
int axes_by_chunk(const RopeAppendArgs& a, int v) {
  for (int i = 0; i < a.rope.rot_dim / 2; ++i)
    if (a.rope.pair_axis[i] != a.rope.pair_axis[i - i % v]) return 0;
  return 1;
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
  a.rope.whole_axes = axes_by_chunk(a, v);
  if (is_bf16)
    return whole_chunks(a, 2) ? launch_rope_typed<__nv_bfloat16, true>(a, stream)
                              : launch_rope_typed<__nv_bfloat16, false>(a, stream);
  return whole_chunks(a, 4) ? launch_rope_typed<float, true>(a, stream)
                            : launch_rope_typed<float, false>(a, stream);
}

bool append_fp8_block_supported(const RopeAppendArgs& a) {
  return a.head_dim % 16 == 0 && a.head_dim <= 128 && a.rope.rot_dim % 16 == 0;
}

cudaError_t launch_kv_append_fp8_block(const RopeAppendArgs& args, cudaStream_t stream) {
  if (args.num_tokens == 0) return cudaSuccess;
  if (args.num_tokens > 0x7fffffff) return cudaErrorInvalidValue;
  RopeAppendArgs a = args;
  a.rope.whole_axes = axes_by_chunk(a, 8);
  const int64_t windows = (a.num_tokens + kWindow - 1) / kWindow;
  // few windows: a head to a CTA, for latency; many: 4 heads share slots,
  // positions and table (a chunk of 2,048 tokens: 13.0 us before the exact
  // codes, and with 2 heads to a CTA 16.5 us)
  const bool few = windows * 2 * a.num_kv_heads <= 152 * 4;
  const int64_t kv_ctas = windows * 2 * (few ? a.num_kv_heads : (a.num_kv_heads + 3) / 4);
  const int units = a.head_dim / 16;
  const int slots = head_slots<kQueryHeads>(std::max(a.num_q_heads, 1), units, kAppendThreads);
  const int tokens = kAppendThreads / (units * slots);
  const int64_t q_ctas = a.q ? (a.num_tokens + tokens - 1) / tokens : 0;
  if (kv_ctas + q_ctas > 0x7fffffff) return cudaErrorInvalidValue;
  auto* kernel = few ? kv_append_fp8_block_kernel<1> : kv_append_fp8_block_kernel<4>;
  kernel<<<(unsigned)(kv_ctas + q_ctas), kAppendThreads, 0, stream>>>(a, (int)kv_ctas, units, slots);
  return cudaGetLastError();
}

}  // namespace pkv
