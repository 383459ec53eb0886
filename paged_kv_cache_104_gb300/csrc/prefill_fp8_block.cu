// Chunked-prefill attention over the block-scaled fp8 cache, on tcgen05
// (sm_103a).
//
// What it computes: chunk row i of one sequence, at absolute position prior +
// i, attends keys 0 .. prior + i, K and V read as decode(code) * 2^e with an
// exponent per block of 16 tokens and KV head.  As in the bf16 prefill a CTA
// carries two streams of 128 query rows that share every K/V tile of 128 keys
// (two query heads of one KV head over the same rows, or one head over two
// query tiles when the GQA group is odd); S_h and O_h (128 columns each) of the
// two streams fill TMEM, P_h lies in the columns of its S_h, and the streams
// take turns on the tensor core.
//
// How the 8-bit cache is fed to it.
//  * Q K^T needs no conversion: K's codes are operands of kind::f8f6f4 as they
//    lie, gathered by TMA (one 16-row x 128-byte box per block).  A query row,
//    scaled by a power of two to a largest element in [128, 256), is split
//    into two E4M3 numbers, hi = E4M3(q) and lo = E4M3(q - hi): a bf16 has 8
//    significant bits and the pair holds 4 + 4, exactly so within 2^-9 of the
//    row's maximum and to 2^-10 absolute below.  S = hi K^T + lo K^T runs at
//    the time of one 16-bit product.
//  * P V: P is f16, V's codes are widened to f16 (exact) by four converter
//    warps, from staging tiles that 1-D bulk copies fill (a block and head is
//    2 KiB in one piece) into the 128B-swizzled tiles the MMAs read.  P's 11 bits
//    are three more than the result has: a weight is off by 2^-11 at most, below
//    2^-14 of the row's largest by 2^-25 of that; l sums the weights in fp32.
//  * The scales act in the softmax, where they are uniform over 16 columns:
//    key j of a block with scales 2^ek, 2^ev has the score t_j 2^ek and the
//    output weight p_j = 2^(s_j + ev - M), M the running maximum of s_j + ev
//    (raised lazily); O += p_j code_j, and the softmax sum is l += p_j 2^(E -
//    ev), E the first tile's largest ev; the result is O 2^E / l.  One
//    exponential serves both sums, at one FMA per block more than without
//    scales.  A block whose ev is more than 40 off E could lose its weight in
//    l to the fp32 range of p (an all-zero V block has the smallest ev there
//    is): from the first tile with such a block on, l is summed from
//    exponentials of its own.
//  * A NaN value code would reach rows that do not see its key (0 * NaN).  In
//    the tiles with masked entries it is zeroed, its key noted, and the rows
//    that see the key come out as NaN.
// Roles (512 threads):
//   warps 0-3 / 4-7   softmax of stream A / B: thread r owns query row r
//   warp 8            TMEM allocator and MMA issuer of both streams
//   warp 9 / 10       producers: K's boxes and the scales / V's copies
//   warps 11, 13-15   V converters
//   warp 12           none: it shares a scheduler with the issuer, whose two
//                     softmax warps lagged the others by 400 cycles a tile
//                     with a converter there (141.5 us against 139.6 us)
// The issuer's own instructions count: with descriptors formed and a warp vote
// taken at every wait it needed 1,500 cycles for a stream's 1,024 cycles of
// products (161 us).  Two issuers, one a stream, let the streams fall into
// step, both in their softmax or both at the tensor core (192 us).
// Both pools' tiles are three stages deep in their fp8 form (K's ring is read
// by the MMAs, V's by the converters), so 96 KiB are in flight or in use.
// Measured on the way (2,048 tokens over 4,096, 32/8 heads): both pools
// converted to bf16 by cp.async producers 280 us, to f16 185 us (with the
// loads left out 141 us: bound by their latency at 32 KiB in flight).
//
// Splitting the keys.  Where the work items fill the SMs badly, a cluster of 2
// to 8 CTAs shares an item's key tiles.  At the end every CTA reads the
// others' sums through distributed shared memory, scales its O to the common
// one, and sends each CTA its share of the columns, which adds them up and
// writes them.
// Every mbarrier wait is bounded; on time-out the kernel records an error,
// stops issuing work, lets its copies land, frees its TMEM and returns.
#include <cuda.h>

#include <algorithm>
#include <climits>
#include <map>
#include <mutex>

#include "common.cuh"
#include "host_cache.h"
#include "launch.h"
#include "tc_common.cuh"
#include "tmap.h"

namespace pkv {
namespace {

constexpr int BM = 128, BN = 128, HD = 128;
constexpr int kTile8 = BN * HD;              // an fp8 tile, 16 KiB
constexpr int kTile16 = 2 * kTile8;          // an f16 tile, two 64-column halves
constexpr int kHalf16 = kTile8;
constexpr int kBlk8 = kBlockSize * HD;       // one block and head, 2 KiB
constexpr int kBlkPerTile = BN / kBlockSize;
constexpr int NSK = 3, NSV = 2, NST = 3;     // K ring, V (f16) ring, V staging ring
constexpr int OFF_Q = 0;                     // [stream][hi, lo]; the bf16 rows land in the V ring
constexpr int OFF_K = 2 * kTile16;
constexpr int OFF_V = OFF_K + NSK * kTile8;
constexpr int OFF_ST = OFF_V + NSV * kTile16;
constexpr int OFF_SCALES = OFF_ST + NST * kTile8;
// the scales of a tile's 8 blocks, as the softmax uses them
struct TileScales {
  float k[kBlkPerTile];    // scale * log2e * 2^ek
  float v[kBlkPerTile];    // ev
  float l[kBlkPerTile];    // 2^(E - ev)
  int wide;                // a block's ev is far from E
  int e;                   // E
  int pad[6];
};
// Deeper than the K ring: a K stage is free again when its products are done,
// but the softmax reads l after it has handed over P, so tile j's scales are
// done with when both streams have handed over P of tile j + 1, which S of tile
// j + 2, and so K's stage of that tile becoming free, follows.
constexpr int kScaleSlots = NSK + 2;
constexpr int kWideSpread = 40;
constexpr int OFF_BAR = OFF_SCALES + kScaleSlots * (int)sizeof(TileScales);
// split keys: [stream][row] (reference of l, l)
constexpr int OFF_ROWS = OFF_BAR + 256;
constexpr int SMEM_BYTES = OFF_ROWS + 2 * BM * 8;
constexpr int kSoftThreads = 256;
constexpr int kThreads = 512;
constexpr int W_MMA = 8, W_KPROD = 9, W_VPROD = 10, W_NONE = 12;
// registers per thread after the split (setmaxnreg), against the launch budget
constexpr int kRegsSoft = 200, kRegsRest = 56;
constexpr int kRegsLaunch = (65536 / kThreads) & ~7;   // 128
static_assert(kRegsSoft * kSoftThreads + kRegsRest * (kThreads - kSoftThreads) <=
                  kRegsLaunch * kThreads,
              "the register split must fit in what the CTA was launched with");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t COL_S = 0, COL_O = 2 * BN;
constexpr float kLazy = 8.0f;

static_assert(NSV * kTile16 == 2 * BM * HD * 2, "the bf16 queries fit the V ring");
static_assert(SMEM_BYTES <= 227 * 1024, "one CTA per SM");
// the merge's fp32 columns: 7 CTAs of 32 are the most
static_assert(7 * 2 * BM * 32 * 4 <= OFF_SCALES, "the merge lies in the tiles' place");

enum {
  B_Q = 0,
  B_QC,                   // the queries are split
  B_KF,                   // [NSK]
  B_KE = B_KF + NSK,
  B_STF = B_KE + NSK,     // [NST]
  B_STE = B_STF + NST,
  B_VF = B_STE + NST,     // [NSV]
  B_VE = B_VF + NSV,
  B_SF = B_VE + NSV,      // [stream]
  B_PF = B_SF + 2,        // [stream][half]
  B_OD = B_PF + 4,        // [stream]
  B_COUNT = B_OD + 2
};
static_assert(B_COUNT * 8 + 12 <= 256, "barrier area");

// Position in a ring of N stages: the slot, and the parity of its current use
// (a division by 3 in every tile costs the issuer more than the products do)
template <int N>
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1;
    }
  }
};

struct Params {
  PrefillArgs a;
  int total_len;
  int q_tiles;
  int rows_mode;          // 1: a CTA's streams are two query tiles of one head
  int splits;             // CTAs (a cluster) that share an item's key tiles
};

// the value 2^(b - 127) of a scale byte, 0 included
__device__ __forceinline__ float scale_value(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

// w with its NaN codes replaced by +0; *found is set when there are any
__device__ __forceinline__ uint32_t drop_nan(uint32_t w, bool* found) {
  const uint32_t top = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // 0x7f carries
  if (top == 0) return w;
  *found = true;
  return w & ~((top >> 7) * 0xffu);
}

// A wait for the roles that run ahead (producer, converters): it sleeps
// between polls and leaves the issue slots to the softmax.  Bounded and
// abort-aware as the others.
__device__ __forceinline__ bool wait_idle(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (unsigned int it = 0; it < kWaitLimitIters; ++it) {
    if (*abort_flag) return false;
    __nanosleep(100);
    if (mbar_try_wait(bar, parity)) return true;
    if (clock64() - t0 > kWaitLimitCycles) break;
  }
  record_error(err, DEVERR_TIMEOUT);
  *abort_flag = 1;
  return false;
}

// 16 columns of 32 bits of this thread's lane
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void tma_box8(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                         int row) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(row)
      : "memory");
}
// S = (hi + lo) K^T in eight products of 32 dims, then the commit to `bar`: one
// elected lane, one block (an election and descriptors formed for every
// product made the issuer the bound).  A step adds 32 bytes to the operands'
// addresses (2 in a descriptor's 16-byte units, which cannot carry out of the
// address field), lo lies 16 KiB behind hi.
__device__ __forceinline__ void issue_qk8(uint32_t d_tmem, uint64_t q_desc, uint64_t k_desc,
                                          uint32_t idesc, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e, t, f;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 f, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 1024;\n\tadd.s64 b, %2, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 1026;\n\tadd.s64 b, %2, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 1028;\n\tadd.s64 b, %2, 4;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 1030;\n\tadd.s64 b, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}" ::"r"(
          d_tmem),
      "l"(q_desc), "l"(k_desc), "r"(idesc), "r"(bar)
      : "memory");
}
// O (+)= P V over 64 keys in four products of 16: P from TMEM, 8 columns a
// step, V's rows 2 KiB a step.
__device__ __forceinline__ void issue_pv4(uint32_t d_tmem, uint32_t p_tmem, uint64_t v_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, t, f;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 f, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n\t"
      "add.u32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.u32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.u32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t}" ::"r"(d_tmem),
      "r"(p_tmem), "l"(v_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// f16 pair to E4M3 codes, to nearest even, saturating
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t u) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(u));
  return d;
}
// instruction descriptor, fp32 accumulate, both operands format 0: E4M3 in
// kind::f8f6f4, f16 in kind::f16
__host__ __device__ constexpr uint32_t idesc0(bool b_mn_major, int m, int n) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// address of addr in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer(uint32_t addr, int rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(addr), "r"(rank));
  return d;
}
__device__ __forceinline__ float2 ld_peer2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];"
               : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_peer4(uint32_t addr, float x, float y, float z, float w) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(x), "f"(y), "f"(z),
               "f"(w)
               : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
prefill_fp8_block_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_COUNT);
  int* abort_i = reinterpret_cast<int*>(tmem_slot + 1);
  volatile int* abort_flag = abort_i;
  int* nan_key = abort_i + 1;   // the first key whose value row holds a NaN
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const PrefillArgs& a = p.a;
  // swizzled operand tiles need a 1 KiB-aligned base (the same in every CTA)
  if (sbase & 1023u) {
    if (threadIdx.x == 0) record_error(a.err, DEVERR_SMEM_LAYOUT);
    return;
  }

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the item: stream hh covers head[hh], query rows qrow[hh] .. + 127; both
  // read KV head g; this CTA takes key tiles t0 .. t1 - 1
  const int tq = (int)gridDim.y - 1 - (int)blockIdx.y;   // heaviest query tiles first
  const int rank = (int)blockIdx.z;                       // in the cluster
  const int head0 = p.rows_mode ? (int)blockIdx.x : 2 * (int)blockIdx.x;
  const int head1 = p.rows_mode ? head0 : head0 + 1;
  const int qrow0 = p.rows_mode ? 2 * tq * BM : tq * BM;
  const int qrow1 = p.rows_mode ? qrow0 + BM : qrow0;
  const int g = head0 / (a.num_q_heads / a.num_kv_heads);
  const int all_tiles = (a.prior_len + min(a.chunk_len, qrow1 + BM) - 1) / BN + 1;
  const int t0 = (int)((int64_t)all_tiles * rank / p.splits);
  const int n_tiles = (int)((int64_t)all_tiles * (rank + 1) / p.splits) - t0;

  if (warp == W_KPROD && lane == 0) {
    mbar_init(bar(B_Q), 1);
    mbar_init(bar(B_QC), kSoftThreads);
    for (int s = 0; s < NSK; ++s) {
      mbar_init(bar(B_KF + s), 1);
      mbar_init(bar(B_KE + s), 4);               // one arrival per stream-B softmax warp
    }
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar(B_STF + s), 1);
      mbar_init(bar(B_STE + s), 4);              // one arrival per converter warp
    }
    for (int s = 0; s < NSV; ++s) {
      mbar_init(bar(B_VF + s), 4);
      mbar_init(bar(B_VE + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_SF + i), 1);
      mbar_init(bar(B_PF + 2 * i), 4);           // one arrival per softmax warp
      mbar_init(bar(B_PF + 2 * i + 1), 4);
      mbar_init(bar(B_OD + i), 1);
    }
    *abort_i = 0;
    *nan_key = INT_MAX;
    fence_mbar_init();
    // the queries at once: what comes first needs nothing else
    if (n_tiles > 0) {
      mbar_arrive_expect_tx(bar(B_Q), 2 * kTile16);
      for (int hh = 0; hh < 2; ++hh) {
        const uint32_t dst = sbase + OFF_V + hh * kTile16;
        tma_load_3d(dst, &tm_q, bar(B_Q), 0, hh ? head1 : head0, hh ? qrow1 : qrow0);
        tma_load_3d(dst + kHalf16, &tm_q, bar(B_Q), 64, hh ? head1 : head0, hh ? qrow1 : qrow0);
      }
    }
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
  }
  if (warp == W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= kSoftThreads / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == W_KPROD || warp == W_VPROD) {
      // ------------------------------------------------------------- producers
      const bool is_v = warp == W_VPROD;
      const uint8_t* vpool = static_cast<const uint8_t*>(a.v_cache);
      const int nblk_seq = (p.total_len + kBlockSize - 1) / kBlockSize;
      // a window of 32 blocks (4 tiles), one per lane: ids, and with K the
      // scale bytes, K's in bits 0-7 and V's in 8-15 (-1 behind the end)
      auto load_ids = [&](int win) {
        const int idx = win * 32 + lane;
        int blk = 0;
        if (idx < nblk_seq) {
          blk = __ldg(a.block_table_row + idx);
          if (blk < 0 || (int64_t)blk >= a.num_blocks) {
            record_error(a.err, DEVERR_BLOCK_RANGE);
            blk = 0;
          }
        }
        return blk;
      };
      auto load_scales = [&](int win, int blk) {
        if (is_v || win * 32 + lane >= nblk_seq) return -1;
        const int64_t i = (int64_t)blk * a.num_kv_heads + g;
        return (int)__ldg(a.k_bscale + i) | (int)__ldg(a.v_bscale + i) << 8;
      };
      int ids = n_tiles > 0 ? load_ids(t0 / 4) : 0;
      int sc = load_scales(t0 / 4, ids);
      int ids_next = 0, sc_next = -1;            // requested behind the first tile
      int e_ref = 0, sent = 0;
      bool go = true;
      static_assert(NSK == NST, "both producers' rings turn alike");
      Ring<NSK> ring;
      Ring<kScaleSlots> sr;
      const int full0 = is_v ? B_STF : B_KF, empty0 = is_v ? B_STE : B_KE;
      for (int jj = 0; jj < n_tiles; ++jj, ring.next(), sr.next()) {
        const int j = t0 + jj;
        const bool turn = jj > 0 && j % 4 == 0;
        if (turn) {
          ids = ids_next;
          sc = sc_next;
        }
        const int blk = __shfl_sync(0xffffffffu, ids, (j % 4) * kBlkPerTile + (lane & 7));
        const int nb = min(kBlkPerTile, nblk_seq - j * kBlkPerTile);
        const int64_t tile = (int64_t)blk * a.num_kv_heads + g;
        if (jj >= NSK) go = wait_idle(bar(empty0 + ring.slot), ring.parity ^ 1, abort_flag, a.err);
        go = __all_sync(0xffffffffu, go && !*abort_flag);
        if (!go) break;                          // leave the loop as a warp
        const uint32_t full = bar(full0 + ring.slot);
        if (is_v) {
          if (lane == 0) mbar_arrive_expect_tx(full, nb * kBlk8);
          __syncwarp();
          if (lane < nb)
            bulk_g2s_hint(sbase + OFF_ST + ring.slot * kTile8 + lane * kBlk8, vpool + tile * kBlk8,
                          kBlk8, full, policy_evict_normal());
        } else {
          // the tile's scales, which its stage's barrier publishes
          const int both = __shfl_sync(0xffffffffu, sc, (j % 4) * kBlkPerTile + (lane & 7));
          int ev = both < 0 ? INT_MIN : (both >> 8) - 127;
          if (jj == 0) e_ref = __reduce_max_sync(0xffffffffu, ev);
          if (both < 0) ev = e_ref;              // no key of this block counts
          const int off = e_ref - ev;
          const bool wide = __any_sync(0xffffffffu, abs(off) > kWideSpread);
          TileScales* ts = reinterpret_cast<TileScales*>(smem + OFF_SCALES) + sr.slot;
          if (lane < kBlkPerTile) {
            ts->k[lane] = a.scale * 1.4426950408889634f * scale_value(both < 0 ? 127u : both & 0xffu);
            ts->v[lane] = (float)ev;
            ts->l[lane] = __uint_as_float((uint32_t)(127 + max(-100, min(100, off))) << 23);
            if (lane == 0) {
              ts->wide = wide;
              ts->e = e_ref;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(full, nb * kBlk8);
          __syncwarp();
          if (lane < nb)
            tma_box8(sbase + OFF_K + ring.slot * kTile8 + lane * kBlk8, &tm_k, full,
                     (int)(tile * kBlockSize));
        }
        ++sent;
        if (jj == 0 || turn) {
          ids_next = load_ids(j / 4 + 1);
          sc_next = load_scales(j / 4 + 1, ids_next);
        }
      }
      if (!go && lane == 0) {                    // let the copies in flight land
        for (int jj = max(0, sent - NSK); jj < sent; ++jj)
          mbar_wait(bar(full0 + jj % NSK), (jj / NSK) & 1, nullptr);
      }
      __syncwarp();
    } else if (warp > W_VPROD && warp != W_NONE) {
      // ------------------------------------------------------------- V converters
      // thread (rs, cc) takes the 16 codes of chunk cc in row rs of every
      // block.  They are 32 bytes of a swizzled f16 row; the threads of its two
      // 64-column halves store their two 16-byte chunks in opposite order, so
      // no banks conflict.
      const int pt = (warp < W_NONE ? 0 : warp - W_NONE) * 32 + lane;
      const int rs = pt >> 3, cc = pt & 7, half = cc >> 2;
      const uint32_t ch = 2 * (cc & 3);
      const uint32_t thr_dst = half * kHalf16 + rs * 128;
      const uint32_t sw_first = ((ch + half) ^ (rs & 7)) << 4;
      const uint32_t sw_second = ((ch + 1 - half) ^ (rs & 7)) << 4;
      const int masked_from = (a.prior_len + qrow0 + 1) / BN;   // tiles with a masked entry
      bool go = true;
      Ring<NST> tr;
      Ring<NSV> vr;
      for (int jj = 0; jj < n_tiles; ++jj, tr.next(), vr.next()) {
        const int j = t0 + jj;
        // the V ring first holds the queries
        go = jj > 0 || wait_fast(bar(B_QC), 0, abort_flag, a.err);
        if (go) go = wait_idle(bar(B_STF + tr.slot), tr.parity, abort_flag, a.err);
        if (go && jj >= NSV) go = wait_idle(bar(B_VE + vr.slot), vr.parity ^ 1, abort_flag, a.err);
        go = __all_sync(0xffffffffu, go && !*abort_flag);
        if (!go) break;                          // leave the loop as a warp
        const uint32_t src = sbase + OFF_ST + tr.slot * kTile8 + pt * 16;
        const uint32_t dst = sbase + OFF_V + vr.slot * kTile16 + thr_dst;
        if (j >= masked_from) {
          // NaN codes and rows behind the sequence become zeros where they are
          // staged: rare, so its code stays short
#pragma unroll 1
          for (int b = 0; b < kBlkPerTile; ++b) {
            const int key = j * BN + b * kBlockSize + rs;
            uint4 x = lds16(src + b * kBlk8);
            bool found = false;
            x.x = drop_nan(x.x, &found);
            x.y = drop_nan(x.y, &found);
            x.z = drop_nan(x.z, &found);
            x.w = drop_nan(x.w, &found);
            if (key >= p.total_len) x = make_uint4(0u, 0u, 0u, 0u);
            else if (found) atomicMin(nan_key, key);
            sts16(src + b * kBlk8, x);
          }
        }
#pragma unroll 1
        for (int b4 = 0; b4 < kBlkPerTile; b4 += 4) {
          uint4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = lds16(src + (b4 + i) * kBlk8);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {half ? x[i].z : x[i].x, half ? x[i].w : x[i].y,
                                   half ? x[i].x : x[i].z, half ? x[i].y : x[i].w};
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[2 * k] = e4m3x2_to_f16x2((uint16_t)(w[k] & 0xffffu));
              o[2 * k + 1] = e4m3x2_to_f16x2((uint16_t)(w[k] >> 16));
            }
            const uint32_t d = dst + (b4 + i) * (kBlockSize * 128);
            sts16(d + sw_first, make_uint4(o[0], o[1], o[2], o[3]));
            sts16(d + sw_second, make_uint4(o[4], o[5], o[6], o[7]));
          }
        }
        fence_proxy_async_smem();                // make the tile visible to the tensor core
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(B_STE + tr.slot));
          mbar_arrive(bar(B_VF + vr.slot));
        }
      }
    } else if (warp == W_MMA && n_tiles > 0) {
      // ------------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = idesc0(false, BM, BN);
      constexpr uint32_t idesc_pv = idesc0(true, BM, HD);
      const uint64_t q_desc = make_sw128_desc(sbase + OFF_Q, 16, 1024);
      const uint64_t k_desc = make_sw128_desc(sbase + OFF_K, 16, 1024);
      const uint64_t v_desc = make_sw128_desc(sbase + OFF_V, kHalf16, 1024);
      auto issue_qk = [&](int hh, int stage) {
        issue_qk8(tmem + COL_S + hh * BN, q_desc + hh * (kTile16 / 16),
                  k_desc + stage * (kTile8 / 16), idesc_qk, bar(B_SF + hh));
      };
      auto issue_pv = [&](int hh, int stage, uint32_t accumulate, int half) {
        issue_pv4(tmem + COL_O + hh * HD, tmem + COL_S + hh * BN + half * 32,
                  v_desc + stage * (kTile16 / 16) + half * (64 * 128 / 16), idesc_pv, accumulate);
      };
      // The streams alternate: while one's softmax runs, the other's products
      // do.  Q K_{j+1}^T rewrites S_h, which holds P_h, right behind P_h V_j:
      // products issued by one thread execute in issue order.  A lane that
      // gives up a wait keeps issuing (every address stays valid) until the
      // vote at the tile's end.
      bool ok = true;
      auto wait_for = [&](int b, uint32_t parity) {
        ok &= wait_fast(bar(b), parity, abort_flag, a.err);
        __syncwarp();
      };
      Ring<NSK> kr;
      Ring<NSV> vr;
      wait_for(B_QC, 0);
      wait_for(B_KF, 0);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc_fence_after();
        issue_qk(0, 0);
        issue_qk(1, 0);
        for (int jj = 0; jj < n_tiles && ok; ++jj, vr.next()) {
          const bool more = jj + 1 < n_tiles;
          kr.next();                             // of tile jj + 1
          // ahead of the softmax, where this warp waits anyway
          wait_for(B_VF + vr.slot, vr.parity);
          if (more) wait_for(B_KF + kr.slot, kr.parity);
#pragma unroll 1
          for (int hh = 0; hh < 2; ++hh) {
            wait_for(B_PF + 2 * hh, jj & 1);
            tc_fence_after();
            issue_pv(hh, vr.slot, jj > 0 ? 1u : 0u, 0);
            wait_for(B_PF + 2 * hh + 1, jj & 1);
            tc_fence_after();
            issue_pv(hh, vr.slot, 1u, 1);
            if (more)
              issue_qk(hh, kr.slot);
            else
              commit_e(bar(B_OD + hh));
          }
          commit_e(bar(B_VE + vr.slot));         // V no longer needed
          ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        }
      }
      if (!ok) mbar_wait(bar(B_Q), 0, nullptr);  // after an abort, let the Q load land
    }
    __syncwarp();
    if (p.splits > 1) {                          // the merge's two barriers
      cluster_sync();
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    // ------------------------------------------------------------- softmax (stream hh)
    const int hh = warp >> 2;
    const int r = tid & 127;                // query row in the tile, TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t col_s = COL_S + hh * BN, col_o = COL_O + hh * HD;
    const int q0 = hh ? qrow1 : qrow0, head = hh ? head1 : head0;
    const int row_pos = a.prior_len + q0 + r;
    float q_up = 1.f;                       // what brings products back to the query's size
    const bool queries = q0 + (r & ~31) < a.chunk_len;   // the warp has rows of the chunk
    if (n_tiles > 0 && wait_fast(bar(B_Q), 0, abort_flag, a.err)) {
      if (queries) {
        // This row's query becomes its hi and lo rows.  Short loops: the code runs
        // once, and fetching it is what takes the time.
        const uint32_t src = sbase + OFF_V + hh * kTile16 + r * 128;
        const uint32_t dst = sbase + OFF_Q + hh * kTile16 + r * 128;
        auto piece = [&](int i) {             // elements 8 i .. 8 i + 7
          return lds16(src + (i >> 3) * kHalf16 + (((i & 7) ^ (r & 7)) << 4));
        };
        uint32_t top = 0;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const uint4 x = piece(i);
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                       __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
        }
        // 2^(7 - exponent of the row's largest element), of zeros and of
        // infinities or NaN 1
        top = max(top & 0xffffu, top >> 16) >> 7;
        const int ex = top == 255 ? 7 : max(-119, min((int)top - 127, 126));
        const float down = __uint_as_float((uint32_t)(127 + 7 - ex) << 23);
        q_up = __uint_as_float((uint32_t)(127 + ex - 7) << 23);
        // an infinite or NaN element makes the row's scores NaN
        const uint32_t bad = top == 255 ? 0x7f7f7f7fu : 0u;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {         // 16 elements: a chunk of hi and one of lo
          const uint4 x = piece(2 * i), y = piece(2 * i + 1);
          const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h2[2], l2[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // f16 holds the scaled element exactly, or to 2^-25
              const __half2 u = __floats2half2_rn(bf16lo(w[2 * k + e]) * down,
                                                  bf16hi(w[2 * k + e]) * down);
              h2[e] = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&u));
              const uint32_t back = e4m3x2_to_f16x2((uint16_t)h2[e]);
              const __half2 d = __hsub2(u, *reinterpret_cast<const __half2*>(&back));
              l2[e] = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&d));
            }
            hi[k] = (h2[0] | h2[1] << 16) | bad;
            lo[k] = l2[0] | l2[1] << 16;
          }
          const uint32_t at = dst + ((i ^ (r & 7)) << 4);
          sts16(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          sts16(at + kTile8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
      } else {                              // zeros: no score, no rescaling
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int i = 0; i < 8; ++i) {
          sts16(sbase + OFF_Q + hh * kTile16 + r * 128 + i * 16, zero);
          sts16(sbase + OFF_Q + hh * kTile16 + kTile8 + r * 128 + i * 16, zero);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(B_QC));
    }
    // M, in log2 units, and l
    float m_run = -INFINITY, l_run = 0.f;
    bool wide = false;                      // once true, l is summed against
    float ms_run = -INFINITY;               // a running maximum of its own
    Ring<NSK> kr;
    Ring<kScaleSlots> sr;
    for (int jj = 0; jj < n_tiles; ++jj, kr.next(), sr.next()) {
      wait_fast(bar(B_SF + hh), jj & 1, abort_flag, a.err);
      __syncwarp();
      tc_fence_after();
      // the S_B commit follows both streams' Q K^T: this K stage can be refilled
      if (hh == 1 && lane == 0) mbar_arrive(bar(B_KE + kr.slot));
      const int k0 = (t0 + jj) * BN;
      const TileScales* ts =
          reinterpret_cast<const TileScales*>(smem + OFF_SCALES) + sr.slot;
      // the whole S row into registers: four loads in flight, one wait
      float t[BN / 32][32];
#pragma unroll
      for (int c = 0; c < BN / 32; ++c) tmem_ld32(lane_base + col_s + c * 32, t[c]);
      // blocks' factors from products to scores; never 0, so that a masked
      // score stays -inf
      float kq[kBlkPerTile], ev[kBlkPerTile];
#pragma unroll
      for (int b = 0; b < kBlkPerTile; b += 4) {
        const float4 k = *reinterpret_cast<const float4*>(ts->k + b);
        const float4 v = *reinterpret_cast<const float4*>(ts->v + b);
        kq[b] = fmaxf(k.x * q_up, 1e-38f), kq[b + 1] = fmaxf(k.y * q_up, 1e-38f);
        kq[b + 2] = fmaxf(k.z * q_up, 1e-38f), kq[b + 3] = fmaxf(k.w * q_up, 1e-38f);
        ev[b] = v.x, ev[b + 1] = v.y, ev[b + 2] = v.z, ev[b + 3] = v.w;
      }
      const bool tile_wide = ts->wide;
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < BN / 32; ++c) reg_fence(t[c]);
      if (k0 + BN - 1 > a.prior_len + q0) {   // causal mask needed: bit i stands for column i
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) {
          const int last = row_pos - k0 - c * 32;
          const uint32_t seen = last < 0 ? 0u : 0xffffffffu >> (31 - min(last, 31));
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(seen >> i & 1u)) t[c][i] = -INFINITY;
        }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int b = 0; b < kBlkPerTile; ++b) {
        const float* x = &t[b / 2][(b & 1) * 16];
        float m0 = fmax3(x[0], x[1], x[2]), m1 = fmax3(x[3], x[4], x[5]);
        m0 = fmax3(m0, x[6], x[7]);
        m1 = fmax3(m1, x[8], x[9]);
        m0 = fmax3(m0, x[10], x[11]);
        m1 = fmax3(m1, x[12], x[13]);
        m0 = fmax3(m0, x[14], x[15]);
        mx = fmaxf(mx, fmaf(fmaxf(m0, m1), kq[b], ev[b]));
      }
      if (tile_wide || wide) {
        // from here on l = sum 2^(s - ms); before, it was sum 2^(s + E - M).
        // Rare, so it reads S again block by block and keeps the code short.
        if (!wide && jj > 0) ms_run = m_run - (float)ts->e;
        wide = true;
#pragma unroll 1
        for (int b = 0; b < kBlkPerTile; ++b) {
          float x[16];
          tmem_ld16(lane_base + col_s + b * 16, x);
          tmem_wait_ld();
          reg_fence(x);
          const float k = fmaxf(ts->k[b] * q_up, 1e-38f);
          float m2 = ms_run;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            x[i] = k0 + b * 16 + i > row_pos ? -INFINITY : x[i] * k;
            m2 = fmaxf(m2, x[i]);
          }
          const float m0 = m2 == -INFINITY ? 0.f : m2;   // no key yet: every weight is 0
          l_run *= ms_run == m2 ? 1.f : fast_exp2(ms_run - m2);
          ms_run = m2;
#pragma unroll
          for (int i = 0; i < 16; ++i) l_run += fast_exp2(x[i] - m0);
        }
      }
      float m_new = m_run;
      if (mx > m_run + kLazy || m_run == -INFINITY) m_new = mx;
      const float alpha = (m_new == m_run) ? 1.f : fast_exp2(m_run - m_new);
      if (jj >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
        // O holds P V of the tiles before; the S_h commit of this tile was
        // issued behind their last product, so that product is complete and
        // O can be rescaled in place
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < HD / 16; ++c) {
          float o[16];
          tmem_ld16(lane_base + col_o + c * 16, o);
          tmem_wait_ld();
          reg_fence(o);
          uint32_t u[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i] * alpha);
          tmem_st16(lane_base + col_o + c * 16, u);
        }
      }
      // p = 2^(s + ev - M), written as f16 pairs over the first 64 columns of
      // S; a row that has seen no key (its keys are in another CTA) has p = 0
      const float m_ref = m_new == -INFINITY ? 0.f : m_new;
      float2 sums[kBlkPerTile];              // of the blocks' weights, even and odd columns
#pragma unroll
      for (int c = 0; c < BN / 32; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int b = 2 * c + h;
          const float n = ev[b] - m_ref;
          const float2 k2 = make_float2(kq[b], kq[b]), n2 = make_float2(n, n);
          float2 part[2];
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 x = ffma2(make_float2(t[c][16 * h + i], t[c][16 * h + i + 1]), k2, n2);
            const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            part[(i >> 1) & 1] = i < 4 ? pp : fadd2(part[(i >> 1) & 1], pp);
            const __half2 ph = __floats2half2_rn(pp.x, pp.y);
            pk[8 * h + i / 2] = *reinterpret_cast<const uint32_t*>(&ph);
          }
          sums[b] = fadd2(part[0], part[1]);
        }
        tmem_st16(lane_base + col_s + c * 16, pk);
        if (c & 1) {                        // a half of P is in TMEM
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_PF + 2 * hh + (c >> 1)));
        }
      }
      // l, while the products run
      if (!wide) {
        l_run *= alpha;
#pragma unroll
        for (int b = 0; b < kBlkPerTile; ++b)
          l_run = fmaf(sums[b].x + sums[b].y, ts->l[b], l_run);
      }
      m_run = m_new;
    }
    if (n_tiles > 0) {
      wait_fast(bar(B_OD + hh), 0, abort_flag, a.err);
      __syncwarp();
      tc_fence_after();
    }
    // l stands for l 2^ref, O for O 2^M = O 2^ref unit unit2.  The results take
    // 1 / l and then the unit, which may leave the normal range when V's scales
    // do (in two factors where it is an exponential, which flushes there).
    const int e = n_tiles > 0 ? (reinterpret_cast<const TileScales*>(smem + OFF_SCALES))->e : 0;
    const float ref = wide ? ms_run : m_run - (float)e;
    const float unit = !wide ? scale_value((uint32_t)(e + 127))
                       : m_run == -INFINITY ? 0.f   // no key of the row in this CTA
                                            : fast_exp2(0.5f * (m_run - ms_run));
    const float unit2 = wide ? unit : 1.f;
    if (n_tiles > 0 && row_pos >= *nan_key)
      l_run = __int_as_float(0x7fffffff);   // the row sees a NaN value
    const bool row_ok = (q0 + r) < a.chunk_len;
    if (p.splits == 1) {
      // The rows leave through this stream's query tiles, which its products
      // are done with: 16-byte chunks XORed by the row, then whole rows of
      // the warp's 32, two to a store.  (Each thread storing its own row, 32
      // lines to a store, took 5,400 cycles.)
      const float inv = 1.f / l_run;
      const uint32_t tile = sbase + OFF_Q + hh * kTile16;
#pragma unroll 1
      for (int c = 0; c < HD; c += 32) {
        float o[32];
        tmem_ld32(lane_base + col_o + c, o);
        tmem_wait_ld();
        reg_fence(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = o[i] * inv * unit * unit2;
#pragma unroll
        for (int i = 0; i < 32; i += 8)
          sts16(tile + r * 256 + ((((c + i) / 8) ^ (r & 15)) << 4),
                make_uint4(pack_bf16(o[i], o[i + 1]), pack_bf16(o[i + 2], o[i + 3]),
                           pack_bf16(o[i + 4], o[i + 5]), pack_bf16(o[i + 6], o[i + 7])));
      }
      __syncwarp();
      const int r0 = r - lane + (lane >> 4), chunk = lane & 15;
      __nv_bfloat16* base = static_cast<__nv_bfloat16*>(a.out) +
                            ((int64_t)q0 * a.num_q_heads + head) * HD + chunk * 8;
#pragma unroll 4
      for (int i = 0; i < 32; i += 2) {
        const int row = r0 + i;
        const uint4 v = lds16(tile + row * 256 + ((chunk ^ (row & 15)) << 4));
        if (q0 + row < a.chunk_len)
          *reinterpret_cast<uint4*>(base + (int64_t)row * a.num_q_heads * HD) = v;
      }
    } else {
      const uint32_t row_at = sbase + OFF_ROWS + (hh * BM + r) * 8;
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(row_at), "f"(ref), "f"(l_run) : "memory");
      cluster_sync();                       // every CTA's stats are there, its tiles are done with
      // CTA k adds up columns k W .. k W + W - 1, W = 2^w the columns over the
      // largest power of two of CTAs.  It gets each CTA's part of the results in
      // fp32, four columns of 128 rows in a piece of 2 KiB, rows side by side.
      // (These 128 KiB a CTA, at some 25 bytes a cycle, are the longest part of a
      // short call: 77 rows over 500 keys take 13.2 us; 12.0 us with f16 parts,
      // whose rounding would stand beside that of P.)
      const int w = 7 - (31 - __clz(p.splits));
      const int owners = HD >> w;
      float f = 0.f;                        // a row's share over l
      if (row_ok) {
        float2 stat[8];                     // all on their way before the first is used
#pragma unroll
        for (int k = 0; k < 8; ++k)
          stat[k] = k < p.splits ? ld_peer2(peer(row_at, k)) : make_float2(-INFINITY, 0.f);
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, stat[k].x);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < p.splits) sum = fmaf(fast_exp2(stat[k].x - top), stat[k].y, sum);
        if (n_tiles > 0) f = fast_exp2(ref - top) / sum;
      }
#pragma unroll 1
      for (int c = 0; c < HD; c += 16) {
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = 0.f;
        if (n_tiles > 0) {
          tmem_ld16(lane_base + col_o + c, o);
          tmem_wait_ld();
          reg_fence(o);
        }
        // W is at least 16: the 16 columns have one owner
        const int piece = ((rank * 2 + hh) << (w - 2)) + ((c & ((1 << w) - 1)) >> 2);
        const uint32_t at = peer(sbase + piece * (BM * 16) + r * 16, c >> w);
        if (row_ok) {
          // f first: the unit may leave the normal range when V's scales do
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = o[i] * f * unit * unit2;
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            st_peer4(at + i / 4 * (BM * 16), o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
      }
      cluster_sync();
      // this CTA's columns of the chunk's rows, eight to a thread
      const int shift = w - 3, groups = rank < owners ? 1 << shift : 0;
      const int rows0 = min(BM, a.chunk_len - qrow0), rows1 = max(0, min(BM, a.chunk_len - qrow1));
#pragma unroll 1
      for (int i = tid; i < (rows0 + rows1) * groups; i += kSoftThreads) {
        const int row = i >> shift, c8 = i & (groups - 1);
        const int h = row >= rows0 ? 1 : 0, rr = row - (h ? rows0 : 0);
        float acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k < p.splits) {
            const uint32_t at = sbase + (((k * 2 + h) << (w - 2)) + 2 * c8) * (BM * 16) + rr * 16;
            const uint4 x = lds16(at), y = lds16(at + BM * 16);
            acc[0] += __uint_as_float(x.x);
            acc[1] += __uint_as_float(x.y);
            acc[2] += __uint_as_float(x.z);
            acc[3] += __uint_as_float(x.w);
            acc[4] += __uint_as_float(y.x);
            acc[5] += __uint_as_float(y.y);
            acc[6] += __uint_as_float(y.z);
            acc[7] += __uint_as_float(y.w);
          }
        }
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) +
                             ((int64_t)((h ? qrow1 : qrow0) + rr) * a.num_q_heads +
                              (h ? head1 : head0)) * HD + (rank << w) + c8 * 8;
        *reinterpret_cast<uint4*>(dst) =
            make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                       pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7]));
      }
    }
  }
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols));
  }
}

constexpr int kMaxSplits = 8;     // the portable cluster

// Clusters of s CTAs (1 .. kMaxSplits) that run at once, at [s].  Of 152 SMs
// clusters of 8 reach 120 only: they lie within a GPC.  Asked once per context.
struct ClusterSlots {
  int at[kMaxSplits + 1] = {};
};
cudaError_t cluster_slots(int num_sms, ClusterSlots* out) {
  static std::mutex mu;
  static std::map<uint64_t, ClusterSlots> known;
  const uint64_t ctx = current_context_id();
  std::lock_guard<std::mutex> lock(mu);
  auto it = known.find(ctx);
  if (ctx != 0 && it != known.end()) {
    *out = it->second;
    return cudaSuccess;
  }
  out->at[1] = num_sms;
  for (int s = 2; s <= kMaxSplits; ++s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, 1, s);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        cudaOccupancyMaxActiveClusters(&out->at[s], prefill_fp8_block_kernel, &cfg);
    if (e != cudaSuccess) return e;
  }
  if (ctx != 0) {
    if (known.size() > 256) known.clear();   // stale contexts: start over
    known[ctx] = *out;
  }
  return cudaSuccess;
}

// CTAs to an item: the number by which the longest share of the GPU ends first.
// Items go to the slots heaviest first, back and forth; an item costs its
// tiles (1.56 us measured) and 6.5 us, when it is split 9.6 us and 0.45 us a CTA
// (short chunks; where 128 rows meet, their fp32 sums take up to 2 us more).
// (640 rows of 32 heads over 16,384 keys are 80 items: one CTA each leaves 72
// SMs idle.)  The choice is the best of all splits, in us: 128 rows over 1,024
// keys 15.9 (8 CTAs, as many as SMs would hold: 26.8), 640 over 16,384 169 (one:
// 209), 768 over 16,768 196 (one: 215), 1,024 rows of 4 heads over 5,120 27.9 (8:
// 39.8), 200 of 8 heads over 32,200 63 (one: 389).
int choose_splits(const Params& p, int n_x, int n_t, const ClusterSlots& slots) {
  const int64_t n = (int64_t)n_x * n_t;
  if (n > 4 * (int64_t)slots.at[1]) return 1;          // many items even out by themselves
  const int rows = p.rows_mode ? 2 * BM : BM;
  auto tiles = [&](int64_t item) {                      // heaviest first
    const int64_t end = (n_t - item / n_x) * rows;      // behind the item's last row
    return (int)((p.a.prior_len + std::min<int64_t>(p.a.chunk_len, end) - 1) / BN + 1);
  };
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int s = 1; s <= std::min(kMaxSplits, tiles(0)); ++s) {
    const int64_t k = slots.at[s];
    if (k < 1) continue;
    // the longest slot is a first or last one, or beside the last lap's end
    const int64_t rem = n % k, ends[] = {0, k - 1, rem - 1, rem, k - rem - 1, k - rem};
    int64_t cost = 0;
    for (int64_t i : ends) {
      int64_t sum = 0;
      for (int64_t lap = 0; i >= 0 && i < k && lap * k < n; ++lap) {
        const int64_t item = lap * k + (lap % 2 ? k - 1 - i : i);
        if (item < n) sum += (tiles(item) + s - 1) / s * 156 + (s == 1 ? 650 : 960 + 45 * s);
      }
      cost = std::max(cost, sum);
    }
    if (cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return best;
}

}  // namespace

cudaError_t launch_prefill_fp8_block(const PrefillArgs& a, int num_sms, cudaStream_t stream) {
  Params p;
  p.a = a;
  p.total_len = a.prior_len + a.chunk_len;
  p.q_tiles = (a.chunk_len + BM - 1) / BM;
  if (p.q_tiles == 0) return cudaSuccess;
  // two query tiles of one head to a CTA when the group is odd
  p.rows_mode = (a.num_q_heads / a.num_kv_heads) % 2;
  CUtensorMap tm_q, tm_k;
  if (!encode_rows_map_bf16(&tm_q, a.q, a.chunk_len, a.num_q_heads) ||
      !encode_pool_map_u8(&tm_k, a.k_cache, a.num_blocks * a.num_kv_heads * kBlockSize))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_dynamic_smem(prefill_fp8_block_kernel, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int n_x = p.rows_mode ? a.num_q_heads : a.num_q_heads / 2;
  const int n_t = p.rows_mode ? (p.q_tiles + 1) / 2 : p.q_tiles;
  ClusterSlots slots;
  e = cluster_slots(num_sms, &slots);
  if (e != cudaSuccess) return e;
  p.splits = choose_splits(p, n_x, n_t, slots);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_x, n_t, p.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = p.splits;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefill_fp8_block_kernel, p, tm_q, tm_k);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pkv
