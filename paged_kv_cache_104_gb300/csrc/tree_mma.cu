// Attention of drafted tokens over the paged bf16 cache, on tcgen05 (sm_103a).
//
// What it computes: for row (drafted token i, query head h of KV head g) of a
// sequence, over the keys the row sees (the whole context, and the drafted
// tokens of its mask), out = sum_n softmax(scale q . k_n) v_n and the logarithm
// of the softmax sum.
//
// What bounds it: every stored key and value is read once for all rows of its
// sequence, 512 B for 512 R multiply-adds (R rows of a KV head), so up to about
// R = 256 rows (64 drafted tokens of a group of 4) HBM is the bound.  Measured,
// 32 query and 8 KV heads, with the merge: 64 sequences of 2,301 with 16 drafted
// tokens 106 us (5.8 TB/s, 86% of a plain copy's rate), 8 of 32,001 with 64 drafted
// 192-200 us (5.3-5.5 TB/s and 1,340-1,390 TFLOP/s: the tensor pipe is busy 64% of
// the time, the rest is softmax between a side's two products, as tensor memory
// holds one S for each side), one of 777 with 8 drafted 10.4 us (latency).
//
// Work.  A stream is one (sequence, KV head, 256 rows), cut into tiles of 128
// keys; the tiles of the whole batch are shared out by weight to one persistent
// CTA per SM (tree_common.cuh).  A CTA's part of a stream is an item; a stream
// that falls to several CTAs leaves fp32 partials (unnormalised O, max, sum),
// at most two per CTA, that a second kernel joins.
//
// Two softmax warpgroups ("sides") work in turn on S and O accumulators of
// their own, so the tensor core and the loads run on while one exponentiates:
//   more than 128 rows: side s takes rows 128 s .. of every tile;
//   up to 128 rows:     side s takes every other tile, and the two join at the
//                       item's end through TMEM (thread r of either side can
//                       read row r of both accumulators);
//   two KV heads:       short sequences of up to 128 rows go in pairs of KV heads,
//                       one to a side, whose items start and end once for both.
// Each way the products alternate between the sides ("steps").
//
// Roles (384 threads):
//   warps 0-3 / 4-7  softmax of side 0 / 1: thread r owns row r (TMEM lane r);
//                    warps whose rows do not exist only pass barriers on
//   warp 8           K/V producer: one 4 KiB TMA copy per cache block (K and V
//                    tiles through one ring of five 32 KiB slots)
//   warp 9           tcgen05 issuer: S = Q K^T from shared memory, O += P V with
//                    P (bf16) in TMEM over its S.  P is rounded to bf16, the
//                    values' type, as the product's operands have one type: up
//                    to 2^-8 of each weight, 1.3e-3 to 1.6e-3 of the result's
//                    norm for normal values, next to 1.7e-3 for its own
//                    rounding (P as a sum of two bf16 would take the product
//                    twice).  The sum l takes the unrounded weights, as lse
//                    needs them; the rounded ones would be a second sum.
//   warp 10          checks the drafted tokens' values: a row of V that holds an
//                    infinity or NaN would reach, as 0 x inf, rows that do not
//                    see it.  Such rows are cleared in shared memory and added
//                    by the softmax threads to the rows that see them; rows of
//                    the last block past the sequence's end are cleared too.
//   warp 11          works out the plan, hands the items to the others through
//                    a ring of four, and loads their queries
// Every mbarrier wait is bounded; on time-out the kernel records an error,
// stops issuing work, lets its copies land, frees its TMEM and returns.
#include <climits>

#include <cuda.h>

#include "common.cuh"
#include "host_cache.h"
#include "launch.h"
#include "tc_common.cuh"
#include "tmap.h"
#include "tree_common.cuh"

namespace pkv {
namespace {

constexpr int BM = 128, BN = kTreeTile, HD = 128;
constexpr int QHALF = BM * 128;               // 64 columns of 128 query rows, 16 KiB
constexpr int Q_BYTES = 2 * QHALF;
constexpr int TILE = BN * HD * 2;             // a K or V tile, 32 KiB: [8 rows][half][8 x 128 B]
constexpr int GROUP8 = 2048;                  // 8 rows of a tile
constexpr int NS = 5;                         // ring slots
constexpr int NI = 4;                         // items in flight
constexpr int NCK = 4;                        // V tiles on their way to the guard
constexpr int OFF_Q = 0;                      // two 32 KiB buffers
constexpr int OFF_KV = 2 * Q_BYTES;
constexpr int OFF_ML = OFF_KV + NS * TILE;    // [side][row] (max, sum) exchange
constexpr int OFF_ITEM = OFF_ML + 2 * BM * 8;
constexpr int OFF_BAD = OFF_ITEM + NI * 64;   // drafted tokens whose V was cleared, per item slot
constexpr int OFF_BAR = OFF_BAD + NI * 16;
constexpr int kSoft = 256, kThreadsT = 384;
constexpr int W_KV = 8, W_MMA = 9, W_FIX = 10, W_PLAN = 11;
constexpr int kRegsSoft = 200, kRegsRest = 96;
static_assert(kRegsSoft * kSoft + kRegsRest * (kThreadsT - kSoft) <= ((65536 / kThreadsT) & ~7) * kThreadsT,
              "the register split must fit in what the CTA was launched with");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t COL_S = 0, COL_O = 2 * BN;  // per side: S (P over its first 64 columns), O
constexpr float kLazy = 8.0f;                  // the maximum is raised when it grows by more than 2^8

enum {
  TB_QF = 0,               // [2] queries loaded
  TB_QE = TB_QF + 2,       // [2] queries no longer read
  TB_F = TB_QE + 2,        // [NS] tile loaded
  TB_E = TB_F + NS,        // [NS] tile no longer read
  TB_IF = TB_E + NS,       // [NI] item there
  TB_IE = TB_IF + NI,      // [NI] item no longer read
  TB_CK = TB_IE + NI,      // [NCK] V tile to be checked loaded (its TB_F follows the check)
  TB_SF = TB_CK + NCK,     // [side] S complete
  TB_PF = TB_SF + 2,       // [side][half] P written
  TB_OD = TB_PF + 4,       // [side] O complete, where the sides have rows of their own
  TB_OJ = TB_OD + 2,       // both O complete, where they share their rows
  TB_ML,                   // both sides' (max, sum) written
  TB_JD,                   // both sides' O read by both
  TB_COUNT
};
constexpr int SMEM_BYTES = OFF_BAR + TB_COUNT * 8 + 16;
static_assert(SMEM_BYTES <= 227 * 1024, "one CTA per SM");
static_assert(sizeof(TreeItem) <= 64, "an item's slot");

// What CTA c left of a stream that starts in it and goes on in others.
struct MergeDesc {
  int pieces;      // 0: nothing to join
  int b, g, row0, rows, q_tok;
  int heads;       // 2: rows of KV head g, then of g + 1
  int pad;
};

struct TreeMmaParams {
  TreeArgs a;
  int q_bufs;                // 2: no item has more than 128 rows, or two KV heads
  MergeDesc* desc;           // [CTA]
  char* partials;            // [CTA][2] of piece_bytes: O [rows][128], then (max, sum) [rows]
  int64_t piece_bytes;
  int piece_rows;
  bool wide;                 // out is 32-byte aligned
  bool whole;                // streams are not cut
};

// The order of an item's tiles in the ring, as the products need them: with
// `both` K0 V0 K1 V1 .., else K0 K1 V0 K2 V1 K3 .. (side s's Q K^T of its next
// tile is issued behind its P V of this one).  A pair's tiles are numbered
// alternately: 2 j + s is tile j of side s's KV head.
struct Order {
  bool both;   // both sides take every tile
  int n;       // tiles of K (and of V)
  __device__ int v(int j) const { return both ? 2 * j + 1 : (j < n - 1 ? 2 * j + 2 : 2 * n - 1); }
  __device__ int side_steps(int side) const { return both ? n : (n + 1 - side) >> 1; }
};

__device__ __forceinline__ void store32(char* to, const uint32_t (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// Adds p V to the row's O (TMEM column o_col) for the drafted tokens `left`
// whose values were cleared, p = 2^(scaled score - base) from q and k in
// global memory.  The whole warp, each lane its row; not the usual path.
__device__ __noinline__ void add_cleared(const TreeArgs& a, const TreeItem& it, int g, unsigned long long left,
                                         float base, uint32_t o_col, int out_row) {
  const unsigned long long any = __reduce_or_sync(0xffffffffu, (uint32_t)left) |
                                 (unsigned long long)__reduce_or_sync(0xffffffffu, (uint32_t)(left >> 32)) << 32;
  for (unsigned long long todo = any; todo; todo &= todo - 1) {
    const int d = __ffsll((long long)todo) - 1, pos = it.ctx + d;
    const bool mine = left >> d & 1;
    int blk = __ldg(a.block_table + (int64_t)it.b * a.max_blocks_per_seq + pos / kBlockSize);
    if (blk < 0 || (int64_t)blk >= a.num_blocks) blk = 0;
    const int64_t at = (((int64_t)blk * a.num_kv_heads + g) * kBlockSize + pos % kBlockSize) * HD;
    const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(a.k_cache) + at;
    const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(a.v_cache) + at;
    const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)out_row * HD;
    float s = 0.f;
    if (mine)
      for (int i = 0; i < HD; ++i) s = fmaf(__bfloat162float(qr[i]), __bfloat162float(kr[i]), s);
    const float pw = fast_exp2(fmaf(s, a.scale * 1.4426950408889634f, -base));
#pragma unroll 1
    for (int c = 0; c < HD; c += 32) {
      float o[32];
      __syncwarp();
      tmem_ld32(o_col + c, o);
      tmem_wait_ld();
      reg_fence(o);
      if (mine)
#pragma unroll
        for (int q = 0; q < 32; ++q) o[q] = fmaf(pw, __bfloat162float(vr[c + q]), o[q]);
      __syncwarp();
      tmem_st32(o_col + c, o);
      tmem_wait_st();
    }
  }
}

template <bool PAIRS>
__global__ void __launch_bounds__(kThreadsT, 1)
tree_mma_kernel(const __grid_constant__ TreeMmaParams p, const __grid_constant__ CUtensorMap tm_q,
                const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sbase = smem_u32(smem);
  const TreeArgs& a = p.a;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + TB_COUNT);
  int* abort_i = reinterpret_cast<int*>(tmem_slot + 1);
  volatile int* abort_flag = abort_i;
  unsigned long long* bad_v = reinterpret_cast<unsigned long long*>(smem + OFF_BAD);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  if (sbase & 1023u) {   // swizzled operand tiles need a 1 KiB-aligned base
    if (threadIdx.x == 0) {
      record_error(a.err, DEVERR_SMEM_LAYOUT);
      p.desc[blockIdx.x].pieces = 0;
    }
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.num_q_heads / a.num_kv_heads, log_group = 31 - __clz(group);   // a power of two

  if (tid == 0) {
    for (int i = 0; i < TB_COUNT; ++i) {
      int count = 1;
      if (i >= TB_IE && i < TB_CK) count = 3 + kSoft / 32;   // issuer, producer, guard, softmax warps
      if (i >= TB_PF && i < TB_OD) count = 4;
      if (i >= TB_ML) count = kSoft / 32;
      mbar_init(bar(i), count);
    }
    *abort_i = 0;
    fence_mbar_init();
  }
  if (warp == W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  TreePlan<true, PAIRS> plan(a, warp == W_PLAN, p.whole);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The k-th item, for a warp that consumes items (false: none, or aborted).
  auto item_at = [&](int k, TreeItem& it) {
    bool ok = wait_or_abort(bar(TB_IF + k % NI), (k / NI) & 1, abort_flag, a.err);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    it = *reinterpret_cast<const TreeItem*>(smem + OFF_ITEM + (k % NI) * 64);
    return it.n > 0;
  };
  auto item_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(TB_IE + k % NI));
  };
  // a whole warp waits and agrees
  auto warp_wait = [&](int b, uint32_t parity) {
    return (bool)__all_sync(0xffffffffu, wait_fast(bar(b), parity, abort_flag, a.err));
  };
  auto order_of = [&](const TreeItem& it) { return Order{it.rows > BM, PAIRS ? it.n * it.heads : it.n}; };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == W_PLAN) {
      // ---------------------------------------------------------------- plan and queries
      MergeDesc d{};
      int made = 0, loaded = 0;        // items handed out; queries asked for
      bool last = false;
      TreeItem it;
      long long since = clock64();
      while (!last || loaded < made - 1) {
        bool moved = false;
        if (!last && (made < NI || __all_sync(0xffffffffu, mbar_try_wait(bar(TB_IE + made % NI), ((made / NI) - 1) & 1)))) {
          it = plan.next();
          last = it.n == 0;
          if (it.pieces > 0) d = MergeDesc{it.pieces, it.b, it.g, it.row0, it.rows, it.q_tok, it.heads, 0};
          if (lane == 0) *reinterpret_cast<TreeItem*>(smem + OFF_ITEM + (made % NI) * 64) = it;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(TB_IF + made % NI));
          ++made;
          moved = true;
        }
        if (loaded < made - (last ? 1 : 0)) {
          const int qb = loaded % p.q_bufs;
          if (loaded < p.q_bufs ||
              __all_sync(0xffffffffu, mbar_try_wait(bar(TB_QE + qb), ((loaded / p.q_bufs) - 1) & 1))) {
            // an item's slot is written again only once its queries were used
            const TreeItem x = *reinterpret_cast<const TreeItem*>(smem + OFF_ITEM + (loaded % NI) * 64);
            if (lane == 0) {
              const bool pair = PAIRS && x.heads == 2;
              const int sides = pair || x.rows > BM ? 2 : 1;
              mbar_arrive_expect_tx(bar(TB_QF + qb), sides * Q_BYTES);
              for (int s = 0; s < sides; ++s)
                for (int h = 0; h < 2; ++h)
                  tma_load_3d(sbase + OFF_Q + (qb + s) * Q_BYTES + h * QHALF, &tm_q, bar(TB_QF + qb), 64 * h,
                              (x.g + (pair ? s : 0)) * group,
                              x.q_tok + ((x.row0 + (pair ? 0 : s * BM)) >> log_group));
            }
            __syncwarp();
            ++loaded;
            moved = true;
          }
        }
        const long long now = clock64();
        if (moved) since = now;
        if (__any_sync(0xffffffffu, *abort_flag || now - since > kWaitLimitCycles)) {
          if (!*abort_flag) record_error(a.err, DEVERR_TIMEOUT);
          *abort_flag = 1;
          break;
        }
      }
      __syncwarp();
      if (*abort_flag)   // let the queries' copies still in flight land
        for (int k = max(0, loaded - p.q_bufs); k < loaded; ++k)
          mbar_wait(bar(TB_QF + k % p.q_bufs), (k / p.q_bufs) & 1, nullptr);
      if (lane == 0) p.desc[blockIdx.x] = d;
    } else if (warp == W_KV) {
      // ---------------------------------------------------------------- K/V producer
      if (lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
      }
      // K and V that are read once leave the L2 first; those of a sequence
      // whose rows are several streams are read again
      const uint64_t once = policy_evict_first(), again = policy_evict_normal();
      uint64_t policy = once;
      int pos = 0, checks = 0;        // ring position; V tiles sent to the guard
      uint32_t history = 0;           // which of the last positions went to the guard
      TreeItem it;
      bool ok = !kWithholdCopies;     // (a test's build: the others' waits run out, nothing is in flight)
      for (int k = 0; ok && item_at(k, it); ++k) {
        const int32_t* row = a.block_table + (int64_t)it.b * a.max_blocks_per_seq;
        const int blocks = (it.len + kBlockSize - 1) / kBlockSize;
        // block ids of four tiles, one per lane
        auto ids_of = [&](int window) {
          const int idx = window * 32 + lane;
          int blk = 0;
          if (idx < blocks && idx < (it.t0 + it.n) * 8) {
            blk = __ldg(row + idx);
            if (blk < 0 || (int64_t)blk >= a.num_blocks) {
              record_error(a.err, DEVERR_BLOCK_RANGE);
              blk = 0;
            }
          }
          return blk;
        };
        int window = it.t0 >> 2;
        int ids = ids_of(window), next_ids = ids_of(window + 1);
        const bool both = it.rows > BM;
        const int pair = PAIRS ? it.heads - 1 : 0, tiles = it.n << pair;
        auto load = [&](bool is_v, int j) {
          const int t = it.t0 + (j >> pair), slot = pos % NS;
          if (pos >= NS) ok = warp_wait(TB_E + slot, ((pos / NS) - 1) & 1);
          if (!ok) return;
          if (is_v && (t >> 2) > window) {   // V follows K: nobody needs the older window
            ids = next_ids;
            next_ids = ids_of(++window + 1);
          }
          const int mine = __shfl_sync(0xffffffffu, (t >> 2) > window ? next_ids : ids, (t & 3) * 8 + (lane & 7));
          const int nb = min(8, blocks - 8 * t);
          const bool check = is_v && (t + 1) * BN > it.ctx;
          const uint32_t full = bar(check ? TB_CK + checks % NCK : TB_F + slot);
          if (lane == 0) mbar_arrive_expect_tx(full, nb * 2 * GROUP8);
          __syncwarp();
          if (lane < nb)
            tma_load_4d(sbase + OFF_KV + slot * TILE + lane * 2 * GROUP8, is_v ? &tm_v : &tm_k, full, 0, 0, 0,
                        2 * (mine * a.num_kv_heads + it.g + (j & pair)), policy);
          history = history << 1 | (check ? 1u : 0u);
          checks += check;
          ++pos;
        };
        policy = (it.len - it.ctx) * group <= kTreeRows ? once : again;
        load(false, 0);
        if (!both && tiles > 1 && ok) load(false, 1);
        for (int j = 0; j < tiles && ok; ++j) {
          load(true, j);
          const int kj = both ? j + 1 : j + 2;
          if (kj < tiles && ok) load(false, kj);
        }
        item_done(k);
      }
      if (*abort_flag) {   // let the copies already issued land
        for (int i = max(0, pos - NS); i < pos; ++i)
          if (!(history >> (pos - 1 - i) & 1)) mbar_wait(bar(TB_F + i % NS), (i / NS) & 1, nullptr);
        for (int i = max(0, checks - NCK); i < checks; ++i) mbar_wait(bar(TB_CK + i % NCK), (i / NCK) & 1, nullptr);
      }
    } else if (warp == W_MMA) {
      // ---------------------------------------------------------------- issuer
      constexpr uint32_t idesc_qk = make_idesc(false, BM, BN);
      constexpr uint32_t idesc_pv = make_idesc(true, BM, HD);
      // What this warp does between two products can leave the tensor core
      // idle: descriptors are formed once, ring positions counted up, and only
      // S (per step) and O (per item) are committed; the softmax threads free
      // the ring's slots, which those commits tell them are read.
      const uint64_t k_desc = make_sw128_desc(sbase + OFF_KV, 16, GROUP8);
      const uint64_t v_desc = make_sw128_desc(sbase + OFF_KV, 1024, GROUP8);
      const uint64_t q_desc = make_sw128_desc(sbase + OFF_Q, 16, 1024);
      int slot = 0;                   // ring position: slot and parity
      uint32_t par = 0, p_par[2] = {0, 0};
      TreeItem it;
      bool ok = true;
      auto tile_there = [&](int sl, uint32_t pr) {
        ok = ok && warp_wait(TB_F + sl, pr);
        tc_fence_after();
      };
      auto step = [&] {
        if (++slot == NS) {
          slot = 0;
          par ^= 1;
        }
      };
      auto qk = [&](int side, uint64_t q, int sl) {
        if (!ok) return;
        mma_ss8_e(tmem + COL_S + side * BN, q, k_desc + (uint32_t)(sl * (TILE >> 4)), idesc_qk, QHALF >> 4, 1024 >> 4);
        commit_e(bar(TB_SF + side));
      };
      auto pv = [&](int side, int sl, bool first, int ks) {
        for (int half = 0; half < 2; ++half) {
          ok = ok && warp_wait(TB_PF + 2 * side + half, p_par[side]);
          if (!ok) return;
          tc_fence_after();
          mma_ts4_e(tmem + COL_O + side * HD, tmem + COL_S + side * BN + half * 32,
                    v_desc + (uint32_t)(sl * (TILE >> 4) + half * (8 * GROUP8 >> 4)), idesc_pv, 2 * GROUP8 >> 4,
                    (!first || half) ? 1u : 0u, ks - 4 * half);
        }
        p_par[side] ^= 1;
      };
      for (int k = 0; ok && item_at(k, it); ++k) {
        // the same in every lane, and known to be: descriptors stay in uniform registers
        const int heads = PAIRS ? __shfl_sync(0xffffffffu, it.heads, 0) : 1, n = __shfl_sync(0xffffffffu, it.n, 0) * heads;
        const bool both = __shfl_sync(0xffffffffu, it.rows, 0) > BM;
        // 16-key products of the item's last tile; 8 in the others
        const int last_ks = __shfl_sync(0xffffffffu, (min(BN, it.len - (it.t0 + it.n - 1) * BN) + 15) / 16, 0);
        const int qb = k % p.q_bufs;
        ok = warp_wait(TB_QF + qb, (k / p.q_bufs) & 1);
        const uint64_t q0 = q_desc + (uint32_t)(qb * (Q_BYTES >> 4)), q1 = q0 + (both || heads == 2 ? Q_BYTES >> 4 : 0);
        tile_there(slot, par);
        qk(0, q0, slot);
        if (both) {
          qk(1, q1, slot);
          step();
          for (int j = 0; j < n && ok; ++j) {
            const bool more = j + 1 < n;
            const int vs = slot, ks = more ? 8 : last_ks;
            const uint32_t vp = par;
            step();
            if (j == n - 1 && ok) commit_e(bar(TB_QE + qb));   // every Q K^T of the item is behind this
            tile_there(vs, vp);
            pv(0, vs, j == 0, ks);
            if (more) {
              tile_there(slot, par);
              qk(0, q0, slot);
            } else if (ok) {
              commit_e(bar(TB_OD));
            }
            pv(1, vs, j == 0, ks);
            if (more) {
              qk(1, q1, slot);
              step();
            } else if (ok) {
              commit_e(bar(TB_OD + 1));
            }
          }
        } else {
          step();
          if (n > 1) {
            tile_there(slot, par);
            qk(1, q1, slot);
            step();
          }
          for (int s = 0; s < n && ok; ++s) {
            const int side = s & 1;
            if (s + 2 == max(n, 2) && ok) commit_e(bar(TB_QE + qb));
            tile_there(slot, par);
            pv(side, slot, s < 2, s >= n - heads ? last_ks : 8);
            step();
            if (s + 2 < n) {
              tile_there(slot, par);
              qk(side, side ? q1 : q0, slot);
              step();
            } else if (heads == 2 && ok) {
              commit_e(bar(TB_OD + side));
            }
          }
          if (heads == 1 && ok) commit_e(bar(TB_OJ));
        }
        item_done(k);
      }
    } else if (warp == W_FIX) {
      // ---------------------------------------------------------------- guard of the drafted tokens' values
      int base = 0, checks = 0;
      TreeItem it;
      bool ok = true;
      for (int k = 0; ok && item_at(k, it); ++k) {
        const Order ord = order_of(it);
        const int pair = PAIRS ? it.heads - 1 : 0;
        unsigned long long bad[2] = {0, 0};
        for (int j = (max(it.t0, it.ctx / BN) - it.t0) << pair; j < it.n << pair; ++j) {
          const int t = it.t0 + (j >> pair), at = base + ord.v(j);
          // (a barrier of its own: this warp does not follow every turn of the ring)
          ok = warp_wait(TB_CK + checks % NCK, (checks / NCK) & 1);
          ++checks;
          if (!ok) break;
          unsigned char* tile = smem + OFF_KV + (at % NS) * TILE;
          const int r0 = max(it.ctx - t * BN, 0), r1 = min(it.len - t * BN, BN);
          // two rows at a time, 16 bytes per lane (chunk lane & 15: which half
          // and where in it does not matter to a check or a clear)
          auto chunk = [&](int r) {
            return reinterpret_cast<uint4*>(tile + (r >> 3) * GROUP8 + ((lane >> 3) & 1) * 1024 + (r & 7) * 128 +
                                            (lane & 7) * 16);
          };
          for (int r = r0; r < r1; r += 2) {
            const int mine = r + (lane >> 4);
            bool odd = false;
            if (mine < r1) {
              const uint4 x = *chunk(mine);
              const uint32_t words[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)   // all exponent bits of either half set
                odd |= (words[i] & 0x7f80u) == 0x7f80u || (words[i] & 0x7f800000u) == 0x7f800000u;
            }
            const uint32_t votes = __ballot_sync(0xffffffffu, odd);
            const bool clear = lane < 16 ? (votes & 0xffffu) != 0 : (votes >> 16) != 0;
            if (clear && mine < r1) *chunk(mine) = make_uint4(0, 0, 0, 0);
            const int d = t * BN + r - it.ctx;
            const unsigned long long found = (votes & 0xffffu ? 1ull << d : 0) | (votes >> 16 ? 2ull << d : 0);
            if (j & pair) bad[1] |= found;
            else bad[0] |= found;
          }
          // rows of the last block behind the sequence
          for (int r = r1 + (lane >> 4); r < ((r1 + 15) & ~15); r += 2) *chunk(r) = make_uint4(0, 0, 0, 0);
          if (lane == 0) bad_v[2 * (k % NI) + (j & pair)] = j & pair ? bad[1] : bad[0];
          fence_proxy_async_smem();       // the clears become visible to the tensor core
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(TB_F + at % NS));
        }
        base += 2 * ord.n;
        item_done(k);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    // ---------------------------------------------------------------- softmax
    const int side = warp >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t col_s = COL_S + side * BN, col_o = COL_O + side * HD;
    const float sl2 = a.scale * 1.4426950408889634f;
    float2* ml = reinterpret_cast<float2*>(smem + OFF_ML);
    uint32_t count = 0, own = 0, joints = 0;   // steps, items of the two kinds so far
    int base_slot = 0;                         // ring slot of the item's first tile
    const bool leader = (tid & 127) == 0;
    auto release = [&](int at) { mbar_arrive(bar(TB_E + at % NS)); };
    TreeItem it;
    for (int k = 0; item_at(k, it); ++k) {
      const Order ord = order_of(it);
      const int row = r + (ord.both ? side * BM : 0);      // of the stream
      const bool pair = PAIRS && it.heads == 2;                     // this side's KV head is its own
      const bool live = row < it.rows;
      const bool warp_live = (warp & 3) * 32 + (ord.both ? side * BM : 0) < it.rows;
      uint64_t bits = 0;
      if (live) {
        TreeSeq s;
        s.len = it.len;
        s.drafted = it.len - it.ctx;
        s.row0 = it.q_tok;
        bits = tree_bits(a, s, (it.row0 + row) >> log_group);
      }
      float m_run = -INFINITY, l_run = 0.f;                // maximum in scaled log2 units
      const int steps = ord.side_steps(side);
      for (int i = 0; i < steps; ++i, ++count) {
        wait_fast(bar(TB_SF + side), count & 1, abort_flag, a.err);
        // S complete: the step's K tile is read, and so is the V tile of the
        // side's step before, whose product was issued ahead of it (where the
        // sides share the tiles, side 1 is the later one)
        if (leader && ord.both && side == 1) {
          if (i > 0) release(base_slot + 2 * i - 1);
          release(base_slot + 2 * i);
        } else if (leader && !ord.both) {
          if (i > 0) {
            release(base_slot + 4 * i + 2 * side - 2);
            release(base_slot + 4 * i + 2 * side - 1);
          } else {
            release(base_slot + side);
          }
        }
        __syncwarp();
        tc_fence_after();
        if (!warp_live) {                                  // rows that do not exist
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(TB_PF + 2 * side));
            mbar_arrive(bar(TB_PF + 2 * side + 1));
          }
          continue;
        }
        const int t = it.t0 + (ord.both || pair ? i : 2 * i + side), k0 = t * BN;
        if (k0 + BN > it.ctx) {
          // Drafted tokens among the keys: those that the row does not see
          // become -inf in TMEM, 32 keys at a time (in the registers of the
          // loop below it would be 400 more instructions for every CTA to
          // fetch).  Drafted token d is key ctx + d.
#pragma unroll 1
          for (int c = 0; c < BN / 32; ++c) {
            const int d = k0 + 32 * c - it.ctx;            // drafted token of the first key
            uint32_t see;
            if (d >= 64) see = 0;
            else if (d >= 0) see = (uint32_t)(bits >> d);
            else if (d > -32) see = (uint32_t)(bits << -d) | ((1u << -d) - 1);
            else see = 0xffffffffu;
            if (__all_sync(0xffffffffu, see == 0xffffffffu || !live)) continue;
            float x[32];
            tmem_ld32(lane_base + col_s + c * 32, x);
            tmem_wait_ld();
            reg_fence(x);
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (!((see >> q) & 1)) x[q] = -INFINITY;
            tmem_st32(lane_base + col_s + c * 32, x);
          }
          tmem_wait_st();
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto max32 = [&](const float (&x)[32]) {
#pragma unroll
          for (int q = 0; q < 32; q += 8) {
            mx4[0] = fmax3(mx4[0], x[q], x[q + 4]);
            mx4[1] = fmax3(mx4[1], x[q + 1], x[q + 5]);
            mx4[2] = fmax3(mx4[2], x[q + 2], x[q + 6]);
            mx4[3] = fmax3(mx4[3], x[q + 3], x[q + 7]);
          }
        };
        // the maximum so far, and O scaled to it
        float m_new, base, alpha;
        auto raise = [&] {
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
          m_new = m_run;
          if (mx > m_run + kLazy || m_run == -INFINITY) m_new = mx;
          base = m_new == -INFINITY ? 0.f : m_new;         // nothing seen so far: all weights 0
          alpha = (m_new == m_run) ? 1.f : fast_exp2(m_run - base);
          if (i >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // this step's S was issued behind the last product into O, so that
            // product is complete and O can be rescaled in place
            __syncwarp();
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
              float o[32];
              tmem_ld32(lane_base + col_o + c * 32, o);
              tmem_wait_ld();
              reg_fence(o);
#pragma unroll
              for (int q = 0; q < 32; ++q) o[q] *= alpha;
              tmem_st32(lane_base + col_o + c * 32, o);
            }
            tmem_wait_st();
          }
        };
        float2 sum2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                          make_float2(0.f, 0.f)};
        // P of 32 keys into TMEM, half a tile at a time to the issuer
        auto exp32 = [&](const float (&x)[32], int c) {
          const float2 sl2x2 = make_float2(sl2, sl2), negm = make_float2(-base, -base);
          uint32_t pk[16];
#pragma unroll
          for (int q = 0; q < 32; q += 2) {
            const float2 y = ffma2(make_float2(x[q], x[q + 1]), sl2x2, negm);
            const float2 pp = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            sum2[(q >> 1) & 3] = fadd2(sum2[(q >> 1) & 3], pp);
            pk[q / 2] = pack_bf16(pp.x, pp.y);
          }
          tmem_st16(lane_base + col_s + c * 16, pk);
          if (c & 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(TB_PF + 2 * side + (c >> 1)));
          }
        };
        // the whole row in registers, four loads in flight (32 keys at a time,
        // twice from TMEM, a step took 2,700 cycles instead of 1,300)
        float x[BN / 32][32];
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) tmem_ld32(lane_base + col_s + c * 32, x[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) reg_fence(x[c]);
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) max32(x[c]);
        raise();
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) exp32(x[c], c);
        const float2 s01 = fadd2(sum2[0], sum2[1]), s23 = fadd2(sum2[2], sum2[3]);
        l_run = l_run * alpha + ((s01.x + s23.x) + (s01.y + s23.y));
        m_run = m_new;
      }
      // ---- the item's result.  Where the sides shared the rows' keys, each
      // thread joins both for half of its row's columns.
      const bool joint = !ord.both && !pair, two = ord.side_steps(1) > 0;
      wait_or_abort(bar(joint ? TB_OJ : TB_OD + side), (joint ? joints : own) & 1, abort_flag, a.err);
      // the item's last V tiles are read
      if (leader && (pair || side == (joint ? 0 : 1))) {
        if (ord.n > 1 && (joint || (pair && side == 0))) release(base_slot + 2 * ord.n - 2);
        if (!pair || side == 1) release(base_slot + 2 * ord.n - 1);
      }
      base_slot = (base_slot + 2 * ord.n) % NS;
      __syncwarp();
      tc_fence_after();
      const int g = it.g + (pair ? side : 0);
      const int out_row = (it.q_tok + ((it.row0 + row) >> log_group)) * a.num_q_heads + g * group +
                          (row & (group - 1));             // rows of q, times heads
      if ((it.t0 + it.n) * BN > it.ctx && warp_live) {
        // drafted tokens whose values the products left out, of this side's tiles
        unsigned long long left = live ? bad_v[2 * (k % NI) + (pair ? side : 0)] & bits : 0;
        if (joint && left) {
          const int edge = min(max(it.ctx / BN * BN + BN - it.ctx, 0), 64);   // drafted tokens of the first such tile
          const unsigned long long early = edge >= 64 ? ~0ull : (1ull << edge) - 1;
          left &= ((it.ctx / BN - it.t0) & 1) == side ? early : ~early;
        }
        if (__any_sync(0xffffffffu, left != 0))
          add_cleared(a, it, g, left, m_run == -INFINITY ? 0.f : m_run, lane_base + col_o, out_row);
      }
      float w0 = 1.f, w1 = 1.f, m = m_run, l = l_run;
      if (joint) {
        ml[side * BM + r] = make_float2(m_run, l_run);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(TB_ML));
        wait_or_abort(bar(TB_ML), joints & 1, abort_flag, a.err);
        __syncwarp();
        tc_fence_after();
        const float2 s0 = ml[r], s1 = ml[BM + r];
        m = fmaxf(s0.x, s1.x);
        const float base = m == -INFINITY ? 0.f : m;
        w0 = fast_exp2(s0.x - base);
        w1 = fast_exp2(s1.x - base);
        l = w0 * s0.y + w1 * s1.y;
      }
      if (warp_live) {
        const bool none = l == 0.f;                        // the row sees none of these keys
        const bool whole = it.slot < 0;
        char* piece = p.partials + ((int64_t)blockIdx.x * 2 + it.slot) * p.piece_bytes;
        const int piece_row = row + (pair && side ? it.rows : 0);
        char* to = whole ? static_cast<char*>(a.out) + (int64_t)out_row * (HD * 2) : piece + piece_row * (HD * 4);
        const float inv = none ? 0.f : 1.f / l;
        const int col0 = joint ? side * 64 : 0, cols = joint ? 64 : HD;
#pragma unroll 1
        for (int c = col0; c < col0 + cols; c += 32) {
          __syncwarp();                                    // the TMEM loads are the whole warp's
          float o[32];
          tmem_ld32(lane_base + (joint ? COL_O : col_o) + c, o);
          if (joint && two) {
            float o2[32];
            tmem_ld32(lane_base + COL_O + HD + c, o2);
            tmem_wait_ld();
            reg_fence(o);
            reg_fence(o2);
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = w0 * o[q] + w1 * o2[q];
          } else {
            tmem_wait_ld();
            reg_fence(o);   // side 0 alone: w0 = 1
          }
          if (!live) continue;
          // 32 bytes a store (a sector; 16 took twice as long) where out is so aligned
          if (whole) {
#pragma unroll
            for (int q = 0; q < 32; q += 16) {
              uint32_t v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = none ? 0u : pack_bf16(o[q + 2 * i] * inv, o[q + 2 * i + 1] * inv);
              store32(to + (c + q) * 2, v, p.wide);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 32; q += 8) {
              uint32_t v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(o[q + i]);
              store32(to + (c + q) * 4, v, true);
            }
          }
        }
        if (live && (!joint || side == 0)) {
          if (!whole)
            reinterpret_cast<float2*>(piece + (int64_t)p.piece_rows * HD * 4)[piece_row] = make_float2(m, l);
          else if (a.lse)
            a.lse[out_row] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (joint) {   // on to the next item once nobody reads this one's accumulators
        if (lane == 0) mbar_arrive(bar(TB_JD));
        wait_or_abort(bar(TB_JD), joints & 1, abort_flag, a.err);
        ++joints;
      } else {
        ++own;
      }
      item_done(k);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == W_MMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

// Joins the partials of the stream that starts in CTA blockIdx.x and goes on
// in the next ones: a warp per row, four dims per lane,
//   M = max m_i, out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// FEW (CTAs of at most four tiles): the latency of its loads counts, so the
// pieces' (m, l) are asked for before it is known how many there are, and O of
// the first eight together (12.2 -> 10.6 us for 8 drafted tokens over 777).  In
// large batches the one would be 40 MB of reads, and the other halves the warps
// that fit (198 -> 200 us for 8 sequences of 32,001).
template <bool FEW>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeMmaParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const TreeArgs& a = p.a;
  const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5);
  // the stream's first piece is its CTA's second partial, the others the first of theirs
  auto piece = [&](int i) { return p.partials + ((int64_t)(blockIdx.x + i) * 2 + (i == 0)) * p.piece_bytes; };
  auto stat = [&](int i) { return reinterpret_cast<const float2*>(piece(i) + (int64_t)p.piece_rows * HD * 4)[row]; };
  float2 mine = make_float2(-INFINITY, 0.f);
  // inside the workspace, if not this stream's
  if (FEW && row < p.piece_rows && blockIdx.x + lane < gridDim.x) mine = stat(lane);
  const MergeDesc d = p.desc[blockIdx.x];
  if (d.pieces == 0 || row >= d.rows * d.heads) return;
  if (!FEW && lane < d.pieces) mine = stat(lane);
  if (lane >= d.pieces) mine = make_float2(-INFINITY, 0.f);
  auto value = [&](int i) { return reinterpret_cast<const float4*>(piece(i))[row * (HD / 4) + lane]; };
  constexpr int kFirst = FEW ? 8 : 4;
  float4 o[kFirst];
#pragma unroll
  for (int i = 0; i < kFirst; ++i)
    if (i < d.pieces) o[i] = value(i);
  float m = mine.x;
  for (int i = 32 + lane; i < d.pieces; i += 32) m = fmaxf(m, stat(i).x);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float2 s, float4 x) {
    const float w = fast_exp2(s.x - base);
    l = fmaf(w, s.y, l);
    if (s.y != 0.f) {   // a piece of which the row sees nothing holds no O
      acc.x = fmaf(w, x.x, acc.x);
      acc.y = fmaf(w, x.y, acc.y);
      acc.z = fmaf(w, x.z, acc.z);
      acc.w = fmaf(w, x.w, acc.w);
    }
  };
#pragma unroll
  for (int i = 0; i < kFirst; ++i) {
    const float2 s = make_float2(__shfl_sync(0xffffffffu, mine.x, i), __shfl_sync(0xffffffffu, mine.y, i));
    if (i < d.pieces) add(s, o[i]);
  }
#pragma unroll 4
  for (int i = kFirst; i < d.pieces; ++i) add(stat(i), value(i));
  const bool none = l == 0.f;
  const float inv = 1.f / l;
  const int group = a.num_q_heads / a.num_kv_heads;
  const bool second = row >= d.rows;                       // the pair's other KV head
  const int of = d.row0 + row - (second ? d.rows : 0);
  const int64_t at = (int64_t)(d.q_tok + of / group) * a.num_q_heads + (d.g + second) * group + of % group;
  uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at * HD) + lane;
  *out = none ? make_uint2(0, 0)
              : make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (a.lse && lane == 0) a.lse[at] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

// Rows of a partial: up to 256, of one KV head or of a pair.
static int64_t piece_rows(int64_t rows, bool pairs) {
  const int64_t most = pairs ? 2 * rows : rows;
  return most < kTreeRows ? most : kTreeRows;
}

size_t tree_workspace_bytes(int group, int max_draft) {
  const size_t piece = (piece_rows((int64_t)max_draft * group, true) * (HD + 2) * 4 + 255) & ~(size_t)255;
  return 2 * (size_t)kTreeMaxCtas * piece + kTreeMaxCtas * sizeof(MergeDesc);
}

cudaError_t launch_tree_attention_mma(const TreeArgs& a, int num_sms, cudaStream_t stream) {
  const int group = a.num_q_heads / a.num_kv_heads;
  const int64_t rows = (int64_t)a.max_draft * group;
  TreeMmaParams p;
  p.a = a;
  p.wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  p.desc = static_cast<MergeDesc*>(a.workspace);
  p.partials = static_cast<char*>(a.workspace) + kTreeMaxCtas * sizeof(MergeDesc);
  CUtensorMap tm_q, tm_k, tm_v;
  const int64_t tiles = a.num_blocks * a.num_kv_heads;
  if (!encode_group_rows_map_bf16(&tm_q, a.q, a.num_rows, a.num_q_heads, group) ||
      !encode_latent_block_map(&tm_k, a.k_cache, tiles) || !encode_latent_block_map(&tm_v, a.v_cache, tiles))
    return cudaErrorInvalidValue;
  const int64_t row_tiles = (rows + kTreeRows - 1) / kTreeRows;
  const int64_t stages = (int64_t)a.num_seqs * a.num_kv_heads * row_tiles * ((a.max_seq_len + BN - 1) / BN);
  int grid = num_sms < kTreeMaxCtas ? num_sms : kTreeMaxCtas;
  const bool few = stages <= 4 * grid;
  // Short sequences are not cut: nothing to write in parts, and no second kernel
  // (4 sequences of 300 to 500 with 64 drafted tokens 23.4 -> 17.0 us, 50 of 131 to
  // 393 with 9 drafted, 8 query heads and one KV head 14.9 -> 11.8, 80 of 300 to 500
  // with 16 45.4 -> 36.6, one of 200 with 8 10.1 -> 8.6), but where a few of three or
  // four tiles and few rows leave CTAs without any (one of 500 with 8 drafted tokens
  // 10.2 cut, 10.8 whole); of eight tiles, 16 of 1,000 with 8 take 21.3 cut, 24.0 whole.
  p.whole = a.max_seq_len <= 2 * BN || (a.max_seq_len <= 4 * BN && (stages >= grid || rows > BM));
  // a batch that may have enough tiles, and whose KV heads and rows go in pairs
  const bool pairs = stages >= kTreePairTiles * grid && !(a.num_kv_heads & 1);
  p.q_bufs = rows <= BM && !pairs ? 2 : 1;
  p.piece_rows = (int)piece_rows(rows, pairs);
  p.piece_bytes = ((int64_t)p.piece_rows * (HD + 2) * 4 + 255) & ~255ll;
  if (stages < grid) grid = (int)stages;
  const auto kernel = pairs ? tree_mma_kernel<true> : tree_mma_kernel<false>;
  cudaError_t e = allow_dynamic_smem(kernel, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreadsT, SMEM_BYTES, stream>>>(p, tm_q, tm_k, tm_v);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.whole) return e;               // no partials
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, (p.piece_rows + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<true>, p)
             : cudaLaunchKernelEx(&cfg, tree_merge_kernel<false>, p);
}

}  // namespace pkv
