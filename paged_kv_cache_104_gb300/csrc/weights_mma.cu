// The attention each stored token got, added up, on tcgen05 (sm_103a, bf16).
//
//   weights[b][g][n] += sum over the rows of sequence b that see token n, and
//                       the query heads h of KV head g, of e^(scale q . k_n - lse)
//
// What bounds it: every stored key is read once, 256 B for 128 R multiply-adds
// and R exponentials (R rows of a KV head): HBM up to about 170 rows, the
// exponentials behind that.  Measured, 8 KV heads: 64 sequences of 2,301 with one
// row of four heads 49-50 us, 8 of 32,001 with 32 such rows 86 us, 6.2 to 6.3
// TB/s (92-94% of a plain copy's rate); on CUDA cores 593 and 4,877 us.
//
// The products are formed with the keys as the M side, S^T = K Q^T (128 keys x
// up to 256 rows), so that a thread holds all rows of one key: the sum over the
// rows stays in the thread, and one thread owns a token's running sum: no
// atomics and no partials, the same bits every time.  The tiles of 128 keys of
// the whole batch are shared out by weight to one persistent CTA per SM
// (tree_common.cuh); where a KV head has more than 256 rows, a CTA passes its
// tiles again for the next 256, the same thread on the same key.  The weights
// are those of the attention, whose streams start and end at a higher cost than
// here, so that short sequences next to long ones get more CTAs than they need:
// 64 of 2 to 128 tokens and one of 32,001, one row of four heads each, take 20.2 us
// (floor 11.3).
//
// Roles (352 threads):
//   warps 0-3 / 4-7  every other tile each: thread r owns key r (TMEM lane r)
//   warp 8           key producer: one 4 KiB TMA copy per cache block, a ring of
//                    five 32 KiB tiles
//   warp 9           tcgen05 issuer, two S^T accumulators of 256 columns
//   warp 10          works out the plan, hands the passes to the others through
//                    a ring of four, and loads their queries, lse and masks
// Every mbarrier wait is bounded; on time-out the kernel records an error,
// stops issuing work, lets its copies land, frees its TMEM and returns.
#include <cuda.h>

#include "common.cuh"
#include "host_cache.h"
#include "launch.h"
#include "tc_common.cuh"
#include "tmap.h"
#include "tree_common.cuh"

namespace pkv {
namespace {

constexpr int BK = kTreeTile, HD = 128;
constexpr int Q_BYTES = 128 * HD * 2;          // 128 query rows, 32 KiB
constexpr int TILE = BK * HD * 2;              // a K tile, 32 KiB: [8 rows][half][8 x 128 B]
constexpr int GROUP8 = 2048;                   // 8 rows of a tile
constexpr int NS = 5;                          // ring slots
constexpr int NI = 4;                          // passes in flight
constexpr int OFF_Q = 0;
constexpr int OFF_K = 2 * Q_BYTES;
constexpr int OFF_LSE = OFF_K + NS * TILE;     // 256 floats: a pass's rows (or two of 128 rows)
constexpr int OFF_MASK = OFF_LSE + kTreeRows * 4;    // [2][64] words
constexpr int OFF_SKIP = OFF_MASK + 2 * kMaxDraft * 8;   // [2]: has the pass a row that adds nothing?
constexpr int OFF_PASS = OFF_SKIP + 16;
constexpr int OFF_BAR = OFF_PASS + NI * 64;
constexpr int kSoft = 256, kThreadsW = 352;
constexpr int W_KEYS = 8, W_MMA = 9, W_PLAN = 10;
constexpr uint32_t kTmemCols = 512;

enum {
  WB_QF = 0,               // [2] queries, lse and masks there
  WB_QE = WB_QF + 2,       // [2] ... no longer read
  WB_F = WB_QE + 2,        // [NS] tile loaded
  WB_E = WB_F + NS,        // [NS] tile no longer read
  WB_PF = WB_E + NS,       // [NI] pass there
  WB_PE = WB_PF + NI,      // [NI] pass no longer read
  WB_SF = WB_PE + NI,      // [side] S complete
  WB_SE = WB_SF + 2,       // [side] S read
  WB_COUNT = WB_SE + 2
};
constexpr int SMEM_BYTES = OFF_BAR + WB_COUNT * 8 + 16;
static_assert(SMEM_BYTES <= 227 * 1024, "one CTA per SM");

struct WeightParams {
  TreeArgs a;
  int q_bufs;                // 2: no pass has more than 128 rows
};

__global__ void __launch_bounds__(kThreadsW, 1)
weights_mma_kernel(const __grid_constant__ WeightParams p, const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sbase = smem_u32(smem);
  const TreeArgs& a = p.a;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + WB_COUNT);
  int* abort_i = reinterpret_cast<int*>(tmem_slot + 1);
  volatile int* abort_flag = abort_i;
  auto bar = [&](int i) { return smem_u32(bars + i); };
  if (sbase & 1023u) {   // swizzled operand tiles need a 1 KiB-aligned base
    if (threadIdx.x == 0) record_error(a.err, DEVERR_SMEM_LAYOUT);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.num_q_heads / a.num_kv_heads;
  const int log_group = 31 - __clz(group);      // a power of two
  int* skips = reinterpret_cast<int*>(smem + OFF_SKIP);
  const int q_half = (p.q_bufs == 2 ? 1 : 2) * (Q_BYTES / 2);   // bytes of 64 columns of a pass's queries

  if (tid == 0) {
    for (int i = 0; i < WB_COUNT; ++i) {
      int count = 1;
      if (i >= WB_QE && i < WB_F) count = 1 + kSoft / 32;    // issuer, summing warps
      if (i >= WB_PE && i < WB_SF) count = 2 + kSoft / 32;   // producer, issuer, summing warps
      if (i >= WB_SE) count = 4;
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
  TreePlan<false> plan(a, warp == W_PLAN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The k-th pass, for a warp that consumes passes (false: none, or aborted).
  auto pass_at = [&](int k, TreeItem& it) {
    bool ok = wait_or_abort(bar(WB_PF + k % NI), (k / NI) & 1, abort_flag, a.err);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    it = *reinterpret_cast<const TreeItem*>(smem + OFF_PASS + (k % NI) * 64);
    return it.n > 0;
  };
  auto pass_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(WB_PE + k % NI));
  };
  auto warp_wait = [&](int b, uint32_t parity) {
    return (bool)__all_sync(0xffffffffu, wait_fast(bar(b), parity, abort_flag, a.err));
  };

  if (warp == W_PLAN) {
    // ------------------------------------------------------------------ plan, queries
    int made = 0, loaded = 0;        // passes handed out; queries asked for
    bool last = false;
    TreeItem it;
    it.rows = 0;
    int row0 = 0;
    long long since = clock64();
    while (!last || loaded < made - 1) {
      bool moved = false;
      if (!last && (made < NI || __all_sync(0xffffffffu, mbar_try_wait(bar(WB_PE + made % NI), ((made / NI) - 1) & 1)))) {
        if (row0 >= it.rows) {       // the item's rows are handed out: the next one
          it = plan.next();
          row0 = 0;
          last = it.n == 0;
        }
        TreeItem pass = it;
        pass.row0 = row0;
        pass.rows = min(it.rows - row0, kTreeRows);
        row0 += kTreeRows;
        if (lane == 0) *reinterpret_cast<TreeItem*>(smem + OFF_PASS + (made % NI) * 64) = pass;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(WB_PF + made % NI));
        ++made;
        moved = true;
      }
      if (loaded < made - (last ? 1 : 0)) {
        const int qb = loaded % p.q_bufs;
        if (loaded < p.q_bufs ||
            __all_sync(0xffffffffu, mbar_try_wait(bar(WB_QE + qb), ((loaded / p.q_bufs) - 1) & 1))) {
          // a pass's slot is written again only once its queries were used
          const TreeItem x = *reinterpret_cast<const TreeItem*>(smem + OFF_PASS + (loaded % NI) * 64);
          const int tok0 = x.row0 >> log_group, drafted = x.len - x.ctx;
          float* lse = reinterpret_cast<float*>(smem + OFF_LSE) + qb * 128;
          unsigned long long* words = reinterpret_cast<unsigned long long*>(smem + OFF_MASK) + qb * kMaxDraft;
          bool skip = false;
          for (int r = lane; r < x.rows; r += 32) {
            const int row = x.row0 + r;
            const float v = a.lse[(int64_t)(x.q_tok + (row >> log_group)) * a.num_q_heads + x.g * group +
                                  (row & (group - 1))];
            lse[r] = v * 1.4426950408889634f;
            skip |= v == -INFINITY;
          }
          skip = __any_sync(0xffffffffu, skip);
          if (lane == 0) skips[qb] = skip;
          TreeSeq s;
          s.len = x.len;
          s.drafted = drafted;
          s.row0 = x.q_tok;
          for (int t = lane; t < (x.rows + group - 1) >> log_group; t += 32) words[t] = tree_bits(a, s, tok0 + t);
          __syncwarp();
          if (lane == 0) {
            const int parts = x.rows > 128 ? 2 : 1;
            mbar_arrive_expect_tx(bar(WB_QF + qb), parts * Q_BYTES);
            for (int i = 0; i < parts; ++i)
              for (int h = 0; h < 2; ++h)
                tma_load_3d(sbase + OFF_Q + qb * Q_BYTES + h * q_half + i * (Q_BYTES / 2), &tm_q, bar(WB_QF + qb),
                            64 * h, x.g * group, x.q_tok + tok0 + (i * 128 >> log_group));
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
        mbar_wait(bar(WB_QF + k % p.q_bufs), (k / p.q_bufs) & 1, nullptr);
  } else if (warp == W_KEYS) {
    // ------------------------------------------------------------------ key producer
    if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
    // keys that are read once leave the L2 first; those of several passes are read again
    const uint64_t once = policy_evict_first(), again = policy_evict_normal();
    int pos = 0;                     // ring position
    TreeItem it;
    bool ok = !kWithholdCopies;      // (a test's build: the others' waits run out, nothing is in flight)
    for (int k = 0; ok && pass_at(k, it); ++k) {
      const int32_t* row = a.block_table + (int64_t)it.b * a.max_blocks_per_seq;
      const int blocks = (it.len + kBlockSize - 1) / kBlockSize;
      const uint64_t policy = (it.len - it.ctx) * group <= kTreeRows ? once : again;
      auto ids_of = [&](int window) {   // block ids of four tiles, one per lane
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
      for (int t = it.t0; t < it.t0 + it.n; ++t, ++pos) {
        const int slot = pos % NS;
        if (pos >= NS) ok = warp_wait(WB_E + slot, ((pos / NS) - 1) & 1);
        if (!ok) break;
        if ((t >> 2) > window) {
          ids = next_ids;
          next_ids = ids_of(++window + 1);
        }
        const int mine = __shfl_sync(0xffffffffu, ids, (t & 3) * 8 + (lane & 7));
        const int nb = min(8, blocks - 8 * t);
        if (lane == 0) mbar_arrive_expect_tx(bar(WB_F + slot), nb * 2 * GROUP8);
        __syncwarp();
        if (lane < nb)
          tma_load_4d(sbase + OFF_K + slot * TILE + lane * 2 * GROUP8, &tm_k, bar(WB_F + slot), 0, 0, 0,
                      2 * (mine * a.num_kv_heads + it.g), policy);
      }
      pass_done(k);
    }
    if (*abort_flag)   // let the copies already issued land
      for (int i = max(0, pos - NS); i < pos; ++i) mbar_wait(bar(WB_F + i % NS), (i / NS) & 1, nullptr);
  } else if (warp == W_MMA) {
    // ------------------------------------------------------------------ issuer
    const uint64_t k_desc = make_sw128_desc(sbase + OFF_K, 16, GROUP8);
    const uint64_t q_desc = make_sw128_desc(sbase + OFF_Q, 16, 1024);
    int slot = 0;                    // ring position: slot and parity
    uint32_t par = 0, uses[2] = {0, 0};
    TreeItem it;
    bool ok = true;
    for (int k = 0; ok && pass_at(k, it); ++k) {
      it.n = __shfl_sync(0xffffffffu, it.n, 0);         // known to be the same in every lane
      it.rows = __shfl_sync(0xffffffffu, it.rows, 0);
      const int qb = k % p.q_bufs;
      const uint32_t idesc = make_idesc(false, BK, (it.rows + 15) & ~15);
      ok = warp_wait(WB_QF + qb, (k / p.q_bufs) & 1);
      const uint64_t q = q_desc + (uint32_t)(qb * (Q_BYTES >> 4));
      for (int j = 0; j < it.n && ok; ++j) {
        const int side = j & 1;
        if (uses[side] > 0) ok = warp_wait(WB_SE + side, (uses[side] - 1) & 1);
        if (ok) ok = warp_wait(WB_F + slot, par);
        if (!ok) break;
        tc_fence_after();
        mma_ss8_e(tmem + side * kTreeRows, k_desc + (uint32_t)(slot * (TILE >> 4)), q, idesc, 1024 >> 4, q_half >> 4);
        commit_e(bar(WB_SF + side));   // the summing warps free the tile's slot
        ++uses[side];
        if (++slot == NS) {
          slot = 0;
          par ^= 1;
        }
      }
      if (ok) commit_e(bar(WB_QE + qb));
      pass_done(k);
    }
  } else {
    // ------------------------------------------------------------------ sums over the rows
    const int side = warp >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + side * kTreeRows;
    const float sl2 = a.scale * 1.4426950408889634f;
    uint32_t count = 0;
    int base = 0;                    // ring slot of the pass's first tile
    TreeItem it;
    for (int k = 0; pass_at(k, it); ++k) {
      const int qb = k % p.q_bufs;
      wait_or_abort(bar(WB_QF + qb), (k / p.q_bufs) & 1, abort_flag, a.err);
      __syncwarp();
      const float* lse = reinterpret_cast<const float*>(smem + OFF_LSE) + qb * 128;
      const unsigned long long* words = reinterpret_cast<const unsigned long long*>(smem + OFF_MASK) + qb * kMaxDraft;
      const bool skip = skips[qb] != 0;
      float* line = a.weights + ((int64_t)it.b * a.num_kv_heads + it.g) * a.weights_len;
      for (int j = side; j < it.n; j += 2, ++count) {
        const int key = (it.t0 + j) * BK + r, d = key - it.ctx;
        const bool there = key < it.len;
        const float old = there ? line[key] : 0.f;
        // does some row not see some key of this warp?
        const bool masked = __any_sync(0xffffffffu, d >= 0);
        wait_fast(bar(WB_SF + side), count & 1, abort_flag, a.err);
        if (r == 0) mbar_arrive(bar(WB_E + (base + j) % NS));
        __syncwarp();
        tc_fence_after();
        float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // 2^(s sl2 - lse) of two rows
        auto weight2 = [&](float x, float y, float lse_x, float lse_y) {
          const float2 z = ffma2(make_float2(x, y), make_float2(sl2, sl2), make_float2(-lse_x, -lse_y));
          return make_float2(fast_exp2(z.x), fast_exp2(z.y));
        };
        const int plain = masked || skip ? 0 : it.rows & ~31;   // rows whose sums need no care
        for (int c = 0; c < plain; c += 32) {
          float x[32];
          tmem_ld32(lane_base + c, x);
          tmem_wait_ld();
          reg_fence(x);
#pragma unroll
          for (int q = 0; q < 32; q += 4) {
            const float4 e = *reinterpret_cast<const float4*>(lse + c + q);
            sum[q >> 1 & 2] = fadd2(sum[q >> 1 & 2], weight2(x[q], x[q + 1], e.x, e.y));
            sum[(q >> 1 & 2) + 1] = fadd2(sum[(q >> 1 & 2) + 1], weight2(x[q + 2], x[q + 3], e.z, e.w));
          }
        }
        // the rest eight rows at a time: those behind the last, those that do
        // not see this key and those whose lse is -inf (their scores may be
        // NaN) add nothing.  A key of the context is seen by
        // all, the pass's first token in bit 0.  (The words looked up row by row,
        // short sequences took two to three times as long: 64 of 1 to 300 with 16
        // drafted tokens 29 us, against 14.8.)
        uint64_t seers = ~0ull;
        if (masked && d >= 0) {
          seers = 0;
          if (d < kMaxDraft) {
            const int tokens = it.rows >> log_group;
#pragma unroll 4
            for (int i = 0; i < tokens; ++i) seers |= ((words[i] >> d) & 1) << i;
          }
        }
#pragma unroll 1
        for (int c = plain; c < it.rows; c += 8) {
          float x[8];
          tmem_ld8(lane_base + c, x);
          tmem_wait_ld();
          reg_fence(x);
#pragma unroll
          for (int q = 0; q < 8; q += 2) {
            const float2 e = *reinterpret_cast<const float2*>(lse + c + q);
            const float2 y = weight2(x[q], x[q + 1], e.x, e.y);
            const bool see0 = c + q < it.rows && (seers >> ((c + q) >> log_group) & 1) && e.x != -INFINITY;
            const bool see1 = c + q + 1 < it.rows && (seers >> ((c + q + 1) >> log_group) & 1) && e.y != -INFINITY;
            sum[q >> 1] = fadd2(sum[q >> 1], make_float2(see0 ? y.x : 0.f, see1 ? y.y : 0.f));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(WB_SE + side));
        const float2 s01 = fadd2(sum[0], sum[1]), s23 = fadd2(sum[2], sum[3]);
        if (there) line[key] = old + ((s01.x + s23.x) + (s01.y + s23.y));
      }
      base = (base + it.n) % NS;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(WB_QE + qb));
      pass_done(k);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

}  // namespace

cudaError_t launch_kv_add_weights_mma(const TreeArgs& a, int num_sms, cudaStream_t stream) {
  const int group = a.num_q_heads / a.num_kv_heads;
  WeightParams p;
  p.a = a;
  p.q_bufs = (int64_t)a.max_draft * group <= 128 ? 2 : 1;
  CUtensorMap tm_q, tm_k;
  if (!encode_group_rows_map_bf16(&tm_q, a.q, a.num_rows, a.num_q_heads, group) ||
      !encode_latent_block_map(&tm_k, a.k_cache, a.num_blocks * a.num_kv_heads))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_dynamic_smem(weights_mma_kernel, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int64_t stages = (int64_t)a.num_seqs * a.num_kv_heads * ((a.max_seq_len + BK - 1) / BK);
  const int grid = (int)(stages < num_sms ? stages : num_sms);
  weights_mma_kernel<<<grid, kThreadsW, SMEM_BYTES, stream>>>(p, tm_q, tm_k);
  return cudaGetLastError();
}

}  // namespace pkv
