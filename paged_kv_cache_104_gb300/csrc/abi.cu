// C ABI of libpagedkv.so: argument validation, workspace layout, dispatch to
// the kernel launchers, and the per-device error word.  The declarations and
// their contracts are in include/pagedkv.h.
#include <climits>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <mutex>

#include "host_cache.h"
#include "launch.h"
#include "pagedkv.h"

namespace {

constexpr int kMaxDevices = 64;

// One error word per device: kernels record the first device-side error here.
__device__ int g_pkv_error_word;

// Per device: the context the cached state was resolved in, the device-side
// address of the error word and the SM count.  Resolved on the first call
// with that device current, and again after the context changes (a device
// reset destroys the primary context and the module with it).  Guarded by a
// mutex: host threads may make their first calls at the same time.
struct DeviceState {
  uint64_t ctx;
  int* err;
  int num_sms;
};
DeviceState g_dev[kMaxDevices];
std::mutex g_dev_mu;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int elem_bytes(pkv_dtype d) { return d == PKV_BF16 ? 2 : 4; }

bool dtype_ok(pkv_dtype d) { return d == PKV_F32 || d == PKV_BF16; }

pkv_status device_state(int** err, int* num_sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PKV_ECUDA;
  std::lock_guard<std::mutex> lock(g_dev_mu);
  DeviceState& s = g_dev[dev];
  uint64_t ctx = pkv::current_context_id();
  if (!s.err || ctx == 0 || ctx != s.ctx) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_pkv_error_word) != cudaSuccess) return PKV_ECUDA;
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return PKV_ECUDA;
    s.num_sms = sms;
    s.err = static_cast<int*>(p);
    s.ctx = pkv::current_context_id();   // now that the runtime made one current
  }
  *err = s.err;
  *num_sms = s.num_sms;
  return PKV_OK;
}

int max_splits_for(int max_seq_len, int split_tokens = pkv::kSplitTokens) {
  return (max_seq_len + split_tokens - 1) / split_tokens;
}

// Partial slots per (sequence, query head) row: a sequence of n tokens gives
// at most ceil(n / split_tokens) partials in splits, and at most one more in
// the balanced walk (each CTA's share of at least split_tokens tokens may
// start inside a sequence).  One slot: no partials at all.
int partial_slots_for(int max_seq_len, int split_tokens = pkv::kSplitTokens) {
  const int s = max_splits_for(max_seq_len, split_tokens);
  return s <= 1 ? 1 : s + 1;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

size_t partials_bytes(int num_seqs, int num_q_heads, int head_dim, int slots) {
  if (slots <= 1) return 0;
  const size_t rows = (size_t)num_seqs * num_q_heads * slots;
  return align256(rows * head_dim * sizeof(float)) + align256(rows * 2 * sizeof(float)) +
         align256((size_t)num_seqs * num_q_heads * sizeof(int));
}

// The decode workspace, in order: fp32 partial rows [rows][head_dim], their
// (m, l) pairs [rows][2], and the partial count per (sequence, head) [count],
// rows = num_seqs * num_q_heads * partial slots.
struct Partials {
  float* acc;
  float* ml;
  int* np;
};
Partials carve_partials(void* workspace, size_t rows, int head_dim) {
  char* ws = static_cast<char*>(workspace);
  const size_t acc_b = align256(rows * head_dim * sizeof(float));
  const size_t ml_b = align256(rows * 2 * sizeof(float));
  return {reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + acc_b),
          reinterpret_cast<int*>(ws + acc_b + ml_b)};
}

// Shape checks shared by decode and prefill.
pkv_status check_heads(int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                       pkv_dtype dtype) {
  if (!dtype_ok(dtype)) return PKV_EDTYPE;
  if (num_q_heads < 1 || num_kv_heads < 1 || head_dim < 1 || block_size < 1) return PKV_EINVAL;
  if (num_q_heads % num_kv_heads != 0) return PKV_EINVAL;
  if (block_size != pkv::kBlockSize) return PKV_EUNSUPPORTED;
  const int group = num_q_heads / num_kv_heads;
  if (!pkv::decode_supported(dtype == PKV_BF16, head_dim, group) &&
      !pkv::decode_mma_supported(dtype == PKV_BF16, head_dim, group))
    return PKV_EUNSUPPORTED;
  return PKV_OK;
}

}  // namespace

extern "C" {

int pkv_abi_version(void) { return 2; }

}  // extern "C"

namespace {
// the span record of later side-by-side calls (pkv_set_span_buffer)
std::atomic<unsigned long long*> g_span_buf{nullptr};
}  // namespace

extern "C" {

pkv_status pkv_set_span_buffer(unsigned long long* buf) {
  if (reinterpret_cast<uintptr_t>(buf) & 7u) return PKV_EINVAL;
  g_span_buf.store(buf);
  return PKV_OK;
}

const char* pkv_status_str(pkv_status s) {
  switch (s) {
    case PKV_OK: return "ok";
    case PKV_EINVAL: return "invalid argument";
    case PKV_EDTYPE: return "unknown dtype";
    case PKV_ERANGE: return "size out of range";
    case PKV_ECUDA: return "CUDA runtime error";
    case PKV_EUNSUPPORTED: return "unsupported shape";
  }
  return "unknown status";
}

pkv_status pkv_get_device_error(int* code, int clear) {
  if (!code) return PKV_EINVAL;
  int* err = nullptr;
  int sms = 0;
  pkv_status st = device_state(&err, &sms);
  if (st != PKV_OK) return st;
  if (cudaDeviceSynchronize() != cudaSuccess) return PKV_ECUDA;
  if (cudaMemcpy(code, err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return PKV_ECUDA;
  if (clear && cudaMemset(err, 0, sizeof(int)) != cudaSuccess) return PKV_ECUDA;
  return PKV_OK;
}

pkv_status pkv_kv_append(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                         const int64_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
                         int num_kv_heads, int head_dim, int block_size, pkv_dtype dtype,
                         pkv_stream_t stream) {
  if (!dtype_ok(dtype)) return PKV_EDTYPE;
  if (num_tokens < 0 || num_blocks < 1 || num_kv_heads < 1 || head_dim < 1 || block_size < 1)
    return PKV_EINVAL;
  if (block_size != pkv::kBlockSize) return PKV_EUNSUPPORTED;
  const int row_bytes = head_dim * elem_bytes(dtype);
  if (row_bytes % 16 != 0) return PKV_EUNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !slot_mapping) return PKV_EINVAL;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return PKV_EINVAL;
  int* err = nullptr;
  int sms = 0;
  pkv_status st = device_state(&err, &sms);
  if (st != PKV_OK) return st;
  pkv::AppendArgs a{k_new, v_new, k_cache, v_cache, slot_mapping, num_tokens, num_blocks,
                    num_kv_heads, row_bytes, err};
  return pkv::launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

}  // extern "C"

namespace {

// One token stride of a rotating append: 0 is the contiguous layout.
bool token_stride(int64_t given, int64_t heads, int head_dim, int elem, int64_t* out) {
  const int64_t least = heads * head_dim;
  *out = given == 0 ? least : given;
  return *out >= least && (*out * elem) % 16 == 0;
}

// Validates a rotating append and fills its launch arguments (num_tokens > 0).
pkv_status rope_append_prepare(const pkv_rope_append_args& x, pkv::RopeAppendArgs* out) {
  const int elem = elem_bytes(x.dtype);
  if (!x.k_new || !x.v_new || !x.k_cache || !x.v_cache || !x.slot_mapping) return PKV_EINVAL;
  if (!x.q != !x.q_out) return PKV_EINVAL;
  if (x.q && x.num_q_heads < 1) return PKV_EINVAL;
  for (const void* p : {(const void*)x.q_out, x.q, x.k_new, x.v_new, (const void*)x.k_cache,
                        (const void*)x.v_cache, (const void*)x.cos_sin})
    if (!aligned16(p)) return PKV_EINVAL;
  if (reinterpret_cast<uintptr_t>(x.slot_mapping) & 7u) return PKV_EINVAL;
  pkv::RopeAppendArgs a{};
  const int hq = x.q ? x.num_q_heads : 0;
  if (!token_stride(x.k_stride, x.num_kv_heads, x.head_dim, elem, &a.k_stride) ||
      !token_stride(x.v_stride, x.num_kv_heads, x.head_dim, elem, &a.v_stride) ||
      (x.q && (!token_stride(x.q_stride, hq, x.head_dim, elem, &a.q_stride) ||
               !token_stride(x.q_out_stride, hq, x.head_dim, elem, &a.q_out_stride))))
    return PKV_EINVAL;
  if (x.q == x.q_out && a.q_stride != a.q_out_stride) return PKV_EINVAL;
  if (x.cos_sin) {
    if (!x.positions || (reinterpret_cast<uintptr_t>(x.positions) & 3u) || x.num_positions < 1)
      return PKV_EINVAL;
    if (x.num_axes < 1 || x.num_axes > PKV_MAX_ROPE_AXES || (x.num_axes > 1 && !x.pair_axis))
      return PKV_EINVAL;
    if (x.rot_dim < 2 || x.rot_dim % 2 != 0 || x.rot_dim > x.head_dim) return PKV_EINVAL;
    if (x.rot_dim > PKV_MAX_ROT_DIM) return PKV_EUNSUPPORTED;
    a.rope.cos_sin = x.cos_sin;
    a.rope.num_positions = x.num_positions;
    a.rope.positions = x.positions;
    a.rope.num_axes = x.num_axes;
    a.rope.rot_dim = x.rot_dim;
    a.rope.interleaved = x.interleaved != 0;
    for (int i = 0; x.pair_axis && i < x.rot_dim / 2; ++i) {
      if (x.pair_axis[i] >= x.num_axes) return PKV_EINVAL;
      a.rope.pair_axis[i] = x.pair_axis[i];
    }
  }
  a.q_out = x.q_out;
  a.q = x.q;
  a.k_new = x.k_new;
  a.v_new = x.v_new;
  a.k_cache = x.k_cache;
  a.v_cache = x.v_cache;
  a.k_scale = x.k_scale;
  a.v_scale = x.v_scale;
  a.slot_mapping = x.slot_mapping;
  a.num_tokens = x.num_tokens;
  a.num_blocks = x.num_blocks;
  a.num_q_heads = hq;
  a.num_kv_heads = x.num_kv_heads;
  a.head_dim = x.head_dim;
  *out = a;
  return PKV_OK;
}

// Sizes every rotating append checks before its pointers.
pkv_status rope_append_sizes(const pkv_rope_append_args& x) {
  if (!dtype_ok(x.dtype)) return PKV_EDTYPE;
  if (x.num_tokens < 0 || x.num_blocks < 1 || x.num_kv_heads < 1 || x.head_dim < 1 ||
      x.block_size < 1)
    return PKV_EINVAL;
  if (x.block_size != pkv::kBlockSize) return PKV_EUNSUPPORTED;
  if (x.num_tokens > INT_MAX) return PKV_ERANGE;
  return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_kv_append_rope(const pkv_rope_append_args* x, pkv_stream_t stream) {
  if (!x) return PKV_EINVAL;
  pkv_status st = rope_append_sizes(*x);
  if (st != PKV_OK) return st;
  if ((x->head_dim * elem_bytes(x->dtype)) % 16 != 0 || x->head_dim > PKV_MAX_APPEND_HEAD_DIM)
    return PKV_EUNSUPPORTED;
  if (x->num_tokens == 0) return PKV_OK;
  if (!x->cos_sin) return PKV_EINVAL;
  pkv::RopeAppendArgs a;
  st = rope_append_prepare(*x, &a);
  if (st != PKV_OK) return st;
  int sms = 0;
  st = device_state(&a.err, &sms);
  if (st != PKV_OK) return st;
  return pkv::launch_kv_append_rope(a, x->dtype == PKV_BF16,
                                    reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

pkv_status pkv_kv_append_fp8_block(const pkv_rope_append_args* x, pkv_stream_t stream) {
  if (!x) return PKV_EINVAL;
  pkv_status st = rope_append_sizes(*x);
  if (st != PKV_OK) return st;
  if (x->dtype != PKV_BF16) return PKV_EUNSUPPORTED;
  if (x->num_tokens == 0) return PKV_OK;
  if (!x->k_scale || !x->v_scale || (x->q && !x->cos_sin)) return PKV_EINVAL;
  if (x->head_dim % 16 != 0 || x->head_dim > 128) return PKV_EUNSUPPORTED;
  pkv::RopeAppendArgs a;
  st = rope_append_prepare(*x, &a);
  if (st != PKV_OK) return st;
  if (!pkv::append_fp8_block_supported(a)) return PKV_EUNSUPPORTED;
  int sms = 0;
  st = device_state(&a.err, &sms);
  if (st != PKV_OK) return st;
  return pkv::launch_kv_append_fp8_block(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

size_t pkv_decode_workspace_bytes(int num_seqs, int num_q_heads, int head_dim, int max_seq_len) {
  if (num_seqs < 1 || num_q_heads < 1 || head_dim < 1 || max_seq_len < 1) return 0;
  return partials_bytes(num_seqs, num_q_heads, head_dim, partial_slots_for(max_seq_len));
}

}  // extern "C"

namespace {

// Shared by paged_decode_attention and its fused-append form (k_new != null).
// Validates a decode call and fills its launch arguments; launches nothing.
pkv_status decode_prepare(pkv::DecodeArgs* out_args, int* out_sms, void* out, const void* q,
                          const void* k_new, const void* v_new, const void* k_cache,
                          const void* v_cache, const int32_t* block_table,
                          const int32_t* seq_lens, int num_seqs, int max_blocks_per_seq,
                          int max_seq_len, int64_t num_blocks, int num_q_heads, int num_kv_heads,
                          int head_dim, int block_size, float scale, void* workspace,
                          size_t workspace_bytes, pkv_dtype dtype) {
  pkv_status st = check_heads(num_q_heads, num_kv_heads, head_dim, block_size, dtype);
  if (st != PKV_OK) return st;
  if (num_seqs < 0 || max_blocks_per_seq < 1 || max_seq_len < 1 || num_blocks < 1)
    return PKV_EINVAL;
  if (num_seqs == 0) return PKV_OK;
  if (num_seqs > PKV_MAX_SEQS) return PKV_ERANGE;
  if ((int64_t)max_seq_len > (int64_t)max_blocks_per_seq * block_size) return PKV_EINVAL;
  if (!isfinite(scale)) return PKV_EINVAL;
  if (!out || !q || !k_cache || !v_cache || !block_table || !seq_lens) return PKV_EINVAL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return PKV_EINVAL;
  const size_t need = pkv_decode_workspace_bytes(num_seqs, num_q_heads, head_dim, max_seq_len);
  if (workspace_bytes < need) return PKV_ERANGE;
  if ((int64_t)num_seqs * num_kv_heads * max_splits_for(max_seq_len) >= (int64_t)INT_MAX)
    return PKV_ERANGE;  // the kernels' unit list is indexed by int
  if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))) return PKV_EINVAL;
  int* err = nullptr;
  int sms = 0;
  st = device_state(&err, &sms);
  if (st != PKV_OK) return st;
  const int s = partial_slots_for(max_seq_len);
  const Partials part = carve_partials(workspace, (size_t)num_seqs * num_q_heads * s, head_dim);
  pkv::DecodeArgs a{};
  a.out = out;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.ws_acc = need ? part.acc : nullptr;
  a.ws_ml = need ? part.ml : nullptr;
  a.ws_np = need ? part.np : nullptr;
  a.err = err;
  a.num_seqs = num_seqs;
  a.bt_stride = max_blocks_per_seq;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_seq_len = max_seq_len;
  a.max_splits = s;
  a.split_tokens = pkv::kSplitTokens;
  a.num_blocks = num_blocks;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.scale = scale;
  a.chunk_prior = -1;
  a.is_bf16 = dtype == PKV_BF16;
  a.k_new = k_new;
  a.v_new = v_new;
  *out_args = a;
  *out_sms = sms;
  return PKV_OK;
}

// Launches a prepared decode; sm_budget bounds its persistent grid, and
// dependent launches it as the programmatic dependent of the stream's
// previous kernel (tensor-core path only).
pkv_status decode_launch(const pkv::DecodeArgs& a, int sm_budget, bool dependent,
                         cudaStream_t s_) {
  if (a.num_seqs == 0) return PKV_OK;   // nothing was prepared: an empty batch
  const cudaError_t e =
      pkv::decode_mma_supported(a.is_bf16, a.head_dim, a.num_q_heads / a.num_kv_heads)
          ? pkv::launch_paged_decode_mma(a, sm_budget, s_, dependent)
          : pkv::launch_paged_decode(a, sm_budget, s_);
  return e == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

pkv_status decode_impl(void* out, const void* q, const void* k_new, const void* v_new,
                       const void* k_cache, const void* v_cache, const int32_t* block_table,
                       const int32_t* seq_lens, int num_seqs, int max_blocks_per_seq,
                       int max_seq_len, int64_t num_blocks, int num_q_heads, int num_kv_heads,
                       int head_dim, int block_size, float scale, void* workspace,
                       size_t workspace_bytes, pkv_dtype dtype, pkv_stream_t stream) {
  pkv::DecodeArgs a{};
  int sms = 0;
  const pkv_status st = decode_prepare(&a, &sms, out, q, k_new, v_new, k_cache, v_cache,
                                       block_table, seq_lens, num_seqs, max_blocks_per_seq,
                                       max_seq_len, num_blocks, num_q_heads, num_kv_heads,
                                       head_dim, block_size, scale, workspace, workspace_bytes,
                                       dtype);
  if (st != PKV_OK) return st;
  return decode_launch(a, sms, false, reinterpret_cast<cudaStream_t>(stream));
}

// Validates a chunked-prefill call; launches nothing.
pkv_status prefill_check(const void* out, const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* block_table_row, int max_blocks, int prior_len,
                         int chunk_len, int64_t num_blocks, int num_q_heads, int num_kv_heads,
                         int head_dim, int block_size, float scale, pkv_dtype dtype) {
  pkv_status st = check_heads(num_q_heads, num_kv_heads, head_dim, block_size, dtype);
  if (st != PKV_OK) return st;
  if (max_blocks < 1 || prior_len < 0 || chunk_len < 0 || num_blocks < 1) return PKV_EINVAL;
  if (chunk_len == 0) return PKV_OK;
  if ((int64_t)prior_len + chunk_len > (int64_t)max_blocks * block_size) return PKV_EINVAL;
  if (!isfinite(scale)) return PKV_EINVAL;
  if (!out || !q || !k_cache || !v_cache || !block_table_row) return PKV_EINVAL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(block_table_row) & 3u))
    return PKV_EINVAL;
  if (!(dtype == PKV_BF16 && head_dim == 128) && chunk_len > PKV_MAX_SEQS) return PKV_ERANGE;
  return PKV_OK;
}

// Launches a checked chunked prefill (chunk_len > 0).  persistent_ctas > 0
// asks the two-head tensor-core kernel for that many persistent CTAs.
pkv_status prefill_launch(void* out, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_table_row, int max_blocks, int prior_len,
                          int chunk_len, int64_t num_blocks, int num_q_heads, int num_kv_heads,
                          int head_dim, float scale, pkv_dtype dtype, int persistent_ctas,
                          cudaStream_t s) {
  int* err = nullptr;
  int sms = 0;
  pkv_status st = device_state(&err, &sms);
  if (st != PKV_OK) return st;
  if (dtype == PKV_BF16 && head_dim == 128) {
    pkv::PrefillArgs a{out, q, k_cache, v_cache, block_table_row, max_blocks, prior_len, chunk_len,
                       num_blocks, num_q_heads, num_kv_heads, scale, err};
    return pkv::launch_prefill_pair(a, s, persistent_ctas) == cudaSuccess ? PKV_OK : PKV_ECUDA;
  }
  // CUDA-core path: every chunk row is one query over its causal prefix, run
  // as a single split so no workspace is needed.
  const int total = prior_len + chunk_len;
  pkv::DecodeArgs a{};
  a.out = const_cast<void*>(out);
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table_row;
  a.seq_lens = nullptr;
  a.err = err;
  a.num_seqs = chunk_len;
  a.bt_stride = 0;
  a.max_blocks_per_seq = max_blocks;
  a.max_seq_len = total;
  a.max_splits = 1;
  a.split_tokens = ((total + pkv::kSplitTokens - 1) / pkv::kSplitTokens) * pkv::kSplitTokens;
  a.num_blocks = num_blocks;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.scale = scale;
  a.chunk_prior = prior_len;
  a.is_bf16 = dtype == PKV_BF16;
  return pkv::launch_paged_decode(a, sms, s) == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

}  // namespace

extern "C" {

pkv_status pkv_paged_decode_attention(void* out, const void* q, const void* k_cache,
                                      const void* v_cache, const int32_t* block_table,
                                      const int32_t* seq_lens, int num_seqs,
                                      int max_blocks_per_seq, int max_seq_len,
                                      int64_t num_blocks, int num_q_heads, int num_kv_heads,
                                      int head_dim, int block_size, float scale,
                                      void* workspace, size_t workspace_bytes, pkv_dtype dtype,
                                      pkv_stream_t stream) {
  return decode_impl(out, q, nullptr, nullptr, k_cache, v_cache, block_table, seq_lens, num_seqs,
                     max_blocks_per_seq, max_seq_len, num_blocks, num_q_heads, num_kv_heads,
                     head_dim, block_size, scale, workspace, workspace_bytes, dtype, stream);
}

pkv_status pkv_paged_decode_attention_append(void* out, const void* q, const void* k_new,
                                             const void* v_new, void* k_cache, void* v_cache,
                                             const int32_t* block_table, const int32_t* seq_lens,
                                             int num_seqs, int max_blocks_per_seq,
                                             int max_seq_len, int64_t num_blocks,
                                             int num_q_heads, int num_kv_heads, int head_dim,
                                             int block_size, float scale, void* workspace,
                                             size_t workspace_bytes, pkv_dtype dtype,
                                             pkv_stream_t stream) {
  if (!dtype_ok(dtype)) return PKV_EDTYPE;
  if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0) return PKV_EINVAL;
  if (!pkv::decode_mma_supported(dtype == PKV_BF16, head_dim, num_q_heads / num_kv_heads))
    return PKV_EUNSUPPORTED;
  if (num_seqs > 0 && (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)))
    return PKV_EINVAL;
  return decode_impl(out, q, k_new, v_new, k_cache, v_cache, block_table, seq_lens, num_seqs,
                     max_blocks_per_seq, max_seq_len, num_blocks, num_q_heads, num_kv_heads,
                     head_dim, block_size, scale, workspace, workspace_bytes, dtype, stream);
}

pkv_status pkv_kv_append_fp8(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                             const float* k_scale, const float* v_scale,
                             const int64_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
                             int num_kv_heads, int head_dim, int block_size, pkv_stream_t stream) {
  if (num_tokens < 0 || num_blocks < 1 || num_kv_heads < 1 || head_dim < 1 || block_size < 1)
    return PKV_EINVAL;
  if (block_size != pkv::kBlockSize || head_dim % 16 != 0) return PKV_EUNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !slot_mapping || !k_scale || !v_scale)
    return PKV_EINVAL;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) ||
      (reinterpret_cast<uintptr_t>(k_scale) & 3u) || (reinterpret_cast<uintptr_t>(v_scale) & 3u))
    return PKV_EINVAL;
  int* err = nullptr;
  int sms = 0;
  pkv_status st = device_state(&err, &sms);
  if (st != PKV_OK) return st;
  pkv::AppendFp8Args a{k_new, v_new, k_cache, v_cache, k_scale, v_scale, slot_mapping,
                       num_tokens, num_blocks, num_kv_heads, head_dim, err};
  return pkv::launch_kv_append_fp8(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

}  // extern "C"

namespace {

// Validates a decode call over an fp8 cache (either kind of scale) and fills
// its launch arguments but for the scales (scales_ok: given and aligned);
// num_seqs 0 in them: nothing to do.
pkv_status fp8_decode_prepare(pkv::DecodeArgs* out_args, int* sms, bool scales_ok,
                              int split_tokens, void* out, const void* q, const void* k_cache,
                              const void* v_cache, const int32_t* block_table,
                              const int32_t* seq_lens, int num_seqs,
                              int max_blocks_per_seq, int max_seq_len, int64_t num_blocks,
                              int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                              float scale, void* workspace, size_t workspace_bytes) {
  *out_args = pkv::DecodeArgs{};
  if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0 || head_dim < 1 ||
      block_size < 1)
    return PKV_EINVAL;
  if (block_size != pkv::kBlockSize ||
      !pkv::decode_mma_supported(1, head_dim, num_q_heads / num_kv_heads))
    return PKV_EUNSUPPORTED;
  if (num_seqs < 0 || max_blocks_per_seq < 1 || max_seq_len < 1 || num_blocks < 1)
    return PKV_EINVAL;
  if (num_seqs == 0) return PKV_OK;
  if (num_seqs > PKV_MAX_SEQS) return PKV_ERANGE;
  if ((int64_t)max_seq_len > (int64_t)max_blocks_per_seq * block_size) return PKV_EINVAL;
  if (!isfinite(scale)) return PKV_EINVAL;
  if (!out || !q || !k_cache || !v_cache || !block_table || !seq_lens || !scales_ok)
    return PKV_EINVAL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return PKV_EINVAL;
  const int s = partial_slots_for(max_seq_len, split_tokens);
  const size_t need = partials_bytes(num_seqs, num_q_heads, head_dim, s);
  if (workspace_bytes < need) return PKV_ERANGE;
  if ((int64_t)num_seqs * num_kv_heads * max_splits_for(max_seq_len, split_tokens) >= (int64_t)INT_MAX)
    return PKV_ERANGE;  // the kernels' unit list is indexed by int
  if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))) return PKV_EINVAL;
  int* err = nullptr;
  const pkv_status st = device_state(&err, sms);
  if (st != PKV_OK) return st;
  const Partials part = carve_partials(workspace, (size_t)num_seqs * num_q_heads * s, head_dim);
  pkv::DecodeArgs a{};
  a.out = out;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.ws_acc = need ? part.acc : nullptr;
  a.ws_ml = need ? part.ml : nullptr;
  a.ws_np = need ? part.np : nullptr;
  a.err = err;
  a.num_seqs = num_seqs;
  a.bt_stride = max_blocks_per_seq;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_seq_len = max_seq_len;
  a.max_splits = s;
  a.split_tokens = split_tokens;
  a.num_blocks = num_blocks;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.scale = scale;
  a.chunk_prior = -1;
  a.is_bf16 = 1;
  *out_args = a;
  return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_paged_decode_attention_fp8(void* out, const void* q, const void* k_cache,
                                          const void* v_cache, const float* k_scale,
                                          const float* v_scale, const int32_t* block_table,
                                          const int32_t* seq_lens, int num_seqs,
                                          int max_blocks_per_seq, int max_seq_len,
                                          int64_t num_blocks, int num_q_heads, int num_kv_heads,
                                          int head_dim, int block_size, float scale,
                                          void* workspace, size_t workspace_bytes,
                                          pkv_stream_t stream) {
  pkv::DecodeArgs a;
  const bool scales_ok = k_scale && v_scale && !(reinterpret_cast<uintptr_t>(k_scale) & 3u) &&
                         !(reinterpret_cast<uintptr_t>(v_scale) & 3u);
  int sms = 0;
  const pkv_status st = fp8_decode_prepare(
      &a, &sms, scales_ok, pkv::kSplitTokens, out, q, k_cache, v_cache, block_table, seq_lens, num_seqs,
      max_blocks_per_seq, max_seq_len, num_blocks, num_q_heads, num_kv_heads, head_dim, block_size,
      scale, workspace, workspace_bytes);
  if (st != PKV_OK || a.num_seqs == 0) return st;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return pkv::launch_paged_decode_fp8(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

size_t pkv_decode_fp8_block_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                            int head_dim, int max_seq_len) {
  if (num_seqs < 1 || num_q_heads < 1 || num_kv_heads < 1 || head_dim < 1 || max_seq_len < 1 ||
      max_seq_len > INT_MAX - pkv::kSplitTokens)
    return 0;
  const int split = pkv::fp8_block_split_tokens(num_seqs, num_kv_heads, max_seq_len);
  return partials_bytes(num_seqs, num_q_heads, head_dim, partial_slots_for(max_seq_len, split));
}

pkv_status pkv_paged_decode_attention_fp8_block(
    void* out, const void* q, const void* k_cache, const void* v_cache, const uint8_t* k_scale,
    const uint8_t* v_scale, const int32_t* block_table, const int32_t* seq_lens, int num_seqs,
    int max_blocks_per_seq, int max_seq_len, int64_t num_blocks, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, float scale, void* workspace, size_t workspace_bytes,
    pkv_stream_t stream) {
  if (max_seq_len > INT_MAX - pkv::kSplitTokens) return PKV_ERANGE;   // rounded up to whole splits
  pkv::DecodeArgs a;
  int sms = 0;
  int split = pkv::kSplitTokens;
  if (num_seqs > 0 && num_q_heads > 0 && num_kv_heads > 0 && head_dim > 0 && max_seq_len > 0) {
    split = pkv::fp8_block_split_tokens(num_seqs, num_kv_heads, max_seq_len);
    // a caller's workspace for a larger batch may be too small for the shorter
    // splits of this one
    while (split < pkv::kSplitTokens &&
           partials_bytes(num_seqs, num_q_heads, head_dim, partial_slots_for(max_seq_len, split)) >
               workspace_bytes)
      split *= 2;
  }
  const pkv_status st = fp8_decode_prepare(
      &a, &sms, k_scale && v_scale, split, out, q, k_cache, v_cache, block_table, seq_lens, num_seqs,
      max_blocks_per_seq, max_seq_len, num_blocks, num_q_heads, num_kv_heads, head_dim, block_size,
      scale, workspace, workspace_bytes);
  if (st != PKV_OK || a.num_seqs == 0) return st;
  a.k_bscale = k_scale;
  a.v_bscale = v_scale;
  a.skip_empty = 1;
  return pkv::launch_paged_decode_fp8_block(a, sms, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

pkv_status pkv_latent_append(const void* c_new, void* c_cache, const int64_t* slot_mapping,
                             int64_t num_tokens, int64_t num_blocks, int rank, int block_size,
                             pkv_stream_t stream) {
  if (num_tokens < 0 || num_blocks < 1 || rank < 1 || block_size < 1) return PKV_EINVAL;
  if (block_size != pkv::kBlockSize || (rank * 2) % 16 != 0) return PKV_EUNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!c_new || !c_cache || !slot_mapping) return PKV_EINVAL;
  if (!aligned16(c_new) || !aligned16(c_cache) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return PKV_EINVAL;
  int* err = nullptr;
  int sms = 0;
  pkv_status st = device_state(&err, &sms);
  if (st != PKV_OK) return st;
  pkv::AppendArgs a{c_new, nullptr, c_cache, nullptr, slot_mapping, num_tokens, num_blocks, 1,
                    rank * 2, err};
  return pkv::launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

size_t pkv_mla_workspace_bytes(int num_seqs, int num_q_heads, int rank, int max_seq_len) {
  if (num_seqs < 1 || num_q_heads < 1 || rank < 1 || max_seq_len < 1) return 0;
  const size_t vec = align256((size_t)num_seqs * num_q_heads * rank * 2);
  return 2 * vec + pkv_decode_workspace_bytes(num_seqs, num_q_heads, rank, max_seq_len);
}

}  // extern "C"

namespace {

// The latent decode call; c_new (optional): each sequence's new latent,
// appended by the query absorption's launch.
pkv_status mla_decode(void* out, const void* q, const void* c_new, const void* w_k,
                      const void* w_v, void* c_cache, const int32_t* block_table,
                      const int32_t* seq_lens, int num_seqs, int max_blocks_per_seq,
                      int max_seq_len, int64_t num_blocks, int num_q_heads, int head_dim, int rank,
                      int block_size, float scale, void* workspace, size_t workspace_bytes,
                      pkv_stream_t stream) {
  if (num_q_heads < 1 || head_dim < 1 || rank < 1 || block_size < 1) return PKV_EINVAL;
  if (block_size != pkv::kBlockSize || num_q_heads != 32 || head_dim != 128 || rank != 128)
    return PKV_EUNSUPPORTED;
  if (num_seqs < 0 || max_blocks_per_seq < 1 || max_seq_len < 1 || num_blocks < 1) return PKV_EINVAL;
  if (num_seqs == 0) return PKV_OK;
  if (num_seqs > PKV_MAX_SEQS) return PKV_ERANGE;
  if ((int64_t)max_seq_len > (int64_t)max_blocks_per_seq * block_size) return PKV_EINVAL;
  if (!isfinite(scale)) return PKV_EINVAL;
  if (!out || !q || !w_k || !w_v || !c_cache || !block_table || !seq_lens || !workspace)
    return PKV_EINVAL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(w_k) || !aligned16(w_v) ||
      !aligned16(c_cache) || (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return PKV_EINVAL;
  if (workspace_bytes < pkv_mla_workspace_bytes(num_seqs, num_q_heads, rank, max_seq_len))
    return PKV_ERANGE;
  if ((int64_t)num_seqs * max_splits_for(max_seq_len) >= (int64_t)INT_MAX)
    return PKV_ERANGE;  // the kernel's unit list is indexed by int
  int* err = nullptr;
  int sms = 0;
  pkv_status st = device_state(&err, &sms);
  if (st != PKV_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t vec = align256((size_t)num_seqs * num_q_heads * rank * 2);
  char* ws = static_cast<char*>(workspace);
  void* q_lat = ws;          // absorbed queries [B][Hq][rank] bf16
  void* z = ws + vec;        // attention over the latent [B][Hq][rank] bf16
  char* part = ws + 2 * vec;
  // 1) q~_h = W_K[h]^T q_h (and, given c_new, each sequence's new latent
  //    placed at position seq_lens[b] - 1)
  const pkv::LatentAppend app{c_new, c_cache, block_table, seq_lens, max_blocks_per_seq,
                              (int)std::min<int64_t>(max_seq_len,
                                                     (int64_t)max_blocks_per_seq * block_size),
                              num_blocks, err};
  if (pkv::launch_gemm_heads(q_lat, q, w_k, num_seqs, num_q_heads, s, c_new ? &app : nullptr) !=
      cudaSuccess)
    return PKV_ECUDA;
  // 2) z_h = softmax(scale q~_h . C^T) C over the latent pool
  const int splits = partial_slots_for(max_seq_len);
  const Partials pp = carve_partials(part, (size_t)num_seqs * num_q_heads * splits, rank);
  pkv::DecodeArgs a{};
  a.out = z;
  a.q = q_lat;
  a.k_cache = c_cache;
  a.v_cache = c_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.ws_acc = pp.acc;
  a.ws_ml = pp.ml;
  a.ws_np = splits > 1 ? pp.np : nullptr;
  a.err = err;
  a.num_seqs = num_seqs;
  a.bt_stride = max_blocks_per_seq;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_seq_len = max_seq_len;
  a.max_splits = splits;
  a.split_tokens = pkv::kSplitTokens;
  a.num_blocks = num_blocks;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = 1;
  a.head_dim = rank;
  a.scale = scale;
  a.chunk_prior = -1;
  a.is_bf16 = 1;
  // 3) merge of the partials fused with o_h = W_V[h] z_h
  if (pkv::launch_decode_mla(a, w_v, out, sms, s) != cudaSuccess) return PKV_ECUDA;
  return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_mla_decode_attention(void* out, const void* q, const void* w_k, const void* w_v,
                                    const void* c_cache, const int32_t* block_table,
                                    const int32_t* seq_lens, int num_seqs, int max_blocks_per_seq,
                                    int max_seq_len, int64_t num_blocks, int num_q_heads,
                                    int head_dim, int rank, int block_size, float scale,
                                    void* workspace, size_t workspace_bytes, pkv_stream_t stream) {
  return mla_decode(out, q, nullptr, w_k, w_v, const_cast<void*>(c_cache), block_table, seq_lens,
                    num_seqs, max_blocks_per_seq, max_seq_len, num_blocks, num_q_heads, head_dim,
                    rank, block_size, scale, workspace, workspace_bytes, stream);
}

pkv_status pkv_mla_decode_attention_append(void* out, const void* q, const void* c_new,
                                           const void* w_k, const void* w_v, void* c_cache,
                                           const int32_t* block_table, const int32_t* seq_lens,
                                           int num_seqs, int max_blocks_per_seq, int max_seq_len,
                                           int64_t num_blocks, int num_q_heads, int head_dim,
                                           int rank, int block_size, float scale, void* workspace,
                                           size_t workspace_bytes, pkv_stream_t stream) {
  if (num_seqs > 0 && (!c_new || !aligned16(c_new))) return PKV_EINVAL;
  return mla_decode(out, q, c_new, w_k, w_v, c_cache, block_table, seq_lens, num_seqs,
                    max_blocks_per_seq, max_seq_len, num_blocks, num_q_heads, head_dim, rank,
                    block_size, scale, workspace, workspace_bytes, stream);
}

pkv_status pkv_chunked_prefill_attention(void* out, const void* q, const void* k_cache,
                                         const void* v_cache, const int32_t* block_table_row,
                                         int max_blocks, int prior_len, int chunk_len,
                                         int64_t num_blocks, int num_q_heads, int num_kv_heads,
                                         int head_dim, int block_size, float scale,
                                         pkv_dtype dtype, pkv_stream_t stream) {
  pkv_status st = prefill_check(out, q, k_cache, v_cache, block_table_row, max_blocks, prior_len,
                                chunk_len, num_blocks, num_q_heads, num_kv_heads, head_dim,
                                block_size, scale, dtype);
  if (st != PKV_OK || chunk_len == 0) return st;
  return prefill_launch(out, q, k_cache, v_cache, block_table_row, max_blocks, prior_len, chunk_len,
                        num_blocks, num_q_heads, num_kv_heads, head_dim, scale, dtype, 0,
                        reinterpret_cast<cudaStream_t>(stream));
}

pkv_status pkv_chunked_prefill_attention_fp8_block(
    void* out, const void* q, const void* k_cache, const void* v_cache, const uint8_t* k_scale,
    const uint8_t* v_scale, const int32_t* block_table_row, int max_blocks, int prior_len,
    int chunk_len, int64_t num_blocks, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, pkv_stream_t stream) {
  pkv_status st = prefill_check(out, q, k_cache, v_cache, block_table_row, max_blocks, prior_len,
                                chunk_len, num_blocks, num_q_heads, num_kv_heads, head_dim,
                                block_size, scale, PKV_BF16);
  if (st != PKV_OK || chunk_len == 0) return st;
  if (!k_scale || !v_scale || !(scale > 0.f)) return PKV_EINVAL;
  if ((int64_t)prior_len + chunk_len > INT_MAX - 4096) return PKV_ERANGE;   // rounded up to tiles
  int* err = nullptr;
  int sms = 0;
  st = device_state(&err, &sms);
  if (st != PKV_OK) return st;
  pkv::PrefillArgs a{out, q, k_cache, v_cache, block_table_row, max_blocks, prior_len, chunk_len,
                     num_blocks, num_q_heads, num_kv_heads, scale, err};
  a.k_bscale = k_scale;
  a.v_bscale = v_scale;
  return pkv::launch_prefill_fp8_block(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKV_OK
             : PKV_ECUDA;
}

}  // extern "C"

namespace {

constexpr int kMaxTreeLen = INT_MAX - 65536;   // positions a little behind the end are formed as ints

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Validates a call of drafted tokens and fills its launch arguments.  *todo
// false: valid, and nothing to launch.
pkv_status tree_prepare(const pkv_tree_args* x, bool attention, pkv::TreeArgs* out, int* sms, bool* todo) {
  *todo = false;
  if (!x) return PKV_EINVAL;
  pkv_status st = check_heads(x->num_q_heads, x->num_kv_heads, x->head_dim, x->block_size, x->dtype);
  if (st != PKV_OK) return st;
  if (x->num_seqs < 0 || x->num_rows < 0 || x->max_blocks_per_seq < 1 || x->max_seq_len < 1 || x->num_blocks < 1 ||
      x->max_draft < 1)
    return PKV_EINVAL;
  if (x->max_draft > PKV_MAX_DRAFT) return PKV_EUNSUPPORTED;
  if (x->num_seqs == 0 || x->num_rows == 0) return PKV_OK;
  if (x->num_seqs > PKV_MAX_SEQS || x->max_seq_len > kMaxTreeLen) return PKV_ERANGE;
  if ((int64_t)x->max_seq_len > (int64_t)x->max_blocks_per_seq * x->block_size) return PKV_EINVAL;
  if (!isfinite(x->scale) || !(x->scale > 0.f)) return PKV_EINVAL;
  if (!x->q || !x->k_cache || !x->block_table || !x->seq_lens || !x->draft_offsets) return PKV_EINVAL;
  if (!aligned16(x->q) || !aligned16(x->k_cache) || misaligned(x->block_table, 4) || misaligned(x->seq_lens, 4) ||
      misaligned(x->draft_offsets, 4) || misaligned(x->tree_mask, 8) || misaligned(x->lse, 4))
    return PKV_EINVAL;
  if (attention) {
    if (!x->out || !x->v_cache || !aligned16(x->out) || !aligned16(x->v_cache)) return PKV_EINVAL;
    const size_t need = x->dtype != PKV_BF16 ? 0   // the fp32 kernel joins its splits in shared memory
                                             : pkv_tree_workspace_bytes(x->num_q_heads, x->num_kv_heads, x->head_dim,
                                                                        x->max_draft, x->max_seq_len);
    if (x->workspace_bytes < need) return PKV_ERANGE;
    if (need > 0 && (!x->workspace || misaligned(x->workspace, 256))) return PKV_EINVAL;
  } else {
    if (!x->weights || !x->lse || misaligned(x->weights, 4)) return PKV_EINVAL;
    if (x->weights_len < x->max_seq_len) return PKV_EINVAL;
  }
  // tiles of all sequences, heads and rows (and what the plan adds for a
  // stream's start and end) are counted in an int
  const int64_t tiles = (x->max_seq_len + 31) / 32;
  const int64_t chunks = ((int64_t)x->max_draft * (x->num_q_heads / x->num_kv_heads) + 31) / 32;
  if ((int64_t)x->num_seqs * x->num_kv_heads * (tiles * chunks + 2 * chunks + 16) >= (int64_t)INT_MAX)
    return PKV_ERANGE;
  if ((int64_t)x->num_rows * x->num_q_heads >= (int64_t)INT_MAX) return PKV_ERANGE;
  int* err = nullptr;
  st = device_state(&err, sms);
  if (st != PKV_OK) return st;
  pkv::TreeArgs a{};
  a.out = x->out;
  a.lse = x->lse;
  a.weights = x->weights;
  a.weights_len = x->weights_len;
  a.q = x->q;
  a.k_cache = x->k_cache;
  a.v_cache = x->v_cache;
  a.block_table = x->block_table;
  a.seq_lens = x->seq_lens;
  a.draft_offsets = x->draft_offsets;
  a.tree_mask = x->tree_mask;
  a.num_seqs = x->num_seqs;
  a.num_rows = x->num_rows;
  a.max_blocks_per_seq = x->max_blocks_per_seq;
  a.max_seq_len = x->max_seq_len;
  a.max_draft = x->max_draft;
  a.num_blocks = x->num_blocks;
  a.num_q_heads = x->num_q_heads;
  a.num_kv_heads = x->num_kv_heads;
  a.head_dim = x->head_dim;
  a.scale = x->scale;
  a.workspace = x->workspace;
  a.err = err;
  *out = a;
  *todo = true;
  return PKV_OK;
}

}  // namespace

extern "C" {

size_t pkv_tree_workspace_bytes(int num_q_heads, int num_kv_heads, int head_dim, int max_draft, int max_seq_len) {
  if (check_heads(num_q_heads, num_kv_heads, head_dim, pkv::kBlockSize, PKV_BF16) != PKV_OK || max_draft < 1 ||
      max_draft > PKV_MAX_DRAFT || max_seq_len < 1 || max_seq_len > kMaxTreeLen)
    return 0;
  return pkv::tree_workspace_bytes(num_q_heads / num_kv_heads, max_draft);
}

pkv_status pkv_paged_tree_attention(const pkv_tree_args* x, pkv_stream_t stream) {
  pkv::TreeArgs a;
  int sms = 0;
  bool todo = false;
  const pkv_status st = tree_prepare(x, true, &a, &sms, &todo);
  if (st != PKV_OK || !todo) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = x->dtype == PKV_BF16 ? pkv::launch_tree_attention_mma(a, sms, s)
                                             : pkv::launch_tree_attention_cc(a, s);
  return e == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

pkv_status pkv_kv_add_weights(const pkv_tree_args* x, pkv_stream_t stream) {
  pkv::TreeArgs a;
  int sms = 0;
  bool todo = false;
  const pkv_status st = tree_prepare(x, false, &a, &sms, &todo);
  if (st != PKV_OK || !todo) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = x->dtype == PKV_BF16 ? pkv::launch_kv_add_weights_mma(a, sms, s)
                                             : pkv::launch_kv_add_weights_cc(a, s);
  return e == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

pkv_status pkv_kv_select(int32_t* kept, int32_t* kept_lens, const float* weights, int64_t weights_len,
                         const int32_t* seq_lens, int num_seqs, int num_kv_heads, int max_seq_len, int budget,
                         int sinks, int recent, pkv_stream_t stream) {
  if (num_seqs < 0 || num_kv_heads < 1 || max_seq_len < 1 || budget < 1 || sinks < 0 || recent < 0)
    return PKV_EINVAL;
  if (sinks > budget || recent > budget - sinks || weights_len < max_seq_len) return PKV_EINVAL;
  if (num_seqs == 0) return PKV_OK;
  if (num_seqs > PKV_MAX_SEQS || (int64_t)num_seqs * num_kv_heads > INT_MAX / 16 ||
      max_seq_len > INT_MAX - 65536)
    return PKV_ERANGE;
  if (!kept || !kept_lens || !weights || !seq_lens) return PKV_EINVAL;
  if (misaligned(kept, 4) || misaligned(kept_lens, 4) || misaligned(weights, 4) || misaligned(seq_lens, 4))
    return PKV_EINVAL;
  int* err = nullptr;
  int sms = 0;
  const pkv_status st = device_state(&err, &sms);
  if (st != PKV_OK) return st;
  pkv::SelectArgs a{kept, kept_lens, weights, weights_len, seq_lens, num_seqs, num_kv_heads, max_seq_len,
                    budget, sinks, recent, err};
  return pkv::launch_kv_select(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PKV_OK : PKV_ECUDA;
}

pkv_status pkv_kv_compact(const pkv_compact_args* x, pkv_stream_t stream) {
  if (!x) return PKV_EINVAL;
  if (x->num_seqs < 0 || x->max_blocks_per_seq < 1 || x->num_blocks < 1 || x->num_kv_heads < 1 ||
      x->kept_len < 0 || x->row_bytes < 1 || x->block_size < 1)
    return PKV_EINVAL;
  if (x->kept_heads != 1 && x->kept_heads != x->num_kv_heads) return PKV_EINVAL;
  if (x->block_size != pkv::kBlockSize || x->row_bytes % 16 != 0 || x->row_bytes > PKV_MAX_COMPACT_ROW_BYTES)
    return PKV_EUNSUPPORTED;
  if (x->num_seqs == 0) return PKV_OK;
  if (x->num_seqs > PKV_MAX_SEQS || (int64_t)x->num_seqs * x->num_kv_heads > INT_MAX / 64 ||
      (int64_t)x->max_blocks_per_seq * x->block_size > INT_MAX - 65536)
    return PKV_ERANGE;
  if (!x->k_cache || !x->v_cache || !x->block_table || !x->seq_lens || !x->kept_lens || (x->kept_len > 0 && !x->kept))
    return PKV_EINVAL;
  if (x->k_cache == x->v_cache || (x->weights && x->weights_len < 1)) return PKV_EINVAL;
  if (!aligned16(x->k_cache) || !aligned16(x->v_cache) || misaligned(x->block_table, 4) ||
      misaligned(x->seq_lens, 4) || misaligned(x->kept, 4) || misaligned(x->kept_lens, 4) ||
      misaligned(x->first, 4) || misaligned(x->weights, 4))
    return PKV_EINVAL;
  int* err = nullptr;
  int sms = 0;
  const pkv_status st = device_state(&err, &sms);
  if (st != PKV_OK) return st;
  pkv::CompactArgs a{x->k_cache, x->v_cache, x->weights, x->weights_len, x->block_table, x->seq_lens,
                     x->kept, x->kept_lens, x->first, x->num_seqs, x->max_blocks_per_seq, x->num_kv_heads,
                     x->kept_heads, x->kept_len, x->row_bytes, x->num_blocks, err};
  return pkv::launch_kv_compact(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PKV_OK
                                                                                              : PKV_ECUDA;
}

pkv_status pkv_decode_prefill_attention(const pkv_decode_prefill_args* x, pkv_stream_t stream) {
  if (!x) return PKV_EINVAL;
  // validate both halves before anything is launched
  if (!dtype_ok(x->dtype)) return PKV_EDTYPE;
  if (x->num_q_heads < 1 || x->num_kv_heads < 1 || x->num_q_heads % x->num_kv_heads != 0)
    return PKV_EINVAL;
  if (!pkv::decode_mma_supported(x->dtype == PKV_BF16, x->head_dim,
                                 x->num_q_heads / x->num_kv_heads))
    return PKV_EUNSUPPORTED;
  if (x->num_seqs > 0 && (!x->k_new || !x->v_new || !aligned16(x->k_new) || !aligned16(x->v_new)))
    return PKV_EINVAL;
  pkv::DecodeArgs d{};
  int sms = 0;
  pkv_status st = decode_prepare(&d, &sms, x->decode_out, x->decode_q, x->k_new, x->v_new,
                                 x->k_cache, x->v_cache, x->block_table, x->seq_lens, x->num_seqs,
                                 x->max_blocks_per_seq, x->max_seq_len, x->num_blocks,
                                 x->num_q_heads, x->num_kv_heads, x->head_dim, x->block_size,
                                 x->scale, x->workspace, x->workspace_bytes, x->dtype);
  if (st != PKV_OK) return st;
  st = prefill_check(x->prefill_out, x->prefill_q, x->k_cache, x->v_cache, x->prefill_block_table,
                     x->prefill_max_blocks, x->prior_len, x->chunk_len, x->num_blocks,
                     x->num_q_heads, x->num_kv_heads, x->head_dim, x->block_size, x->scale,
                     x->dtype);
  if (st != PKV_OK) return st;
  if (x->prefill_sms < 0) return PKV_EINVAL;
  // the chunk's own keys and values: all three pointers or none
  const bool chunk_append = x->chunk_k_new || x->chunk_v_new || x->chunk_slot_mapping;
  if (chunk_append && x->chunk_len > 0 &&
      (!x->chunk_k_new || !x->chunk_v_new || !x->chunk_slot_mapping || !aligned16(x->chunk_k_new) ||
       !aligned16(x->chunk_v_new) || (reinterpret_cast<uintptr_t>(x->chunk_slot_mapping) & 7u)))
    return PKV_EINVAL;
  int* err = nullptr;
  st = device_state(&err, &sms);
  if (st != PKV_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (chunk_append && x->chunk_len > 0) {
    // the chunk's rows first; the prefill (launched next, not as a
    // programmatic dependent) reads them
    pkv::AppendArgs ap{x->chunk_k_new, x->chunk_v_new, x->k_cache, x->v_cache,
                       x->chunk_slot_mapping, x->chunk_len, x->num_blocks, x->num_kv_heads,
                       x->head_dim * elem_bytes(x->dtype), err};
    if (pkv::launch_kv_append(ap, s) != cudaSuccess) return PKV_ECUDA;
  }
  const int p_sms = x->prefill_sms > 0 ? x->prefill_sms : sms / 4;
  pkv::PrefillArgs pa{x->prefill_out, x->prefill_q, x->k_cache, x->v_cache, x->prefill_block_table,
                      x->prefill_max_blocks, x->prior_len, x->chunk_len, x->num_blocks,
                      x->num_q_heads, x->num_kv_heads, x->scale, err};
  if (unsigned long long* span = g_span_buf.load()) {
    pa.span = span;
    d.span = span + 2;
  }
  const bool side_by_side = x->chunk_len > 0 && d.num_seqs > 0 && x->head_dim == 128 &&
                            x->dtype == PKV_BF16 && p_sms < sms &&
                            pkv::prefill_pair_persistent_ok(pa, p_sms);
  if (!side_by_side) {   // one after the other, each on the whole GPU
    if (x->chunk_len > 0) {
      st = prefill_launch(x->prefill_out, x->prefill_q, x->k_cache, x->v_cache,
                          x->prefill_block_table, x->prefill_max_blocks, x->prior_len,
                          x->chunk_len, x->num_blocks, x->num_q_heads, x->num_kv_heads,
                          x->head_dim, x->scale, x->dtype, 0, s);
      if (st != PKV_OK) return st;
    }
    return decode_launch(d, sms, false, s);
  }
  // the prefill's persistent CTAs take p_sms SMs; the decode, launched as its
  // programmatic dependent, runs on the others and finishes after it.  (The
  // prefill launched as the programmatic dependent of the chunk's append,
  // its gathers waiting for that grid, measured 20% slower per layer.)
  if (pkv::launch_prefill_pair(pa, s, p_sms) != cudaSuccess) return PKV_ECUDA;
  return decode_launch(d, sms - p_sms, true, s);
}

}  // extern "C"
