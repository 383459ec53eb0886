// Decode attention over the fp8 cache with one scale per KV head: the kernel
// of decode_fp8_kernel.cuh, its split partials merged by the shared reduce.
#include "decode_fp8_kernel.cuh"

namespace pkv {

cudaError_t launch_paged_decode_fp8(const DecodeArgs& a, int num_sms, cudaStream_t stream) {
  if (a.chunk_prior >= 0 || a.split_tokens % kStageTok != 0 || !a.k_scale || !a.v_scale)
    return cudaErrorInvalidValue;
  DecodeArgs m = a;   // as the kernel is launched
  m.partials_f16 = 1;
  const cudaError_t e = launch_fp8<false>(a, num_sms, stream, &m.balanced);
  if (e != cudaSuccess || a.max_splits <= 1) return e;
  return launch_decode_reduce_bf16_128(m, stream);
}

}  // namespace pkv
