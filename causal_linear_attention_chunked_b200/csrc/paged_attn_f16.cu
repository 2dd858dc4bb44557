// paged_attn_f16.cu -- the first decode launch for fp16 queries.
#include "paged_attn.cuh"

namespace lt {
namespace paged {

cudaError_t launch_f16(const DecodeArgs& a, lt_kv_dtype_t kv, int d, int sms, cudaStream_t s) {
  if (kv == LT_KV_E4M3) return launch_mma<__half, E4M3>(a, d, sms, s);
  if (kv == LT_KV_INT8) return launch_mma<__half, Int8>(a, d, sms, s);
  return launch_mma<__half, __half>(a, d, sms, s);
}

}  // namespace paged
}  // namespace lt
