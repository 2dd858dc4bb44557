// paged_attn_bf16.cu -- the first decode launch for bf16 queries.
#include "paged_attn.cuh"

namespace lt {
namespace paged {

cudaError_t launch_bf16(const DecodeArgs& a, lt_kv_dtype_t kv, int d, int sms, cudaStream_t s) {
  if (kv == LT_KV_E4M3) return launch_mma<__nv_bfloat16, E4M3>(a, d, sms, s);
  if (kv == LT_KV_INT8) return launch_mma<__nv_bfloat16, Int8>(a, d, sms, s);
  return launch_mma<__nv_bfloat16, __nv_bfloat16>(a, d, sms, s);
}

}  // namespace paged
}  // namespace lt
