// paged_attn_f32.cu -- the first decode launch for fp32 queries.
#include "paged_attn.cuh"

namespace lt {
namespace paged {
namespace {

cudaError_t launch_fp32(const DecodeArgs& a, int d, int sms, cudaStream_t s) {
  if (d == 64)
    return a.dv == 64 ? launch_engine<Fp32Engine<64, 64>>(a, sms, s)
                      : launch_engine<Fp32Engine<64, 128>>(a, sms, s);
  return a.dv == 64 ? launch_engine<Fp32Engine<128, 64>>(a, sms, s)
                    : launch_engine<Fp32Engine<128, 128>>(a, sms, s);
}

}  // namespace

cudaError_t launch_f32(const DecodeArgs& a, lt_kv_dtype_t kv, int d, int sms, cudaStream_t s) {
  if (kv == LT_KV_E4M3) return launch_mma_nb<float, E4M3, 1>(a, d, sms, s);
  if (kv == LT_KV_INT8) return launch_mma_nb<float, Int8, 1>(a, d, sms, s);
  return launch_fp32(a, d, sms, s);
}

}  // namespace paged
}  // namespace lt
