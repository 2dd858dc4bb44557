// lt_vec.cuh -- four consecutive elements as one access, widened to fp32 or
// rounded once from it.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lt {

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_float(__nv_bfloat16* p, float x) {
  *p = __float2bfloat16_rn(x);
}
__device__ __forceinline__ void from_float(__half* p, float x) { *p = __float2half_rn(x); }

// the types that an 8-bit cache holds (each user of them decodes into its own)
struct E4M3 {};
struct Int8 {};

// raw storage of four elements of T (8 or 16 bytes)
template <typename T>
struct Quad {
  uint2 r;
};
template <>
struct Quad<float> {
  float4 r;
};

template <typename T>
__device__ __forceinline__ Quad<T> load_quad(const T* p) {
  Quad<T> q;
  q.r = __ldg(reinterpret_cast<const decltype(q.r)*>(p));
  return q;
}

__device__ __forceinline__ void widen(const Quad<float>& q, float* f) {
  f[0] = q.r.x;
  f[1] = q.r.y;
  f[2] = q.r.z;
  f[3] = q.r.w;
}
__device__ __forceinline__ void widen(const Quad<__nv_bfloat16>& q, float* f) {
  f[0] = __uint_as_float(q.r.x << 16);
  f[1] = __uint_as_float(q.r.x & 0xffff0000u);
  f[2] = __uint_as_float(q.r.y << 16);
  f[3] = __uint_as_float(q.r.y & 0xffff0000u);
}
__device__ __forceinline__ void widen(const Quad<__half>& q, float* f) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&q.r.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&q.r.y));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

__device__ __forceinline__ void store_quad(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store_quad(__nv_bfloat16* p, const float* f) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]);
  const __nv_bfloat162 b = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store_quad(__half* p, const float* f) {
  const __half2 a = __floats2half2_rn(f[0], f[1]);
  const __half2 b = __floats2half2_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

// ------------------------------------------------------- two fp32 at a time
// sm_100 multiplies and adds register pairs of fp32 in one instruction, each
// half rounded as by the scalar one.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pack_f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack_f2(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 swap2(F2 a) {
  const float2 t = unpack_f2(a);
  return pack_f2(t.y, t.x);
}

template <typename T>
__device__ __forceinline__ void widen2x2(const Quad<T>& q, F2* f) {
  float x[4];
  widen(q, x);
  f[0] = pack_f2(x[0], x[1]);
  f[1] = pack_f2(x[2], x[3]);
}
template <typename T>
__device__ __forceinline__ void store_quad(T* p, F2 a, F2 b) {
  const float2 x = unpack_f2(a), y = unpack_f2(b);
  const float f[4] = {x.x, x.y, y.x, y.y};
  store_quad(p, f);
}

// The results of the launch before this one on the stream are complete and
// visible after dependency_wait(); dependency_release() lets the launch after
// this one start early (its own wait still covers this whole launch).
__device__ __forceinline__ void dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void dependency_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace lt
