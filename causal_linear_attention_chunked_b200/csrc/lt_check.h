// lt_check.h -- host-side argument checks and the dependent-launch helper of
// the cache, decode and norm-rotation entry points.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "lt_fault.h"
#include "lt_internal.h"

namespace lt {

inline bool aligned_to(const void* p, unsigned a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// the current device, or -1
inline int current_device() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();  // clear the non-sticky error
    return -1;
  }
  return dev;
}

// memory that a kernel on the current device (dev) may use: managed, or device
// memory of that very device (a pointer of another device is refused here
// rather than read over the bus)
inline bool on_device(int dev, const void* p) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeManaged || (at.type == cudaMemoryTypeDevice && at.device == dev);
}

// Lets `kern` use `bytes` of dynamic shared memory, once per device: `done` is
// the kernel's own set of devices (a repeated call costs the host about as
// much as a pointer check).
inline cudaError_t allow_smem(const void* kern, int bytes, std::atomic<uint64_t>& done) {
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

struct Span {
  const void* p;
  size_t n;  // bytes
};

inline bool spans_overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}

inline size_t dtype_size(lt_dtype_t t) { return t == LT_F32 ? 4 : 2; }
inline bool dtype_ok(lt_dtype_t t) { return t == LT_F32 || t == LT_BF16 || t == LT_F16; }
inline bool eight_bit(lt_kv_dtype_t t) { return t == LT_KV_E4M3 || t == LT_KV_INT8; }
inline size_t kv_size(lt_kv_dtype_t t) { return t == LT_KV_F32 ? 4 : eight_bit(t) ? 1 : 2; }
// the cache type that is an exact copy of a tensor type
inline lt_kv_dtype_t kv_of(lt_dtype_t t) {
  return t == LT_F32 ? LT_KV_F32 : t == LT_BF16 ? LT_KV_BF16 : LT_KV_F16;
}

// A token-strided tensor [tokens][H][w]: bytes from its first to its last element.
inline size_t strided_bytes(int64_t tokens, int64_t stride, int64_t H, int64_t w, size_t es) {
  return ((size_t)(tokens - 1) * (size_t)stride + (size_t)(H * w)) * es;
}
// its stride covers a token, keeps 16-byte alignment and a sane extent
inline bool stride_ok(int64_t tokens, int64_t stride, int64_t H, int64_t w, size_t es) {
  if (stride < H * w || (stride * (int64_t)es) % 16 != 0) return false;
  return stride < ((int64_t)1 << 40) && tokens < ((int64_t)1 << 62) / (stride * (int64_t)es);
}

// The checks of a cache that need no CUDA call, then (pointers) those that do.
lt_status_t check_cache(const lt_kv_cache_t* c);
lt_status_t check_cache_pointers(int dev, const lt_kv_cache_t* c);
// the four address ranges of a cache's pools and scales
void cache_spans(const lt_kv_cache_t* c, Span out[4]);

// The caller's workspace, or a stream-ordered one of the same size.
struct Workspace {
  void* p = nullptr;
  bool own = false;
  cudaStream_t stream;
  lt_status_t take(int dev, void* given, size_t given_bytes, size_t need, cudaStream_t s) {
    stream = s;
    if (given) {
      if (given_bytes < need || !aligned_to(given, 16) || !on_device(dev, given))
        return LT_ERR_INVALID_ARG;
      p = given;
      return LT_OK;
    }
    if (injected_workspace_alloc_failure() || cudaMallocAsync(&p, need, s) != cudaSuccess) {
      cudaGetLastError();
      p = nullptr;
      return LT_ERR_CUDA;
    }
    own = true;
    return LT_OK;
  }
  cudaError_t release() {
    if (!own) return cudaSuccess;
    own = false;
    return cudaFreeAsync(p, stream);
  }
};

// Launch `kern` so that it may start while the launch before it on the stream
// still runs; it must wait (griddepcontrol.wait) before it touches that
// launch's results, in every block.
template <typename Args>
inline cudaError_t launch_dependent(void (*kern)(Args), dim3 grid, int threads, size_t smem,
                                    cudaStream_t stream, const Args& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace lt
