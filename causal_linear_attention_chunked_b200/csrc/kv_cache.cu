// kv_cache.cu -- rows of keys and values into a paged cache, quantised as
// they are written, and a batch of sequences read back, packed.
//
// Per row x (one head of one token): scale = max(max|x| / qmax, 2^-126),
// code = round(x / scale), qmax 448 (e4m3) or 127 (int8).  Both divisions are
// the correctly rounded ones, so the codes follow from the inputs alone and
// do not depend on how a row is spread over lanes.  The floor on the scale
// makes a row of zeros read back as zeros without a case of its own.
//
// Bound by memory.  A row is spread over w/8 lanes (the maximum is a 3- or
// 4-step shuffle); each lane moves 8 elements, and holds kU rows in flight.
// A block takes kTok tokens: their slots (or the sequences they belong to)
// are looked up once, in shared memory, and used by all heads.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/lt_linear_attn.h"
#include "lt_check.h"
#include "lt_internal.h"
#include "lt_ptx.cuh"
#include "lt_vec.cuh"

namespace lt {
namespace {

constexpr int kT = 256;   // threads
constexpr int kTok = 32;  // tokens per block
constexpr int kU = 4;     // rows in flight per thread
constexpr float kTiny = 1.17549435e-38f;  // 2^-126

struct Pool {
  void* p;
  float* scale;
  int64_t page, slot, head;  // strides, elements
  int w;                     // row width
};

struct CacheArgs {
  Pool pool[2];  // keys, values
  int num_pages, page_size, H;
  // write
  const void* in[2];
  int64_t stride[2];
  const int32_t* slots;
  int64_t tokens;
  // read
  void* out[2];
  const int32_t* table;
  int64_t table_stride;
  int max_pages;
  const int32_t* cu;
  int B, N;
  int* err;
};

// where a token's rows are: page and slot, or page -1
struct Place {
  int page, slot;
};

// ------------------------------------------------ eight elements <-> codes
// the cache's element types; Code<KV>::Raw is a lane's eight elements
struct E4M3 {};
struct Int8 {};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f) {
  widen(load_quad(p), f);
  widen(load_quad(p + 4), f + 4);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* f) {
  store_quad(p, f);
  store_quad(p + 4, f + 4);
}

__device__ __forceinline__ uint2 encode(const float* y, E4M3) {
  uint2 r;
  const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(y[4], y[5]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t d = __nv_cvt_float2_to_fp8x2(make_float2(y[6], y[7]), __NV_SATFINITE, __NV_E4M3);
  r.x = a | (b << 16);
  r.y = c | (d << 16);
  return r;
}
__device__ __forceinline__ uint2 encode(const float* y, Int8) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[h] |= ((uint32_t)__float2int_rn(y[4 * h + e]) & 0xffu) << (8 * e);
  }
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void decode(uint2 r, float* y, E4M3) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t word = h < 2 ? r.x : r.y;
    const __half2_raw t =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(word >> (16 * (h & 1))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&t));
    y[2 * h] = f.x;
    y[2 * h + 1] = f.y;
  }
}
__device__ __forceinline__ void decode(uint2 r, float* y, Int8) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    y[e] = (float)(int8_t)((e < 4 ? r.x : r.y) >> (8 * (e & 3)));
}

template <typename KV>
struct IsQuant {
  static constexpr bool value = false;
};
template <>
struct IsQuant<E4M3> {
  static constexpr bool value = true;
};
template <>
struct IsQuant<Int8> {
  static constexpr bool value = true;
};
template <typename KV>
__device__ __forceinline__ float qmax() {
  return 448.0f;
}
template <>
__device__ __forceinline__ float qmax<Int8>() {
  return 127.0f;
}

// ------------------------------------------------------------------- write
// blockIdx.y: 0 keys, 1 values
template <typename T, typename KV>
__global__ void __launch_bounds__(kT) lt_kv_write_kernel(const CacheArgs a) {
  __shared__ Place place[kTok];
  const int which = blockIdx.y;
  const Pool pool = a.pool[which];
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  const int nt = (int)min((int64_t)kTok, a.tokens - t0);
  if (threadIdx.x < nt) {
    const int s = a.slots[t0 + threadIdx.x];
    Place pl{-1, 0};
    if (s >= 0 && s / a.page_size < a.num_pages)
      pl = Place{s / a.page_size, s % a.page_size};
    else if (s != -1)
      report_error(a.err, kDevErrBadPage);
    place[threadIdx.x] = pl;
  }
  __syncthreads();
  const int L = pool.w >> 3, RG = kT / L;  // lanes per row, rows at a time
  const int grp = threadIdx.x / L, j = threadIdx.x % L;
  const int rows = nt * a.H;
  const T* in = static_cast<const T*>(a.in[which]) + t0 * a.stride[which] + j * 8;
  const int first = (threadIdx.x & ~31) / L;  // warps stay converged for the shuffles
#pragma unroll 1
  for (int r = grp, rw = first; rw < rows; r += RG * kU, rw += RG * kU) {
    float y[kU][8];
    Place pl[kU];
    int hd[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int row = r + u * RG;
      pl[u].page = -1;
      hd[u] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[u][e] = 0.0f;
      if (row < rows) {
        const int tt = row / a.H;
        hd[u] = row - tt * a.H;
        pl[u] = place[tt];
        if (pl[u].page >= 0) load8(in + (int64_t)tt * a.stride[which] + hd[u] * pool.w, y[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t off = (int64_t)pl[u].page * pool.page + (int64_t)pl[u].slot * pool.slot +
                          (int64_t)hd[u] * pool.head + j * 8;
      if constexpr (!IsQuant<KV>::value) {
        if (pl[u].page >= 0) store8(static_cast<T*>(pool.p) + off, y[u]);
      } else {
        // the largest magnitude as bits: those of a NaN and of an infinity lie
        // above every finite one, so a row that holds any is seen
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(y[u][e]) & 0x7fffffffu);
        for (int o = L >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const bool finite = top < 0x7f800000u;
        const float scale = finite ? fmaxf(__fdiv_rn(__uint_as_float(top), qmax<KV>()), kTiny)
                                   : __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[u][e] = finite ? __fdiv_rn(y[u][e], scale) : 0.0f;
        const uint2 c = encode(y[u], KV());
        if (pl[u].page >= 0) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool.p) + off) = c;
          if (j == 0)
            pool.scale[((int64_t)pl[u].page * a.H + hd[u]) * a.page_size + pl[u].slot] = scale;
        }
      }
    }
  }
}

// -------------------------------------------------------------------- read
template <typename T, typename KV>
__global__ void __launch_bounds__(kT) lt_kv_read_kernel(const CacheArgs a) {
  __shared__ Place place[kTok];
  const int which = blockIdx.y;
  const Pool pool = a.pool[which];
  const int t0 = blockIdx.x * kTok;
  const int nt = min(kTok, a.N - t0);
  if (blockIdx.x == 0 && which == 0) {  // every offset, whichever rows it describes
    for (int s = threadIdx.x; s < a.B; s += kT) {
      const int begin = a.cu[s], end = a.cu[s + 1];
      if ((s == 0 && begin != 0) || begin < 0 || end < begin || end > a.N ||
          (int64_t)end - begin > (int64_t)a.max_pages * a.page_size)
        report_error(a.err, kDevErrBadSeqlens);
    }
  }
  if (threadIdx.x < nt) {
    // the sequence that holds row t: the last s with cu[s] <= t; a row that
    // no sequence holds is left alone
    const int t = t0 + threadIdx.x;
    int lo = 0, hi = a.B;  // cu[lo] <= t < cu[hi], for consistent offsets
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const int begin = a.cu[lo], end = a.cu[lo + 1];
    Place pl{-1, 0};
    if (begin >= 0 && t >= begin && t < end &&
        (int64_t)end - begin <= (int64_t)a.max_pages * a.page_size) {
      const int i = t - begin, page = a.table[(int64_t)lo * a.table_stride + i / a.page_size];
      if (page >= 0 && page < a.num_pages)
        pl = Place{page, i % a.page_size};
      else
        report_error(a.err, kDevErrBadPage);
    }
    place[threadIdx.x] = pl;
  }
  __syncthreads();
  const int L = pool.w >> 3, RG = kT / L;
  const int grp = threadIdx.x / L, j = threadIdx.x % L;
  const int rows = nt * a.H;
  T* out = static_cast<T*>(a.out[which]) + (int64_t)t0 * a.H * pool.w + j * 8;
#pragma unroll 1
  for (int r = grp; r < rows; r += RG * kU) {
    float y[kU][8], scale[kU];
    uint2 c[kU];
    bool live[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int row = r + u * RG;
      live[u] = false;
      if (row < rows) {
        const int tt = row / a.H, h = row - tt * a.H;
        const Place pl = place[tt];
        live[u] = pl.page >= 0;
        if (live[u]) {
          const int64_t off = (int64_t)pl.page * pool.page + (int64_t)pl.slot * pool.slot +
                              (int64_t)h * pool.head + j * 8;
          if constexpr (IsQuant<KV>::value) {
            c[u] = __ldg(reinterpret_cast<const uint2*>(static_cast<uint8_t*>(pool.p) + off));
            scale[u] = __ldg(&pool.scale[((int64_t)pl.page * a.H + h) * a.page_size + pl.slot]);
          } else {
            load8(static_cast<const T*>(pool.p) + off, y[u]);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (!live[u]) continue;
      if constexpr (IsQuant<KV>::value) {
        decode(c[u], y[u], KV());
#pragma unroll
        for (int e = 0; e < 8; ++e) y[u][e] *= scale[u];
      }
      store8(out + (int64_t)(r + u * RG) * pool.w, y[u]);
    }
  }
}

template <typename T, typename KV>
cudaError_t launch_t(const CacheArgs& a, bool write, cudaStream_t s) {
  const int64_t n = write ? a.tokens : a.N;
  const dim3 grid((unsigned)((n + kTok - 1) / kTok), 2);
  if (write)
    lt_kv_write_kernel<T, KV><<<grid, kT, 0, s>>>(a);
  else
    lt_kv_read_kernel<T, KV><<<grid, kT, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_kv(const CacheArgs& a, lt_kv_dtype_t kv, bool write, cudaStream_t s) {
  if (kv == LT_KV_E4M3) return launch_t<T, E4M3>(a, write, s);
  if (kv == LT_KV_INT8) return launch_t<T, Int8>(a, write, s);
  return launch_t<T, T>(a, write, s);
}

cudaError_t launch(const CacheArgs& a, lt_dtype_t t, lt_kv_dtype_t kv, bool write,
                   cudaStream_t s) {
  return t == LT_BF16  ? launch_kv<__nv_bfloat16>(a, kv, write, s)
         : t == LT_F16 ? launch_kv<__half>(a, kv, write, s)
                       : launch_kv<float>(a, kv, write, s);
}

CacheArgs args_of(const lt_kv_cache_t* c) {
  CacheArgs a = {};
  a.pool[0] = Pool{c->k, c->k_scale, c->k_page_stride, c->k_slot_stride, c->k_head_stride, c->d};
  a.pool[1] = Pool{c->v, c->v_scale, c->v_page_stride, c->v_slot_stride, c->v_head_stride, c->dv};
  a.num_pages = c->num_pages;
  a.page_size = c->page_size;
  a.H = c->H_kv;
  return a;
}

// bytes from a pool's first element to its last
size_t pool_bytes(const lt_kv_cache_t* c, bool values) {
  const int64_t pg = values ? c->v_page_stride : c->k_page_stride;
  const int64_t sl = values ? c->v_slot_stride : c->k_slot_stride;
  const int64_t hd = values ? c->v_head_stride : c->k_head_stride;
  const int64_t w = values ? c->dv : c->d;
  return (size_t)((c->num_pages - 1) * pg + (c->page_size - 1) * sl + (c->H_kv - 1) * hd + w) *
         kv_size(c->dtype);
}

}  // namespace

lt_status_t check_cache(const lt_kv_cache_t* c) {
  if (!c) return LT_ERR_INVALID_ARG;
  if (c->dtype < LT_KV_F32 || c->dtype > LT_KV_INT8) return LT_ERR_UNSUPPORTED;
  if ((c->d != 64 && c->d != 128) || (c->dv != 64 && c->dv != 128)) return LT_ERR_UNSUPPORTED;
  if (!c->k || !c->v || !aligned_to(c->k, 16) || !aligned_to(c->v, 16)) return LT_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1 || c->page_size > 65536 || c->H_kv < 1 ||
      c->H_kv > 65535)
    return LT_ERR_INVALID_ARG;
  if ((int64_t)c->num_pages * c->page_size > 0x7fffffff) return LT_ERR_INVALID_ARG;  // slots: int32
  const int64_t es = (int64_t)kv_size(c->dtype);
  const int64_t st[] = {c->k_page_stride, c->k_slot_stride, c->k_head_stride,
                        c->v_page_stride, c->v_slot_stride, c->v_head_stride};
  const int64_t ext[] = {c->num_pages, c->page_size, c->H_kv};
  for (int i = 0; i < 6; ++i) {
    // a stride that no second row uses may be anything that keeps alignment
    const int64_t w = i < 3 ? c->d : c->dv;
    if (st[i] < 0 || (st[i] * es) % 16 != 0 || st[i] > ((int64_t)1 << 44)) return LT_ERR_INVALID_ARG;
    if (ext[i % 3] > 1 && (st[i] < w || st[i] > ((int64_t)1 << 58) / ext[i % 3]))
      return LT_ERR_INVALID_ARG;
  }
  if (eight_bit(c->dtype) ? (!c->k_scale || !c->v_scale || !aligned_to(c->k_scale, 4) ||
                             !aligned_to(c->v_scale, 4))
                          : (c->k_scale || c->v_scale))
    return LT_ERR_INVALID_ARG;
  return LT_OK;
}

lt_status_t check_cache_pointers(const lt_kv_cache_t* c) {
  if (!on_current_device(c->k) || !on_current_device(c->v) ||
      (c->k_scale && !on_current_device(c->k_scale)) ||
      (c->v_scale && !on_current_device(c->v_scale)))
    return LT_ERR_INVALID_ARG;
  return LT_OK;
}

void cache_spans(const lt_kv_cache_t* c, Span out[4]) {
  const size_t rows = (size_t)c->num_pages * c->page_size * c->H_kv;
  out[0] = Span{c->k, pool_bytes(c, false)};
  out[1] = Span{c->v, pool_bytes(c, true)};
  out[2] = Span{c->k_scale, rows * 4};
  out[3] = Span{c->v_scale, rows * 4};
}

}  // namespace lt

extern "C" lt_status_t lt_kv_cache_write(const lt_kv_cache_t* cache, const void* k, const void* v,
                                         const int32_t* slots, int64_t tokens, int64_t k_stride,
                                         int64_t v_stride, lt_stream_t stream, lt_dtype_t dtype) {
  using namespace lt;
  const lt_status_t st = check_cache(cache);
  if (st != LT_OK) return st;
  if (!dtype_ok(dtype) || (!eight_bit(cache->dtype) && cache->dtype != kv_of(dtype)))
    return LT_ERR_UNSUPPORTED;
  const size_t es = dtype_size(dtype);
  if (!k || !v || !slots || tokens < 1 || tokens > (int64_t)kTok * 0x7fffffff ||
      !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(slots, 4) ||
      !stride_ok(tokens, k_stride, cache->H_kv, cache->d, es) ||
      !stride_ok(tokens, v_stride, cache->H_kv, cache->dv, es))
    return LT_ERR_INVALID_ARG;
  Span pools[4];
  cache_spans(cache, pools);
  const Span ins[] = {{k, strided_bytes(tokens, k_stride, cache->H_kv, cache->d, es)},
                      {v, strided_bytes(tokens, v_stride, cache->H_kv, cache->dv, es)},
                      {slots, (size_t)tokens * 4}};
  for (const Span& p : pools)
    for (const Span& i : ins)
      if (spans_overlap(p, i)) return LT_ERR_INVALID_ARG;
  if (check_cache_pointers(cache) != LT_OK || !on_current_device(k) || !on_current_device(v) ||
      !on_current_device(slots))
    return LT_ERR_INVALID_ARG;
  CacheArgs a = args_of(cache);
  a.in[0] = k;
  a.in[1] = v;
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.slots = slots;
  a.tokens = tokens;
  a.err = device_error_word_current();
  if (!a.err) return LT_ERR_CUDA;
  return launch(a, dtype, cache->dtype, true, (cudaStream_t)stream) == cudaSuccess ? LT_OK
                                                                                    : LT_ERR_CUDA;
}

extern "C" lt_status_t lt_kv_cache_read(const lt_kv_cache_t* cache, const int32_t* block_table,
                                        int64_t table_stride, int max_pages,
                                        const int32_t* cu_seqlens, int B, int N, void* k_out,
                                        void* v_out, lt_stream_t stream, lt_dtype_t dtype) {
  using namespace lt;
  const lt_status_t st = check_cache(cache);
  if (st != LT_OK) return st;
  if (!dtype_ok(dtype) || (!eight_bit(cache->dtype) && cache->dtype != kv_of(dtype)))
    return LT_ERR_UNSUPPORTED;
  if (!block_table || !cu_seqlens || !k_out || !v_out || B < 1 || N < 1 || max_pages < 1 ||
      table_stride < max_pages || table_stride > ((int64_t)1 << 40) ||
      !aligned_to(block_table, 4) || !aligned_to(cu_seqlens, 4) || !aligned_to(k_out, 16) ||
      !aligned_to(v_out, 16))
    return LT_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype);
  Span ins[6];
  cache_spans(cache, ins);
  ins[4] = Span{block_table, ((size_t)(B - 1) * table_stride + max_pages) * 4};
  ins[5] = Span{cu_seqlens, ((size_t)B + 1) * 4};
  const Span ko = {k_out, (size_t)N * cache->H_kv * cache->d * es};
  const Span vo = {v_out, (size_t)N * cache->H_kv * cache->dv * es};
  if (spans_overlap(ko, vo)) return LT_ERR_INVALID_ARG;
  for (const Span& i : ins)
    if (spans_overlap(ko, i) || spans_overlap(vo, i)) return LT_ERR_INVALID_ARG;
  if (check_cache_pointers(cache) != LT_OK || !on_current_device(block_table) ||
      !on_current_device(cu_seqlens) || !on_current_device(k_out) || !on_current_device(v_out))
    return LT_ERR_INVALID_ARG;
  CacheArgs a = args_of(cache);
  a.table = block_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.cu = cu_seqlens;
  a.B = B;
  a.N = N;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.err = device_error_word_current();
  if (!a.err) return LT_ERR_CUDA;
  return launch(a, dtype, cache->dtype, false, (cudaStream_t)stream) == cudaSuccess ? LT_OK
                                                                                     : LT_ERR_CUDA;
}
