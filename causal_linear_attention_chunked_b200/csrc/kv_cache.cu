// kv_cache.cu -- rows of keys and values into a paged cache, quantised as
// they are written, and a batch of sequences read back, packed.
//
// Per row x (one head of one token): scale = max(max|x| / qmax, 2^-126),
// code = round(x / scale), qmax 448 (e4m3) or 127 (int8).  Both divisions are
// the correctly rounded ones, so the codes follow from the inputs alone and
// do not depend on how a row is spread over lanes.  The floor on the scale
// makes a row of zeros read back as zeros without a case of its own.
//
// Bound by memory, quantising also close to instruction issue: the maximum of
// a 16-bit row is taken two values at a time, and the quotients by a
// multiplication with corrections (below) whose codes are the division's.
// A row is spread over w/16 lanes (the maximum is a 2- or 3-step shuffle);
// each lane moves two chunks of 8 elements, w/2 apart, so that both the 16-bit
// and the 8-bit side are accessed in whole runs.  Quantising, the warps of the
// blocks that stay on the SMs step through the rows, a step's loads under way
// while the step before is worked on, and look a row's slot up with its values
// (a block per tile of tokens with the lookups in shared memory: 20% slower at
// 16384 tokens of 8 heads of 64).  Copying and reading back, a block does one
// tile of tokens, looks up its places once for all heads, and hides that
// behind other blocks' rows.
//
// Measured on one B200 (plain copy 6.55 TB/s): 32768 bf16 tokens of 8 heads of
// 128, keys and values, into e4m3 pages 38 us, 5.4 TB/s (16384 fp32 tokens 28 us,
// 6.1 TB/s); 64 ragged sequences (270k tokens of 8 heads of 64) back from e4m3 to
// bf16 134 us, 6.3 TB/s.
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

constexpr int kT = 256;      // threads
constexpr int kMaxTok = 64;  // tokens per tile, at most
// quantising: blocks per SM for keys, and as many for values
constexpr int kQuantBlocks = 2;

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
  int tok;  // tokens per tile
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
  uint32_t page_magic;  // quantising: floor(2^(31 + page_shift) / page_size) + 1
  int page_shift;       // ceil(log2(page_size))
  int* err;
};

// where a token's rows are in a pool and its scales: offsets of its first head,
// or -1
struct Place {
  int64_t row;    // elements
  int64_t scale;  // a head's scales are page_size apart
};

// A block's (token, head) rows in order, advanced by a fixed step.
struct RowAt {
  int tt, h, dt, dh, H;
  __device__ __forceinline__ RowAt(int first, int step, int heads) : H(heads) {
    tt = first / heads;
    h = first - tt * heads;
    dt = step / heads;
    dh = step - dt * heads;
  }
  __device__ __forceinline__ void next() {
    tt += dt;
    h += dh;
    if (h >= H) {
      h -= H;
      ++tt;
    }
  }
};

// ------------------------------------------------- chunks of eight elements
template <typename KV>
struct KvMax;
template <>
struct KvMax<E4M3> {
  static constexpr float value = 448.0f;
};
template <>
struct KvMax<Int8> {
  static constexpr float value = 127.0f;
};

template <typename T>
struct Chunk {  // 16-bit elements
  uint4 r;
};
template <>
struct Chunk<float> {
  float4 r[2];
};
template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* p) {
  Chunk<T> c;
  if constexpr (sizeof(T) == 2) {
    c.r = __ldg(reinterpret_cast<const uint4*>(p));
  } else {
    c.r[0] = __ldg(reinterpret_cast<const float4*>(p));
    c.r[1] = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  return c;
}
template <typename T>
__device__ __forceinline__ void widen8(const Chunk<T>& c, F2* f) {
  if constexpr (sizeof(T) == 2) {
    widen2x2(Quad<T>{make_uint2(c.r.x, c.r.y)}, f);
    widen2x2(Quad<T>{make_uint2(c.r.z, c.r.w)}, f + 2);
  } else {
    widen2x2(Quad<float>{c.r[0]}, f);
    widen2x2(Quad<float>{c.r[1]}, f + 2);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const F2* f) {
  if constexpr (sizeof(T) == 2) {
    uint4 r;
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = unpack_f2(f[e]);
      T two[2];
      from_float(&two[0], x.x);
      from_float(&two[1], x.y);
      w[e] = *reinterpret_cast<const uint32_t*>(two);
    }
    *reinterpret_cast<uint4*>(p) = r;
  } else {
    store_quad(p, f[0], f[1]);
    store_quad(p + 4, f[2], f[3]);
  }
}

// Bits of the largest magnitude of a chunk, as fp32.  Those of an infinity and
// of a NaN lie above every finite value's, so a row that holds one is seen.
__device__ __forceinline__ uint32_t top_bits(const Chunk<float>& c) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float f[4] = {c.r[q].x, c.r[q].y, c.r[q].z, c.r[q].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max(m, __float_as_uint(f[e]) & 0x7fffffffu);
  }
  return m;
}
__device__ __forceinline__ uint32_t top_bits(const Chunk<__nv_bfloat16>& c) {
  const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&c.r);
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(__habs2(w[0]), __habs2(w[1])),
                                       __hmax2_nan(__habs2(w[2]), __habs2(w[3])));
  return __float_as_uint(to_float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)))) &
         0x7fffffffu;
}
__device__ __forceinline__ uint32_t top_bits(const Chunk<__half>& c) {
  const __half2* w = reinterpret_cast<const __half2*>(&c.r);
  const __half2 m = __hmax2_nan(__hmax2_nan(__habs2(w[0]), __habs2(w[1])),
                                __hmax2_nan(__habs2(w[2]), __habs2(w[3])));
  return __float_as_uint(to_float(__hmax_nan(__low2half(m), __high2half(m)))) & 0x7fffffffu;
}

// Quotients by multiplication, for codes that are those of the correctly
// rounded quotients.  With v the correctly rounded reciprocal of b, q = x v is
// within two steps of x / b; one correction q + (x - q b) v brings it within
// one, and Markstein's theorem (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990) makes a second, whose
// remainder is exact, the rounded quotient.  The remainder is exact while it
// stays above fp32's smallest numbers: for a row's largest magnitude within
// 2^-60 .. 2^60 that holds for the scale, and for every quotient that does not
// round to code 0 anyway.  Other rows divide.
//
// 16-bit inputs need one correction only: a code goes by two 8-bit (11-bit)
// significands and the difference of their exponents, and over all of those
// (22 differences; more give code 0) one correction gives the same codes (none
// leaves 140 of 352320 bf16 cases different).  For them the reciprocal may be a
// step off, which the correction's last factor does not notice.
//
// What is computed is minus the quotient, p = -(x v), p + (x + p b)(-v): so a
// zero keeps its sign, which x - q b would lose.
__device__ __forceinline__ float near_reciprocal(float b) {
  float v;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(v) : "f"(b));
  return fmaf(v, fmaf(-b, v, 1.0f), v);  // a Newton step
}
template <int kCorrections>
__device__ __forceinline__ F2 minus_quotient(F2 x, F2 b, F2 minus_v) {
  F2 p = mul2(x, minus_v);
#pragma unroll
  for (int i = 0; i < kCorrections; ++i) p = fma2(fma2(p, b, x), minus_v, p);
  return p;
}
// y[0..7] -> -(y / scale), with the row's scale from the bits of its largest
// magnitude (where that is not finite: zeros, and NaN)
template <typename T, typename KV>
__device__ __forceinline__ float minus_quotients(F2* y, uint32_t top) {
  constexpr float kMax = KvMax<KV>::value;
  const float x = __uint_as_float(top);
  if (top - 0x21800000u <= 0x5d800000u - 0x21800000u) {  // 2^-60 .. 2^60
    constexpr float v = 1.0f / kMax;  // rounded by the compiler
    float q = x * v;
    q = fmaf(fmaf(q, -kMax, x), v, q);
    q = fmaf(fmaf(q, -kMax, x), v, q);
    const float r = -(sizeof(T) == 2 ? near_reciprocal(q) : __frcp_rn(q));
    const F2 b = pack_f2(q, q), n = pack_f2(r, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = minus_quotient<sizeof(T) == 2 ? 1 : 2>(y[e], b, n);
    return q;
  }
  if (top >= 0x7f800000u) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = pack_f2(-0.0f, -0.0f);
    return __uint_as_float(0x7fc00000u);
  }
  const float b = fmaxf(__fdiv_rn(x, kMax), kTiny);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 z = unpack_f2(y[e]);
    y[e] = pack_f2(__fdiv_rn(z.x, -b), __fdiv_rn(z.y, -b));
  }
  return b;
}

// the codes of -y[0..3]
__device__ __forceinline__ uint2 encode_minus(const F2* y, E4M3) {
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    h[e] = __nv_cvt_float2_to_fp8x2(unpack_f2(y[e]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2((h[0] | (h[1] << 16)) ^ 0x80808080u, (h[2] | (h[3] << 16)) ^ 0x80808080u);
}
__device__ __forceinline__ uint2 encode_minus(const F2* y, Int8) {
  // 1.5 * 2^23 - y rounds to an integer, ties to even, and leaves it in the
  // low bits as a two's complement number
  const F2 magic = pack_f2(12582912.0f, 12582912.0f), minus = pack_f2(-1.0f, -1.0f);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 a = unpack_f2(fma2(y[2 * h], minus, magic));
    const float2 b = unpack_f2(fma2(y[2 * h + 1], minus, magic));
    const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    w[h] = __byte_perm(lo, hi, 0x5410);
  }
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void decode(uint2 r, F2* y, E4M3) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t word = h < 2 ? r.x : r.y;
    const __half2_raw t =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(word >> (16 * (h & 1))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&t));
    y[h] = pack_f2(f.x, f.y);
  }
}
__device__ __forceinline__ void decode(uint2 r, F2* y, Int8) {
  // the byte, offset by 128, as the low bits of 2^23, less 2^23 + 128: exact
  const F2 bias = pack_f2(-8388736.0f, -8388736.0f);
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t word = (h < 2 ? r.x : r.y) ^ 0x80808080u;
    const uint32_t a = __byte_perm(word, 0x4b000000u, h & 1 ? 0x7442 : 0x7440);
    const uint32_t b = __byte_perm(word, 0x4b000000u, h & 1 ? 0x7443 : 0x7441);
    y[h] = add2(pack_f2(__uint_as_float(a), __uint_as_float(b)), bias);
  }
}

// ---------------------------------------------------------- tokens' places
__device__ __forceinline__ Place place_at(const CacheArgs& a, const Pool& pool, int page,
                                          int slot) {
  return Place{(int64_t)page * pool.page + (int64_t)slot * pool.slot,
               (int64_t)page * a.H * a.page_size + slot};
}

__device__ __forceinline__ Place place_of_slot(const CacheArgs& a, const Pool& pool, int64_t t) {
  const int s = a.slots[t];
  const int page = s / a.page_size;  // (meaningless below 0)
  if (s >= 0 && page < a.num_pages) return place_at(a, pool, page, s - page * a.page_size);
  if (s != -1) report_error(a.err, kDevErrBadPage);
  return Place{-1, 0};
}

__device__ __forceinline__ Place place_of_row(const CacheArgs& a, const Pool& pool, int t) {
  // the sequence that holds row t: the last s with cu[s] <= t; a row that no
  // sequence holds is left alone
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu + mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int begin = __ldg(a.cu + lo), end = __ldg(a.cu + lo + 1);
  if (begin >= 0 && t >= begin && t < end && end <= a.N &&
      (int64_t)end - begin <= (int64_t)a.max_pages * a.page_size) {
    const int i = t - begin, n = i / a.page_size;
    const int page = __ldg(a.table + (int64_t)lo * a.table_stride + n);
    if (page >= 0 && page < a.num_pages) return place_at(a, pool, page, i - n * a.page_size);
    report_error(a.err, kDevErrBadPage);
  }
  return Place{-1, 0};
}

// every offset of a batch, whichever rows it describes
__device__ __forceinline__ void check_offsets(const CacheArgs& a) {
  for (int s = threadIdx.x; s < a.B; s += kT) {
    const int begin = a.cu[s], end = a.cu[s + 1];
    if ((s == 0 && begin != 0) || begin < 0 || end < begin || end > a.N ||
        (int64_t)end - begin > (int64_t)a.max_pages * a.page_size)
      report_error(a.err, kDevErrBadSeqlens);
  }
}

// ----------------------------------------------------------------- kernels
// A block does one tile of tokens: `look` gives a token's place, `work` does the
// tile's rows (its first token, tokens and places).
template <typename Look, typename Work>
__device__ __forceinline__ void one_tile(int64_t n, int tok, const Look& look, const Work& work) {
  __shared__ Place place[kMaxTok];
  const int64_t t0 = (int64_t)blockIdx.x * tok;
  const int nt = (int)min((int64_t)tok, n - t0);
  if (threadIdx.x < nt) place[threadIdx.x] = look(t0 + threadIdx.x);
  __syncthreads();
  work(t0, nt, place);
}

template <typename T, typename KV, int WIDTH>
__device__ __forceinline__ void dequant_rows(const CacheArgs& a, const Pool& pool, T* out,
                                             const Place* place, int nt, RowAt at) {
  constexpr int kU = 4;
  constexpr int L = WIDTH / 16, HALF = WIDTH / 2, RG = kT / L;
  const int j = threadIdx.x % L, n = nt * a.H;
  out += j * 8;
#pragma unroll 1
  for (int r = threadIdx.x / L; r < n; r += RG * kU) {
    uint2 code[kU][2];
    float scale[kU];
    bool live[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      live[u] = false;
      if (r + u * RG < n) {
        const Place pl = place[at.tt];
        live[u] = pl.row >= 0;
        if (live[u]) {
          const uint8_t* p =
              static_cast<const uint8_t*>(pool.p) + pl.row + at.h * pool.head + j * 8;
          code[u][0] = __ldg(reinterpret_cast<const uint2*>(p));
          code[u][1] = __ldg(reinterpret_cast<const uint2*>(p + HALF));
          scale[u] = __ldg(&pool.scale[pl.scale + (int64_t)at.h * a.page_size]);
        }
      }
      at.next();
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (!live[u]) continue;
      const F2 s2 = pack_f2(scale[u], scale[u]);
      T* o = out + (int64_t)(r + u * RG) * WIDTH;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        F2 y[4];
        decode(code[u][c], y, KV());
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], s2);
        store8(o + c * HALF, y);
      }
    }
  }
}

// Quantising: a warp takes 32 / L rows at a time, every so many apart.  A step's
// loads go out as soon as the step before has widened its own, and land while
// its codes are worked out (two steps ahead: no faster, and fp32 rows then do
// not fit the registers that four blocks per SM leave).
template <typename T, typename KV, int WIDTH>
__device__ __forceinline__ void quant_rows(const CacheArgs& a, const Pool& pool, int which) {
  constexpr int L = WIDTH / 16, HALF = WIDTH / 2, RW = 32 / L;  // lanes per row, rows per step
  const int lane = threadIdx.x & 31, j = lane % L;
  const int64_t warp = (int64_t)blockIdx.x * (kT / 32) + (threadIdx.x >> 5);
  const int64_t rows = a.tokens * a.H, step = (int64_t)gridDim.x * (kT / 32) * RW;
  if (warp * RW >= rows) return;
  const int n = (int)((rows - warp * RW + step - 1) / step);  // the warp's steps
  // token and head of this lane's next row to load
  const int64_t r0 = warp * RW + lane / L;
  uint32_t t = (uint32_t)(r0 / a.H), h = (uint32_t)(r0 - (int64_t)t * a.H);
  const uint32_t dt = (uint32_t)(step / a.H), dh = (uint32_t)(step - (int64_t)dt * a.H);
  const T* const in = static_cast<const T*>(a.in[which]) + j * 8;
  const int64_t stride = a.stride[which];
  Chunk<T> x[2];
  int slot, head;
  auto load = [&]() {
    const bool live = t < (uint32_t)a.tokens;
    const uint32_t tt = live ? t : 0;  // (past the last row: the first token's, not stored)
    const T* p = in + tt * stride + h * WIDTH;
    slot = live ? __ldg(a.slots + tt) : -1;
    head = h;
    x[0] = load_chunk(p);
    x[1] = load_chunk(p + HALF);
    t += dt;
    h += dh;
    if (h >= (uint32_t)a.H) {
      h -= a.H;
      ++t;
    }
  };
  load();
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    uint32_t top = max(top_bits(x[0]), top_bits(x[1]));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    F2 y[2][4];
    widen8(x[0], y[0]);
    widen8(x[1], y[1]);
    const int s = slot, hd = head;
    if (i + 1 < n) load();
    const float scale = minus_quotients<T, KV>(y[0], top);
    // s / page_size, exact for 0 <= s < 2^31
    const int page = (int)(((uint64_t)(uint32_t)s * a.page_magic) >> (31 + a.page_shift));
    if (s >= 0 && page < a.num_pages) {
      const int at = s - page * a.page_size;
      uint8_t* out = static_cast<uint8_t*>(pool.p) + page * pool.page + at * pool.slot +
                     hd * pool.head + j * 8;
      *reinterpret_cast<uint2*>(out) = encode_minus(y[0], KV());
      *reinterpret_cast<uint2*>(out + HALF) = encode_minus(y[1], KV());
      if (j == 0) pool.scale[((int64_t)page * a.H + hd) * a.page_size + at] = scale;
    } else if (s != -1) {
      report_error(a.err, kDevErrBadPage);
    }
  }
}
// blockIdx.y: 0 keys, 1 values
template <typename T, typename KV>
__global__ void __launch_bounds__(kT) lt_kv_quant_kernel(const CacheArgs a) {
  const Pool pool = a.pool[blockIdx.y];
  if (pool.w == 64)
    quant_rows<T, KV, 64>(a, pool, blockIdx.y);
  else
    quant_rows<T, KV, 128>(a, pool, blockIdx.y);
}

template <typename T, typename KV, int WIDTH>
__device__ __forceinline__ void dequant_tile(const CacheArgs& a, const Pool& pool, int which) {
  T* out = static_cast<T*>(a.out[which]);
  constexpr int L = WIDTH / 16;
  const RowAt at(threadIdx.x / L, kT / L, a.H);
  one_tile(
      a.N, a.tok, [&](int64_t t) { return place_of_row(a, pool, (int)t); },
      [&](int64_t t0, int nt, const Place* place) {
        dequant_rows<T, KV, WIDTH>(a, pool, out + t0 * a.H * WIDTH, place, nt, at);
      });
}
template <typename T, typename KV>
__global__ void __launch_bounds__(kT) lt_kv_dequant_kernel(const CacheArgs a) {
  const Pool pool = a.pool[blockIdx.y];
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(a);
  if (pool.w == 64)
    dequant_tile<T, KV, 64>(a, pool, blockIdx.y);
  else
    dequant_tile<T, KV, 128>(a, pool, blockIdx.y);
}

// Rows as they are, in 16-byte pieces: into the cache, or out of it.  Strides
// and widths are in bytes here, whatever the type.
template <bool kWrite>
__global__ void __launch_bounds__(kT) lt_kv_copy_kernel(const CacheArgs a) {
  constexpr int kU = 4;
  const int which = blockIdx.y;
  const Pool pool = a.pool[which];
  if (!kWrite && blockIdx.x == 0 && which == 0) check_offsets(a);
  const int L = pool.w >> 4, RG = kT / L;  // lanes per row, rows at a time
  const int grp = threadIdx.x / L, j = threadIdx.x % L;
  const int64_t stride = a.stride[which];
  const RowAt first(grp, RG, a.H);
  one_tile(
      kWrite ? a.tokens : (int64_t)a.N, a.tok,
      [&](int64_t t) { return kWrite ? place_of_slot(a, pool, t) : place_of_row(a, pool, (int)t); },
      [&](int64_t t0, int nt, const Place* place) {
        const int n = nt * a.H;
        const uint8_t* in = static_cast<const uint8_t*>(a.in[which]) + t0 * stride + j * 16;
        uint8_t* out = static_cast<uint8_t*>(a.out[which]) + t0 * a.H * pool.w + j * 16;
        RowAt at = first;
#pragma unroll 1
        for (int r = grp; r < n; r += RG * kU) {
          uint4 x[kU];
          uint8_t* dst[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            dst[u] = nullptr;
            if (r + u * RG < n) {
              const Place pl = place[at.tt];
              if (pl.row >= 0) {
                uint8_t* row =
                    static_cast<uint8_t*>(pool.p) + pl.row + at.h * pool.head + j * 16;
                const uint8_t* src = kWrite ? in + at.tt * stride + at.h * pool.w : row;
                dst[u] = kWrite ? row : out + (int64_t)(r + u * RG) * pool.w;
                x[u] = __ldg(reinterpret_cast<const uint4*>(src));
              }
            }
            at.next();
          }
#pragma unroll
          for (int u = 0; u < kU; ++u)
            if (dst[u]) *reinterpret_cast<uint4*>(dst[u]) = x[u];
        }
      });
}

template <typename T>
cudaError_t launch_quant(const CacheArgs& a, bool e4m3, bool write, dim3 grid, cudaStream_t s) {
  if (write)
    e4m3 ? lt_kv_quant_kernel<T, E4M3><<<grid, kT, 0, s>>>(a)
         : lt_kv_quant_kernel<T, Int8><<<grid, kT, 0, s>>>(a);
  else
    e4m3 ? lt_kv_dequant_kernel<T, E4M3><<<grid, kT, 0, s>>>(a)
         : lt_kv_dequant_kernel<T, Int8><<<grid, kT, 0, s>>>(a);
  return cudaGetLastError();
}

// Tokens per tile, at most kMaxTok: enough rows for every group of a block's
// threads (at most 64: a row has four lanes or more), few enough that a batch
// spreads over the device, and kTileBytes of the dense side at most (token: its
// bytes there).  32 KB: 49k bf16 tokens of 8 heads of 128 read back in 64.7 us, 270k
// of 64 from e4m3 in 143; 16 KB 67.4 and 162, 64 KB 66.0 and 146.
constexpr int kTileBytes = 32768;
int tile_tokens(int64_t tokens, int heads, int lanes, int64_t token, int sms) {
  const int64_t least = (kT / lanes + heads - 1) / heads, fit = kTileBytes / token;
  const int64_t most = fit < least ? least : fit > kMaxTok ? kMaxTok : fit;
  const int64_t n = tokens / (4 * sms);
  return (int)(n < least ? least : n > most ? most : n);
}

cudaError_t launch(CacheArgs a, lt_dtype_t t, lt_kv_dtype_t kv, bool write, int sms,
                   cudaStream_t s) {
  const int64_t n = write ? a.tokens : a.N;
  const int row = (a.pool[0].w > a.pool[1].w ? a.pool[0].w : a.pool[1].w) * (int)kv_size(kv);
  const int64_t token = (int64_t)a.H * (row / (int)kv_size(kv)) * (int64_t)dtype_size(t);
  a.tok = tile_tokens(n, a.H, row / 16, token, sms);
  dim3 grid((unsigned)((n + a.tok - 1) / a.tok), 2);
  if (eight_bit(kv) && write) {
    while ((1 << a.page_shift) < a.page_size) ++a.page_shift;
    a.page_magic = (uint32_t)(((uint64_t)1 << (31 + a.page_shift)) / a.page_size + 1);
    // as many blocks as stay on the SMs, fewer where they would have no row
    const int64_t rows = n * a.H, per = kT / (row / 16), most = kQuantBlocks * sms;
    grid.x = (unsigned)(rows > per * most ? most : (rows + per - 1) / per);
  }
  if (eight_bit(kv)) {
    const bool e4m3 = kv == LT_KV_E4M3;
    return t == LT_BF16  ? launch_quant<__nv_bfloat16>(a, e4m3, write, grid, s)
           : t == LT_F16 ? launch_quant<__half>(a, e4m3, write, grid, s)
                         : launch_quant<float>(a, e4m3, write, grid, s);
  }
  const int es = (int)kv_size(kv);
  for (int i = 0; i < 2; ++i) {
    a.pool[i].page *= es;
    a.pool[i].slot *= es;
    a.pool[i].head *= es;
    a.pool[i].w *= es;
    a.stride[i] *= es;
  }
  if (write)
    lt_kv_copy_kernel<true><<<grid, kT, 0, s>>>(a);
  else
    lt_kv_copy_kernel<false><<<grid, kT, 0, s>>>(a);
  return cudaGetLastError();
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
    if (st[i] < 0 || (st[i] * es) % 16 != 0 || st[i] > ((int64_t)1 << 44))
      return LT_ERR_INVALID_ARG;
    if (ext[i % 3] > 1 && (st[i] < w || st[i] > ((int64_t)1 << 58) / ext[i % 3]))
      return LT_ERR_INVALID_ARG;
  }
  if (eight_bit(c->dtype) ? (!c->k_scale || !c->v_scale || !aligned_to(c->k_scale, 4) ||
                             !aligned_to(c->v_scale, 4))
                          : (c->k_scale || c->v_scale))
    return LT_ERR_INVALID_ARG;
  return LT_OK;
}

lt_status_t check_cache_pointers(int dev, const lt_kv_cache_t* c) {
  if (!on_device(dev, c->k) || !on_device(dev, c->v) ||
      (c->k_scale && !on_device(dev, c->k_scale)) ||
      (c->v_scale && !on_device(dev, c->v_scale)))
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
  if (!k || !v || !slots || tokens < 1 || tokens > 0x7fffffff ||
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
  const int dev = current_device();
  if (check_cache_pointers(dev, cache) != LT_OK || !on_device(dev, k) || !on_device(dev, v) ||
      !on_device(dev, slots))
    return LT_ERR_INVALID_ARG;
  CacheArgs a = args_of(cache);
  a.in[0] = k;
  a.in[1] = v;
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.slots = slots;
  a.tokens = tokens;
  a.err = device_error_word_current();
  const int sms = device_sm_count();
  if (!a.err || sms <= 0) return LT_ERR_CUDA;
  return launch(a, dtype, cache->dtype, true, sms, (cudaStream_t)stream) == cudaSuccess
             ? LT_OK
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
  if (!block_table || !cu_seqlens || !k_out || !v_out || B < 1 || B > (1 << 30) || N < 1 ||
      max_pages < 1 || table_stride < max_pages || table_stride > ((int64_t)1 << 40) ||
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
  const int dev = current_device();
  if (check_cache_pointers(dev, cache) != LT_OK || !on_device(dev, block_table) ||
      !on_device(dev, cu_seqlens) || !on_device(dev, k_out) || !on_device(dev, v_out))
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
  const int sms = device_sm_count();
  if (!a.err || sms <= 0) return LT_ERR_CUDA;
  return launch(a, dtype, cache->dtype, false, sms, (cudaStream_t)stream) == cudaSuccess
             ? LT_OK
             : LT_ERR_CUDA;
}
