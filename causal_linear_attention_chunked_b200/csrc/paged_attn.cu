// paged_attn.cu -- softmax attention of one new token per sequence over a
// paged key-value cache.
//
// For sequence b, KV head g and its query heads h (G per KV head), over the
// keys j that the window keeps:
//     out_h = sum_j p_j V_j / sum_j p_j,   p_j = exp(scale q_h . K_j).
// One pass over the cache: with m the largest score so far, each tile adds
// exp2(s_j - m) and exp2(s_j - m) V_j to a running sum and accumulator, which
// are rescaled when m grows.  Pieces of a sequence join by the same rule.
//
// Bound by memory: every key and value is read once, for G <= 16 query heads,
// 2G flops per byte of a 16-bit cache.
//
// Split: the cache of all (sequence, KV head) pairs, cut into tiles of kTile
// tokens and laid end to end, is dealt out in equal runs to the warps of one
// launch with a fixed number of blocks, whatever the lengths: a batch of very
// different sequences and one long sequence load the SMs alike, and the
// workspace does not grow with either.  A warp owns its run: its own ring of
// tiles in shared memory, filled with 16-byte asynchronous copies, its own
// running maximum and sum; no barrier between warps.  A pair that lies inside
// one run is finished by its warp.  A pair that several runs share leaves one
// partial result per run, and a second launch, which starts early and waits
// for the first, joins them in run order, so results do not depend on timing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/lt_linear_attn.h"
#include "lt_check.h"
#include "lt_internal.h"
#include "lt_ptx.cuh"
#include "lt_vec.cuh"

namespace lt {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct E4M3 {
  uint8_t b;
};
struct Int8 {
  int8_t b;
};

struct DecodeArgs {
  const void* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  int64_t kpg, ksl, khd, vpg, vsl, vhd;  // pool strides, bytes
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  int B, Hq, Hkv, G, nhb;  // nhb: blocks of query heads per KV head
  int hb;                  // query heads per block (the engine's kHeads)
  int num_pages, page_size, max_pages, window;
  int tile;       // tokens per tile
  int warps;      // runs the tiles are dealt to
  int min_tiles;  // shortest run
  float scale;
  void* out;
  float* lse;
  float* part;  // [warps][2][hb][dv] partial accumulators
  float* ml;    // [warps][2][hb][2] their maximum and sum
  int dv, dtype;
  int* err;
};

// ------------------------------------------------------------ the schedule
struct Seq {
  int first, len;  // keys [first, len) take part
  int tiles;
  bool bad;
};
__device__ __forceinline__ Seq seq_of(const DecodeArgs& a, int b) {
  Seq s;
  s.len = a.lens[b];
  // (positions up to a tile past the end stay inside 32 bits)
  s.bad = s.len < 0 || (int64_t)s.len > min((int64_t)a.max_pages * a.page_size, (int64_t)0x7fffff00);
  if (s.bad) s.len = 0;
  s.first = a.window ? max(0, s.len - a.window) : 0;
  s.tiles = (s.len - s.first + a.tile - 1) / a.tile;
  return s;
}

// tiles per run, from the tiles of all pairs
__device__ __forceinline__ int64_t run_length(const DecodeArgs& a, int64_t total) {
  return max((total + a.warps - 1) / a.warps, (int64_t)a.min_tiles);
}

// --------------------------------------------------------------- copies
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;  // the rest of the 16 bytes is zero-filled
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  const int n = live ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Position of 16-byte chunk c of row r in a tile whose rows are RB bytes:
// chunks are permuted within 128 bytes so that eight consecutive rows' chunk c
// lie in eight different bank groups.
template <int RB>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  constexpr int kPer = RB >= 128 ? 1 : 128 / RB;        // rows per 128 bytes
  constexpr int kMask = (RB >= 128 ? 8 : RB / 16) - 1;  // chunks permuted among
  return (uint32_t)(r * RB + ((c ^ ((r / kPer) & kMask)) << 4));
}

__device__ __forceinline__ float exp2_fast(float x) { return ex2_approx(x); }

// What an engine is told of a tile in shared memory.
struct TileAt {
  uint32_t k, v;     // shared addresses of the two tiles
  const float* ks;   // scales of the tile's tokens (8-bit caches)
  const float* vs;
  uint32_t mask;     // tokens that take part
};

// ------------------------------------------------- tensor-core instructions
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float* c, const uint32_t* a, uint32_t b0,
                                                   uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__half>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 t = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}

__device__ __forceinline__ void store_pair(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}
template <typename T>
__device__ __forceinline__ void store_pair(T* p, float a, float b) {
  *reinterpret_cast<uint32_t*>(p) = pack2<T>(a, b);
}

// Where an engine leaves a pair's result: rows of out and lse, or of the
// partial accumulators with their maximum and sum.
template <typename T>
struct Sink {
  bool partial;
  T* out;       // [heads][dv]
  float* lse;   // [heads] or nullptr
  float* part;  // [heads][dv]
  float* ml;    // [heads][2]
};

// the sum's reciprocal; no key with a weight above zero gives zeros
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
// log of the sum, of weights relative to 2^m
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// --------------------------------------------------- engine: tensor cores
template <typename KT>
struct KvTraits {  // 16-bit caches: the cache's own type, 16 tokens per tile
  using Math = KT;
  static constexpr int kBytes = 2, kTile = 16;
  static constexpr bool kQuant = false;
};
template <>
struct KvTraits<E4M3> {
  using Math = __half;  // every e4m3 value is an fp16 value
  static constexpr int kBytes = 1, kTile = 32;
  static constexpr bool kQuant = true;
};
template <>
struct KvTraits<Int8> {
  using Math = __half;
  static constexpr int kBytes = 1, kTile = 32;
  static constexpr bool kQuant = true;
};

// two bytes (the low half of w) -> two fp16 values, exactly
__device__ __forceinline__ uint32_t widen2(uint32_t w, E4M3) {
  const __half2_raw t = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
  return *reinterpret_cast<const uint32_t*>(&t);
}
// four bytes -> (bytes 0, 1) and (bytes 2, 3), or with kSplit (0, 2) and (1, 3)
template <bool kSplit>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi, E4M3 t) {
  if (kSplit) w = __byte_perm(w, 0, 0x3120);
  lo = widen2(w, t);
  hi = widen2(w >> 16, t);
}
// an integer byte x as the fp16 value 1024 + (x + 128) (its bits are 0x6400 plus
// the offset byte), less 1152: exact
template <bool kSplit>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi, Int8) {
  w ^= 0x80808080u;
  uint32_t a = __byte_perm(w, 0x64646464u, kSplit ? 0x4240 : 0x4140);
  uint32_t b = __byte_perm(w, 0x64646464u, kSplit ? 0x4341 : 0x4342);
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// Legacy mma on purpose: the 16 rows of the instruction are the query heads of
// one KV head (G of them live), a tcgen05 tile of 128 rows would be nearly
// empty, and the work is bound by memory: per 16 tokens of a 16-bit cache of
// width 128 a warp issues 32 mma and 16 ldmatrix for 8 KB read.
//
// Scores S = Q K^T: A = Q (heads x d, in registers), B = K (ldmatrix of the
// token rows).  S's registers are the second product's A layout, so P V needs
// no exchange; B = V by transposing ldmatrix.
//
// 8-bit caches are widened to fp16 in registers.  A lane's four bytes of a key
// row are four neighbouring d, where the instruction's B layout has two pairs
// eight apart: Q's registers are filled in the same order instead.  A lane's
// transposed word of V holds two columns of two tokens: one tile of even and
// one of odd columns.  Key scales multiply the scores; value scales go into
// the weights, relative to a power of two A >= every scale seen, so that the
// fp16 weights stay at most 2^kShift.  Q is scaled by a power of two per head
// into [1, 2), so that no bf16 query leaves fp16's range.
//
// kShift: fp16 weights are held times 2^12 (it cancels in the division), so
// that weights down to 2^-26 of the largest keep fp16's full precision; 2^12 *
// 65504 * 2^31 keys stay inside fp32.  bf16 has fp32's range and needs none.
template <typename QT_, typename KT, int D, int DV>
struct MmaEngine {
  using QT = QT_;
  using Kv = KvTraits<KT>;
  using MT = typename Kv::Math;
  static constexpr int kD = D, kHeads = 16, kTile = Kv::kTile, kWarps = 8;
  static constexpr int kKRow = D * Kv::kBytes, kVRow = DV * Kv::kBytes;  // bytes
  static constexpr bool kQuant = Kv::kQuant;
  static constexpr int kExtra = 0;  // shared bytes per warp beside the ring
  static constexpr float kShift = sizeof(MT) == 2 && !__is_same(MT, __nv_bfloat16) ? 12.0f : 0.0f;
  static constexpr int NT = kTile / 8;
  uint32_t qf[D / 16][4];
  float o[DV / 8][4];
  float m[2], l[2], sl2[2];
  uint32_t vtop;  // A's bits
  int heads;

  __device__ __forceinline__ void init(uint8_t*) {}

  __device__ __forceinline__ void begin(const QT* q, int nheads, float scale) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    heads = nheads;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.0f;
    sl2[0] = sl2[1] = scale * kLog2e;
    vtop = 0x00800000u;
#pragma unroll
    for (int j = 0; j < DV / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int h = r + 8 * half;
      const bool live = h < nheads;
      const uint32_t* row = reinterpret_cast<const uint32_t*>(q + (size_t)h * D);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        // pairs of elements, in words of two
        const int w0 = kQuant ? 8 * s + 2 * c : 8 * s + c;
        const int w1 = kQuant ? w0 + 1 : w0 + 4;
        qf[s][half] = live ? __ldg(row + w0) : 0u;
        qf[s][2 + half] = live ? __ldg(row + w1) : 0u;
      }
      if constexpr (kQuant) {
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 x = unpack(qf[s][2 * e + half]);
            top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t ex = min(max(__float_as_uint(top) >> 23, 7u), 247u);
        const float down = __uint_as_float((254u - ex) << 23);
        sl2[half] *= __uint_as_float(ex << 23);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 x = unpack(qf[s][2 * e + half]);
            qf[s][2 * e + half] = pack2<__half>(x.x * down, x.y * down);
          }
      }
    }
  }

  __device__ __forceinline__ static float2 unpack(uint32_t w) {
    if constexpr (__is_same(QT, __nv_bfloat16))
      return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
      return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }

  __device__ __forceinline__ void tile(const TileAt& t) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
    if constexpr (!kQuant) {
      const int row = (lane & 7) + ((lane >> 4) << 3), ch = (lane >> 3) & 1;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t b[4];
        ldsm4(b, t.k + chunk_at<kKRow>(row, 2 * i + ch));
        mma<MT>(s[0], qf[i], b[0], b[1]);
        mma<MT>(s[1], qf[i], b[2], b[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t w[4];
          ldsm4(w, t.k + chunk_at<kKRow>(8 * n + (lane & 7), 4 * i + (lane >> 3)));
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t b0, b1;
            widen4<false>(w[x], b0, b1, KT());
            mma<MT>(s[n], qf[4 * i + x], b0, b1);
          }
        }
    }
    // scores in units of log 2; tokens that take no part get -infinity
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float2 ks = make_float2(1.0f, 1.0f);
      if constexpr (kQuant) ks = *reinterpret_cast<const float2*>(t.ks + 8 * n + 2 * c);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool live = (t.mask >> (8 * n + 2 * c + e)) & 1u;
        const float kf = e ? ks.y : ks.x;
        s[n][e] = live ? s[n][e] * (sl2[0] * kf) : -INFINITY;
        s[n][2 + e] = live ? s[n][2 + e] * (sl2[1] * kf) : -INFINITY;
        mx[0] = fmaxf(mx[0], s[n][e]);
        mx[1] = fmaxf(mx[1], s[n][2 + e]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
    }
    uint32_t top = vtop;
    if constexpr (kQuant) {
      // A: the next power of two of the largest scale, within 2^-126 .. 2^126
      uint32_t v = (t.mask >> lane) & 1u ? __float_as_uint(t.vs[lane]) & 0x7fffffffu : 0u;
      v = __reduce_max_sync(0xffffffffu, v);
      v = v >= 0x7e800000u ? 0x7e800000u : (v + 0x7fffffu) & 0x7f800000u;
      top = max(top, v);
    }
    const float inv_a = __uint_as_float(0x7f000000u - top);
    if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1] || top != vtop)) {
      const float fa = kQuant ? __uint_as_float(vtop) * inv_a : 1.0f;
      float f[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        f[r] = mx[r] == m[r] ? 1.0f : exp2_fast(m[r] - mx[r]);
        l[r] *= f[r];
        f[r] *= fa;
        m[r] = mx[r];
      }
      vtop = top;
#pragma unroll
      for (int j = 0; j < DV / 8; ++j) {
        o[j][0] *= f[0];
        o[j][1] *= f[0];
        o[j][2] *= f[1];
        o[j][3] *= f[1];
      }
    }
    const float base[2] = {(m[0] == -INFINITY ? 0.0f : m[0]) - kShift,
                           (m[1] == -INFINITY ? 0.0f : m[1]) - kShift};
    uint32_t pf[kTile / 16][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float2 vs = make_float2(1.0f, 1.0f);
      if constexpr (kQuant) {
        vs = *reinterpret_cast<const float2*>(t.vs + 8 * n + 2 * c);
        vs.x *= inv_a;
        vs.y *= inv_a;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p0 = exp2_fast(s[n][2 * r] - base[r]);
        const float p1 = exp2_fast(s[n][2 * r + 1] - base[r]);
        l[r] += p0 + p1;
        pf[n >> 1][2 * (n & 1) + r] = pack2<MT>(p0 * vs.x, p1 * vs.y);
      }
    }
    if constexpr (!kQuant) {
      const int row = lane & 15, ch = lane >> 4;
#pragma unroll
      for (int j = 0; j < DV / 16; ++j) {
        uint32_t b[4];
        ldsm4t(b, t.v + chunk_at<kVRow>(row, 2 * j + ch));
        mma<MT>(o[2 * j], pf[0], b[0], b[1]);
        mma<MT>(o[2 * j + 1], pf[0], b[2], b[3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < DV / 32; ++j)
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          uint32_t w[4];
          ldsm4t(w, t.v + chunk_at<kVRow>(16 * kt + (lane & 15), 2 * j + (lane >> 4)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t e0, o0, e1, o1;
            widen4<true>(w[2 * x], e0, o0, KT());
            widen4<true>(w[2 * x + 1], e1, o1, KT());
            mma<MT>(o[4 * j + 2 * x], pf[kt], e0, e1);
            mma<MT>(o[4 * j + 2 * x + 1], pf[kt], o0, o1);
          }
        }
    }
  }

  __device__ __forceinline__ void finish(const Sink<QT>& out) {
    const int lane = threadIdx.x & 31, c = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float sum = l[r];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int h = (lane >> 2) + 8 * r;
      if (h >= heads) continue;
      const float mm = m[r] - kShift;
      float f = kQuant ? __uint_as_float(vtop) : 1.0f;
      if (out.partial) {
        if (c == 0) *reinterpret_cast<float2*>(out.ml + 2 * h) = make_float2(mm, sum);
        put(out.part + (size_t)h * DV, r, f);
      } else {
        if (c == 0 && out.lse) out.lse[h] = log_sum(mm, sum);
        put(out.out + (size_t)h * DV, r, f * inverse_sum(sum));
      }
    }
  }

  template <typename P>
  __device__ __forceinline__ void put(P* row, int r, float f) {
    const int c = threadIdx.x & 3;
    if constexpr (!kQuant) {
#pragma unroll
      for (int j = 0; j < DV / 8; ++j)
        store_pair(row + 8 * j + 2 * c, o[j][2 * r] * f, o[j][2 * r + 1] * f);
    } else {
#pragma unroll
      for (int j = 0; j < DV / 16; ++j) {
        const float y[4] = {o[2 * j][2 * r] * f, o[2 * j + 1][2 * r] * f, o[2 * j][2 * r + 1] * f,
                            o[2 * j + 1][2 * r + 1] * f};
        store_quad(row + 16 * j + 4 * c, y);
      }
    }
  }
};

// ----------------------------------------------------- engine: fp32 FMA
__device__ __forceinline__ void shared4(uint32_t addr, float* f, float) {
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
               : "r"(addr)
               : "memory");
}
template <typename KT>
__device__ __forceinline__ void shared4(uint32_t addr, float* f, KT) {
  uint32_t w, a, b;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(addr) : "memory");
  widen4<false>(w, a, b, KT());
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  f[0] = x.x;
  f[1] = x.y;
  f[2] = y.x;
  f[3] = y.y;
}

// fp32 queries: scores with two lanes per token (each half of the row's
// quads), then the weights through shared memory, each lane owning DV/32
// columns of the accumulator.  Up to eight query heads share a tile.
template <typename KT, int D, int DV>
struct FmaEngine {
  using QT = float;
  static constexpr int kBytes = sizeof(KT);
  static constexpr int kD = D, kHeads = 8, kTile = 16, kWarps = 4;
  static constexpr int kKRow = D * kBytes, kVRow = DV * kBytes;
  static constexpr bool kQuant = kBytes == 1;
  static constexpr int kExtra = kHeads * (D + kTile) * 4;  // queries, weights
  static constexpr int NC = DV / 32;                       // columns per lane
  float* qs;  // [kHeads][D]
  float* ps;  // [kHeads][kTile]
  float acc[kHeads][NC];
  float m[kHeads], l[kHeads];
  float sl2;
  int heads;

  __device__ __forceinline__ void init(uint8_t* extra) {
    qs = reinterpret_cast<float*>(extra);
    ps = qs + kHeads * D;
  }

  __device__ __forceinline__ void begin(const float* q, int nheads, float scale) {
    const int lane = threadIdx.x & 31;
    heads = nheads;
    sl2 = scale * kLog2e;
    __syncwarp();
    for (int i = lane; i < nheads * D; i += 32) qs[i] = __ldg(q + i);
    __syncwarp();
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.0f;
#pragma unroll
      for (int i = 0; i < NC; ++i) acc[h][i] = 0.0f;
    }
  }

  // four values at element e of row r
  template <int RB>
  __device__ __forceinline__ static void load4(uint32_t base, int r, int e, float* f) {
    const int byte = e * kBytes;
    shared4(base + chunk_at<RB>(r, byte >> 4) + (byte & 15), f, KT());
  }

  __device__ __forceinline__ void tile(const TileAt& t) {
    const int lane = threadIdx.x & 31, tok = lane >> 1, half = lane & 1;
    float s[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) s[h] = 0.0f;
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
      const int e = 4 * (2 * i + half);
      float k[4];
      load4<kKRow>(t.k, tok, e, k);
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
        if (h < heads) {
          const float4 q = *reinterpret_cast<const float4*>(qs + h * D + e);
          s[h] = fmaf(q.x, k[0], fmaf(q.y, k[1], fmaf(q.z, k[2], fmaf(q.w, k[3], s[h]))));
        }
    }
    const bool live = (t.mask >> tok) & 1u;
    const float kf = sl2 * (kQuant ? t.ks[tok] : 1.0f), vf = kQuant ? t.vs[tok] : 1.0f;
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (h < heads) {
        float x = s[h] + __shfl_xor_sync(0xffffffffu, s[h], 1);
        x = live ? x * kf : -INFINITY;
        float mx = fmaxf(m[h], x);
#pragma unroll
        for (int off = 2; off < 32; off <<= 1)
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        if (mx > m[h]) {
          const float f = exp2f(m[h] - mx);
          l[h] *= f;
#pragma unroll
          for (int i = 0; i < NC; ++i) acc[h][i] *= f;
          m[h] = mx;
        }
        const float p = exp2f(x - (mx == -INFINITY ? 0.0f : mx));
        l[h] += p;
        // a token that takes no part has zero-filled values, whatever its scale
        if (half == 0) ps[h * kTile + tok] = live ? p * vf : 0.0f;
      }
    __syncwarp();
#pragma unroll 2
    for (int j = 0; j < kTile; j += 4) {
      float v[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if constexpr (NC == 4) {
          load4<kVRow>(t.v, j + u, 4 * lane, v[u]);
        } else {  // two columns: this lane's half of a quad
          float x[4];
          load4<kVRow>(t.v, j + u, 4 * (lane >> 1), x);
          v[u][0] = half ? x[2] : x[0];
          v[u][1] = half ? x[3] : x[1];
        }
      }
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
        if (h < heads) {
          const float4 p = *reinterpret_cast<const float4*>(ps + h * kTile + j);
#pragma unroll
          for (int i = 0; i < NC; ++i)
            acc[h][i] = fmaf(p.x, v[0][i],
                             fmaf(p.y, v[1][i], fmaf(p.z, v[2][i], fmaf(p.w, v[3][i], acc[h][i]))));
        }
    }
  }

  __device__ __forceinline__ void finish(const Sink<float>& out) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
      if (h < heads) {
        float sum = l[h];
#pragma unroll
        for (int off = 2; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const float f = out.partial ? 1.0f : inverse_sum(sum);
        float* row = (out.partial ? out.part : out.out) + (size_t)h * DV + NC * lane;
#pragma unroll
        for (int i = 0; i < NC; ++i) row[i] = acc[h][i] * f;
        if (lane == 0) {
          if (out.partial)
            *reinterpret_cast<float2*>(out.ml + 2 * h) = make_float2(m[h], sum);
          else if (out.lse)
            out.lse[h] = log_sum(m[h], sum);
        }
      }
  }
};

// ------------------------------------------------------------ first launch
template <typename E>
struct Ring {
  static constexpr int kK = E::kTile * E::kKRow, kV = E::kTile * E::kVRow;
  static constexpr int kScale = E::kQuant ? E::kTile * 4 : 0;
  static constexpr int kStage = (kK + kV + 2 * kScale + 16 + 127) / 128 * 128;
  // about 24 KB per warp (48 KB for the fp32 engine's four warps): with eight
  // warps, the bytes in flight that cover the memory latency of an SM's share
  static constexpr int kWant = 8 * 24576 / E::kWarps / kStage;
  static constexpr int kStages = kWant < 3 ? 3 : kWant > 8 ? 8 : kWant;
  static constexpr int kWarpBytes = kStage * kStages + (E::kExtra + 127) / 128 * 128;
  static constexpr int kBytes = kWarpBytes * E::kWarps;
  static_assert(kBytes <= 220 * 1024, "shared memory");
};

// a tile of a run: sequence b, unit u of it (KV head and block of query
// heads), tile t of the unit
struct Cursor {
  int b, u, t;
  Seq s;
  __device__ __forceinline__ void next(const DecodeArgs& a, int units) {
    if (++t < s.tiles) return;
    t = 0;
    if (++u < units) return;
    u = 0;
    while (b + 1 < a.B) {
      s = seq_of(a, ++b);
      if (s.tiles) return;
    }
  }
};

// a tile whose table entries have been asked for: lane i holds row i % kTile's
struct Lookup {
  int page, slot, g;
  bool in;
};

template <typename E>
__global__ void __launch_bounds__(E::kWarps * 32, 1)
    lt_paged_decode_kernel(const DecodeArgs a) {
  using R = Ring<E>;
  using QT = typename E::QT;
  constexpr int kThreads = E::kWarps * 32, TILE = E::kTile, S = R::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t before[kThreads];     // tiles of the sequences before this thread's
  __shared__ int64_t warp_sum[E::kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  dependency_release();

  // each thread adds a run of sequences' tiles; a scan gives the runs' starts
  const int per = (a.B + kThreads - 1) / kThreads;
  int64_t sum = 0;
  for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) {
    const Seq s = seq_of(a, b);
    if (s.bad && blockIdx.x == 0) report_error(a.err, kDevErrBadSeqlens);
    sum += s.tiles;
  }
  int64_t scan = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, scan, off);
    if (lane >= off) scan += x;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  int64_t total = 0, mine = 0;
#pragma unroll
  for (int w = 0; w < E::kWarps; ++w) {
    if (w < warp) mine += warp_sum[w];
    total += warp_sum[w];
  }
  before[tid] = mine + scan - sum;
  __syncthreads();

  const int units = a.Hkv * a.nhb;
  total *= units;
  const int64_t run = run_length(a, total);
  const int gw = warp * gridDim.x + blockIdx.x;  // runs spread over the SMs first
  const int64_t start = gw * run, end = min(start + run, total);
  if (start >= end) return;

  Cursor cc;
  {
    int lo = 0, hi = kThreads;  // the last thread whose sequences begin at or before start
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] * units <= start)
        lo = mid;
      else
        hi = mid;
    }
    int64_t rem = start - before[lo] * units;
    cc.b = lo * per;
    cc.s = seq_of(a, cc.b);
    while (cc.b + 1 < a.B && rem >= (int64_t)cc.s.tiles * units) {
      rem -= (int64_t)cc.s.tiles * units;
      cc.s = seq_of(a, ++cc.b);
    }
    cc.u = (int)(rem / cc.s.tiles);
    cc.t = (int)(rem - (int64_t)cc.u * cc.s.tiles);
  }
  Cursor pc = cc;

  uint8_t* ring = smem + warp * R::kWarpBytes;
  const uint32_t ring_u = smem_u32(ring);
  E eng;
  eng.init(ring + R::kStage * S);

  const int row = lane & (TILE - 1);
  auto look = [&](const Cursor& c) {
    Lookup p;
    const int pos = c.s.first + c.t * TILE + row;
    p.in = pos < c.s.len;
    const int idx = pos / a.page_size;
    p.slot = pos - idx * a.page_size;
    p.page = p.in ? __ldg(a.table + (int64_t)c.b * a.table_stride + idx) : 0;
    p.g = c.u / a.nhb;
    return p;
  };
  auto issue = [&](int stage, const Lookup& p) {
    bool live = p.in;
    if (live && (p.page < 0 || p.page >= a.num_pages)) {
      report_error(a.err, kDevErrBadPage);
      live = false;
    }
    uint32_t mask = __ballot_sync(0xffffffffu, live);
    if (TILE < 32) mask &= (1u << (TILE & 31)) - 1u;
    const int64_t page = live ? p.page : 0, slot = live ? p.slot : 0;
    const int64_t ko = page * a.kpg + slot * a.ksl + p.g * a.khd;
    const int64_t vo = page * a.vpg + slot * a.vsl + p.g * a.vhd;
    const uint32_t dst = ring_u + stage * R::kStage;
    constexpr int kc = E::kKRow / 16, vc = E::kVRow / 16;  // chunks per row
#pragma unroll
    for (int i = 0; i < TILE * kc / 32; ++i) {
      const int r = i * (32 / kc) + lane / kc, c = lane % kc;
      const int64_t off = __shfl_sync(0xffffffffu, ko, r);
      copy16(dst + chunk_at<E::kKRow>(r, c), a.k + off + c * 16, (mask >> r) & 1u);
    }
#pragma unroll
    for (int i = 0; i < TILE * vc / 32; ++i) {
      const int r = i * (32 / vc) + lane / vc, c = lane % vc;
      const int64_t off = __shfl_sync(0xffffffffu, vo, r);
      copy16(dst + R::kK + chunk_at<E::kVRow>(r, c), a.v + off + c * 16, (mask >> r) & 1u);
    }
    if constexpr (E::kQuant) {
      const int64_t at = (page * a.Hkv + p.g) * a.page_size + slot;
      if (lane < TILE) {
        copy4(dst + R::kK + R::kV + lane * 4, a.ks + at, live);
        copy4(dst + R::kK + R::kV + R::kScale + lane * 4, a.vs + at, live);
      }
    }
    if (lane == 0)
      *reinterpret_cast<uint32_t*>(ring + stage * R::kStage + R::kK + R::kV + 2 * R::kScale) = mask;
  };

  const int64_t count = end - start;
  int64_t issued = 0;
  Lookup pend = look(pc);
  auto feed = [&](int stage) {
    if (issued < count) {
      issue(stage, pend);
      if (++issued < count) {
        pc.next(a, units);
        pend = look(pc);
      }
    }
    copy_commit();
  };
#pragma unroll 1
  for (int s = 0; s < S - 1; ++s) feed(s);

  int stage = 0, seg_t = cc.t;
  bool first_seg = true;
#pragma unroll 1
  for (int64_t i = 0; i < count; ++i) {
    if (i == 0 || cc.t == 0) {  // a new unit
      const int g = cc.u / a.nhb, blk = cc.u - g * a.nhb;
      const int h0 = g * a.G + blk * E::kHeads;
      eng.begin(static_cast<const QT*>(a.q) + ((size_t)cc.b * a.Hq + h0) * E::kD,
                min(E::kHeads, a.G - blk * E::kHeads), a.scale);
      seg_t = cc.t;
    }
    copy_wait<S - 2>();
    __syncwarp();  // every lane's copies of this tile have landed, and the last tile is read
    feed(stage == 0 ? S - 1 : stage - 1);
    const uint8_t* st = ring + stage * R::kStage;
    TileAt t;
    t.k = ring_u + stage * R::kStage;
    t.v = t.k + R::kK;
    t.ks = reinterpret_cast<const float*>(st + R::kK + R::kV);
    t.vs = reinterpret_cast<const float*>(st + R::kK + R::kV + R::kScale);
    t.mask = *reinterpret_cast<const uint32_t*>(st + R::kK + R::kV + 2 * R::kScale);
    eng.tile(t);
    if (++stage == S) stage = 0;
    const bool unit_done = cc.t + 1 == cc.s.tiles;
    if (unit_done || i + 1 == count) {
      const int g = cc.u / a.nhb, blk = cc.u - g * a.nhb;
      const int h0 = g * a.G + blk * E::kHeads;
      Sink<QT> out;
      out.partial = !(unit_done && seg_t == 0);
      const size_t orow = (size_t)cc.b * a.Hq + h0;
      out.out = static_cast<QT*>(a.out) + orow * a.dv;
      out.lse = a.lse ? a.lse + orow : nullptr;
      const size_t piece = (size_t)gw * 2 + (first_seg ? 0 : 1);
      out.part = a.part + piece * a.hb * a.dv;
      out.ml = a.ml + piece * a.hb * 2;
      eng.finish(out);
      first_seg = false;
    }
    if (i + 1 < count) cc.next(a, units);
  }
  copy_wait<0>();
}

// ----------------------------------------------------------- second launch
// One block per (query head, sequence): nothing to do where one warp had the
// whole pair; else the pieces, in run order.
constexpr int kJoin = 256;

__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  int64_t s = 0;
#pragma unroll
  for (int w = 0; w < kJoin / 32; ++w) s += red[w];
  return s;
}

__global__ void __launch_bounds__(kJoin) lt_paged_join_kernel(const DecodeArgs a) {
  __shared__ int64_t red[kJoin / 32];
  __shared__ float fred[kJoin / 32];
  __shared__ float acc_s[kJoin], l_s[kJoin];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  int64_t all = 0, pre = 0;
  for (int i = tid; i < a.B; i += kJoin) {
    const int n = seq_of(a, i).tiles;
    all += n;
    if (i < b) pre += n;
  }
  all = block_sum(all, red);
  pre = block_sum(pre, red);
  const Seq s = seq_of(a, b);
  const int units = a.Hkv * a.nhb;
  const int g = h / a.G, hh = h - g * a.G, blk = hh / a.hb, r = hh - blk * a.hb;
  const int64_t run = run_length(a, all * units);
  const int64_t from = pre * units + (int64_t)(g * a.nhb + blk) * s.tiles;
  const int64_t w0 = from / run, w1 = s.tiles ? (from + s.tiles - 1) / run : w0;
  // every block waits, so that this launch ends after the first one has
  dependency_wait();
  if (s.bad) return;
  const size_t orow = (size_t)b * a.Hq + h;
  const int groups = kJoin / a.dv, col = tid % a.dv, grp = tid / a.dv;
  float res = 0.0f, lse = -INFINITY;
  if (s.tiles) {
    if (w0 == w1) return;
    const int n = (int)(w1 - w0 + 1);
    // piece i of the pair: slot 1 only of a warp that began with another pair
    const int slot0 = from > w0 * run ? 1 : 0;
    auto piece = [&](int i) { return (size_t)(w0 + i) * 2 + (i == 0 ? slot0 : 0); };
    float mx = -INFINITY;
    for (int i = tid; i < n; i += kJoin) mx = fmaxf(mx, a.ml[(piece(i) * a.hb + r) * 2]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if ((tid & 31) == 0) fred[tid >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoin / 32; ++w) mx = fmaxf(mx, fred[w]);
    const float base = mx == -INFINITY ? 0.0f : mx;
    float o = 0.0f, l = 0.0f;
#pragma unroll 4
    for (int i = grp; i < n; i += groups) {
      const size_t p = piece(i) * a.hb + r;
      const float2 ml = *reinterpret_cast<const float2*>(a.ml + p * 2);
      const float f = exp2f(ml.x - base);
      l = fmaf(f, ml.y, l);
      o = fmaf(f, a.part[p * a.dv + col], o);
    }
    acc_s[tid] = o;
    l_s[tid] = l;
    __syncthreads();
    o = l = 0.0f;
    for (int q = 0; q < groups; ++q) {
      o += acc_s[q * a.dv + col];
      l += l_s[q * a.dv + col];
    }
    res = o * inverse_sum(l);
    lse = log_sum(mx, l);
  }
  if (grp != 0) return;
  const size_t at = orow * a.dv + col;
  if (a.dtype == LT_F32)
    static_cast<float*>(a.out)[at] = res;
  else if (a.dtype == LT_BF16)
    from_float(static_cast<__nv_bfloat16*>(a.out) + at, res);
  else
    from_float(static_cast<__half*>(a.out) + at, res);
  if (a.lse && col == 0) a.lse[orow] = lse;
}

// ------------------------------------------------------------------- host
template <typename E>
cudaError_t launch_e(DecodeArgs a, int sms, cudaStream_t stream) {
  auto kern = lt_paged_decode_kernel<E>;
  constexpr int smem = Ring<E>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  a.tile = E::kTile;
  kern<<<sms, E::kWarps * 32, smem, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(lt_paged_join_kernel, dim3(a.Hq, a.B), kJoin, 0, stream, a);
}

template <typename QT, typename KT>
cudaError_t launch_w(const DecodeArgs& a, int d, int sms, cudaStream_t s) {
  if constexpr (sizeof(QT) == 4) {
    if (d == 64)
      return a.dv == 64 ? launch_e<FmaEngine<KT, 64, 64>>(a, sms, s)
                        : launch_e<FmaEngine<KT, 64, 128>>(a, sms, s);
    return a.dv == 64 ? launch_e<FmaEngine<KT, 128, 64>>(a, sms, s)
                      : launch_e<FmaEngine<KT, 128, 128>>(a, sms, s);
  } else {
    if (d == 64)
      return a.dv == 64 ? launch_e<MmaEngine<QT, KT, 64, 64>>(a, sms, s)
                        : launch_e<MmaEngine<QT, KT, 64, 128>>(a, sms, s);
    return a.dv == 64 ? launch_e<MmaEngine<QT, KT, 128, 64>>(a, sms, s)
                      : launch_e<MmaEngine<QT, KT, 128, 128>>(a, sms, s);
  }
}

template <typename QT>
cudaError_t launch_q(const DecodeArgs& a, lt_kv_dtype_t kv, int d, int sms, cudaStream_t s) {
  if (kv == LT_KV_E4M3) return launch_w<QT, E4M3>(a, d, sms, s);
  if (kv == LT_KV_INT8) return launch_w<QT, Int8>(a, d, sms, s);
  return launch_w<QT, QT>(a, d, sms, s);
}

// query heads per unit, and warps (runs) on a device
int heads_per_unit(lt_dtype_t t, int G) {
  const int most = t == LT_F32 ? 8 : 16;  // the engines' kHeads
  return G < most ? G : most;
}
int run_count(lt_dtype_t t, int sms) { return sms * (t == LT_F32 ? 4 : 8); }

size_t workspace_floats(lt_dtype_t t, int G, int dv, int sms) {
  return (size_t)run_count(t, sms) * 2 * heads_per_unit(t, G) * (dv + 2);
}

}  // namespace
}  // namespace lt

extern "C" lt_status_t lt_paged_attn_decode_plan(int H_q, int H_kv, int d, int dv,
                                                 lt_dtype_t dtype, lt_kv_dtype_t kv_dtype,
                                                 int num_sms, size_t* workspace_bytes) {
  using namespace lt;
  if (!dtype_ok(dtype) || kv_dtype < LT_KV_F32 || kv_dtype > LT_KV_INT8 ||
      (!eight_bit(kv_dtype) && kv_dtype != kv_of(dtype)))
    return LT_ERR_UNSUPPORTED;
  if ((d != 64 && d != 128) || (dv != 64 && dv != 128)) return LT_ERR_UNSUPPORTED;
  if (!workspace_bytes || H_q < 1 || H_kv < 1 || H_q > 65535 || H_q % H_kv != 0)
    return LT_ERR_INVALID_ARG;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return LT_ERR_CUDA;
  *workspace_bytes = workspace_floats(dtype, H_q / H_kv, dv, num_sms) * sizeof(float);
  return LT_OK;
}

extern "C" lt_status_t lt_paged_attn_decode(const void* q, const lt_kv_cache_t* cache,
                                            const int32_t* block_table, int64_t table_stride,
                                            int max_pages, const int32_t* seq_lens, int B, int H_q,
                                            float scale, int window, void* out, float* lse,
                                            void* workspace, size_t workspace_bytes,
                                            lt_stream_t stream, lt_dtype_t dtype) {
  using namespace lt;
  const lt_status_t st = check_cache(cache);
  if (st != LT_OK) return st;
  if (!dtype_ok(dtype) || (!eight_bit(cache->dtype) && cache->dtype != kv_of(dtype)))
    return LT_ERR_UNSUPPORTED;
  if (!q || !block_table || !seq_lens || !out || B < 1 || B > 65535 || H_q < 1 || H_q > 65535 ||
      H_q % cache->H_kv != 0 || max_pages < 1 || table_stride < max_pages ||
      table_stride > ((int64_t)1 << 40) || window < 0 || !isfinite(scale))
    return LT_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(block_table, 4) ||
      !aligned_to(seq_lens, 4) || !aligned_to(lse, 4))
    return LT_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype);
  Span ins[8];
  cache_spans(cache, ins);
  ins[4] = Span{q, (size_t)B * H_q * cache->d * es};
  ins[5] = Span{block_table, ((size_t)(B - 1) * table_stride + max_pages) * 4};
  ins[6] = Span{seq_lens, (size_t)B * 4};
  ins[7] = Span{workspace, workspace_bytes};
  const Span o = {out, (size_t)B * H_q * cache->dv * es}, ls = {lse, (size_t)B * H_q * 4};
  if (spans_overlap(o, ls)) return LT_ERR_INVALID_ARG;
  for (const Span& i : ins)
    if (spans_overlap(o, i) || spans_overlap(ls, i)) return LT_ERR_INVALID_ARG;
  for (int i = 0; i < 7; ++i)
    if (spans_overlap(ins[7], ins[i])) return LT_ERR_INVALID_ARG;
  if (check_cache_pointers(cache) != LT_OK || !on_current_device(q) ||
      !on_current_device(block_table) || !on_current_device(seq_lens) || !on_current_device(out) ||
      (lse && !on_current_device(lse)))
    return LT_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  int* err = device_error_word_current();
  if (sms <= 0 || !err) return LT_ERR_CUDA;
  DecodeArgs a = {};
  a.G = H_q / cache->H_kv;
  a.hb = heads_per_unit(dtype, a.G);
  a.nhb = (a.G + a.hb - 1) / a.hb;
  a.warps = run_count(dtype, sms);
  Workspace w;
  const lt_status_t sw =
      w.take(workspace, workspace_bytes,
             workspace_floats(dtype, a.G, cache->dv, sms) * sizeof(float), (cudaStream_t)stream);
  if (sw != LT_OK) return sw;
  const int64_t ks = (int64_t)kv_size(cache->dtype);
  a.q = q;
  a.k = static_cast<const uint8_t*>(cache->k);
  a.v = static_cast<const uint8_t*>(cache->v);
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.kpg = cache->k_page_stride * ks;
  a.ksl = cache->k_slot_stride * ks;
  a.khd = cache->k_head_stride * ks;
  a.vpg = cache->v_page_stride * ks;
  a.vsl = cache->v_slot_stride * ks;
  a.vhd = cache->v_head_stride * ks;
  a.table = block_table;
  a.table_stride = table_stride;
  a.lens = seq_lens;
  a.B = B;
  a.Hq = H_q;
  a.Hkv = cache->H_kv;
  a.num_pages = cache->num_pages;
  a.page_size = cache->page_size;
  a.max_pages = max_pages;
  a.window = window;
  a.min_tiles = 2;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.dv = cache->dv;
  a.dtype = (int)dtype;
  a.part = static_cast<float*>(w.p);
  a.ml = a.part + (size_t)a.warps * 2 * a.hb * a.dv;
  a.err = err;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = dtype == LT_BF16  ? launch_q<__nv_bfloat16>(a, cache->dtype, cache->d, sms, s)
                  : dtype == LT_F16 ? launch_q<__half>(a, cache->dtype, cache->d, sms, s)
                                    : launch_q<float>(a, cache->dtype, cache->d, sms, s);
  const cudaError_t f = w.release();
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}
