// paged_attn.cuh -- softmax attention of one new token per sequence over a
// paged key-value cache: the first launch, and the schedule that both share.
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
// Split: all sequences' tiles of 16 or 32 tokens, laid end to end, are dealt out
// in equal runs to the blocks of one launch, one per SM, whatever the lengths:
// a batch of very different sequences and one long sequence load the SMs
// alike, and the workspace does not grow with either.  Inside a block the
// warps share out the units (KV head and block of query heads) of its run, so
// that the heads of a token, neighbours in memory, are read at about the same
// time (an 8-bit row is only 64 or 128 bytes).  A warp has its own ring of
// tiles in shared memory, filled with 16-byte asynchronous copies, and its own
// running maximum and sum; no barrier between warps.  A unit of a sequence
// that one warp had whole is finished by it.  Where several warps of a block
// share it, each leaves a piece, and the block joins them at its end; where
// several blocks share it, each leaves one, and a second launch (which starts
// early and waits for the first) joins those.  The order of joining follows
// from the lengths alone, so results do not depend on timing.
//
// Measured on one B200 (plain copy 6.55 TB/s, reads alone up to 7.1), 32 query
// over 8 KV heads of 128: 64 ragged sequences (270k tokens) bf16 171 us, 6.5 TB/s;
// e4m3 101 us, 5.6 TB/s, replayed from a graph, and up to 112 in seconds of
// back-to-back calls, where the widening of the codes and the weights' two terms
// keep the issue slots busy at a lower clock; one sequence of 65536 tokens, bf16, 51
// us, of which 10 are the two launches' starts and ends.  Runs of (sequence, KV head)
// pairs instead of whole columns read the e4m3 rows of one token at different times:
// 30% slower.  Bulk copies of single rows are slower than 16-byte copies below 256
// bytes a row (128-byte rows 4.5 against 7.0 TB/s).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/lt_linear_attn.h"
#include "lt_check.h"
#include "lt_internal.h"
#include "lt_ptx.cuh"
#include "lt_vec.cuh"

namespace lt {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What the engines and the workspace's sizes go by.  Query heads that a warp has at
// once (a unit: up to so many of one KV head's G): one or two blocks of 8.
constexpr int heads_at_once(bool f32, int G) { return f32 || G <= 8 ? 8 : 16; }
// Tokens per tile: 8 KB per tile, so that short rows share a tile's bookkeeping
// (e4m3 rows of 128 in tiles of 16, with 16 warps, issued a third more
// instructions per token).  kv_bytes: of a value in the cache.
constexpr int tile_tokens(int kv_bytes, int d, int dv) {
  return (d + dv) * kv_bytes <= 256 ? 32 : 16;
}
// Warps per block, for units of up to `heads` query heads.  8-bit rows of 64: tiles
// are 4 KB, and a warp's chain of steps per tile is no shorter, so twice the warps
// where their registers do (64 sequences, 270k tokens of 8 heads, e4m3: 75.0 us
// with 8, 62.5 with 16).  Not for 9 heads or more, which spill in the 128 registers
// of 16 warps (the same sequences, 16 heads over 1: 23.6 us with 8, 26.8 with 16; 80
// over 8: 500 and 530; 256 over 4, of 16 units, 202 and 190), nor fp32 queries.
constexpr int block_warps(bool f32, int kv_bytes, int d, int dv, int heads) {
  return kv_bytes == 4 ? 4 : (d + dv) * kv_bytes <= 128 && !f32 && heads == 8 ? 16 : 8;
}

// A piece of a pair: unnormalised sums of values [heads][dv], and the maximum
// and sum of weights [heads][2].
struct Pieces {
  float* part;
  float* ml;
};
// A sequence that several blocks share, for the second launch: its first block
// and their number (0: none here).
struct Shared {
  int b, block, blocks, pad;
};

struct DecodeArgs {
  const void* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  uint32_t kpg, ksl, khd, vpg, vsl, vhd;  // pool strides, in 16 bytes
  int same;                               // the two pools' strides are the same
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  int B, Hq, Hkv, G, nhb;  // nhb: blocks of query heads per KV head
  int hb;                  // query heads per block of them
  int num_pages, page_size, window;
  uint32_t page_magic;  // floor(2^(31 + page_shift) / page_size) + 1
  int page_shift;       // ceil(log2(page_size))
  int max_len;          // keys that a table row has pages for
  int units, k_shift;   // Hkv * nhb; log2 of the warps per unit (-1: they do not divide)
  int by_seq;           // shared[] goes by sequence (else by first block)
  float scale;
  void* out;
  float* lse;
  Pieces warp, block;  // [blocks][warps][2] and [blocks][2][units] pieces of hb heads
  Shared* shared;      // [min(B, blocks)]
  int dv, dtype;
  int* err;
};

// ------------------------------------------------------------ the schedule
struct Seq {
  int first, len;  // keys [first, len) take part
  int tiles;
};
template <int TILE>
__device__ __forceinline__ Seq seq_of(const DecodeArgs& a, int len) {
  Seq s;
  s.len = len < 0 || len > a.max_len ? 0 : len;
  s.first = a.window ? max(0, s.len - a.window) : 0;
  s.tiles = (s.len - s.first + TILE - 1) / TILE;
  return s;
}

// pos / page_size for 0 <= pos < 2^31: with m = page_magic, m page_size exceeds
// 2^(31 + s) by at most page_size <= 2^s, so pos m / 2^(31 + s) exceeds the
// quotient by less than 1 / page_size
__device__ __forceinline__ int page_of(const DecodeArgs& a, int pos) {
  return (int)(((uint64_t)(uint32_t)pos * a.page_magic) >> (31 + a.page_shift));
}

// --------------------------------------------------------------- copies
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
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
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
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
// chunk c + dc of the same row, at being chunk c's address and dc a multiple of
// a power of two above c: the permutation is an exclusive or, so one suffices
// (tiles begin at multiples of 128 bytes)
__device__ __forceinline__ uint32_t chunk_on(uint32_t at, int dc) {
  return (at ^ ((dc & 7) << 4)) + ((dc & ~7) << 4);
}
// A warp copies a tile 512 bytes at a time: row and chunk of this lane in the
// first step, and step i's address from the first one's.
template <int RB>
__device__ __forceinline__ uint32_t step_at(uint32_t first, int i) {
  constexpr int kRows = 512 / RB;  // rows per step
  constexpr int kPer = RB >= 128 ? 1 : 128 / RB;
  constexpr int kMask = (RB >= 128 ? 8 : RB / 16) - 1;
  return (first ^ (((i * kRows / kPer) & kMask) << 4)) + i * 512;
}

__device__ __forceinline__ float exp2_fast(float x) { return ex2_approx(x); }

// What an engine is told of a tile in shared memory.
struct TileAt {
  uint32_t k, v;     // shared addresses of the two tiles (multiples of 128)
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
// the transpose of an 8 x 8 tile of 16-bit values held one word per lane
__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
  return r;
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

// two values of a word
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (__is_same(T, __nv_bfloat16))
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
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

// one more piece: values x, maximum and sum ml; what is joined so far (o, l,
// relative to 2^mx) and the piece both go by the larger maximum (exp2f: a factor
// below fp32's normal numbers counts too, beside values as large)
__device__ __forceinline__ void add_piece(float4& o, float& l, float& mx, float2 ml, float4 x) {
  const float top = fmaxf(mx, ml.x), base = top == -INFINITY ? 0.0f : top;
  const float f = exp2f(mx - base), g = exp2f(ml.x - base);
  mx = top;
  l = fmaf(g, ml.y, f * l);
  o.x = fmaf(g, x.x, f * o.x);
  o.y = fmaf(g, x.y, f * o.y);
  o.z = fmaf(g, x.z, f * o.z);
  o.w = fmaf(g, x.w, f * o.w);
}

// --------------------------------------------------- engine: tensor cores
template <typename KT>
struct KvTraits {  // 16-bit caches: the cache's own type
  using Math = KT;
  static constexpr int kBytes = 2;
  static constexpr bool kQuant = false;
};
template <>
struct KvTraits<E4M3> {
  using Math = __half;  // every e4m3 value is an fp16 value
  static constexpr int kBytes = 1;
  static constexpr bool kQuant = true;
};
template <>
struct KvTraits<Int8> {
  using Math = __half;
  static constexpr int kBytes = 1;
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

// Legacy mma on purpose: a KV head has G query heads, so a tcgen05 tile of 128
// rows would be nearly empty, and the work is bound by memory.  The tokens are
// the 16 rows of the instruction and the query heads its 8 columns, so that
// few of its lanes idle: per 16 tokens of a 16-bit cache of width 128 a warp
// issues 24 mma (bf16: 32) and 16 ldmatrix for 8 KB read.  kNB blocks of 8 heads
// share a tile's registers.
//
// Scores S^T = K Q^T: A = K (ldmatrix of the token rows), B = Q (in registers).
// Values O^T = V^T P^T: A = V by transposing ldmatrix, B = the weights, whose
// 8 x 8 tiles are turned from S^T's layout by movmatrix.
//
// The weights go in as several terms of the product's type, each the rounded
// rest of those before (a product each), so that they keep 32 bits: three bf16
// terms hold all 24 bits of one, two fp16 terms all but the last (2^-23 off at
// most), which is enough beside a 16-bit output, and fp32 outputs take three.
// One term fewer (one for bf16 queries over 8-bit caches) turned up to one output
// in twenty to the neighbouring bf16 value and saved 1 to 7%: 64 ragged sequences,
// 270k tokens of 8 heads of 128, bf16 171 us against 170, e4m3 101 against 99,
// int8 112 against 104.
//
// 8-bit caches are widened to fp16 in registers.  A lane's four bytes of a key
// row are four neighbouring d, where the instruction's A layout has two pairs
// eight apart: Q's registers are filled in the same order instead.  A lane's
// transposed word of V holds two columns of two tokens: the even columns are
// rows 0 .. 7 of the product, the odd ones rows 8 .. 15.  Key scales multiply
// the scores; value scales go into the weights, relative to a power of two A
// >= every scale seen, so that the fp16 weights stay at most 2^kShift (and what
// falls below fp16's smallest numbers is under 2^-37 of the largest value row).  Q
// is scaled by a power of two per head, its largest entry to 2^12: no bf16 query
// leaves fp16's range, and what falls below it is under 2^-37 of that entry.
// fp32 queries (8-bit caches only) are three fp16 terms, which hold all 24 bits.
//
// kShift: fp16 weights are held times 2^12, so that weights down to 2^-26 of the
// largest keep fp16's full precision; 2^12 * 65504 * 2^31 keys stay inside fp32.
// bf16 has fp32's range and needs none.  finish() takes it out of sums and values
// again, and A last, so that neither takes a result out of fp32's range.
//
// The maximum moves only when some score passes it: one vote per tile instead
// of a reduction.
template <typename QT_, typename KT, int D, int DV, int kNB>
struct MmaEngine {
  using QT = QT_;
  using Kv = KvTraits<KT>;
  using MT = typename Kv::Math;
  static constexpr bool kQuant = Kv::kQuant;
  static constexpr bool kHalf = !__is_same(MT, __nv_bfloat16);
  static constexpr bool kWide = __is_same(QT, float);  // fp32 queries
  static constexpr int kTerms = kWide ? 3 : 1;
  static constexpr int kWeightTerms = !kHalf || kWide ? 3 : 2;
  static_assert(!kWide || kQuant, "fp32 caches have an engine of their own");
  static constexpr int kD = D, kHeads = 8 * kNB;
  static constexpr int kWarps = block_warps(kWide, Kv::kBytes, D, DV, kHeads);
  static constexpr int kTile = tile_tokens(Kv::kBytes, D, DV);
  static constexpr int kHalves = kTile / 16;
  static constexpr int kKRow = D * Kv::kBytes, kVRow = DV * Kv::kBytes;  // bytes
  static constexpr float kShift = kHalf ? 12.0f : 0.0f, kUnshift = kHalf ? 1.0f / 4096 : 1.0f;
  uint32_t qf[kTerms][kNB][D / 16][2];
  float o[kNB][DV / 16][4];
  // per head 2c, 2c + 1 of each block (c the lane's index among four)
  float m[kNB][2], l[kNB][2], sl2[kNB][2];
  uint32_t vtop;  // A's bits
  int heads;

  __device__ __forceinline__ void begin(const QT* q, int nheads, float scale) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    heads = nheads;
    vtop = 0x00800000u;
#pragma unroll
    for (int b = 0; b < kNB; ++b) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[b][e] = -INFINITY;
        l[b][e] = 0.0f;
        sl2[b][e] = scale * kLog2e;
      }
#pragma unroll
      for (int j = 0; j < DV / 16; ++j) o[b][j][0] = o[b][j][1] = o[b][j][2] = o[b][j][3] = 0.0f;
      const int h = 8 * b + (lane >> 2);
      const bool live = h < nheads;
      const QT* row = q + (size_t)h * D;
      if constexpr (!kQuant) {
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qf[0][b][s][e] =
                live ? __ldg(reinterpret_cast<const uint32_t*>(row + 16 * s + 8 * e + 2 * c)) : 0u;
      } else {
        float2 x[D / 16][2];
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[s][e] = live ? load_pair(row + 16 * s + 4 * c + 2 * e) : make_float2(0.0f, 0.0f);
            top = fmaxf(top, fmaxf(fabsf(x[s][e].x), fabsf(x[s][e].y)));
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // times 2^(127 - ex) 2^kUp: the largest entry in [1, 2) 2^kUp
        constexpr uint32_t kUp = 12;
        const uint32_t ex = min(max(__float_as_uint(top) >> 23, 13u), 253u);
        const float down = __uint_as_float((254u + kUp - ex) << 23);
        const float up = __uint_as_float((ex - kUp) << 23);
#pragma unroll
        for (int e = 0; e < 2; ++e) sl2[b][e] *= __shfl_sync(0xffffffffu, up, 8 * c + 4 * e);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float2 y = make_float2(x[s][e].x * down, x[s][e].y * down);
#pragma unroll
            for (int n = 0; n < kTerms; ++n) {
              qf[n][b][s][e] = pack2<__half>(y.x, y.y);
              const float2 z = unpack2<__half>(qf[n][b][s][e]);
              y.x -= z.x;
              y.y -= z.y;
            }
          }
      }
    }
  }

  // two neighbouring queries
  __device__ __forceinline__ static float2 load_pair(const QT* p) {
    if constexpr (kWide)
      return __ldg(reinterpret_cast<const float2*>(p));
    else
      return unpack2<QT>(__ldg(reinterpret_cast<const uint32_t*>(p)));
  }

  using Scores = float[kNB][kHalves][4];

  // the maximum (and A) moved: what is summed so far goes by the new ones
  __device__ __forceinline__ void rescale(const Scores& s, uint32_t top) {
    top = __reduce_max_sync(0xffffffffu, top);
    const float fa = kQuant ? __uint_as_float(vtop) * __uint_as_float(0x7f000000u - top) : 1.0f;
    vtop = top;
#pragma unroll
    for (int b = 0; b < kNB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = m[b][e];
#pragma unroll
        for (int y = 0; y < kHalves; ++y) mx = fmaxf(mx, fmaxf(s[b][y][e], s[b][y][2 + e]));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        float f = mx == m[b][e] ? 1.0f : exp2_fast(m[b][e] - mx);
        m[b][e] = mx;
        l[b][e] *= f;
        f *= fa;
#pragma unroll
        for (int j = 0; j < DV / 16; ++j) {
          o[b][j][e] *= f;
          o[b][j][2 + e] *= f;
        }
      }
  }

  // S^T of 16 tokens, times the heads' factors; `at`: see tile()
  __device__ __forceinline__ void scores(float (*s)[4], uint32_t at) {
    // even and odd steps: two chains of products; the queries' further terms,
    // small beside the first, in a chain of their own
    float s2[kNB][4], small[kNB][4];
#pragma unroll
    for (int b = 0; b < kNB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[b][e] = s2[b][e] = small[b][e] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 16; i += 2) {
      uint32_t a0[4], a1[4];
      if constexpr (!kQuant) {
        ldsm4(a0, chunk_on(at, 2 * i));
        ldsm4(a1, chunk_on(at, 2 * i + 2));
      } else {
        uint32_t w[4];
        ldsm4(w, chunk_on(at, i));
        widen4<false>(w[0], a0[0], a0[2], KT());
        widen4<false>(w[1], a0[1], a0[3], KT());
        widen4<false>(w[2], a1[0], a1[2], KT());
        widen4<false>(w[3], a1[1], a1[3], KT());
      }
#pragma unroll
      for (int n = 0; n < kTerms; ++n)
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
          mma<MT>(n ? small[b] : s[b], a0, qf[n][b][i][0], qf[n][b][i][1]);
          mma<MT>(n ? small[b] : s2[b], a1, qf[n][b][i + 1][0], qf[n][b][i + 1][1]);
        }
    }
#pragma unroll
    for (int b = 0; b < kNB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[b][e] += s2[b][e];
        if constexpr (kTerms > 1) s[b][e] += small[b][e];
        s[b][e] *= sl2[b][e & 1];
      }
  }

  // O^T += V^T P^T of the tile, w its weights' tiles.  The sum of a tile starts
  // from zero, its small terms first, and is added to the rest by plain
  // additions: the instruction's own cut what they lose, all to one side
  // (means of 16384 keys in one chain of products: off by 1e-4).
  using Weights = uint32_t[kHalves][kWeightTerms][kNB][2];
  __device__ __forceinline__ void values(uint32_t at, const Weights& w) {
#pragma unroll
    for (int j = 0; j < DV / 16; j += 2) {
      float sum[2][kNB][4] = {};
#pragma unroll
      for (int y = 0; y < kHalves; ++y) {
        const uint32_t row = at + y * 16 * kVRow;
        uint32_t a0[4], a1[4];
        if constexpr (!kQuant) {
          ldsm4t(a0, chunk_on(row, 2 * j));
          ldsm4t(a1, chunk_on(row, 2 * j + 2));
        } else {
          uint32_t x[4];
          ldsm4t(x, chunk_on(row, j));
          widen4<true>(x[0], a0[0], a0[1], KT());
          widen4<true>(x[1], a0[2], a0[3], KT());
          widen4<true>(x[2], a1[0], a1[1], KT());
          widen4<true>(x[3], a1[2], a1[3], KT());
        }
#pragma unroll
        for (int n = kWeightTerms - 1; n >= 0; --n)
#pragma unroll
          for (int b = 0; b < kNB; ++b) {
            mma<MT>(sum[0][b], a0, w[y][n][b][0], w[y][n][b][1]);
            mma<MT>(sum[1][b], a1, w[y][n][b][0], w[y][n][b][1]);
          }
      }
#pragma unroll
      for (int b = 0; b < kNB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[b][j][e] += sum[0][b][e];
          o[b][j + 1][e] += sum[1][b][e];
        }
    }
  }

  __device__ __forceinline__ void tile(const TileAt& t) {
    const int lane = threadIdx.x & 31, r = lane >> 2;
    // where this lane points the loads of four 8 x 8 tiles: tokens of the first
    // two chunks of K's rows, and of V's (its 16-bit tiles turned token-first)
    const uint32_t k_at = t.k + chunk_at<kKRow>(lane & 15, lane >> 4);
    const uint32_t v_at =
        t.v + (kQuant ? chunk_at<kVRow>(lane & 15, lane >> 4)
                      : chunk_at<kVRow>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1));
    Scores s;  // in units of log 2
    float vs[kHalves][2];
    uint32_t top = vtop;
#pragma unroll
    for (int y = 0; y < kHalves; ++y) {
      float x[kNB][4];
      scores(x, k_at + y * 16 * kKRow);
      if constexpr (kQuant) {
        const float k0 = t.ks[16 * y + r], k1 = t.ks[16 * y + r + 8];
#pragma unroll
        for (int b = 0; b < kNB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[b][e] *= e < 2 ? k0 : k1;
        vs[y][0] = t.vs[16 * y + r];
        vs[y][1] = t.vs[16 * y + r + 8];
        // (the scales of tokens that take no part are zeros)
        top = max(top, __float_as_uint(vs[y][0]) & 0x7fffffffu);
        top = max(top, __float_as_uint(vs[y][1]) & 0x7fffffffu);
      }
#pragma unroll
      for (int b = 0; b < kNB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[b][y][e] = x[b][e];
    }
    if constexpr (kQuant)  // A: the next power of two, within 2^-126 .. 2^126
      top = top >= 0x7e800000u ? 0x7e800000u : (top + 0x7fffffu) & 0x7f800000u;
    if (t.mask != (kTile == 32 ? 0xffffffffu : (1u << (kTile & 31)) - 1u)) {
      // tokens that take no part get -infinity
#pragma unroll
      for (int y = 0; y < kHalves; ++y)
#pragma unroll
        for (int b = 0; b < kNB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((t.mask >> (16 * y + r + (e & 2 ? 8 : 0))) & 1u)) s[b][y][e] = -INFINITY;
    }
    bool moved = top != vtop;
#pragma unroll
    for (int b = 0; b < kNB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(s[b][0][e], s[b][0][2 + e]);
#pragma unroll
        for (int y = 1; y < kHalves; ++y) mx = fmaxf(mx, fmaxf(s[b][y][e], s[b][y][2 + e]));
        moved |= mx > m[b][e];
      }
    if (__any_sync(0xffffffffu, moved)) rescale(s, top);
    const float inv_a = __uint_as_float(0x7f000000u - vtop);
    Weights w;
#pragma unroll
    for (int b = 0; b < kNB; ++b) {
      const float base[2] = {(m[b][0] == -INFINITY ? 0.0f : m[b][0]) - kShift,
                             (m[b][1] == -INFINITY ? 0.0f : m[b][1]) - kShift};
#pragma unroll
      for (int y = 0; y < kHalves; ++y)
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // token r, token r + 8
          float p0 = exp2_fast(s[b][y][2 * u] - base[0]);
          float p1 = exp2_fast(s[b][y][2 * u + 1] - base[1]);
          l[b][0] += p0;
          l[b][1] += p1;
          if constexpr (kQuant) {
            const float f = vs[y][u] * inv_a;
            p0 *= f;
            p1 *= f;
          }
#pragma unroll
          for (int n = 0; n < kWeightTerms; ++n) {
            const uint32_t two = pack2<MT>(p0, p1);
            const float2 x = unpack2<MT>(two);
            w[y][n][b][u] = transpose8(two);
            p0 -= x.x;
            p1 -= x.y;
          }
        }
    }
    values(v_at, w);
  }

  __device__ __forceinline__ void finish(const Sink<QT>& out) {
    const int lane = threadIdx.x & 31, c = lane & 3;
#pragma unroll
    for (int b = 0; b < kNB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[b][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const int h = 8 * b + 2 * c + e;
        if (h >= heads) continue;
        sum *= kUnshift;
        if (out.partial) {
          if (lane < 4) *reinterpret_cast<float2*>(out.ml + 2 * h) = make_float2(m[b][e], sum);
          put(out.part + (size_t)h * DV, b, e, kUnshift);
        } else {
          if (lane < 4 && out.lse) out.lse[h] = log_sum(m[b][e], sum);
          put(out.out + (size_t)h * DV, b, e, kUnshift * inverse_sum(sum));
        }
      }
  }

  // head e's row: its values times f, and A
  template <typename P>
  __device__ __forceinline__ void put(P* row, int b, int e, float f) {
    const int r = (threadIdx.x & 31) >> 2;
    const float top = kQuant ? __uint_as_float(vtop) : 1.0f;
#pragma unroll
    for (int j = 0; j < DV / 16; ++j) {
      const float x = o[b][j][e] * f * top, y = o[b][j][2 + e] * f * top;
      if constexpr (kQuant) {
        store_pair(row + 16 * j + 2 * r, x, y);
      } else {
        from_float(row + 16 * j + r, x);
        from_float(row + 16 * j + r + 8, y);
      }
    }
  }
};

// ---------------------------------------------------- engine: fp32 caches
// Tensor cores in bf16, every factor in three terms, which hold all 24 bits of
// one: x = hi + mid + lo, hi the first 8 bits (cut), mid the rest rounded to 8, lo
// what is left.  Of the nine products of terms the six largest are taken; the others
// are at most 2^-22 of |x y|, 2^-25 in the mean and either way, which is what fp32
// arithmetic itself rounds off.  (Two terms of tf32, three products, took as many
// instructions but were 2^-21 off: a single key did not come back as its value.)
// Sums as in MmaEngine.  Plain fp32 multiplications bound this kernel at 3 TB/s for 4
// query heads per KV head; so it reads 5.6 TB/s (32 sequences, 153k tokens of 8
// heads of 128: 225 us), held by the splitting of keys and values beside memory.
// Subtracting after widening the packed terms, and the five small products in
// one chain, were 3% slower each.
//
// The same two products as MmaEngine: S^T = K Q^T with A = K, O^T = V^T P^T with A
// = V^T.  32-bit tiles have no ldmatrix, so rows and columns are numbered to make a
// lane's share four neighbouring values, read at once and without bank
// conflicts: of S^T, row g is token 4 (g & 1) + g / 2 of its eight, and a lane's
// four d of a step are 16 s + 4 c ..; of V^T, rows g and g + 8 of two products are
// a lane's four columns.
struct Bf16Terms {
  uint32_t t[3];  // of two values, packed
};
// h - x, h a bf16 (mixed operands: no widening of the packed terms)
__device__ __forceinline__ float less(uint32_t h, float x) {
  float r;
  asm("sub.f32.bf16 %0, %1, %2;" : "=f"(r) : "h"((uint16_t)h), "f"(x));
  return r;
}
__device__ __forceinline__ Bf16Terms split_terms(float x, float y) {
  Bf16Terms r;
  r.t[0] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  // minus the rest, of 16 bits; its first 8, rounded; and the 8 that are left
  x = less(r.t[0], x);
  y = less(r.t[0] >> 16, y);
  const uint32_t c = pack2<__nv_bfloat16>(x, y);
  r.t[1] = c ^ 0x80008000u;
  x = less(c, x);
  y = less(c >> 16, y);
  r.t[2] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  return r;
}
__device__ __forceinline__ void shared4(uint32_t addr, float* f) {
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
               : "r"(addr)
               : "memory");
}

template <int D, int DV>
struct Fp32Engine {
  using QT = float;
  static constexpr int kD = D, kHeads = heads_at_once(true, 1);
  static constexpr int kWarps = block_warps(true, 4, D, DV, 8), kTile = tile_tokens(4, D, DV);
  static_assert(kTile == 16, "a tile is one step of the products");
  static constexpr int kKRow = D * 4, kVRow = DV * 4;  // bytes
  static constexpr bool kQuant = false;
  uint32_t qf[D / 16][2][3];  // of head g = lane / 4, d 16 s + 4 c ..
  float o[DV / 32][2][4];
  float m[2], l[2];  // heads 2 c, 2 c + 1
  float sl2;
  int heads;
  const float* query;

  __device__ __forceinline__ void begin(const float* q, int nheads, float scale) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    heads = nheads;
    query = q;
    sl2 = scale * kLog2e;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[e] = -INFINITY;
      l[e] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < DV / 32; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) o[j][e >> 2][e & 3] = 0.0f;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const float4 x = g < nheads ? __ldg(reinterpret_cast<const float4*>(q + g * D + 16 * s) + c)
                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const Bf16Terms a = split_terms(x.x, x.y), b = split_terms(x.z, x.w);
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        qf[s][0][n] = a.t[n];
        qf[s][1][n] = b.t[n];
      }
    }
  }

  // the five smaller products of terms, in two sums: of the middle terms with the
  // first, and the rest
  __device__ __forceinline__ static void mma_small(float* small, float* tiny,
                                                   const uint32_t (*a)[4], const uint32_t* b0,
                                                   const uint32_t* b1) {
    mma<__nv_bfloat16>(tiny, a[2], b0[0], b1[0]);
    mma<__nv_bfloat16>(small, a[1], b0[0], b1[0]);
    mma<__nv_bfloat16>(tiny, a[0], b0[2], b1[2]);
    mma<__nv_bfloat16>(small, a[0], b0[1], b1[1]);
    mma<__nv_bfloat16>(tiny, a[1], b0[1], b1[1]);
  }

  // q . K of one head and row of the tile at k, by plain multiplications: for the scores
  // whose terms hold a NaN, which an infinity leaves among its own, where the
  // products may be infinities of one sign (a key of weight 0, say).
  __device__ __noinline__ static float plain_score(const float* q, uint32_t k, int row) {
    float sum = 0.0f;
#pragma unroll 1
    for (int i = 0; i < D / 4; ++i) {
      float x[4];
      shared4(k + chunk_at<kKRow>(row, i), x);
#pragma unroll
      for (int n = 0; n < 4; ++n) sum = fmaf(__ldg(q + 4 * i + n), x[n], sum);
    }
    return sum;
  }

  __device__ __forceinline__ void tile(const TileAt& t) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int tok = ((g & 1) << 2) | (g >> 1);  // row g's token, of each eight
    float s[4] = {}, s2[4] = {}, small[4] = {}, tiny[4] = {};
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      float x[4], y[4];  // tokens tok and tok + 8
      shared4(t.k + chunk_at<kKRow>(tok, 4 * i + c), x);
      shared4(t.k + chunk_at<kKRow>(tok + 8, 4 * i + c), y);
      uint32_t a[3][4];
      const Bf16Terms p[4] = {split_terms(x[0], x[1]), split_terms(y[0], y[1]),
                              split_terms(x[2], x[3]), split_terms(y[2], y[3])};
#pragma unroll
      for (int n = 0; n < 3; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[n][e] = p[e].t[n];
      mma_small(small, tiny, a, qf[i][0], qf[i][1]);
      mma<__nv_bfloat16>(i & 1 ? s2 : s, a[0], qf[i][0][0], qf[i][1][0]);
    }
    const bool live0 = (t.mask >> tok) & 1u, live1 = (t.mask >> (tok + 8)) & 1u;
    bool moved = false, nan = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[e] += s2[e] + (small[e] + tiny[e]);
      nan |= isnan(s[e]);
    }
    if (__any_sync(0xffffffffu, nan)) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (isnan(s[e]) && 2 * c + (e & 1) < heads)
          s[e] = plain_score(query + (2 * c + (e & 1)) * D, t.k, tok + 4 * (e & 2));
      __syncwarp();
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s[e] = live0 ? s[e] * sl2 : -INFINITY;
      s[2 + e] = live1 ? s[2 + e] * sl2 : -INFINITY;
      moved |= fmaxf(s[e], s[2 + e]) > m[e];
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(m[e], fmaxf(s[e], s[2 + e]));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float f = mx == m[e] ? 1.0f : exp2f(m[e] - mx);
        m[e] = mx;
        l[e] *= f;
#pragma unroll
        for (int j = 0; j < DV / 32; ++j)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            o[j][y][e] *= f;
            o[j][y][2 + e] *= f;
          }
      }
    }
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[e] = exp2f(s[e] - (m[e & 1] == -INFINITY ? 0.0f : m[e & 1]));
      l[e & 1] += p[e];
    }
    // the weights of head g and tokens 2 c, 2 c + 1 of each eight, from the
    // lanes of those tokens' rows (token t is row 2 (t & 3) + t / 4)
    Bf16Terms w[2];
    float pv[2][2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int from = 2 * c + z, src = 4 * (2 * (from & 3) + (from >> 2)) + (g >> 1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float a = __shfl_sync(0xffffffffu, p[2 * u], src);
        const float b = __shfl_sync(0xffffffffu, p[2 * u + 1], src);
        pv[u][z] = g & 1 ? b : a;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) w[u] = split_terms(pv[u][0], pv[u][1]);
#pragma unroll
    for (int j = 0; j < DV / 32; ++j) {
      float x[4][4];  // tokens 2 c, 2 c + 1 of each eight, columns 32 j + 4 g ..
#pragma unroll
      for (int e = 0; e < 4; ++e)
        shared4(t.v + chunk_at<kVRow>(8 * (e >> 1) + 2 * c + (e & 1), 8 * j + g), x[e]);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        uint32_t a[3][4];
        const Bf16Terms p4[4] = {
            split_terms(x[0][2 * z], x[1][2 * z]), split_terms(x[0][2 * z + 1], x[1][2 * z + 1]),
            split_terms(x[2][2 * z], x[3][2 * z]), split_terms(x[2][2 * z + 1], x[3][2 * z + 1])};
#pragma unroll
        for (int n = 0; n < 3; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) a[n][e] = p4[e].t[n];
        float sum[4] = {}, tiny[4] = {};
        mma_small(sum, tiny, a, w[0].t, w[1].t);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += tiny[e];
        mma<__nv_bfloat16>(sum, a[0], w[0].t[0], w[1].t[0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][z][e] += sum[e];
      }
    }
  }

  __device__ __forceinline__ void finish(const Sink<float>& out) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[e];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      const int h = 2 * c + e;
      if (h >= heads) continue;
      const float f = out.partial ? 1.0f : inverse_sum(sum);
      float* row = (out.partial ? out.part : out.out) + (size_t)h * DV + 4 * g;
#pragma unroll
      for (int j = 0; j < DV / 32; ++j) {
        const float y[4] = {o[j][0][e] * f, o[j][0][2 + e] * f, o[j][1][e] * f,
                            o[j][1][2 + e] * f};
        store_quad(row + 32 * j, y);
      }
      if (lane < 4) {
        if (out.partial)
          *reinterpret_cast<float2*>(out.ml + 2 * h) = make_float2(m[e], sum);
        else if (out.lse)
          out.lse[h] = log_sum(m[e], sum);
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
  static constexpr int kWarpBytes = kStage * kStages;
  static constexpr int kBytes = kWarpBytes * E::kWarps;
  static_assert(kBytes <= 220 * 1024, "shared memory");
};

// A tile of a block's run of columns [c0, c1) (a column: one tile of one
// sequence, for every unit): unit u, column c0 + col, tile t of sequence b.
struct Cursor {
  int b, u, t, col;
  Seq s;
};

// a tile whose table entries have been asked for: lane i holds row i % kTile's
struct Lookup {
  int page, slot, g;
  bool in;
};

// A warp's pieces of units that it shares with others of its block: [0] of the
// segment that its part began with, [1] of the one that it ended with.
struct Left {
  int from;  // the sequence's first column
  int b, u, tiles;
  bool any;
};

// The code before a warp's first load runs once and cold: it is kept short
// (32-bit columns, one copy of the search: 10.6 -> 9.0 us for 1024 tokens).
template <typename E>
__global__ void __launch_bounds__(E::kWarps * 32, 1)
    lt_paged_decode_kernel(const DecodeArgs a) {
  using R = Ring<E>;
  using QT = typename E::QT;
  constexpr int W = E::kWarps, kThreads = W * 32, TILE = E::kTile, S = R::kStages;
  static_assert(W <= 16, "the pieces of a block's warps fit one warp's lanes");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int before[kThreads];  // columns of the sequences before this thread's
  __shared__ int warp_sum[W];
  __shared__ Left left[2 * W];
  __shared__ int order[2 * W], group0[2 * W + 1], groups;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  dependency_wait();     // launched early: what came before on the stream is done now
  dependency_release();  // the second launch may come and wait

  // each thread adds a run of sequences' tiles; a scan gives the runs' starts
  const int per = (a.B + kThreads - 1) / kThreads;
  int sum = 0;
#pragma unroll 1
  for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) {
    const int len = a.lens[b];
    if ((len < 0 || len > a.max_len) && blockIdx.x == 0) report_error(a.err, kDevErrBadSeqlens);
    sum += seq_of<TILE>(a, len).tiles;
  }
  int scan = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, scan, off);
    if (lane >= off) scan += x;
  }
  if (lane == 31) warp_sum[warp] = scan;
  if (tid < 2 * W) left[tid].any = false;
  __syncthreads();
  int total = 0, mine = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) mine += warp_sum[w];
    total += warp_sum[w];
  }
  before[tid] = mine + scan - sum;
  __syncthreads();

  // the block's columns, and this warp's tiles of them in the order (unit,
  // column): whole parts of units where the units divide the warps
  const int run = max((int)((unsigned)(total + gridDim.x - 1) / gridDim.x), 1);
  const int c0 = blockIdx.x * run, c1 = min(c0 + run, total), ncol = max(c1 - c0, 0);
  int col0, u0, count;
  if (a.k_shift >= 0) {
    const int p = (ncol + (1 << a.k_shift) - 1) >> a.k_shift;
    u0 = warp >> a.k_shift;
    col0 = (warp - (u0 << a.k_shift)) * p;
    count = min(p, ncol - col0);
  } else {
    const int all = a.units * ncol, p = (all + W - 1) / W, start = warp * p;
    u0 = start / max(ncol, 1);
    col0 = start - u0 * ncol;
    count = min(p, all - start);
  }

  if (count > 0) {
    // the sequences and tiles of the warp's first column and, where its part
    // may go on into another unit, of the block's
    Cursor first = {}, cc = {};
#pragma unroll 1
    for (int pass = a.k_shift >= 0 ? 1 : 0; pass < 2; ++pass) {
      const int col = pass ? col0 : 0;
      int lo = 0, hi = kThreads;  // the last thread whose sequences begin at or before it
#pragma unroll 1
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= c0 + col)
          lo = mid;
        else
          hi = mid;
      }
      int rem = c0 + col - before[lo];
      cc.b = lo * per;
      cc.s = seq_of<TILE>(a, a.lens[cc.b]);
#pragma unroll 1
      while (cc.b + 1 < a.B && rem >= cc.s.tiles) {
        rem -= cc.s.tiles;
        cc.s = seq_of<TILE>(a, a.lens[++cc.b]);
      }
      cc.t = rem;
      cc.col = col;
      if (pass == 0) first = cc;
    }
    cc.u = u0;
    auto next = [&](Cursor& c) {
      ++c.t;
      if (++c.col == ncol) {
        const int u = c.u + 1;
        c = first;
        c.u = u;
      } else if (c.t == c.s.tiles) {
        c.t = 0;
        do c.s = seq_of<TILE>(a, a.lens[++c.b]);
        while (c.s.tiles == 0 && c.b + 1 < a.B);
      }
    };
    Cursor pc = cc;

    uint8_t* ring = smem + warp * R::kWarpBytes;
    const uint32_t ring_u = smem_u32(ring);
    E eng;

    const int row = lane & (TILE - 1);
    constexpr uint32_t kFull = TILE == 32 ? 0xffffffffu : (1u << (TILE & 31)) - 1u;
    constexpr int kc = E::kKRow / 16, vc = E::kVRow / 16;  // chunks per row
    const uint8_t *k_lane = a.k + lane % kc * 16, *v_lane = a.v + lane % vc * 16;
    const uint32_t k_first = chunk_at<E::kKRow>(lane / kc, lane % kc);
    const uint32_t v_first = chunk_at<E::kVRow>(lane / vc, lane % vc);
    auto look = [&](const Cursor& c) {
      Lookup p;
      const int pos = c.s.first + c.t * TILE + row;
      p.in = pos < c.s.len;
      const int idx = page_of(a, pos);
      p.slot = pos - idx * a.page_size;
      p.page = p.in ? __ldg(a.table + (int64_t)c.b * a.table_stride + idx) : 0;
      p.g = a.nhb == 1 ? c.u : c.u / a.nhb;
      return p;
    };
    auto issue = [&](int stage, const Lookup& p) {
      bool live = p.in;
      if (live && (p.page < 0 || p.page >= a.num_pages)) {
        report_error(a.err, kDevErrBadPage);
        live = false;
      }
      const uint32_t mask = __ballot_sync(0xffffffffu, live) & kFull;
      const uint32_t page = live ? p.page : 0, slot = live ? p.slot : 0;
      const uint32_t ko = page * a.kpg + slot * a.ksl + p.g * a.khd;
      const uint32_t vo = a.same ? ko : page * a.vpg + slot * a.vsl + p.g * a.vhd;
      const uint32_t dst = ring_u + stage * R::kStage;
      if (mask == kFull && a.same && E::kKRow == E::kVRow) {  // nearly always
#pragma unroll
        for (int i = 0; i < TILE * kc / 32; ++i) {
          const int r = i * (32 / kc) + lane / kc;
          const uint64_t off = (uint64_t)__shfl_sync(0xffffffffu, ko, r) * 16;
          copy16(step_at<E::kKRow>(dst + k_first, i), k_lane + off);
          copy16(step_at<E::kKRow>(dst + k_first, i) + R::kK, v_lane + off);
        }
      } else {
#pragma unroll
        for (int i = 0; i < TILE * kc / 32; ++i) {
          const int r = i * (32 / kc) + lane / kc;
          const uint64_t off = (uint64_t)__shfl_sync(0xffffffffu, ko, r) * 16;
          copy16(step_at<E::kKRow>(dst + k_first, i), k_lane + off, (mask >> r) & 1u);
        }
#pragma unroll
        for (int i = 0; i < TILE * vc / 32; ++i) {
          const int r = i * (32 / vc) + lane / vc;
          const uint64_t off = (uint64_t)__shfl_sync(0xffffffffu, vo, r) * 16;
          copy16(step_at<E::kVRow>(dst + R::kK + v_first, i), v_lane + off, (mask >> r) & 1u);
        }
      }
      if constexpr (E::kQuant) {
        const int64_t at = ((int64_t)page * a.Hkv + p.g) * a.page_size + slot;
        if (lane < TILE) {
          copy4(dst + R::kK + R::kV + lane * 4, a.ks + at, live);
          copy4(dst + R::kK + R::kV + R::kScale + lane * 4, a.vs + at, live);
        }
      }
      if (lane == 0)
        *reinterpret_cast<uint32_t*>(ring + stage * R::kStage + R::kK + R::kV + 2 * R::kScale) =
            mask;
    };

    const int n = count;
    int issued = 0;
    Lookup pend = look(pc);
    auto feed = [&](int stage) {
      if (issued < n) {
        issue(stage, pend);
        if (++issued < n) {
          next(pc);
          pend = look(pc);
        }
      }
      copy_commit();
    };
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) feed(s);

    int stage = 0;
    int seg = cc.col;  // the segment's first column
    bool first_seg = true;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      if (i == 0 || cc.t == 0 || cc.col == 0) {  // a new unit or sequence
        const int g = cc.u / a.nhb, blk = cc.u - g * a.nhb;
        const int h0 = g * a.G + blk * E::kHeads;
        eng.begin(static_cast<const QT*>(a.q) + ((size_t)cc.b * a.Hq + h0) * E::kD,
                  min(E::kHeads, a.G - blk * E::kHeads), a.scale);
        seg = cc.col;
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
      const bool seq_done = cc.t + 1 == cc.s.tiles;
      if (seq_done || cc.col + 1 == ncol || i + 1 == n) {
        const int from = c0 + cc.col - cc.t, to = from + cc.s.tiles;
        const bool had_block = c0 + seg == max(from, c0) && c0 + cc.col + 1 == min(to, c1);
        const int g = cc.u / a.nhb, blk = cc.u - g * a.nhb;
        const size_t orow = (size_t)cc.b * a.Hq + g * a.G + blk * E::kHeads;
        Sink<QT> out;
        out.partial = !(had_block && from >= c0 && to <= c1);
        out.out = static_cast<QT*>(a.out) + orow * a.dv;
        out.lse = a.lse ? a.lse + orow : nullptr;
        const int slot = first_seg ? 0 : 1;
        const Pieces to_where = had_block ? a.block : a.warp;
        const size_t piece =
            (had_block ? ((size_t)blockIdx.x * 2 + (from < c0 ? 0 : 1)) * a.units + cc.u
                       : ((size_t)blockIdx.x * W + warp) * 2 + slot) * a.hb;
        out.part = to_where.part + piece * a.dv;
        out.ml = to_where.ml + piece * 2;
        eng.finish(out);
        if (!had_block && lane == 0)
          left[2 * warp + slot] = Left{from, cc.b, cc.u, cc.s.tiles, true};
        first_seg = false;
        // (the last column's sequence, of which every unit says the same)
        if (!a.by_seq && cc.u == 0 && cc.col + 1 == ncol && lane == 0)
          a.shared[blockIdx.x] =
              Shared{cc.b, (int)blockIdx.x,
                     from >= c0 && to > c1 ? (to - 1) / run - (int)blockIdx.x + 1 : 0, 0};
      }
      if (i + 1 < n) next(cc);
    }
    copy_wait<0>();
  }

  // sequences of no keys: zeros, from one block each
#pragma unroll 1
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int len = a.lens[b];
    if (len != 0) continue;
    for (int i = tid; i < a.Hq * a.dv; i += kThreads)
      from_float(static_cast<QT*>(a.out) + (size_t)b * a.Hq * a.dv + i, 0.0f);
    if (a.lse)
      for (int i = tid; i < a.Hq; i += kThreads) a.lse[(size_t)b * a.Hq + i] = -INFINITY;
  }

  // what the second launch has to do: by sequence (block b says it of sequence
  // b; one sequence per thread then), or by block, of the sequence that begins
  // in its columns and goes on (said above, by the warp that came upon it)
  if (tid == 0 && a.by_seq && blockIdx.x < a.B) {
    const int b = blockIdx.x, from = before[b], tiles = seq_of<TILE>(a, a.lens[b]).tiles;
    const int at = from / run, n = tiles ? (from + tiles - 1) / run - at + 1 : 0;
    a.shared[b] = Shared{b, at, n > 1 ? n : 0, 0};
  }
  if (tid == 0 && !a.by_seq && ncol == 0) a.shared[blockIdx.x] = Shared{0, 0, 0, 0};

  // ---- the pieces of this block's warps, joined
  __syncthreads();
  if (warp == 0) {  // lane p: piece p, in the order of the tiles
    const bool any = lane < 2 * W && left[lane].any;
    const uint32_t valid = __ballot_sync(0xffffffffu, any);
    const uint32_t below = valid & ((1u << lane) - 1u);
    const int prev = below ? 31 - __clz(below) : 0;
    const bool lead = any && (!below || left[lane].from != left[prev].from ||
                              left[lane].u != left[prev].u);
    const uint32_t leads = __ballot_sync(0xffffffffu, lead);
    if (any) order[__popc(below)] = lane;
    if (lead) group0[__popc(leads & ((1u << lane) - 1u))] = __popc(below);
    if (lane == 0) {
      groups = __popc(leads);
      group0[__popc(leads)] = __popc(valid);
    }
  }
  __syncthreads();
  const int cols = a.dv >> 2, per_group = a.hb * cols;
  for (int item = tid; item < groups * per_group; item += kThreads) {
    const int gi = item / per_group, rest = item - gi * per_group;
    const int h = rest / cols, c4 = rest - h * cols;
    const int p0 = group0[gi], np = group0[gi + 1] - p0;
    const Left f = left[order[p0]];
    const int g = f.u / a.nhb, blk = f.u - g * a.nhb;
    if (h >= a.G - blk * E::kHeads) continue;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f, mx = -INFINITY;
    auto row = [&](int i) { return ((size_t)blockIdx.x * 2 * W + order[p0 + i]) * a.hb + h; };
#pragma unroll 4
    for (int i = 0; i < np; ++i) {
      const size_t p = row(i);
      add_piece(o, l, mx, *reinterpret_cast<const float2*>(a.warp.ml + p * 2),
                *reinterpret_cast<const float4*>(a.warp.part + p * a.dv + c4 * 4));
    }
    if (f.from >= c0 && f.from + f.tiles <= c1) {
      const size_t orow = (size_t)f.b * a.Hq + g * a.G + blk * E::kHeads + h;
      const float r = inverse_sum(l);
      const float y[4] = {o.x * r, o.y * r, o.z * r, o.w * r};
      store_quad(static_cast<QT*>(a.out) + orow * a.dv + c4 * 4, y);
      if (a.lse && c4 == 0) a.lse[orow] = log_sum(mx, l);
    } else {
      const size_t p =
          (((size_t)blockIdx.x * 2 + (f.from < c0 ? 0 : 1)) * a.units + f.u) * a.hb + h;
      *reinterpret_cast<float4*>(a.block.part + p * a.dv + c4 * 4) = o;
      if (c4 == 0) *reinterpret_cast<float2*>(a.block.ml + p * 2) = make_float2(mx, l);
    }
  }
}

template <typename E>
cudaError_t launch_engine(const DecodeArgs& a, int sms, cudaStream_t stream) {
  auto kern = lt_paged_decode_kernel<E>;
  constexpr int smem = Ring<E>::kBytes;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(sms), E::kWarps * 32, smem, stream, a);
}

template <typename QT, typename KT, int NB>
cudaError_t launch_mma_nb(const DecodeArgs& a, int d, int sms, cudaStream_t s) {
  if (d == 64)
    return a.dv == 64 ? launch_engine<MmaEngine<QT, KT, 64, 64, NB>>(a, sms, s)
                      : launch_engine<MmaEngine<QT, KT, 64, 128, NB>>(a, sms, s);
  return a.dv == 64 ? launch_engine<MmaEngine<QT, KT, 128, 64, NB>>(a, sms, s)
                    : launch_engine<MmaEngine<QT, KT, 128, 128, NB>>(a, sms, s);
}

template <typename QT, typename KT>
cudaError_t launch_mma(const DecodeArgs& a, int d, int sms, cudaStream_t s) {
  return heads_at_once(false, a.G) == 8 ? launch_mma_nb<QT, KT, 1>(a, d, sms, s)
                                        : launch_mma_nb<QT, KT, 2>(a, d, sms, s);
}

// the first launch, one translation unit per query type
cudaError_t launch_bf16(const DecodeArgs& a, lt_kv_dtype_t kv, int d, int sms, cudaStream_t s);
cudaError_t launch_f16(const DecodeArgs& a, lt_kv_dtype_t kv, int d, int sms, cudaStream_t s);
cudaError_t launch_f32(const DecodeArgs& a, lt_kv_dtype_t kv, int d, int sms, cudaStream_t s);

}  // namespace paged
}  // namespace lt
