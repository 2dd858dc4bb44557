// qk_norm_rope.cu -- root-mean-square norm of every query and key head, gain
// and position rotation in one pass, and its backward pass.
//
// Per row x (one head of one token, d values), r = (mean(x^2) + eps)^(-1/2):
//     forward:  y = x r w,  out = R y
//     backward: g = R^T dout,  u = g w,  dx = r u - x r^3 mean(u x),
//               dw = sum over rows of g x r
// R turns each pair (a, b) by A = position * inv_freq.  A reaches millions of
// turns, so it is formed in turns and reduced in fp64; only the fraction of a
// turn, at most 1/2, goes to fp32 sine and cosine.
//
// Bound by memory.  A warp takes whole tokens, and its angles stay in
// registers for all heads.  The heads of a token are contiguous, so a warp
// moves them in batches of 2 KB with one bulk copy each way, through a ring of
// its own in shared memory (results overwrite their inputs there): enough
// bytes in flight without holding them in registers, and few instructions per
// element, which issue would otherwise bound.  A row is spread over d/8 lanes
// (the norm is a 3- or 4-step shuffle); each lane holds two quads of elements,
// 4j.. and rot/2 + 4j..: whichever way the pairs are laid out, both halves of a
// pair are in one lane, and no value crosses lanes for the rotation.  Products
// run two at a time (f32x2).
//
// Measured on one B200 (plain copy 6.55 TB/s), 32 + 8 heads of 128, replayed from a
// graph: 32768 bf16 tokens forward 108 us, 6.2 TB/s; 16384 backward 88 us, 5.7 TB/s (118
// and 98 in seconds of back-to-back calls, whose power lowers the clock: the
// issue slots are 60% busy).  fp32: 16384 tokens forward 123 us, 5.5 TB/s; 8192 backward
// 95 us, 5.3 TB/s.
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
namespace {

constexpr int kT = 256, kW = kT / 32;  // threads, warps

struct NormArgs {
  const void* x[2];    // q, k
  const void* g[2];    // backward: upstream gradients (dense)
  void* out[2];        // forward: outputs (dense); backward: dq, dk
  const void* w[2];    // gains or nullptr
  int64_t stride[2];   // tokens of x, in elements
  int64_t ostride[2];  // tokens of out, in elements
  int H[2];
  const int32_t* positions;
  int64_t n_pos;
  const float* inv_freq;
  int rot;
  int parts;       // warps that share a token's heads
  int64_t tokens;
  float eps;
  int w_f32;       // gains are fp32
  float* partial;  // backward: [block][2][d] sums of the gains' gradients
  int* err;
};

struct GainArgs {
  const float* partial;  // [blocks][2][d]
  void* out[2];          // [d] each, or nullptr
  int blocks, d, dtype;  // dtype of out (lt_dtype_t)
};

// A lane's place: index j in its row, row `grp` of the warp's step, and the
// offsets of its two quads.
template <int D>
struct Lane {
  static constexpr int L = D / 8, RW = 32 / L;  // lanes per row, rows per warp
  int j, grp, qa, qb;
  bool rotated;
  __device__ __forceinline__ explicit Lane(int rot) {
    const int lane = threadIdx.x & 31;
    j = lane % L;
    grp = lane / L;
    rotated = j < (rot >> 3);
    qa = rotated ? 4 * j : 8 * j;
    qb = rotated ? (rot >> 1) + 4 * j : 8 * j + 4;
  }
  // each row's sum over its lanes, of N rows
  template <int N>
  __device__ __forceinline__ static void row_sums(float* x) {
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1)
#pragma unroll
      for (int v = 0; v < N; ++v) x[v] += __shfl_xor_sync(0xffffffffu, x[v], off);
  }
};

// Cosines and sines of a lane's four pairs, as the rotation's products take
// them: halves (i, i + rot/2): c[0..1] and s[0..1] over pairs (0,1), (2,3);
// neighbours: c[p] = (cos, cos), s[p] = (-sin, sin) of pair p.
template <bool IL>
struct Angles {
  F2 c[IL ? 4 : 2], s[IL ? 4 : 2], n[IL ? 4 : 2];  // n = -s
};

// sine and cosine of a fraction of a turn, |t| <= 1/2.  16-bit outputs: the
// hardware functions, within 2^-21 on [-pi, pi], far below half a step of the
// type (2^-11 at least).  fp32: the accurate ones, of the fraction rounded to fp32,
// turned on by what that left out (up to 9e-8 of angle, more than they are off).
template <typename T>
__device__ __forceinline__ void sincos_turn(double t, float* s, float* c) {
  const float f = (float)t;
  if constexpr (sizeof(T) == 2) {
    __sincosf(6.2831853071795865f * f, s, c);
  } else {
    float sf, cf;
    sincospif(2.0f * f, &sf, &cf);
    const float rest = 6.2831853071795865f * (float)(t - (double)f);
    *s = fmaf(cf, rest, sf);
    *c = fmaf(-sf, rest, cf);
  }
}

// the token's angles: the rows of a warp's step compute a share each and
// exchange them
template <typename T, int D, bool IL>
__device__ __forceinline__ void angles_of(const NormArgs& a, const Lane<D>& ln, uint32_t t,
                                          Angles<IL>& out) {
  constexpr int L = Lane<D>::L, RW = Lane<D>::RW, SH = 4 / RW;  // a lane's share
  constexpr double kInvTwoPi = 0.15915494309189533577;
  float c[4], s[4];
  float mc[SH], ms[SH];
  if (ln.rotated) {
    const int pos = __ldg(a.positions + (a.n_pos == a.tokens ? t : t % (uint32_t)a.n_pos));
#pragma unroll
    for (int e = 0; e < SH; ++e) {
      const int i = ln.grp * SH + e;  // which of the lane's four
      const int pair = IL ? (i < 2 ? 2 * ln.j + i : (a.rot >> 2) + 2 * ln.j + i - 2)
                          : 4 * ln.j + i;
      double turns = (double)pos * (double)__ldg(a.inv_freq + pair) * kInvTwoPi;
      turns -= rint(turns);
      sincos_turn<T>(turns, &ms[e], &mc[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < SH; ++e) mc[e] = 1.0f, ms[e] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = __shfl_sync(0xffffffffu, mc[i % SH], (i / SH) * L + ln.j);
    s[i] = __shfl_sync(0xffffffffu, ms[i % SH], (i / SH) * L + ln.j);
  }
  if constexpr (IL) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      out.c[p] = pack_f2(c[p], c[p]);
      out.s[p] = pack_f2(-s[p], s[p]);
      out.n[p] = pack_f2(s[p], -s[p]);
    }
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      out.c[p] = pack_f2(c[2 * p], c[2 * p + 1]);
      out.s[p] = pack_f2(s[2 * p], s[2 * p + 1]);
      out.n[p] = pack_f2(-s[2 * p], -s[2 * p + 1]);
    }
  }
}

// turn the lane's eight values y[0..3] (pairs of neighbours in registers);
// kBack: by the negative angle
template <bool IL, bool kBack>
__device__ __forceinline__ void turn(F2* y, const Angles<IL>& g) {
  if constexpr (IL) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      y[p] = fma2(swap2(y[p]), kBack ? g.n[p] : g.s[p], mul2(y[p], g.c[p]));
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const F2 A = y[p], B = y[2 + p];
      y[p] = fma2(B, kBack ? g.s[p] : g.n[p], mul2(A, g.c[p]));
      y[2 + p] = fma2(A, kBack ? g.n[p] : g.s[p], mul2(B, g.c[p]));
    }
  }
}

template <typename T>
__device__ __forceinline__ void load_gain(const void* w, int w_f32, int qa, int qb, F2* f) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = pack_f2(1.0f, 1.0f);
  } else if (w_f32) {
    widen2x2(load_quad(static_cast<const float*>(w) + qa), f);
    widen2x2(load_quad(static_cast<const float*>(w) + qb), f + 2);
  } else {
    widen2x2(load_quad(static_cast<const T*>(w) + qa), f);
    widen2x2(load_quad(static_cast<const T*>(w) + qb), f + 2);
  }
}

// sum over the lane's eight products of x and y
__device__ __forceinline__ float dot8(const F2* x, const F2* y) {
  F2 s = mul2(x[0], y[0]);
#pragma unroll
  for (int e = 1; e < 4; ++e) s = fma2(x[e], y[e], s);
  const float2 t = unpack_f2(s);
  return t.x + t.y;
}

// -------------------------------------------------------------- the batches
constexpr int kBatchBytes = 2048, kStages = 3, kBlocks = 2;  // (blocks per SM)
constexpr int kRows = 2;  // rows of a warp's lanes worked on at a time
// A warp's ring: kStages stages of kIn batches (x; backward also the upstream
// gradient) of kStep heads.  More bytes under way do not pay: at 2 x 16384
// tokens of 32 + 8 bf16 heads of 128, 16 warps per SM with 2 KB x 3 stages
// take 113 us, 4 KB x 3 128, 8 KB x 3 141 (and 2 KB x 4 with 24 warps 129):
// reads and writes of DRAM then alternate in longer bursts.
template <typename T, int D, bool kBack>
struct Ring {
  static constexpr int kIn = kBack ? 2 : 1;
  static constexpr int kStep = kBatchBytes / (D * (int)sizeof(T));  // heads per batch
  static constexpr int kBatch = kStep * D;                          // elements
  static constexpr int kWarp = kStages * kIn * kBatch;
  static constexpr int kBytes = kW * kWarp * (int)sizeof(T);
};
constexpr uint64_t kWaitNs = 1000000000ull;  // a wait gives up after 1 s

// A warp's batches in order: units (token, part) unit, + step, ..., and of each
// the token's batches part, + parts, ... (the queries' first, then the keys').
struct Walk {
  uint32_t unit, t;
  int b;
  __device__ __forceinline__ void place(const NormArgs& a) {
    t = a.parts == 1 ? unit : unit / (uint32_t)a.parts;
    b = (int)(unit - t * (uint32_t)a.parts);
  }
  __device__ __forceinline__ void next(const NormArgs& a, int nb, uint32_t step) {
    b += a.parts;
    if (b >= nb) {
      unit += step;
      place(a);
    }
  }
};

// Batch b of token t: queries or keys (ph), its first head and their number.
template <int STEP>
struct Batch {
  int ph, h0, n;
  __device__ __forceinline__ Batch(const NormArgs& a, int b, int nbq) {
    ph = b >= nbq;
    h0 = (ph ? b - nbq : b) * STEP;
    n = min(STEP, (ph ? a.H[1] : a.H[0]) - h0);
  }
};

// Forward (kBack false) and backward.  Backward, each lane also sums its eight
// columns' gain gradients over its rows; the block's rows of lanes are added in
// order at the end, and the launch below adds the blocks in order.
template <typename T, int D, bool IL, bool kBack>
__global__ void __launch_bounds__(kT, kBlocks) lt_norm_rope_kernel(const NormArgs a) {
  using LN = Lane<D>;
  using R = Ring<T, D, kBack>;
  constexpr int STEP = R::kStep, RG = kW * LN::RW, S = kStages;
  // forward, 16-bit: twice the rows where a batch has them (2 x 8192 tokens of 32 +
  // 8 heads of 128: 57.4 -> 56.1 us); the others have no registers left for it
  constexpr int kMoreRows = kBack || sizeof(T) == 4 ? kRows : 2 * kRows;
  static_assert(STEP % (kMoreRows * LN::RW) == 0, "rows at a time stay inside a batch");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kW][S];
  __shared__ volatile int abort_flag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T* const ring = reinterpret_cast<T*>(smem) + warp * R::kWarp;
  uint64_t* const full = bars[warp];
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncthreads();

  const LN ln(a.rot);
  const int nbq = (a.H[0] + STEP - 1) / STEP, nb = nbq + (a.H[1] + STEP - 1) / STEP;
  const uint32_t units = (uint32_t)a.tokens * a.parts, step = gridDim.x * kW;
  Walk use, load;
  use.unit = warp * gridDim.x + blockIdx.x;
  use.place(a);
  load = use;

  // ask for the next batch of `load` (every lane keeps count, the first issues)
  int issued = 0, lstage = 0;
  auto fetch = [&]() {
    if (load.unit >= units) return;
    if (lane == 0) {
      const Batch<STEP> bt(a, load.b, nbq);
      const uint32_t bytes = (uint32_t)(bt.n * D * sizeof(T));
      T* const dst = ring + lstage * (R::kIn * R::kBatch);
      mbar_arrive_expect_tx(&full[lstage], kBack ? 2 * bytes : bytes);
      bulk_load(dst,
                static_cast<const T*>(bt.ph ? a.x[1] : a.x[0]) +
                    (int64_t)load.t * (bt.ph ? a.stride[1] : a.stride[0]) + bt.h0 * D,
                bytes, &full[lstage]);
      if (kBack)
        bulk_load(dst + R::kBatch,
                  static_cast<const T*>(bt.ph ? a.g[1] : a.g[0]) +
                      ((int64_t)load.t * (bt.ph ? a.H[1] : a.H[0]) + bt.h0) * D,
                  bytes, &full[lstage]);
    }
    ++issued;
    if (++lstage == S) lstage = 0;
    load.next(a, nb, step);
  };
  for (int i = 0; i < S - 1; ++i) fetch();

  F2 w[2][4], dw[2][4];
  load_gain<T>(a.w[0], a.w_f32, ln.qa, ln.qb, w[0]);
  load_gain<T>(a.w[1], a.w_f32, ln.qa, ln.qb, w[1]);
#pragma unroll
  for (int e = 0; e < 4; ++e) dw[0][e] = dw[1][e] = F2{0};

  Angles<IL> ang;
  uint32_t have = ~0u;  // the token whose angles `ang` holds
  int done = 0, stage = 0, parity = 0;
#pragma unroll 1
  for (; use.unit < units; ++done) {
    const Batch<STEP> bt(a, use.b, nbq);
    if (a.rot && have != use.t) {
      angles_of<T, D, IL>(a, ln, use.t, ang);
      have = use.t;
    }
    F2 cw[4], cd[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      cw[e] = bt.ph ? w[1][e] : w[0][e];
      cd[e] = F2{0};
    }
    if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], parity, &abort_flag, a.err, kWaitNs)))
      break;
    T* const batch = ring + stage * (R::kIn * R::kBatch);
    T* row = batch + ln.grp * D;
    int hw = 0;
    // Rows hw .. of the batch, kV per lane at a time: their shuffles and roots
    // overlap.  Heads past the last are whatever the stage held: computed, not
    // stored.
    auto rows = [&](auto at_a_time) {
      constexpr int kV = decltype(at_a_time)::value;
      const int h = hw + ln.grp;
      F2 x[kV][4], g[kV][4];
      float rr[kV];
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const T* const r = row + v * (LN::RW * D);
        widen2x2(*reinterpret_cast<const Quad<T>*>(r + ln.qa), x[v]);
        widen2x2(*reinterpret_cast<const Quad<T>*>(r + ln.qb), x[v] + 2);
        if constexpr (kBack) {
          widen2x2(*reinterpret_cast<const Quad<T>*>(r + R::kBatch + ln.qa), g[v]);
          widen2x2(*reinterpret_cast<const Quad<T>*>(r + R::kBatch + ln.qb), g[v] + 2);
        }
        rr[v] = dot8(x[v], x[v]);
      }
      LN::template row_sums<kV>(rr);
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        rr[v] = rsqrtf(rr[v] * (1.0f / D) + a.eps);
        const F2 r2 = pack_f2(rr[v], rr[v]);
        if constexpr (!kBack) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[v][e] = mul2(mul2(x[v][e], r2), cw[e]);
          if (ln.rotated) turn<IL, false>(x[v], ang);
        } else {
          if (ln.rotated) turn<IL, true>(g[v], ang);
          const bool live = h + v * LN::RW < bt.n;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[v][e] = mul2(x[v][e], r2);  // n = x r
            if (live) cd[e] = fma2(g[v][e], x[v][e], cd[e]);
            g[v][e] = mul2(g[v][e], cw[e]);  // u
          }
        }
      }
      if constexpr (kBack) {
        // dx = r (u - n mean(u n)), dw += g n
        float m[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) m[v] = dot8(g[v], x[v]);
        LN::template row_sums<kV>(m);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
          m[v] *= -1.0f / D;
          const F2 m2 = pack_f2(m[v], m[v]), r2 = pack_f2(rr[v], rr[v]);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[v][e] = mul2(r2, fma2(x[v][e], m2, g[v][e]));
        }
      }
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        store_quad(row + v * (LN::RW * D) + ln.qa, x[v][0], x[v][1]);
        store_quad(row + v * (LN::RW * D) + ln.qb, x[v][2], x[v][3]);
      }
      hw += kV * LN::RW;
      row += kV * LN::RW * D;
    };
#pragma unroll 1
    while (hw < bt.n) {
      if (kMoreRows > kRows && bt.n - hw > kRows * LN::RW)
        rows(std::integral_constant<int, kMoreRows>());
      else
        rows(std::integral_constant<int, kRows>());
    }
    fence_proxy_async_smem();  // the results, before the copy unit reads them
    __syncwarp();
    if (lane == 0) {
      const int64_t os = kBack ? (bt.ph ? a.ostride[1] : a.ostride[0])
                               : (int64_t)(bt.ph ? a.H[1] : a.H[0]) * D;
      bulk_store(static_cast<T*>(bt.ph ? a.out[1] : a.out[0]) + (int64_t)use.t * os + bt.h0 * D,
                 batch, (uint32_t)(bt.n * D * sizeof(T)));
      bulk_commit_group();
      bulk_wait_read_but_last();  // the batch before this one has left its stage
    }
    if constexpr (kBack) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (bt.ph)
          dw[1][e] = add2(dw[1][e], cd[e]);
        else
          dw[0][e] = add2(dw[0][e], cd[e]);
      }
    }
    if (++stage == S) {
      stage = 0;
      parity ^= 1;
    }
    use.next(a, nb, step);
    fetch();
  }
  // a wait that gave up: the loads still under way must land before the block ends
  for (; done < issued; ++done) {
    int none = 0;
    mbar_wait(&full[stage], parity, &none, nullptr, kWaitNs);
    if (++stage == S) {
      stage = 0;
      parity ^= 1;
    }
  }
  if (lane == 0) bulk_wait_all();  // the stores read shared memory
  if constexpr (kBack) {
    dependency_release();
    if (!a.partial) return;
    __shared__ __align__(16) float red[RG][D];  // (written two floats at a time)
    const int grp = warp * LN::RW + ln.grp;
#pragma unroll
    for (int ph = 0; ph < 2; ++ph) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float2*>(&red[grp][(e < 2 ? ln.qa : ln.qb) + 2 * (e & 1)]) =
            unpack_f2(dw[ph][e]);
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += kT) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < RG; ++q) s += red[q][c];
        a.partial[((size_t)blockIdx.x * 2 + ph) * D + c] = s;
      }
    }
  }
}

// columns of the blocks' sums added in block order: 32 columns per block, 32
// runs of blocks each, then the runs
__global__ void __launch_bounds__(1024) lt_norm_rope_gain_kernel(const GainArgs a) {
  __shared__ float red[32][33];
  dependency_wait();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  float s = 0.0f;
  for (int b = run; b < a.blocks; b += 32) s += a.partial[(size_t)b * 2 * a.d + c];
  red[run][threadIdx.x & 31] = s;
  __syncthreads();
  if (run == 0) {
    float t = 0.0f;
#pragma unroll
    for (int q = 0; q < 32; ++q) t += red[q][threadIdx.x];
    const int ph = c / a.d, col = c - ph * a.d;
    if (a.out[ph]) {
      if (a.dtype == LT_F32)
        static_cast<float*>(a.out[ph])[col] = t;
      else if (a.dtype == LT_BF16)
        static_cast<__nv_bfloat16*>(a.out[ph])[col] = __float2bfloat16_rn(t);
      else
        static_cast<__half*>(a.out[ph])[col] = __float2half_rn(t);
    }
  }
}

template <typename T, int D, bool IL, bool kBack>
cudaError_t launch_t(const NormArgs& a, int blocks, cudaStream_t stream) {
  constexpr int smem = Ring<T, D, kBack>::kBytes;
  auto kern = lt_norm_rope_kernel<T, D, IL, kBack>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  kern<<<blocks, kT, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, bool kBack>
cudaError_t launch_d(const NormArgs& a, int blocks, int d, int il, cudaStream_t s) {
  if (d == 64)
    return il ? launch_t<T, 64, true, kBack>(a, blocks, s)
              : launch_t<T, 64, false, kBack>(a, blocks, s);
  return il ? launch_t<T, 128, true, kBack>(a, blocks, s)
            : launch_t<T, 128, false, kBack>(a, blocks, s);
}

template <bool kBack>
cudaError_t launch(const NormArgs& a, int blocks, int d, int il, lt_dtype_t dtype,
                   cudaStream_t s) {
  return dtype == LT_BF16  ? launch_d<__nv_bfloat16, kBack>(a, blocks, d, il, s)
         : dtype == LT_F16 ? launch_d<__half, kBack>(a, blocks, d, il, s)
                           : launch_d<float, kBack>(a, blocks, d, il, s);
}

// Warps that share a token's heads: one where the tokens alone fill the warps that
// a launch has on the device, more where they are few (a decode step), up to one
// per batch.  Counting half of those warps: 600 tokens of 32 + 8 bf16 heads of 128
// forward 7.1 us against 5.0, backward 12.9 against 9.5; 256 tokens 4.4 against 3.7 and
// 8.4 against 7.1.  Rounding up instead of down: 2300 tokens 11.7 us against 9.6.
int token_parts(int64_t tokens, int H_q, int H_kv, int d, lt_dtype_t dtype, int sms) {
  const int step = kBatchBytes / (d * (int)dtype_size(dtype));  // Ring::kStep
  const int batches = (H_q + step - 1) / step + (H_kv + step - 1) / step;
  const int64_t want = (int64_t)sms * kBlocks * kW / tokens;
  return want < 1 ? 1 : want > batches ? batches : (int)want;
}

// blocks of a launch: kBlocks per SM; few units take a block each
int64_t block_count(int64_t units, int sms) {
  return units < kBlocks * sms ? units : kBlocks * sms;
}

// the checks that forward and backward share, without any CUDA call
lt_status_t check(const void* q, const void* k, const void* qw, const void* kw,
                  const int32_t* positions, int64_t n_pos, const float* inv_freq, int rot,
                  int interleaved, int64_t tokens, int H_q, int H_kv, int d, int64_t q_stride,
                  int64_t k_stride, float eps, lt_dtype_t dtype, lt_dtype_t w_dtype) {
  if (!dtype_ok(dtype) || (w_dtype != LT_F32 && w_dtype != dtype)) return LT_ERR_UNSUPPORTED;
  if (!q || !k) return LT_ERR_INVALID_ARG;
  if (tokens < 1 || H_q < 1 || H_kv < 1 || H_q > 65535 || H_kv > 65535) return LT_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return LT_ERR_INVALID_ARG;
  if (!(eps > 0.0f) || !isfinite(eps)) return LT_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return LT_ERR_UNSUPPORTED;
  if (rot < 0 || rot > d || rot % 8 != 0) return LT_ERR_UNSUPPORTED;
  if (rot > 0 && (!positions || !inv_freq || n_pos < 1 || tokens % n_pos != 0))
    return LT_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype);
  if (tokens > 0x7fffffff || !stride_ok(tokens, q_stride, H_q, d, es) ||
      !stride_ok(tokens, k_stride, H_kv, d, es))
    return LT_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(qw, 16) || !aligned_to(kw, 16) ||
      !aligned_to(positions, 4) || !aligned_to(inv_freq, 4))
    return LT_ERR_INVALID_ARG;
  return LT_OK;
}

bool disjoint(const Span* outs, int no, const Span* ins, int ni) {
  for (int o = 0; o < no; ++o) {
    for (int i = 0; i < ni; ++i)
      if (spans_overlap(outs[o], ins[i])) return false;
    for (int p = o + 1; p < no; ++p)
      if (spans_overlap(outs[o], outs[p])) return false;
  }
  return true;
}

// Two token-strided outputs whose address ranges interleave: legal exactly as
// slices of one tensor -- the same stride, and each token's rows apart.
bool slices_disjoint(const Span& a, int64_t a_stride, size_t a_row, const Span& b, int64_t b_stride,
                     size_t b_row, size_t es) {
  if (!spans_overlap(a, b)) return true;
  if (a_stride != b_stride) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const size_t period = (size_t)a_stride * es;
  const size_t off = x <= y ? (y - x) % period : period - 1 - (x - y - 1) % period;  // b past a
  return off >= a_row && off + b_row <= period;
}

}  // namespace
}  // namespace lt

extern "C" lt_status_t lt_qk_norm_rope(const void* q, const void* k, const void* q_weight,
                                       const void* k_weight, const int32_t* positions,
                                       int64_t n_pos, const float* inv_freq, int rot,
                                       int interleaved, void* q_out, void* k_out, int64_t tokens,
                                       int H_q, int H_kv, int d, int64_t q_stride,
                                       int64_t k_stride, float eps, lt_stream_t stream,
                                       lt_dtype_t dtype, lt_dtype_t w_dtype) {
  using namespace lt;
  const lt_status_t st = check(q, k, q_weight, k_weight, positions, n_pos, inv_freq, rot,
                               interleaved, tokens, H_q, H_kv, d, q_stride, k_stride, eps, dtype,
                               w_dtype);
  if (st != LT_OK) return st;
  if (!q_out || !k_out || !aligned_to(q_out, 16) || !aligned_to(k_out, 16))
    return LT_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype), ws = dtype_size(w_dtype);
  const Span ins[] = {{q, strided_bytes(tokens, q_stride, H_q, d, es)},
                      {k, strided_bytes(tokens, k_stride, H_kv, d, es)},
                      {q_weight, d * ws},
                      {k_weight, d * ws},
                      {rot ? positions : nullptr, (size_t)n_pos * 4},
                      {rot ? inv_freq : nullptr, (size_t)rot * 2}};
  const Span outs[] = {{q_out, (size_t)tokens * H_q * d * es},
                       {k_out, (size_t)tokens * H_kv * d * es}};
  if (!disjoint(outs, 2, ins, 6)) return LT_ERR_INVALID_ARG;
  const int dev = current_device();
  for (const Span& s : ins)
    if (s.p && !on_device(dev, s.p)) return LT_ERR_INVALID_ARG;
  for (const Span& s : outs)
    if (!on_device(dev, s.p)) return LT_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LT_ERR_CUDA;
  NormArgs a = {};
  a.x[0] = q;
  a.x[1] = k;
  a.out[0] = q_out;
  a.out[1] = k_out;
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.stride[0] = q_stride;
  a.stride[1] = k_stride;
  a.H[0] = H_q;
  a.H[1] = H_kv;
  a.positions = positions;
  a.n_pos = n_pos;
  a.inv_freq = inv_freq;
  a.rot = rot;
  a.tokens = tokens;
  a.eps = eps;
  a.w_f32 = w_dtype == LT_F32;
  a.parts = token_parts(tokens, H_q, H_kv, d, dtype, sms);
  a.err = device_error_word_current();
  if (!a.err) return LT_ERR_CUDA;
  const int blocks = (int)block_count(tokens * a.parts, sms);
  return launch<false>(a, blocks, d, interleaved, dtype, (cudaStream_t)stream) == cudaSuccess
             ? LT_OK
             : LT_ERR_CUDA;
}

extern "C" lt_status_t lt_qk_norm_rope_bwd_plan(int d, int num_sms, size_t* workspace_bytes) {
  if (!workspace_bytes) return LT_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return LT_ERR_UNSUPPORTED;
  if (num_sms <= 0) num_sms = lt::device_sm_count();
  if (num_sms <= 0) return LT_ERR_CUDA;
  // (a launch has at most two blocks per SM, however a token's heads are shared)
  *workspace_bytes = (size_t)lt::kBlocks * num_sms * 2 * d * sizeof(float);
  return LT_OK;
}

extern "C" lt_status_t lt_qk_norm_rope_bwd(
    const void* dq_out, const void* dk_out, const void* q, const void* k, const void* q_weight,
    const void* k_weight, const int32_t* positions, int64_t n_pos, const float* inv_freq, int rot,
    int interleaved, void* dq, void* dk, void* dq_weight, void* dk_weight, int64_t tokens, int H_q,
    int H_kv, int d, int64_t q_stride, int64_t k_stride, int64_t dq_stride, int64_t dk_stride,
    float eps, void* workspace, size_t workspace_bytes, lt_stream_t stream, lt_dtype_t dtype,
    lt_dtype_t w_dtype) {
  using namespace lt;
  const lt_status_t st = check(q, k, q_weight, k_weight, positions, n_pos, inv_freq, rot,
                               interleaved, tokens, H_q, H_kv, d, q_stride, k_stride, eps, dtype,
                               w_dtype);
  if (st != LT_OK) return st;
  if (!dq_out || !dk_out || !dq || !dk || !aligned_to(dq_out, 16) || !aligned_to(dk_out, 16) ||
      !aligned_to(dq, 16) || !aligned_to(dk, 16) || !aligned_to(dq_weight, 4) ||
      !aligned_to(dk_weight, 4))
    return LT_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype), ws = dtype_size(w_dtype);
  if (!stride_ok(tokens, dq_stride, H_q, d, es) || !stride_ok(tokens, dk_stride, H_kv, d, es))
    return LT_ERR_INVALID_ARG;
  const bool gains = dq_weight || dk_weight;
  const size_t nq = (size_t)H_q * d, nk = (size_t)H_kv * d;
  const Span ins[] = {{dq_out, tokens * nq * es},
                      {dk_out, tokens * nk * es},
                      {q, strided_bytes(tokens, q_stride, H_q, d, es)},
                      {k, strided_bytes(tokens, k_stride, H_kv, d, es)},
                      {q_weight, d * ws},
                      {k_weight, d * ws},
                      {rot ? positions : nullptr, (size_t)n_pos * 4},
                      {rot ? inv_freq : nullptr, (size_t)rot * 2},
                      {gains ? workspace : nullptr, workspace_bytes}};  // (used for the gains alone)
  for (int i = 0; i < 8; ++i)
    if (spans_overlap(ins[8], ins[i])) return LT_ERR_INVALID_ARG;
  const Span sq = {dq, strided_bytes(tokens, dq_stride, H_q, d, es)};
  const Span sk = {dk, strided_bytes(tokens, dk_stride, H_kv, d, es)};
  const Span wq = {dq_weight, d * ws}, wk = {dk_weight, d * ws};
  const Span a1[] = {sq, wq, wk}, a2[] = {sk, wq, wk};
  if (!disjoint(a1, 3, ins, 9) || !disjoint(a2, 3, ins, 9) ||
      !slices_disjoint(sq, dq_stride, nq * es, sk, dk_stride, nk * es, es))
    return LT_ERR_INVALID_ARG;
  const int dev = current_device();
  for (int i = 0; i < 8; ++i)
    if (ins[i].p && !on_device(dev, ins[i].p)) return LT_ERR_INVALID_ARG;
  if (!on_device(dev, dq) || !on_device(dev, dk) ||
      (dq_weight && !on_device(dev, dq_weight)) || (dk_weight && !on_device(dev, dk_weight)))
    return LT_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LT_ERR_CUDA;
  int* err = device_error_word_current();
  if (!err) return LT_ERR_CUDA;
  const int parts = token_parts(tokens, H_q, H_kv, d, dtype, sms);
  const int64_t blocks = block_count(tokens * parts, sms);
  Workspace w;
  if (gains) {
    const lt_status_t sw = w.take(dev, workspace, workspace_bytes,
                                  (size_t)kBlocks * sms * 2 * d * sizeof(float),
                                  (cudaStream_t)stream);
    if (sw != LT_OK) return sw;
  }
  NormArgs a = {};
  a.x[0] = q;
  a.x[1] = k;
  a.g[0] = dq_out;
  a.g[1] = dk_out;
  a.out[0] = dq;
  a.out[1] = dk;
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.stride[0] = q_stride;
  a.stride[1] = k_stride;
  a.ostride[0] = dq_stride;
  a.ostride[1] = dk_stride;
  a.H[0] = H_q;
  a.H[1] = H_kv;
  a.positions = positions;
  a.n_pos = n_pos;
  a.inv_freq = inv_freq;
  a.rot = rot;
  a.tokens = tokens;
  a.eps = eps;
  a.w_f32 = w_dtype == LT_F32;
  a.parts = parts;
  a.err = err;
  a.partial = static_cast<float*>(w.p);
  cudaError_t e = launch<true>(a, (int)blocks, d, interleaved, dtype, (cudaStream_t)stream);
  if (e == cudaSuccess && gains) {
    GainArgs ga = {};
    ga.partial = a.partial;
    ga.out[0] = dq_weight;
    ga.out[1] = dk_weight;
    ga.blocks = (int)blocks;
    ga.d = d;
    ga.dtype = (int)w_dtype;
    e = launch_dependent(lt_norm_rope_gain_kernel, dim3(2 * d / 32), 1024, 0,
                         (cudaStream_t)stream, ga);
  }
  const cudaError_t f = w.release();
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}
