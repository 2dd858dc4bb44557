// qk_norm_rope.cu -- root-mean-square norm of every query and key head, gain
// and position rotation in one pass, and its backward pass.
//
// Per row x (one head of one token, d values), r = (mean(x^2) + eps)^(-1/2):
//     forward:  y = x r w,  out = R y
//     backward: g = R^T dout,  u = g w,  dx = r u - x r^3 mean(u x),
//               dw = sum over rows of g x r
// R turns each pair (a, b) by A = position * inv_freq.  A reaches millions of
// turns, so it is formed in turns and reduced in fp64; only the fraction of a
// turn, at most 1/2, goes to fp32 sine and cosine.  They depend on the token
// and the pair alone: a block computes them once for its tokens, in shared
// memory, and all heads of those tokens use them.
//
// Bound by memory (about 8 flops per 2-byte element).  A row is spread over
// d/8 lanes so that the norm is a 3- or 4-step shuffle, and each lane holds
// two quads of elements, 4j.. and rot/2 + 4j..: whichever way the pairs are
// laid out, both halves of a pair are in one lane, and no value crosses lanes
// for the rotation.  Every thread has kU rows in flight.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/lt_linear_attn.h"
#include "lt_check.h"
#include "lt_internal.h"
#include "lt_vec.cuh"

namespace lt {
namespace {

constexpr int kT = 256;   // threads
constexpr int kMaxTB = 8; // tokens per block (sets the table of angles)

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
  int rot, tb;
  int64_t tokens;
  float eps;
  int w_f32;      // gains are fp32
  float* partial;  // backward: [block][2][d] sums of the gains' gradients
};

struct GainArgs {
  const float* partial;  // [blocks][2][d]
  void* out[2];          // [d] each, or nullptr
  int blocks, d, dtype;  // dtype of out (lt_dtype_t)
};

// positions of the block's tokens x frequencies -> cosines and sines
// [tokens][rot/2]
__device__ __forceinline__ void fill_angles(const NormArgs& a, int64_t t0, int nt, float* cosv,
                                            float* sinv) {
  const int half = a.rot >> 1;
  constexpr double kInvTwoPi = 0.15915494309189533577;
  for (int i = threadIdx.x; i < nt * half; i += kT) {
    const int tt = i / half, p = i - tt * half;
    const int64_t t = t0 + tt;
    const int pos = a.positions[a.n_pos == a.tokens ? t : t % a.n_pos];
    double turns = (double)pos * (double)a.inv_freq[p] * kInvTwoPi;
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * (float)turns, &s, &c);
    cosv[i] = c;
    sinv[i] = s;
  }
}

// the lane's two quads: the rotated lanes hold both halves of their pairs
struct Lane {
  int qa, qb;  // element offsets of the quads
  bool rotated;
};
__device__ __forceinline__ Lane lane_of(int j, int rot) {
  Lane l;
  l.rotated = j < (rot >> 3);
  l.qa = l.rotated ? 4 * j : 8 * j;
  l.qb = l.rotated ? (rot >> 1) + 4 * j : 8 * j + 4;
  return l;
}

// turn the lane's pairs in y[0..7] by the token's angles (sign -1: back);
// j is the lane's index in its row
template <bool IL>
__device__ __forceinline__ void turn(float* y, const float* c, const float* s, int j, int rot,
                                     float sign) {
  if (IL) {
    const float2 c0 = *reinterpret_cast<const float2*>(c + 2 * j);
    const float2 s0 = *reinterpret_cast<const float2*>(s + 2 * j);
    const float2 c1 = *reinterpret_cast<const float2*>(c + (rot >> 2) + 2 * j);
    const float2 s1 = *reinterpret_cast<const float2*>(s + (rot >> 2) + 2 * j);
    const float cc[4] = {c0.x, c0.y, c1.x, c1.y}, ss[4] = {s0.x, s0.y, s1.x, s1.y};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float A = y[2 * p], B = y[2 * p + 1], sn = sign * ss[p];
      y[2 * p] = A * cc[p] - B * sn;
      y[2 * p + 1] = B * cc[p] + A * sn;
    }
  } else {
    const float4 c4 = *reinterpret_cast<const float4*>(c + 4 * j);
    const float4 s4 = *reinterpret_cast<const float4*>(s + 4 * j);
    const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float A = y[p], B = y[p + 4], sn = sign * ss[p];
      y[p] = A * cc[p] - B * sn;
      y[p + 4] = B * cc[p] + A * sn;
    }
  }
}

template <typename T>
__device__ __forceinline__ void load_gain(const void* w, int w_f32, const Lane& l, float* f) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 1.0f;
  } else if (w_f32) {
    widen(load_quad(static_cast<const float*>(w) + l.qa), f);
    widen(load_quad(static_cast<const float*>(w) + l.qb), f + 4);
  } else {
    widen(load_quad(static_cast<const T*>(w) + l.qa), f);
    widen(load_quad(static_cast<const T*>(w) + l.qb), f + 4);
  }
}

template <int L>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// row index of a block's (token, head) list, advanced by a fixed step
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

template <typename T, int D, bool IL>
__global__ void __launch_bounds__(kT) lt_norm_rope_kernel(const NormArgs a) {
  constexpr int L = D / 8, RG = kT / L, kU = 4;
  extern __shared__ float4 smem4[];
  float* cosv = reinterpret_cast<float*>(smem4);
  const int half = a.rot >> 1;
  float* sinv = cosv + a.tb * half;
  const int64_t t0 = (int64_t)blockIdx.x * a.tb;
  const int nt = (int)min((int64_t)a.tb, a.tokens - t0);
  const int grp = threadIdx.x / L, j = threadIdx.x % L;
  const Lane ln = lane_of(j, a.rot);
  if (half) {
    fill_angles(a, t0, nt, cosv, sinv);
    __syncthreads();
  }
#pragma unroll 1
  for (int ph = 0; ph < 2; ++ph) {
    const int H = a.H[ph], rows = nt * H;
    const T* x = static_cast<const T*>(a.x[ph]) + t0 * a.stride[ph];
    T* out = static_cast<T*>(a.out[ph]) + t0 * (int64_t)(H * D);
    float w[8];
    load_gain<T>(a.w[ph], a.w_f32, ln, w);
    RowAt at(grp, RG, H);
    // a warp's groups take as many turns as its first one, so that its
    // shuffles stay converged; a group past the last row works on zeros
    const int first = (threadIdx.x & ~31) / L;
#pragma unroll 1
    for (int r = grp, rw = first; rw < rows; r += RG * kU, rw += RG * kU) {
      Quad<T> qa[kU], qb[kU];
      int tt[kU], hh[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        tt[u] = at.tt;
        hh[u] = at.h;
        qa[u] = Quad<T>{};
        qb[u] = Quad<T>{};
        if (r + u * RG < rows) {
          const T* p = x + (int64_t)at.tt * a.stride[ph] + at.h * D;
          qa[u] = load_quad(p + ln.qa);
          qb[u] = load_quad(p + ln.qb);
        }
        at.next();
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float y[8];
        widen(qa[u], y);
        widen(qb[u], y + 4);
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
        const float rr = 1.0f / sqrtf(row_sum<L>(ss) * (1.0f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * rr * w[e];
        if (r + u * RG < rows) {
          if (ln.rotated) turn<IL>(y, cosv + tt[u] * half, sinv + tt[u] * half, j, a.rot, 1.0f);
          T* p = out + (int64_t)tt[u] * (H * D) + hh[u] * D;
          store_quad(p + ln.qa, y);
          store_quad(p + ln.qb, y + 4);
        }
      }
    }
  }
}

// One block walks token blocks blockIdx.x, + gridDim.x, ...; each thread sums
// its eight columns' gain gradients over its rows, the block's row groups are
// added in order at the end, and the launch below adds the blocks in order.
template <typename T, int D, bool IL>
__global__ void __launch_bounds__(kT) lt_norm_rope_bwd_kernel(const NormArgs a) {
  constexpr int L = D / 8, RG = kT / L, kU = 2;
  extern __shared__ float4 smem4[];
  __shared__ float red[RG][D];
  float* cosv = reinterpret_cast<float*>(smem4);
  const int half = a.rot >> 1;
  float* sinv = cosv + a.tb * half;
  const int grp = threadIdx.x / L, j = threadIdx.x % L;
  const Lane ln = lane_of(j, a.rot);
  const int first = (threadIdx.x & ~31) / L;
  float dw[2][8] = {};
  for (int64_t t0 = (int64_t)blockIdx.x * a.tb; t0 < a.tokens;
       t0 += (int64_t)gridDim.x * a.tb) {
    const int nt = (int)min((int64_t)a.tb, a.tokens - t0);
    if (half) {
      __syncthreads();  // the last token block's angles are no longer read
      fill_angles(a, t0, nt, cosv, sinv);
      __syncthreads();
    }
#pragma unroll
    for (int ph = 0; ph < 2; ++ph) {
      const int H = a.H[ph], rows = nt * H;
      const T* x = static_cast<const T*>(a.x[ph]) + t0 * a.stride[ph];
      const T* g = static_cast<const T*>(a.g[ph]) + t0 * (int64_t)(H * D);
      T* out = static_cast<T*>(a.out[ph]) + t0 * a.ostride[ph];
      float w[8];
      load_gain<T>(a.w[ph], a.w_f32, ln, w);
      RowAt at(grp, RG, H);
#pragma unroll 1
      for (int r = grp, rw = first; rw < rows; r += RG * kU, rw += RG * kU) {
        Quad<T> xa[kU], xb[kU], ga[kU], gb[kU];
        int tt[kU], hh[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          tt[u] = at.tt;
          hh[u] = at.h;
          xa[u] = xb[u] = ga[u] = gb[u] = Quad<T>{};
          if (r + u * RG < rows) {
            const T* p = x + (int64_t)at.tt * a.stride[ph] + at.h * D;
            const T* q = g + (int64_t)at.tt * (H * D) + at.h * D;
            xa[u] = load_quad(p + ln.qa);
            xb[u] = load_quad(p + ln.qb);
            ga[u] = load_quad(q + ln.qa);
            gb[u] = load_quad(q + ln.qb);
          }
          at.next();
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const bool live = r + u * RG < rows;
          float xv[8], gv[8];
          widen(xa[u], xv);
          widen(xb[u], xv + 4);
          widen(ga[u], gv);
          widen(gb[u], gv + 4);
          if (live && ln.rotated)
            turn<IL>(gv, cosv + tt[u] * half, sinv + tt[u] * half, j, a.rot, -1.0f);
          float ss = 0.0f, ux = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss = fmaf(xv[e], xv[e], ss);
            ux = fmaf(gv[e] * w[e], xv[e], ux);
          }
          const float rr = 1.0f / sqrtf(row_sum<L>(ss) * (1.0f / D) + a.eps);
          // n = x r: dx = r (u - n mean(u n)), dw += g n
          const float m = row_sum<L>(ux) * rr * (1.0f / D);
          float dx[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float n = xv[e] * rr;
            dx[e] = rr * (gv[e] * w[e] - n * m);
            dw[ph][e] = fmaf(gv[e], n, dw[ph][e]);  // zeros past the last row
          }
          if (live) {
            T* p = out + (int64_t)tt[u] * a.ostride[ph] + hh[u] * D;
            store_quad(p + ln.qa, dx);
            store_quad(p + ln.qb, dx + 4);
          }
        }
      }
    }
  }
  dependency_release();
  if (!a.partial) return;
#pragma unroll
  for (int ph = 0; ph < 2; ++ph) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      red[grp][ln.qa + e] = dw[ph][e];
      red[grp][ln.qb + e] = dw[ph][4 + e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kT) {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < RG; ++q) s += red[q][c];
      a.partial[((size_t)blockIdx.x * 2 + ph) * D + c] = s;
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

template <typename T, int D, bool IL>
cudaError_t launch_t(const NormArgs& a, int blocks, bool bwd, cudaStream_t stream) {
  const size_t smem = (size_t)a.tb * a.rot * sizeof(float);
  if (bwd)
    lt_norm_rope_bwd_kernel<T, D, IL><<<blocks, kT, smem, stream>>>(a);
  else
    lt_norm_rope_kernel<T, D, IL><<<blocks, kT, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_d(const NormArgs& a, int blocks, int d, int il, bool bwd, cudaStream_t s) {
  if (d == 64)
    return il ? launch_t<T, 64, true>(a, blocks, bwd, s) : launch_t<T, 64, false>(a, blocks, bwd, s);
  return il ? launch_t<T, 128, true>(a, blocks, bwd, s) : launch_t<T, 128, false>(a, blocks, bwd, s);
}

cudaError_t launch(const NormArgs& a, int blocks, int d, int il, bool bwd, lt_dtype_t dtype,
                   cudaStream_t s) {
  return dtype == LT_BF16  ? launch_d<__nv_bfloat16>(a, blocks, d, il, bwd, s)
         : dtype == LT_F16 ? launch_d<__half>(a, blocks, d, il, bwd, s)
                           : launch_d<float>(a, blocks, d, il, bwd, s);
}

// tokens per block
int token_block(int64_t tokens, int sms) {
  int tb = kMaxTB;
  while (tb > 1 && (tokens + tb - 1) / tb < sms) tb >>= 1;
  return tb;
}

// blocks of the backward launch: two per SM, at most one per token block
int64_t bwd_blocks(int64_t tokens, int sms) {
  const int tb = token_block(tokens, sms);
  const int64_t n = (tokens + tb - 1) / tb;
  return n < 2 * sms ? n : 2 * sms;
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
  // a block index is 32 bits
  if (tokens > (int64_t)kMaxTB * 0x7fffffff || !stride_ok(tokens, q_stride, H_q, d, es) ||
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
  const Span outs[] = {{q_out, (size_t)tokens * H_q * d * es}, {k_out, (size_t)tokens * H_kv * d * es}};
  if (!disjoint(outs, 2, ins, 6)) return LT_ERR_INVALID_ARG;
  for (const Span& s : ins)
    if (s.p && !on_current_device(s.p)) return LT_ERR_INVALID_ARG;
  for (const Span& s : outs)
    if (!on_current_device(s.p)) return LT_ERR_INVALID_ARG;
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
  a.tb = token_block(tokens, sms);
  const int64_t blocks = (tokens + a.tb - 1) / a.tb;
  return launch(a, (int)blocks, d, interleaved, false, dtype, (cudaStream_t)stream) == cudaSuccess
             ? LT_OK
             : LT_ERR_CUDA;
}

extern "C" lt_status_t lt_qk_norm_rope_bwd_plan(int64_t tokens, int d, int num_sms,
                                                size_t* workspace_bytes) {
  if (!workspace_bytes || tokens < 1) return LT_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return LT_ERR_UNSUPPORTED;
  if (num_sms <= 0) num_sms = lt::device_sm_count();
  if (num_sms <= 0) return LT_ERR_CUDA;
  *workspace_bytes = (size_t)lt::bwd_blocks(tokens, num_sms) * 2 * d * sizeof(float);
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
                      {gains ? workspace : nullptr, workspace_bytes}};
  const Span sq = {dq, strided_bytes(tokens, dq_stride, H_q, d, es)};
  const Span sk = {dk, strided_bytes(tokens, dk_stride, H_kv, d, es)};
  const Span wq = {dq_weight, d * ws}, wk = {dk_weight, d * ws};
  const Span a1[] = {sq, wq, wk}, a2[] = {sk, wq, wk};
  if (!disjoint(a1, 3, ins, 9) || !disjoint(a2, 3, ins, 9) ||
      !slices_disjoint(sq, dq_stride, nq * es, sk, dk_stride, nk * es, es))
    return LT_ERR_INVALID_ARG;
  for (const Span& s : ins)
    if (s.p && s.p != workspace && !on_current_device(s.p)) return LT_ERR_INVALID_ARG;
  if (!on_current_device(dq) || !on_current_device(dk) ||
      (dq_weight && !on_current_device(dq_weight)) || (dk_weight && !on_current_device(dk_weight)))
    return LT_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LT_ERR_CUDA;
  const int64_t blocks = bwd_blocks(tokens, sms);
  Workspace w;
  if (gains) {
    const lt_status_t sw = w.take(workspace, workspace_bytes,
                                  (size_t)blocks * 2 * d * sizeof(float), (cudaStream_t)stream);
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
  a.tb = token_block(tokens, sms);
  a.partial = static_cast<float*>(w.p);
  cudaError_t e = launch(a, (int)blocks, d, interleaved, true, dtype, (cudaStream_t)stream);
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
