// paged_attn.cu -- attention of one new token per sequence over the paged
// cache: the second launch, which joins the pieces that the first one leaves
// (paged_attn.cuh), and the entry points.
#include "paged_attn.cuh"

namespace lt {
namespace paged {
namespace {

// One block per (query head, sequence): nothing to do where one warp had the
// whole pair; else its pieces, weighted by exp2(their maximum - the largest)
// and added in run order.  A piece is read four columns per lane, and the
// block's groups of lanes take the pieces in turn.
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

template <typename T>
__device__ __forceinline__ void store4(void* out, size_t at, const float* f) {
  store_quad(static_cast<T*>(out) + at, f);
}

__global__ void __launch_bounds__(kJoin) lt_paged_join_kernel(const DecodeArgs a) {
  __shared__ int64_t red[kJoin / 32];
  __shared__ float fred[kJoin / 32];
  __shared__ float4 acc_s[kJoin];
  __shared__ float l_s[kJoin];
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
  if (s.bad || (s.tiles && w0 == w1)) return;
  const size_t orow = (size_t)b * a.Hq + h;
  const int lanes = a.dv >> 2, groups = kJoin / lanes, c4 = tid % lanes, grp = tid / lanes;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l = 0.0f, mx = -INFINITY;
  const int n = s.tiles ? (int)(w1 - w0 + 1) : 0;
  // piece i of the pair: slot 1 only of a warp that began with another pair
  const size_t row0 = (size_t)(w0 * 2 + (from > w0 * run ? 1 : 0)) * a.hb + r;
  auto row = [&](int i) { return i == 0 ? row0 : (size_t)(w0 + i) * 2 * a.hb + r; };
  for (int i = tid; i < n; i += kJoin) mx = fmaxf(mx, a.ml[row(i) * 2]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  if ((tid & 31) == 0) fred[tid >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoin / 32; ++w) mx = fmaxf(mx, fred[w]);
  const float base = mx == -INFINITY ? 0.0f : mx;
#pragma unroll 4
  for (int i = grp; i < n; i += groups) {
    const size_t p = row(i);
    const float2 ml = *reinterpret_cast<const float2*>(a.ml + p * 2);
    const float4 x = *reinterpret_cast<const float4*>(a.part + p * a.dv + c4 * 4);
    const float f = exp2f(ml.x - base);
    l = fmaf(f, ml.y, l);
    o.x = fmaf(f, x.x, o.x);
    o.y = fmaf(f, x.y, o.y);
    o.z = fmaf(f, x.z, o.z);
    o.w = fmaf(f, x.w, o.w);
  }
  acc_s[tid] = o;
  l_s[tid] = l;
  __syncthreads();
  if (grp != 0) return;
  for (int q = 1; q < groups; ++q) {
    const float4 x = acc_s[q * lanes + c4];
    o.x += x.x;
    o.y += x.y;
    o.z += x.z;
    o.w += x.w;
    l += l_s[q * lanes + c4];
  }
  const float f = inverse_sum(l);
  const float y[4] = {o.x * f, o.y * f, o.z * f, o.w * f};
  const size_t at = orow * a.dv + c4 * 4;
  if (a.dtype == LT_F32)
    store4<float>(a.out, at, y);
  else if (a.dtype == LT_BF16)
    store4<__nv_bfloat16>(a.out, at, y);
  else
    store4<__half>(a.out, at, y);
  if (a.lse && c4 == 0) a.lse[orow] = log_sum(mx, l);
}

// query heads per unit, and warps (runs) on a device: the engines' kHeads and
// kWarps
int heads_per_unit(lt_dtype_t t, int G) {
  const int most = t == LT_F32 ? 8 : 16;
  return G < most ? G : most;
}
int run_count(lt_dtype_t t, lt_kv_dtype_t kv, int G, int sms) {
  return sms * (t == LT_F32 ? 4 : eight_bit(kv) && G <= 8 ? 16 : 8);
}

size_t workspace_floats(lt_dtype_t t, lt_kv_dtype_t kv, int G, int dv, int sms) {
  return (size_t)run_count(t, kv, G, sms) * 2 * heads_per_unit(t, G) * (dv + 2);
}

}  // namespace
}  // namespace paged
}  // namespace lt

extern "C" lt_status_t lt_paged_attn_decode_plan(int H_q, int H_kv, int d, int dv,
                                                 lt_dtype_t dtype, lt_kv_dtype_t kv_dtype,
                                                 int num_sms, size_t* workspace_bytes) {
  using namespace lt;
  using namespace lt::paged;
  if (!dtype_ok(dtype) || kv_dtype < LT_KV_F32 || kv_dtype > LT_KV_INT8 ||
      (!eight_bit(kv_dtype) && kv_dtype != kv_of(dtype)))
    return LT_ERR_UNSUPPORTED;
  if ((d != 64 && d != 128) || (dv != 64 && dv != 128)) return LT_ERR_UNSUPPORTED;
  if (!workspace_bytes || H_q < 1 || H_kv < 1 || H_q > 65535 || H_q % H_kv != 0)
    return LT_ERR_INVALID_ARG;
  if (num_sms <= 0) num_sms = device_sm_count();
  if (num_sms <= 0) return LT_ERR_CUDA;
  *workspace_bytes = workspace_floats(dtype, kv_dtype, H_q / H_kv, dv, num_sms) * sizeof(float);
  return LT_OK;
}

extern "C" lt_status_t lt_paged_attn_decode(const void* q, const lt_kv_cache_t* cache,
                                            const int32_t* block_table, int64_t table_stride,
                                            int max_pages, const int32_t* seq_lens, int B, int H_q,
                                            float scale, int window, void* out, float* lse,
                                            void* workspace, size_t workspace_bytes,
                                            lt_stream_t stream, lt_dtype_t dtype) {
  using namespace lt;
  using namespace lt::paged;
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
  a.warps = run_count(dtype, cache->dtype, a.G, sms);
  Workspace w;
  const lt_status_t sw =
      w.take(workspace, workspace_bytes,
             workspace_floats(dtype, cache->dtype, a.G, cache->dv, sms) * sizeof(float), (cudaStream_t)stream);
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
  cudaError_t e = dtype == LT_BF16  ? launch_bf16(a, cache->dtype, cache->d, sms, s)
                  : dtype == LT_F16 ? launch_f16(a, cache->dtype, cache->d, sms, s)
                                    : launch_f32(a, cache->dtype, cache->d, sms, s);
  if (e == cudaSuccess)
    e = launch_dependent(lt_paged_join_kernel, dim3(a.Hq, a.B), kJoin, 0, s, a);
  const cudaError_t f = w.release();
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}
