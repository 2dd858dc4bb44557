// paged_attn.cu -- attention of one new token per sequence over the paged
// cache: the second launch, which joins the pieces that the first one leaves
// (paged_attn.cuh), and the entry points.
#include "paged_attn.cuh"

namespace lt {
namespace paged {
namespace {

// Block (x, y): entry x of shared[], query heads y per .. y per + per - 1, with
// an equal share of the threads each.  A head's pieces are joined in an order
// that their number alone sets: four columns per lane, groups of lanes taking
// the pieces in turn, then the groups by halves.  As many loads as possible at
// once: a head's 148 pieces take five dependent steps of 32 groups (16 groups
// that first look for the maximum: 4 us more).  One head per block of 1024
// where the entries are few (one long sequence has a piece in every block of
// the first launch), eight per block of 256 where they are many (and mostly of
// two or three pieces).
constexpr int kJoin = 1024;  // threads, at most

struct JoinArgs {
  DecodeArgs a;
  int per;  // query heads per block
};

template <typename T>
__device__ __forceinline__ void store4(void* out, size_t at, const float* f) {
  store_quad(static_cast<T*>(out) + at, f);
}

__global__ void __launch_bounds__(kJoin) lt_paged_join_kernel(const JoinArgs j) {
  __shared__ float4 acc_s[kJoin];
  __shared__ float l_s[kJoin], m_s[kJoin];
  const DecodeArgs& a = j.a;
  const int share = blockDim.x / j.per, tid = threadIdx.x % share;
  const int h = blockIdx.y * j.per + threadIdx.x / share;
  const int lanes = a.dv >> 2, groups = share / lanes, c4 = tid % lanes, grp = tid / lanes;
  // every block waits, so that this launch ends after the first one has
  dependency_wait();
  dependency_release();  // (all blocks of this launch are on the SMs or done by now)
  const Shared s = a.shared[blockIdx.x];
  const int n = s.blocks;
  if (n == 0) return;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l = 0.0f, mx = -INFINITY;
  if (h < a.Hq) {
    const int g = h / a.G, hh = h - g * a.G, blk = hh / a.hb;
    const int u = g * a.nhb + blk;
    // the first piece is the second of its block, the others the first of theirs
    auto row = [&](int i) {
      return (((size_t)(s.block + i) * 2 + (i == 0 ? 1 : 0)) * a.units + u) * a.hb + hh -
             blk * a.hb;
    };
#pragma unroll 4
    for (int i = grp; i < n; i += groups) {
      const size_t p = row(i);
      add_piece(o, l, mx, *reinterpret_cast<const float2*>(a.block.ml + p * 2),
                *reinterpret_cast<const float4*>(a.block.part + p * a.dv + c4 * 4));
    }
  }
  // the groups of a column, `lanes` threads apart, by halves
  const int at0 = threadIdx.x;
  for (int half = groups >> 1; half > 0; half >>= 1) {
    if (grp >= half && grp < 2 * half) {
      acc_s[at0] = o;
      l_s[at0] = l;
      m_s[at0] = mx;
    }
    __syncthreads();
    if (grp < half) {
      const int p = at0 + half * lanes;
      add_piece(o, l, mx, make_float2(m_s[p], l_s[p]), acc_s[p]);
    }
    __syncthreads();
  }
  if (grp != 0 || h >= a.Hq) return;
  const float f = inverse_sum(l);
  const float y[4] = {o.x * f, o.y * f, o.z * f, o.w * f};
  const size_t orow = (size_t)s.b * a.Hq + h;
  const size_t at = orow * a.dv + c4 * 4;
  if (a.dtype == LT_F32)
    store4<float>(a.out, at, y);
  else if (a.dtype == LT_BF16)
    store4<__nv_bfloat16>(a.out, at, y);
  else
    store4<__half>(a.out, at, y);
  if (a.lse && c4 == 0) a.lse[orow] = log_sum(mx, l);
}

bool pools_within(const lt_kv_cache_t* c, size_t bytes) {
  Span s[4];
  cache_spans(c, s);
  return s[0].n <= bytes && s[1].n <= bytes;
}

int unit_heads(lt_dtype_t t, int G) {
  const int most = heads_at_once(t == LT_F32, G);
  return G < most ? G : most;
}
int warps_of(lt_dtype_t t, lt_kv_dtype_t kv, int d, int dv, int G) {
  const bool f32 = t == LT_F32;
  return block_warps(f32, (int)kv_size(kv), d, dv, heads_at_once(f32, G));
}

// the workspace, one block of the first launch per SM: pieces of its warps
// (two each), of its units (two each), and an entry for the second launch
struct Sizes {
  size_t warp, block;  // pieces
  size_t floats;       // of a piece
  size_t bytes;
};
Sizes sizes_of(lt_dtype_t t, lt_kv_dtype_t kv, int H_q, int H_kv, int d, int dv, int sms) {
  const int G = H_q / H_kv, hb = unit_heads(t, G), nhb = (G + hb - 1) / hb;
  Sizes z;
  z.warp = (size_t)sms * warps_of(t, kv, d, dv, G) * 2;
  z.block = (size_t)sms * 2 * H_kv * nhb;
  z.floats = (size_t)hb * (dv + 2);
  z.bytes = (z.warp + z.block) * z.floats * sizeof(float) + (size_t)sms * sizeof(Shared);
  return z;
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
  *workspace_bytes = sizes_of(dtype, kv_dtype, H_q, H_kv, d, dv, num_sms).bytes;
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
  // pools are addressed in 32 bits of 16 bytes, columns and a block's tiles
  // counted in 31 bits
  const int64_t pages_hold = (int64_t)max_pages * cache->page_size;
  const int most = (int)(pages_hold < 0x7fffff00 ? pages_hold : 0x7fffff00);
  const int64_t columns = (int64_t)B * (most / 16 + 1);
  if (!pools_within(cache, (size_t)64 << 30) || columns > 0x7fff0000 ||
      columns > ((int64_t)1 << 36) / H_q)
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
  const int dev = current_device();
  if (check_cache_pointers(dev, cache) != LT_OK || !on_device(dev, q) ||
      !on_device(dev, block_table) || !on_device(dev, seq_lens) || !on_device(dev, out) ||
      (lse && !on_device(dev, lse)))
    return LT_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  int* err = device_error_word_current();
  if (sms <= 0 || !err) return LT_ERR_CUDA;
  DecodeArgs a = {};
  a.G = H_q / cache->H_kv;
  a.hb = unit_heads(dtype, a.G);
  a.nhb = (a.G + a.hb - 1) / a.hb;
  const Sizes z = sizes_of(dtype, cache->dtype, H_q, cache->H_kv, cache->d, cache->dv, sms);
  Workspace w;
  const lt_status_t sw = w.take(dev, workspace, workspace_bytes, z.bytes, (cudaStream_t)stream);
  if (sw != LT_OK) return sw;
  a.q = q;
  a.k = static_cast<const uint8_t*>(cache->k);
  a.v = static_cast<const uint8_t*>(cache->v);
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  const int64_t ks = (int64_t)kv_size(cache->dtype);
  a.kpg = (uint32_t)(cache->k_page_stride * ks / 16);
  a.ksl = (uint32_t)(cache->k_slot_stride * ks / 16);
  a.khd = (uint32_t)(cache->k_head_stride * ks / 16);
  a.vpg = (uint32_t)(cache->v_page_stride * ks / 16);
  a.vsl = (uint32_t)(cache->v_slot_stride * ks / 16);
  a.vhd = (uint32_t)(cache->v_head_stride * ks / 16);
  a.same = a.kpg == a.vpg && a.ksl == a.vsl && a.khd == a.vhd;
  a.table = block_table;
  a.table_stride = table_stride;
  a.lens = seq_lens;
  a.B = B;
  a.Hq = H_q;
  a.Hkv = cache->H_kv;
  a.num_pages = cache->num_pages;
  a.page_size = cache->page_size;
  a.max_len = most;
  a.units = a.Hkv * a.nhb;
  a.k_shift = -1;
  const int warps = warps_of(dtype, cache->dtype, cache->d, cache->dv, a.G);
  for (int s = 0; (1 << s) <= warps; ++s)
    if (a.units << s == warps) a.k_shift = s;
  while ((1 << a.page_shift) < a.page_size) ++a.page_shift;
  a.page_magic = (uint32_t)(((uint64_t)1 << (31 + a.page_shift)) / a.page_size + 1);
  a.window = window;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.dv = cache->dv;
  a.dtype = (int)dtype;
  float* p = static_cast<float*>(w.p);
  a.warp.part = p;
  a.warp.ml = p + z.warp * a.hb * a.dv;
  p += z.warp * z.floats;
  a.block.part = p;
  a.block.ml = p + z.block * a.hb * a.dv;
  a.shared = reinterpret_cast<Shared*>(p + z.block * z.floats);
  a.by_seq = B <= sms && B <= 128;  // (at most one sequence per thread of any engine)
  a.err = err;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = dtype == LT_BF16  ? launch_bf16(a, cache->dtype, cache->d, sms, s)
                  : dtype == LT_F16 ? launch_f16(a, cache->dtype, cache->d, sms, s)
                                    : launch_f32(a, cache->dtype, cache->d, sms, s);
  if (e == cudaSuccess) {
    const int entries = a.by_seq ? B : sms;
    const bool few = entries * H_q <= 2 * sms;
    const JoinArgs j = {a, few ? 1 : 8};
    e = launch_dependent(lt_paged_join_kernel, dim3(entries, (H_q + j.per - 1) / j.per),
                         few ? kJoin : 256, 0, s, j);
  }
  const cudaError_t f = w.release();
  if (e == cudaSuccess) e = f;
  return e == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}
