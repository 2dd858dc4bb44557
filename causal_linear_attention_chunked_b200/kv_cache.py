"""Queries and keys of an attention layer, and the paged key-value cache of its
softmax layers: norm and rotation, writing and reading the cache, attention of
one new token over it.  Argument marshalling over the C ABI of
include/lt_linear_attn.h, as in ``_binding``; every step of the computation
runs in the CUDA library.

One serving step of a softmax layer:

    q, k = qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq)
    kv_cache_write(cache, k, v, slots)
    out = paged_attn_decode(q, cache, block_table, seq_lens)

Calls run on the tensors' device and, unless ``stream`` is given, on its
current stream.  Tensors that a call allocates (outputs, workspace) belong to
the stream that it runs on.
"""
import contextlib
import ctypes
import math

import torch

from ._binding import KvCacheStruct, _check, _dtype_code, _ptr, lib

_KV_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.float8_e4m3fn: 3,
             torch.int8: 4}
_NO_CTX = contextlib.nullcontext()
_FLOATS = (torch.bfloat16, torch.float16, torch.float32)


class _On:
    """The device and stream of a call: entered around its allocations and
    launch where they are not the current ones already."""

    def __init__(self, device, stream, *tensors):
        if device.type != "cuda":
            raise ValueError("the tensors must be CUDA tensors")
        for t in tensors:
            if t is not None and t.device != device:
                raise ValueError("all tensors must be on one device")
        if stream is None:
            self.handle = ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
            self.ctx = _NO_CTX if torch.cuda.current_device() == device.index \
                else torch.cuda.device(device)
        else:
            if stream.device != device:
                raise ValueError("stream belongs to another device than the tensors")
            self.handle = ctypes.c_void_p(stream.cuda_stream)
            self.ctx = torch.cuda.stream(stream)


def _int32(t, name, dim):
    if t.dtype != torch.int32 or t.dim() != dim or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise TypeError("%s must be an int32 tensor of %d dimension(s), contiguous in its last"
                        % (name, dim))


def _tokens(t, name):
    """(tokens, heads, width, token stride) of [.., heads, width]: heads and
    width contiguous, tokens evenly spaced."""
    if t.dim() not in (3, 4):
        raise ValueError("%s must be [tokens, heads, width] or [B, N, heads, width]" % name)
    H, w = t.shape[-2:]
    if (w > 1 and t.stride(-1) != 1) or (H > 1 and t.stride(-2) != w):
        raise ValueError("%s must be contiguous in its heads and width" % name)
    if t.dim() == 3:
        n, step = t.shape[0], t.stride(0)
    else:
        B, N = t.shape[:2]
        n = B * N
        step = t.stride(1) if N > 1 else t.stride(0)
        if B > 1 and N > 1 and t.stride(0) != N * step:
            raise ValueError("%s must have evenly spaced tokens" % name)
    return n, H, w, step if n > 1 else H * w


def _out(t, shape, dtype, device, name):
    """A given output, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s"
                         % (name, dtype, tuple(shape)))
    return t


def _norm_args(q, k, q_weight, k_weight, positions, inv_freq):
    n, Hq, d, q_step = _tokens(q, "q")
    nk, Hkv, dk, k_step = _tokens(k, "k")
    if nk != n or dk != d or q.shape[:-2] != k.shape[:-2]:
        raise ValueError("q and k must have the same tokens and width")
    if k.dtype != q.dtype or q.dtype not in _FLOATS:
        raise TypeError("q and k must have one dtype (bfloat16, float16 or float32)")
    w_dtype = q.dtype
    given = [w for w in (q_weight, k_weight) if w is not None]
    for w in given:
        w_dtype = given[0].dtype
        if w.shape != (d,) or not w.is_contiguous() or w.dtype != w_dtype or \
                w_dtype not in (torch.float32, q.dtype):
            raise ValueError("weights must be contiguous [d] tensors, both float32 or both of "
                             "q's dtype")
    n_pos = rot = 0
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq are given together")
    if positions is not None:
        if positions.dtype != torch.int32 or not positions.is_contiguous():
            raise TypeError("positions must be a contiguous int32 tensor")
        if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise TypeError("inv_freq must be a contiguous float32 vector")
        n_pos, rot = positions.numel(), 2 * inv_freq.numel()
        if rot and (n_pos == 0 or n % n_pos):
            raise ValueError("the number of tokens must be a multiple of the positions'")
        if rot and q.dim() == 4 and n_pos not in (q.shape[1], n):
            raise ValueError("positions must be [N] or [B, N]")
    return n, Hq, Hkv, d, q_step, k_step, w_dtype, n_pos, rot


def qk_norm_rope(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, eps=1e-6,
                 interleaved=False, q_out=None, k_out=None, stream=None):
    """Root-mean-square norm of every head of q and k, gain, and the rotation by
    the token's position, in one pass: (q_out, k_out), dense, of q's dtype.

    q [.., H_q, d], k [.., H_kv, d] with leading [B, N] or [tokens]; slices of
    a fused projection are taken as they are (evenly spaced tokens).
    q_weight, k_weight: [d] gains (float32 or q's dtype) or None.  positions:
    int32, one per token, or [N] shared by a dense batch; inv_freq: float32
    [rot / 2] angles per position (rot values of each head are rotated, a
    multiple of 8); both None: the norm alone.  interleaved: pairs (2i, 2i + 1)
    instead of (i, i + rot / 2).  See lt_qk_norm_rope."""
    n, Hq, Hkv, d, q_step, k_step, w_dtype, n_pos, rot = _norm_args(q, k, q_weight, k_weight,
                                                                    positions, inv_freq)
    on = _On(q.device, stream, k, q_weight, k_weight, positions, inv_freq, q_out, k_out)
    with on.ctx:
        q_out = _out(q_out, q.shape, q.dtype, q.device, "q_out")
        k_out = _out(k_out, k.shape, q.dtype, q.device, "k_out")
        _check(lib.lt_qk_norm_rope(
            q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(positions), n_pos,
            _ptr(inv_freq), rot, int(bool(interleaved)), q_out.data_ptr(), k_out.data_ptr(), n, Hq,
            Hkv, d, q_step, k_step, float(eps), on.handle, _dtype_code(q.dtype),
            _dtype_code(w_dtype)))
    return q_out, k_out


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, positions=None,
                     inv_freq=None, eps=1e-6, interleaved=False, dq=None, dk=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of qk_norm_rope for upstream
    gradients dq_out, dk_out; the weights' are None where a weight is None.
    dq and dk may be given as slices of a fused gradient.  See
    lt_qk_norm_rope_bwd."""
    n, Hq, Hkv, d, q_step, k_step, w_dtype, n_pos, rot = _norm_args(q, k, q_weight, k_weight,
                                                                    positions, inv_freq)
    for g, x, name in ((dq_out, q, "dq_out"), (dk_out, k, "dk_out")):
        if g.shape != x.shape or g.dtype != q.dtype or not g.is_contiguous():
            raise ValueError("%s must be contiguous, of its input's shape and dtype" % name)
    on = _On(q.device, stream, k, q_weight, k_weight, positions, inv_freq, dq_out, dk_out, dq, dk)
    with on.ctx:
        steps = []
        grads = []
        for t, x, H, name in ((dq, q, Hq, "dq"), (dk, k, Hkv, "dk")):
            if t is None:
                t = torch.empty(x.shape, dtype=q.dtype, device=q.device)
                steps.append(H * d)
            else:
                if t.shape != x.shape or t.dtype != q.dtype:
                    raise ValueError("%s must have its input's shape and dtype" % name)
                steps.append(_tokens(t, name)[3])
            grads.append(t)
        dqw = torch.empty_like(q_weight) if q_weight is not None else None
        dkw = torch.empty_like(k_weight) if k_weight is not None else None
        ws, ws_bytes = None, 0
        if dqw is not None or dkw is not None:
            need = ctypes.c_size_t()
            _check(lib.lt_qk_norm_rope_bwd_plan(n, d, 0, ctypes.byref(need)))
            ws_bytes = need.value
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
        _check(lib.lt_qk_norm_rope_bwd(
            dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), _ptr(q_weight),
            _ptr(k_weight), _ptr(positions), n_pos, _ptr(inv_freq), rot, int(bool(interleaved)),
            grads[0].data_ptr(), grads[1].data_ptr(), _ptr(dqw), _ptr(dkw), n, Hq, Hkv, d, q_step,
            k_step, steps[0], steps[1], float(eps), _ptr(ws), ws_bytes, on.handle,
            _dtype_code(q.dtype), _dtype_code(w_dtype)))
    return grads[0], grads[1], dqw, dkw


class PagedKVCache:
    """A paged key-value cache over the caller's pools.

    k [pages, page_size, H_kv, d], v [pages, page_size, H_kv, dv]: bfloat16,
    float16, float32, float8_e4m3fn or int8; any strides that keep rows
    contiguous and 16-byte aligned.  8-bit caches have k_scale, v_scale
    [pages, H_kv, page_size] float32 (contiguous), one scale per row.  The
    pools are not copied, and stay alive with this object.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or v.dim() != 4 or k.shape[:3] != v.shape[:3]:
            raise ValueError("k and v must be [pages, page_size, H_kv, width] pools of one shape "
                             "but for the width")
        if k.dtype != v.dtype or k.dtype not in _KV_CODES:
            raise TypeError("k and v must have one dtype of bfloat16, float16, float32, "
                            "float8_e4m3fn, int8")
        if k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("the rows of k and v must be contiguous")
        if not k.is_cuda:
            raise ValueError("the pools must be CUDA tensors")
        pages, page_size, H, d = k.shape
        quant = k.dtype in (torch.float8_e4m3fn, torch.int8)
        if quant != (k_scale is not None) or quant != (v_scale is not None):
            raise ValueError("8-bit caches have k_scale and v_scale, others have none")
        for s in (k_scale, v_scale):
            if s is not None and (s.shape != (pages, H, page_size) or s.dtype != torch.float32 or
                                  not s.is_contiguous()):
                raise ValueError("scales must be contiguous float32 [pages, H_kv, page_size]")
        for t in (v, k_scale, v_scale):
            if t is not None and t.device != k.device:
                raise ValueError("all tensors must be on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.dtype, self.device = k.dtype, k.device
        self.num_pages, self.page_size, self.H_kv, self.d, self.dv = pages, page_size, H, d, \
            v.shape[3]
        self._c = KvCacheStruct(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if quant else None,
            v_scale.data_ptr() if quant else None, k.stride(0), k.stride(1), k.stride(2),
            v.stride(0), v.stride(1), v.stride(2), pages, page_size, H, d, v.shape[3],
            _KV_CODES[k.dtype])
        self._ref = ctypes.byref(self._c)
        self._workspace_bytes = {}

    @classmethod
    def empty(cls, num_pages, page_size, H_kv, d, dv=None, dtype=torch.bfloat16, device="cuda"):
        """A cache over new pools, their content unspecified."""
        dv = d if dv is None else dv
        k = torch.empty(num_pages, page_size, H_kv, d, dtype=dtype, device=device)
        v = torch.empty(num_pages, page_size, H_kv, dv, dtype=dtype, device=device)
        ks = vs = None
        if dtype in (torch.float8_e4m3fn, torch.int8):
            ks = torch.empty(num_pages, H_kv, page_size, dtype=torch.float32, device=device)
            vs = torch.empty_like(ks)
        return cls(k, v, ks, vs)


def kv_cache_write(cache, k, v, slots, stream=None):
    """New keys and values into the cache, quantised to 8 bits where it holds 8
    bits.  k [.., H_kv, d], v [.., H_kv, dv] (slices of a fused projection are
    taken as they are); slots: int32, one per token, page * page_size + offset,
    or -1 to skip the token; they must differ.  See lt_kv_cache_write."""
    n, H, d, k_step = _tokens(k, "k")
    nv, Hv, dv, v_step = _tokens(v, "v")
    if nv != n or H != cache.H_kv or Hv != H or d != cache.d or dv != cache.dv:
        raise ValueError("k and v must be [tokens, H_kv, d] and [tokens, H_kv, dv] of the cache")
    if k.dtype != v.dtype:
        raise TypeError("k and v must have one dtype")
    if slots.dtype != torch.int32 or not slots.is_contiguous() or slots.numel() != n:
        raise TypeError("slots must be a contiguous int32 tensor, one per token")
    on = _On(cache.device, stream, k, v, slots)
    with on.ctx:
        _check(lib.lt_kv_cache_write(cache._ref, k.data_ptr(), v.data_ptr(), slots.data_ptr(), n,
                                     k_step, v_step, on.handle, _dtype_code(k.dtype)))


def kv_cache_read(cache, block_table, cu_seqlens, N, dtype=None, k_out=None, v_out=None,
                  stream=None):
    """The sequences of a batch read back from the cache, packed: (k [N, H_kv,
    d], v [N, H_kv, dv]) as linear_attn_fwd and linear_attn_state take packed
    inputs.  block_table: int32 [B, max_pages]; cu_seqlens: int32 [B + 1]
    offsets (on the device), its last entry at most N; rows from it on are left
    as they were.  dtype: of the outputs (default: the cache's own, bfloat16
    for an 8-bit cache).  See lt_kv_cache_read."""
    _int32(block_table, "block_table", 2)
    _int32(cu_seqlens, "cu_seqlens", 1)
    B = cu_seqlens.numel() - 1
    if block_table.shape[0] != B:
        raise ValueError("block_table must have a row per sequence")
    if dtype is None:
        dtype = cache.dtype if cache.dtype in _FLOATS else torch.bfloat16
    on = _On(cache.device, stream, block_table, cu_seqlens, k_out, v_out)
    with on.ctx:
        k_out = _out(k_out, (N, cache.H_kv, cache.d), dtype, cache.device, "k_out")
        v_out = _out(v_out, (N, cache.H_kv, cache.dv), dtype, cache.device, "v_out")
        pages = block_table.shape[1]
        _check(lib.lt_kv_cache_read(cache._ref, block_table.data_ptr(),
                                    block_table.stride(0) if B > 1 else pages, pages,
                                    cu_seqlens.data_ptr(), B, N, k_out.data_ptr(),
                                    v_out.data_ptr(), on.handle, _dtype_code(dtype)))
    return k_out, v_out


def paged_attn_decode(q, cache, block_table, seq_lens, scale=None, window=0, out=None,
                      return_lse=False, stream=None):
    """Softmax attention of one new token per sequence over the cache: out
    [B, H_q, dv] of q's dtype, or (out, lse) with lse [B, H_q] float32.

    q [B, H_q, d]; block_table int32 [B, max_pages]; seq_lens int32 [B], the
    tokens of each sequence in the cache (0 gives zeros, and lse -inf); scale:
    of the scores (default 1 / sqrt(d)); window: the last `window` tokens only
    (0: all).  See lt_paged_attn_decode."""
    if q.dim() != 3 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [B, H_q, d] tensor")
    B, Hq, d = q.shape
    if d != cache.d:
        raise ValueError("q and the cache must have the same width")
    _int32(block_table, "block_table", 2)
    _int32(seq_lens, "seq_lens", 1)
    if block_table.shape[0] != B or seq_lens.numel() != B:
        raise ValueError("block_table and seq_lens must have a row per sequence")
    code = _dtype_code(q.dtype)
    on = _On(cache.device, stream, q, block_table, seq_lens, out)
    with on.ctx:
        out = _out(out, (B, Hq, cache.dv), q.dtype, q.device, "out")
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if return_lse else None
        ws_bytes = cache._workspace_bytes.get((Hq, code))
        if ws_bytes is None:
            need = ctypes.c_size_t()
            _check(lib.lt_paged_attn_decode_plan(Hq, cache.H_kv, d, cache.dv, code,
                                                 _KV_CODES[cache.dtype], 0, ctypes.byref(need)))
            ws_bytes = cache._workspace_bytes[(Hq, code)] = need.value
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
        pages = block_table.shape[1]
        _check(lib.lt_paged_attn_decode(
            q.data_ptr(), cache._ref, block_table.data_ptr(),
            block_table.stride(0) if B > 1 else pages, pages, seq_lens.data_ptr(), B, Hq,
            1.0 / math.sqrt(d) if scale is None else float(scale), int(window), out.data_ptr(),
            _ptr(lse), ws.data_ptr(), ws_bytes, on.handle, code))
    return (out, lse) if return_lse else out
