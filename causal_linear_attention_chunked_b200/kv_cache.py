"""Queries and keys of an attention layer, and the paged key-value cache of its
softmax layers: norm and rotation, writing and reading the cache, attention of
one new token over it.  Argument marshalling over the C ABI of
include/lt_linear_attn.h, as in ``_binding``; every step of the computation
runs in the CUDA library.

One serving step of a softmax layer:

    q, k = qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq)
    kv_cache_write(cache, k, v, slots)
    out = paged_attn_decode(q, cache, block_table, seq_lens)

Calls of no tokens or no sequences do nothing: their outputs are empty (the
gains' gradients zeros).  Calls run on the tensors' device and, unless
``stream`` is given, on its current stream.  Tensors that a call allocates
(outputs, workspace) belong to the stream that it runs on.
"""
import ctypes
import math

import torch

from ._binding import KvCacheStruct, _check, lib

_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}   # lt_dtype_t
_KV_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.float8_e4m3fn: 3,
             torch.int8: 4}
_raw_stream = torch._C._cuda_getCurrentRawStream   # a device's current stream, as a handle
_current_device = torch._C._cuda_getDevice


def _elsewhere(dev, stream, tensors):
    """None where the call can be made as it stands: every tensor on CUDA device
    `dev`, the current one, and no stream named.  Else the context to make it
    in, so that its allocations belong to the stream that it runs on."""
    if dev < 0:
        raise ValueError("the tensors must be CUDA tensors")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device")
    if stream is not None:
        if stream.device_index != dev:
            raise ValueError("stream belongs to another device than the tensors")
        return torch.cuda.stream(stream)
    return None if _current_device() == dev else torch.cuda.device(dev)


def _dtype_code(t):
    code = _CODES.get(t)
    if code is None:
        raise TypeError("unsupported dtype %s (bfloat16, float16 or float32)" % t)
    return code


def _ptr(t):
    return None if t is None else t.data_ptr()


def _int32(t, name, dim):
    if t.dtype != torch.int32 or t.dim() != dim or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise TypeError("%s must be an int32 tensor of %d dimension(s), contiguous in its last"
                        % (name, dim))


def _tokens(t, name):
    """(tokens, heads, width, token stride) of [.., heads, width]: heads and
    width contiguous, tokens evenly spaced."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        n, H, w = shape
        step = stride[0]
    elif len(shape) == 4:
        B, N, H, w = shape
        n = B * N
        step = stride[1] if N > 1 else stride[0]
        if B > 1 and N > 1 and stride[0] != N * step:
            raise ValueError("%s must have evenly spaced tokens" % name)
    else:
        raise ValueError("%s must be [tokens, heads, width] or [B, N, heads, width]" % name)
    if (w > 1 and stride[-1] != 1) or (H > 1 and stride[-2] != w):
        raise ValueError("%s must be contiguous in its heads and width" % name)
    return n, H, w, step if n > 1 else H * w


_grad_enabled = torch.is_grad_enabled


def _no_outputs(*outs):
    """Autograd takes no outputs of the caller's."""
    if any(t is not None for t in outs):
        raise ValueError("an output that the caller gives takes no gradient, and an input requires "
                         "one: leave it out, or call under torch.no_grad()")


def _dense_like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _given(t, shape, dtype, name):
    """Checks an output that the caller passed."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s"
                         % (name, dtype, tuple(shape)))
    return t


def _norm_args(q, k, q_weight, k_weight, positions, inv_freq):
    n, Hq, d, q_step = _tokens(q, "q")
    nk, Hkv, dk, k_step = _tokens(k, "k")
    dims = q.dim()
    if nk != n or dk != d or k.dim() != dims or (dims == 4 and q.shape[0] != k.shape[0]):
        raise ValueError("q and k must have the same tokens and width")
    dtype = q.dtype
    if k.dtype != dtype:
        raise TypeError("q and k must have one dtype")
    code = w_code = _dtype_code(dtype)
    w_dtype = None
    for w in (q_weight, k_weight):
        if w is not None:
            if w_dtype is None:
                w_dtype = w.dtype
            if w.dim() != 1 or w.numel() != d or not w.is_contiguous() or w.dtype != w_dtype or \
                    w_dtype not in (dtype, torch.float32):
                raise ValueError("weights must be contiguous [d] tensors, both float32 or both "
                                 "of q's dtype")
            w_code = _CODES[w_dtype]
    n_pos = rot = 0
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq are given together")
    if positions is not None:
        if positions.dtype != torch.int32 or not positions.is_contiguous():
            raise TypeError("positions must be a contiguous int32 tensor")
        if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise TypeError("inv_freq must be a contiguous float32 vector")
        n_pos, rot = positions.numel(), 2 * inv_freq.numel()
        if rot and n_pos != n and (dims != 4 or n_pos != q.shape[1]):
            raise ValueError("positions must be one per token, or [N] for a [B, N] batch")
    return n, Hq, Hkv, d, q_step, k_step, code, w_code, n_pos, rot


def qk_norm_rope(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, eps=1e-6,
                 interleaved=False, q_out=None, k_out=None, stream=None):
    """Root-mean-square norm of every head of q and k, gain, and the rotation by
    the token's position, in one pass: (q_out, k_out), dense, of q's dtype.

    q [.., H_q, d], k [.., H_kv, d] with leading [B, N] or [tokens]; slices of
    a fused projection are taken as they are (evenly spaced tokens).
    q_weight, k_weight: [d] gains (float32 or q's dtype) or None.  positions:
    int32, one per token, or [N] shared by a [B, N] batch; inv_freq: float32
    [rot / 2] angles per position (rot values of each head are rotated, a
    multiple of 8); both None: the norm alone.  interleaved: pairs (2i, 2i + 1)
    instead of (i, i + rot / 2).  Where q, k or a gain requires a gradient, the
    result has one (by qk_norm_rope_bwd; once).  See lt_qk_norm_rope."""
    n, Hq, Hkv, d, q_step, k_step, code, w_code, n_pos, rot = _norm_args(q, k, q_weight, k_weight,
                                                                         positions, inv_freq)
    dev = q.get_device()
    ctx = _elsewhere(dev, stream, (k, q_weight, k_weight, positions, inv_freq, q_out, k_out))
    if ctx is not None:
        with ctx:
            return qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved,
                                q_out, k_out)
    if _grad_enabled() and (q.requires_grad or k.requires_grad or
                            (q_weight is not None and q_weight.requires_grad) or
                            (k_weight is not None and k_weight.requires_grad) or
                            (inv_freq is not None and inv_freq.requires_grad)):
        _no_outputs(q_out, k_out)
        return _QkNormRope.apply(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved)
    q_out = _dense_like(q) if q_out is None else _given(q_out, q.shape, q.dtype, "q_out")
    k_out = _dense_like(k) if k_out is None else _given(k_out, k.shape, q.dtype, "k_out")
    if n == 0:
        return q_out, k_out
    _check(lib.lt_qk_norm_rope(
        q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(positions), n_pos,
        _ptr(inv_freq), rot, 1 if interleaved else 0, q_out.data_ptr(), k_out.data_ptr(), n, Hq,
        Hkv, d, q_step, k_step, eps, _raw_stream(dev), code, w_code))
    return q_out, k_out


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        ctx.how = eps, interleaved
        return qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        if ctx.needs_input_grad[5]:
            raise RuntimeError("qk_norm_rope has no gradient for inv_freq")
        got = qk_norm_rope_bwd(dq_out.contiguous(), dk_out.contiguous(), *ctx.saved_tensors,
                               *ctx.how)
        return *(g if need else None for g, need in zip(got, ctx.needs_input_grad)), *[None] * 4


_bwd_bytes = {}


def _bwd_workspace(dev, d):
    """Workspace bytes of qk_norm_rope_bwd for heads of d on the current device."""
    n = _bwd_bytes.get((dev, d))
    if n is None:
        need = ctypes.c_size_t()
        _check(lib.lt_qk_norm_rope_bwd_plan(d, 0, need))
        n = _bwd_bytes[(dev, d)] = need.value
    return n


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, positions=None,
                     inv_freq=None, eps=1e-6, interleaved=False, dq=None, dk=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of qk_norm_rope for upstream
    gradients dq_out, dk_out; the weights' are None where a weight is None.
    dq and dk may be given as slices of a fused gradient.  See
    lt_qk_norm_rope_bwd."""
    n, Hq, Hkv, d, q_step, k_step, code, w_code, n_pos, rot = _norm_args(q, k, q_weight, k_weight,
                                                                         positions, inv_freq)
    for g, x, name in ((dq_out, q, "dq_out"), (dk_out, k, "dk_out")):
        if g.shape != x.shape or g.dtype != x.dtype or not g.is_contiguous():
            raise ValueError("%s must be contiguous, of its input's shape and dtype" % name)
    dev = q.get_device()
    ctx = _elsewhere(dev, stream, (k, q_weight, k_weight, positions, inv_freq, dq_out, dk_out, dq,
                                   dk))
    if ctx is not None:
        with ctx:
            return qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq,
                                    eps, interleaved, dq, dk)
    dq_step, dk_step = Hq * d, Hkv * d
    if dq is None:
        dq = _dense_like(q)
    elif dq.shape != q.shape or dq.dtype != q.dtype:
        raise ValueError("dq must have q's shape and dtype")
    else:
        dq_step = _tokens(dq, "dq")[3]
    if dk is None:
        dk = _dense_like(k)
    elif dk.shape != k.shape or dk.dtype != q.dtype:
        raise ValueError("dk must have k's shape and dtype")
    else:
        dk_step = _tokens(dk, "dk")[3]
    dqw = torch.empty_like(q_weight) if q_weight is not None else None
    dkw = torch.empty_like(k_weight) if k_weight is not None else None
    if n == 0:
        return dq, dk, *(w if w is None else w.zero_() for w in (dqw, dkw))
    ws, ws_bytes = None, 0
    if dqw is not None or dkw is not None:
        ws_bytes = _bwd_workspace(dev, d)
        ws = q.new_empty(ws_bytes, dtype=torch.uint8)
    _check(lib.lt_qk_norm_rope_bwd(
        dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), _ptr(q_weight),
        _ptr(k_weight), _ptr(positions), n_pos, _ptr(inv_freq), rot, 1 if interleaved else 0,
        dq.data_ptr(), dk.data_ptr(), _ptr(dqw), _ptr(dkw), n, Hq, Hkv, d, q_step, k_step, dq_step,
        dk_step, eps, _ptr(ws), ws_bytes, _raw_stream(dev), code, w_code))
    return dq, dk, dqw, dkw


class _Pools:
    """A cache's pools as the library takes them: checked, and their places noted."""

    __slots__ = ("k_at", "v_at", "k_scale_at", "v_scale_at", "at", "quant", "struct", "ref", "dev",
                 "dtype", "num_pages", "page_size", "H_kv", "d", "dv", "workspace_bytes")

    def __init__(self, k, v, k_scale, v_scale):
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
        self.quant = quant
        self.k_at, self.v_at = k.data_ptr, v.data_ptr
        self.k_scale_at = k_scale.data_ptr if quant else None
        self.v_scale_at = v_scale.data_ptr if quant else None
        self.at = k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale)
        self.dtype, self.dev = k.dtype, k.get_device()
        self.num_pages, self.page_size, self.H_kv, self.d, self.dv = pages, page_size, H, d, \
            v.shape[3]
        # (a dimension of one entry may have any stride: it is never taken)
        kst, vst = ([s if n > 1 else 0 for s, n in zip(x.stride()[:3], x.shape)] for x in (k, v))
        self.struct = KvCacheStruct(*self.at, *kst, *vst, pages, page_size, H, d, v.shape[3],
                                    _KV_CODES[k.dtype])
        self.ref = ctypes.byref(self.struct)
        self.workspace_bytes = {}

    def stay(self):
        """Whether the pools' memory is where it was."""
        at = self.at
        return self.k_at() == at[0] and self.v_at() == at[1] and \
            (not self.quant or (self.k_scale_at() == at[2] and self.v_scale_at() == at[3]))

    def workspace(self, Hq, code):
        """Workspace bytes of paged_attn_decode for Hq query heads of dtype `code`."""
        n = self.workspace_bytes.get((Hq, code))
        if n is None:
            need = ctypes.c_size_t()
            _check(lib.lt_paged_attn_decode_plan(Hq, self.H_kv, self.d, self.dv, code,
                                                 _KV_CODES[self.dtype], 0, need))
            n = self.workspace_bytes[(Hq, code)] = need.value
        return n


def _pool(name):
    def get(self):
        return self._tensors[name]

    def replace(self, tensor):
        self._tensors[name] = tensor
        self._pools = None
    return property(get, replace)


class PagedKVCache:
    """A paged key-value cache over the caller's pools.

    k [pages, page_size, H_kv, d], v [pages, page_size, H_kv, dv]: bfloat16,
    float16, float32, float8_e4m3fn or int8; any strides that keep rows
    contiguous and 16-byte aligned.  8-bit caches have k_scale, v_scale
    [pages, H_kv, page_size] float32 (contiguous), one scale per row.  The
    pools are not copied, and stay alive with this object.

    k, v, k_scale and v_scale may be set to other pools (larger ones, say): the
    next call takes the pools as they then are, and checks them together.  So it
    does when the memory of one has moved (resize_, set_).  A pool whose shape
    or strides are changed in place, over the same memory, must be set again.
    """

    k, v, k_scale, v_scale = _pool(0), _pool(1), _pool(2), _pool(3)

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self._tensors = [k, v, k_scale, v_scale]
        self._pools = _Pools(k, v, k_scale, v_scale)

    def _now(self):
        """The pools, noted anew where one was replaced or has moved."""
        p = self._pools
        if p is None or not p.stay():
            p = self._pools = _Pools(*self._tensors)
        return p

    _ref = property(lambda self: self._now().ref)
    dtype = property(lambda self: self.k.dtype)
    device = property(lambda self: self.k.device)
    num_pages = property(lambda self: self.k.shape[0])
    page_size = property(lambda self: self.k.shape[1])
    H_kv = property(lambda self: self.k.shape[2])
    d = property(lambda self: self.k.shape[3])
    dv = property(lambda self: self.v.shape[3])

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
    taken as they are, values without their gradients); slots: int32, one per
    token, page * page_size + offset, or -1 to skip the token; they must differ.
    See lt_kv_cache_write."""
    n, H, d, k_step = _tokens(k, "k")
    nv, Hv, dv, v_step = _tokens(v, "v")
    pools = cache._now()
    if nv != n or H != pools.H_kv or Hv != H or d != pools.d or dv != pools.dv:
        raise ValueError("k and v must be [tokens, H_kv, d] and [tokens, H_kv, dv] of the cache")
    if k.dtype != v.dtype:
        raise TypeError("k and v must have one dtype")
    if slots.dtype != torch.int32 or not slots.is_contiguous() or slots.numel() != n:
        raise TypeError("slots must be a contiguous int32 tensor, one per token")
    ctx = _elsewhere(pools.dev, stream, (k, v, slots))
    if ctx is not None:
        with ctx:
            return kv_cache_write(cache, k, v, slots)
    if n == 0:
        return
    _check(lib.lt_kv_cache_write(pools.ref, k.data_ptr(), v.data_ptr(), slots.data_ptr(), n,
                                 k_step, v_step, _raw_stream(pools.dev), _dtype_code(k.dtype)))


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
    pools = cache._now()
    if dtype is None:
        dtype = pools.dtype if pools.dtype in _CODES else torch.bfloat16
    ctx = _elsewhere(pools.dev, stream, (block_table, cu_seqlens, k_out, v_out))
    if ctx is not None:
        with ctx:
            return kv_cache_read(cache, block_table, cu_seqlens, N, dtype, k_out, v_out)
    k_shape, v_shape = (N, pools.H_kv, pools.d), (N, pools.H_kv, pools.dv)
    k_out = cu_seqlens.new_empty(*k_shape, dtype=dtype) if k_out is None \
        else _given(k_out, k_shape, dtype, "k_out")
    v_out = cu_seqlens.new_empty(*v_shape, dtype=dtype) if v_out is None \
        else _given(v_out, v_shape, dtype, "v_out")
    if B == 0 or N == 0:
        return k_out, v_out
    pages = block_table.shape[1]
    _check(lib.lt_kv_cache_read(pools.ref, block_table.data_ptr(),
                                block_table.stride(0) if B > 1 else pages, pages,
                                cu_seqlens.data_ptr(), B, N, k_out.data_ptr(), v_out.data_ptr(),
                                _raw_stream(pools.dev), _dtype_code(dtype)))
    return k_out, v_out


def paged_attn_decode(q, cache, block_table, seq_lens, scale=None, window=0, out=None,
                      return_lse=False, stream=None):
    """Softmax attention of one new token per sequence over the cache: out
    [B, H_q, dv] of q's dtype, or (out, lse) with lse [B, H_q] float32.

    q [B, H_q, d]; block_table int32 [B, max_pages]; seq_lens int32 [B], the
    tokens of each sequence in the cache (0 gives zeros, and lse -inf); scale:
    of the scores (default 1 / sqrt(d)); window: the last `window` tokens only
    (0: all).  There is no backward pass: where q requires a gradient, asking
    for it raises.  See lt_paged_attn_decode."""
    if q.dim() != 3 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [B, H_q, d] tensor")
    B, Hq, d = q.shape
    pools = cache._now()
    if d != pools.d:
        raise ValueError("q and the cache must have the same width")
    _int32(block_table, "block_table", 2)
    _int32(seq_lens, "seq_lens", 1)
    if block_table.shape[0] != B or seq_lens.numel() != B:
        raise ValueError("block_table and seq_lens must have a row per sequence")
    if not -2 ** 31 <= window < 2 ** 31:
        raise ValueError("window must fit 32 bits")
    code = _dtype_code(q.dtype)
    dev = pools.dev
    ctx = _elsewhere(dev, stream, (q, block_table, seq_lens, out))
    if ctx is not None:
        with ctx:
            return paged_attn_decode(q, cache, block_table, seq_lens, scale, window, out,
                                     return_lse)
    if q.requires_grad and _grad_enabled():
        _no_outputs(out)
        return _PagedAttnDecode.apply(q, cache, block_table, seq_lens, scale, window, return_lse)
    out = q.new_empty(B, Hq, pools.dv) if out is None \
        else _given(out, (B, Hq, pools.dv), q.dtype, "out")
    lse = q.new_empty(B, Hq, dtype=torch.float32) if return_lse else None
    if B == 0:
        return (out, lse) if return_lse else out
    ws_bytes = pools.workspace(Hq, code)
    ws = q.new_empty(ws_bytes, dtype=torch.uint8)
    pages = block_table.shape[1]
    _check(lib.lt_paged_attn_decode(
        q.data_ptr(), pools.ref, block_table.data_ptr(),
        block_table.stride(0) if B > 1 else pages, pages, seq_lens.data_ptr(), B, Hq,
        1.0 / math.sqrt(d) if scale is None else scale, window, out.data_ptr(), _ptr(lse),
        ws.data_ptr(), ws_bytes, _raw_stream(dev), code))
    return (out, lse) if return_lse else out


class _PagedAttnDecode(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, cache, block_table, seq_lens, scale, window, return_lse):
        return paged_attn_decode(q, cache, block_table, seq_lens, scale, window, None, return_lse)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("paged_attn_decode has no backward pass")
