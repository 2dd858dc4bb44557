"""Plain 64-bit forms of the norm-and-rotation, cache and decode operators, and
the error bounds that their fp32 arithmetic and one rounding allow.

Units: ``U32`` is half a step of fp32 (2^-24); ``half_step(dtype)`` half a step
of an output type, relative to the value (bf16 2^-8, fp16 2^-11, fp32 2^-24).
"""
import math

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half of the distance between a type's smallest numbers (subnormals)."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


# ------------------------------------------------------------ norm, rotation
def _pairs(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, positions, inv_freq, interleaved, sign=1.0):
    """x [T, H, d] float64, positions [T]."""
    if inv_freq is None or inv_freq.numel() == 0:
        return x.clone()
    rot = 2 * inv_freq.numel()
    ang = positions.double()[:, None] * inv_freq.double()[None, :]
    c, s = torch.cos(ang)[:, None, :], sign * torch.sin(ang)[:, None, :]
    ia, ib = _pairs(rot, interleaved)
    y = x.clone()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def pair_size(y, rot, interleaved):
    """|a| + |b| of each value's pair, at most (what a rotation's rounding goes by)."""
    size = y.abs().clone()
    if rot:
        ia, ib = _pairs(rot, interleaved)
        h = math.sqrt(2.0) * torch.hypot(y[..., ia], y[..., ib])
        size[..., ia] = h
        size[..., ib] = h
    return size


def norm_rope(x, w, positions, inv_freq, eps, interleaved):
    """(value, bound without the last rounding) of x [T, H, d].

    fp32 errors, in U32 of the pair's size: the sum of squares is at most 5
    fused steps and 5 sums (10, halved by the root), the root's reciprocal 2
    steps (4), mean and eps (1), two products (2); the reduced angle in fp32, 2
    pi 2^-26 and its product by 2 pi (3 + 4); sine and cosine 2 steps for fp32
    (4), 2^-21.2 absolute for the 16-bit types (7); two products and a sum (3).
    In all under 30."""
    x = x.double()
    d = x.shape[-1]
    w = torch.ones(d, dtype=torch.float64) if w is None else w.double()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w
    y = rotate(y, positions, inv_freq, interleaved)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    return y, 30 * U32 * pair_size(y, rot, interleaved)


def norm_rope_bwd(g, x, w, positions, inv_freq, eps, interleaved, adds=256):
    """((dx, bound), (dw, bound)).

    dx = r (u - n m): u carries the rotation's and the gain's errors (19 U32 of
    the pair's size), n and r those of the norm (12), m a sum of d products (10
    and what its terms carry: 45 U32 of mean|u n|); so the first term 19 + 12 +
    1, the second 12 + 45 + 12 + 3.  dw: each term carries 19 + 12 + 1 U32 of its
    size, and a sum with at most `adds` roundings in a row (a lane's rows, the
    block's 32 rows of lanes, the blocks)."""
    g, x = g.double(), x.double()
    d = x.shape[-1]
    w1 = torch.ones(d, dtype=torch.float64) if w is None else w.double()
    g = rotate(g, positions, inv_freq, interleaved, -1.0)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    size = pair_size(g, rot, interleaved)
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    n, u = x * r, g * w1
    m = (u * n).mean(-1, keepdim=True)
    m_size = (size * w1.abs() * n.abs()).mean(-1, keepdim=True)
    dx = r * (u - n * m)
    dx_bound = r * U32 * (32 * size * w1.abs() + 80 * n.abs() * m_size)
    dw = (g * n).sum((0, 1))
    dw_bound = (32 + adds) * U32 * (size * n.abs()).sum((0, 1))
    return (dx, dx_bound), (dw, dw_bound)


# -------------------------------------------------------------------- cache
QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def quantise(x, dtype):
    """Codes and scales of rows x [..., w] by the definition, in fp32 division
    (correctly rounded on the CPU): what the library must hold bit for bit."""
    x = x.float()
    ok = torch.isfinite(x).all(-1)
    top = torch.full((), QMAX[dtype])
    safe = torch.where(ok[..., None], x, torch.zeros(()))
    scale = torch.clamp(safe.abs().amax(-1) / top, min=2.0 ** -126)
    y = safe / scale[..., None]
    codes = torch.round(y).to(torch.int8) if dtype == torch.int8 else y.to(dtype)
    return codes, torch.where(ok, scale, torch.full((), math.nan))


def rows_of(pool, scale, table_row, n, page_size):
    """Rows 0 .. n - 1 of one sequence, [n, H, w] float64."""
    i = torch.arange(n)
    page, slot = table_row[i // page_size].long(), i % page_size
    x = pool[page, slot].double()
    if scale is not None:
        x = x * scale[page, :, slot].double()[..., None]
    return x


# ------------------------------------------------------------------- decode
def decode(q, k_pool, v_pool, k_scale, v_scale, table, lens, page_size, scale, window):
    """(out [B, Hq, dv], lse, bound of out before its last rounding, bound of
    lse), everything on the CPU.

    With W = sum p|v| / sum p: a score s = scale q.k carries d + 8 roundings of
    its terms' sizes, and s in units of log 2 a few of its own size; the
    exponential 2^-22; 8-bit caches take q in fp16 relative to the head's
    largest entry, 2^-25 of it.  That moves every weight by a factor within
    e^delta, the quotient by 2 delta W.  The weights for the tensor cores are
    two terms of the cache's 16-bit type, so half a step of it squared (2^-16,
    2^-22); for 8-bit caches fp16, one term for bf16 queries (2^-11), two
    otherwise; for fp32 caches two terms of tf32, the second cut to 11 bits
    (2^-21), as are the products' factors (2^-21 of each term's size, 8 U32, in
    the scores and again in the values).  fp32 queries on 8-bit caches are two
    fp16 terms (2^-22, 4 U32).  Sums over n keys round by n U32 of W, and
    weights under 2^-26 of the largest lose at most 2^-37 each against the
    largest value row."""
    B, Hq, d = q.shape
    Hkv, dv = k_pool.shape[2], v_pool.shape[3]
    out = torch.zeros(B, Hq, dv, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    bound = torch.zeros(B, Hq, dv, dtype=torch.float64)
    lse_bound = torch.zeros(B, Hq, dtype=torch.float64)
    quant = k_scale is not None
    wide = q.dtype == torch.float32
    weight = 2.0 ** -11 if quant and q.dtype == torch.bfloat16 else \
        2.0 ** -22 if quant else 2.0 ** -20 if wide else half_step(q.dtype) ** 2
    for b in range(B):
        n = int(lens[b])
        K = rows_of(k_pool, k_scale, table[b], n, page_size)
        V = rows_of(v_pool, v_scale, table[b], n, page_size)
        if window:
            K, V = K[-window:], V[-window:]
        n = K.shape[0]
        if n == 0:
            continue
        for h in range(Hq):
            g = h * Hkv // Hq
            qh = q[b, h].double()
            s = scale * (K[:, g] @ qh)
            size = abs(scale) * (K[:, g].abs() @ qh.abs())
            delta = ((d + 8 + (16 if wide else 0)) * U32 * size + 8 * U32 * s.abs()).max() + \
                2.0 ** -21
            if quant and q.dtype != torch.float32:
                delta = delta + abs(scale) * qh.abs().max() * 2.0 ** -25 * \
                    K[:, g].abs().sum(-1).max()
            p = torch.softmax(s, 0)
            out[b, h] = p @ V[:, g]
            lse[b, h] = torch.logsumexp(s, 0)
            W = p @ V[:, g].abs()
            bound[b, h] = W * (2 * delta + weight + (n + 32) * U32) + \
                n * 2.0 ** -36 * V[:, g].abs().amax(0)
            lse_bound[b, h] = delta + (n + 32) * U32 + 4 * U32 * lse[b, h].abs()
    return out, lse, bound, lse_bound


def check(got, ref, bound, dtype, what=""):
    """|got - ref| <= bound + half a step of the rounded value, everywhere."""
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref)), what + ": finite places differ"
    tol = bound + half_step(dtype) * (ref.abs() + bound) + smallest(dtype)
    off = (got - ref).abs() / tol
    assert not bool((off > 1).any()), "%s: %.3g times the bound" % (what, float(off.max()))
