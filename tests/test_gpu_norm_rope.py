"""Norm and rotation of queries and keys, and its backward pass, on the GPU
against the 64-bit form (tolerances: the fp32 error bounds of cache_plain plus
half a step of the output type)."""
import ctypes

import pytest
import torch

import cache_plain as plain

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _freq(rot, base=10000.0):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (base ** (-2 * i / max(1, rot))).float()


def _case(T, Hq, Hkv, d, dtype, seed, w_dtype=None, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(T, Hq, d, generator=g) * scale).to(dtype)
    k = (torch.randn(T, Hkv, d, generator=g) * scale).to(dtype)
    wq = (1 + 0.3 * torch.randn(d, generator=g)).to(w_dtype or dtype)
    wk = (1 + 0.3 * torch.randn(d, generator=g)).to(w_dtype or dtype)
    return q, k, wq, wk, g


def _check_fwd(got, q, k, wq, wk, pos, freq, eps, il):
    for x, w, y, name in ((q, wq, got[0], "q"), (k, wk, got[1], "k")):
        ref, bound = plain.norm_rope(x, w, pos, freq, eps, il)
        plain.check(y.reshape(ref.shape), ref, bound, q.dtype, name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [
    # T, Hq, Hkv, d, rot, interleaved, first position
    (1, 1, 1, 64, 64, False, 0), (1, 32, 8, 128, 128, False, 131071), (7, 3, 1, 64, 32, True, 5),
    (130, 5, 5, 128, 16, False, 1000), (33, 8, 2, 64, 8, True, 0), (64, 2, 3, 128, 128, True, 17),
    (300, 40, 1, 64, 0, False, 0), (1201, 8, 8, 64, 64, False, 2 ** 24),
    (9, 7, 2, 128, 56, False, 3),
    (5, 1, 4, 128, 120, True, 2 ** 30),
])
def test_forward(dtype, shape):
    import causal_linear_attention_chunked_b200 as L
    T, Hq, Hkv, d, rot, il, first = shape
    q, k, wq, wk, g = _case(T, Hq, Hkv, d, dtype, 1)
    pos = (first + torch.randint(0, 5000, (T,), generator=g)).int() if rot else None
    freq = _freq(rot) if rot else None
    got = L.qk_norm_rope(q.cuda(), k.cuda(), wq.cuda(), wk.cuda(),
                         pos.cuda() if rot else None, freq.cuda() if rot else None, eps=1e-5,
                         interleaved=il)
    _check_fwd(got, q, k, wq, wk, pos, freq, 1e-5, il)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_fused_slices_shared_positions_and_fp32_gains(dtype):
    """Slices of one projection's output; [N] positions for a [B, N] batch;
    fp32 gains; one token of each row."""
    import causal_linear_attention_chunked_b200 as L
    B, N, Hq, Hkv, d = 3, 37, 8, 2, 128
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(B, N, (Hq + 2 * Hkv) * d, generator=g).to(dtype)
    wq, wk = torch.rand(d, generator=g), torch.rand(d, generator=g)
    freq, pos = _freq(d), torch.arange(100, 100 + N, dtype=torch.int32)
    dev = qkv.cuda()
    cut = lambda x: (x[..., :Hq * d].unflatten(-1, (Hq, d)),
                     x[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d)))
    q, k = cut(qkv)
    for gains in ((wq, wk), (wq, None), (None, None)):
        got = L.qk_norm_rope(*cut(dev), *(w if w is None else w.cuda() for w in gains), pos.cuda(),
                             freq.cuda())
        _check_fwd(got, q.reshape(B * N, Hq, d), k.reshape(B * N, Hkv, d), *gains, pos.repeat(B),
                   freq, 1e-6, False)
    dq, dk = cut(dev)
    got = L.qk_norm_rope(dq[:, 4:5], dk[:, 4:5], wq.cuda(), wk.cuda(), pos[:B].cuda(), freq.cuda())
    _check_fwd(got, q[:, 4], k[:, 4], wq, wk, pos[:B], freq, 1e-6, False)


def test_values_at_the_edges():
    """Rows of zeros, a huge and a tiny row, infinities and NaN: each affects
    its own row only."""
    import causal_linear_attention_chunked_b200 as L
    q, k, wq, wk, _ = _case(8, 2, 1, 64, torch.float32, 3)
    q[0] = 0
    q[1] *= 1e15
    q[2] *= 1e-20
    pos, freq = torch.arange(8, dtype=torch.int32), _freq(64)
    clean = L.qk_norm_rope(q.cuda(), k.cuda(), wq.cuda(), wk.cuda(), pos.cuda(), freq.cuda())
    _check_fwd(clean, q, k, wq, wk, pos, freq, 1e-6, False)
    assert bool((clean[0][0] == 0).all())
    bad = q.clone()
    bad[4, 0, 7] = float("nan")
    bad[5, 1, 9] = float("inf")
    got = L.qk_norm_rope(bad.cuda(), k.cuda(), wq.cuda(), wk.cuda(), pos.cuda(), freq.cuda())[0]
    keep = torch.ones(8, 2, dtype=torch.bool)
    keep[4, 0] = keep[5, 1] = False
    assert torch.equal(got.cpu()[keep], clean[0].cpu()[keep])
    assert bool(torch.isnan(got[4, 0]).all())


BWD = [
    # T, Hq, Hkv, d, rot, interleaved
    (1, 1, 1, 64, 64, False), (1, 8, 2, 128, 128, True), (77, 5, 2, 64, 32, True),
    (300, 8, 8, 128, 96, False), (1500, 3, 1, 64, 64, False), (2049, 1, 1, 128, 0, False),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", BWD)
def test_backward(dtype, shape):
    import causal_linear_attention_chunked_b200 as L
    T, Hq, Hkv, d, rot, il = shape
    q, k, wq, wk, g = _case(T, Hq, Hkv, d, dtype, 4)
    gq = torch.randn(T, Hq, d, generator=g).to(dtype)
    gk = torch.randn(T, Hkv, d, generator=g).to(dtype)
    pos = torch.randint(0, 100000, (T,), generator=g).int() if rot else None
    freq = _freq(rot) if rot else None
    dev = [t if t is None else t.cuda() for t in (gq, gk, q, k, wq, wk, pos, freq)]
    got = L.qk_norm_rope_bwd(*dev, eps=1e-5, interleaved=il)
    again = L.qk_norm_rope_bwd(*dev, eps=1e-5, interleaved=il)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for i, (x, w, gr) in enumerate(((q, wq, gq), (k, wk, gk))):
        (dx, dxb), (dw, dwb) = plain.norm_rope_bwd(gr, x, w, pos, freq, 1e-5, il)
        plain.check(got[i], dx, dxb, dtype, "dx %d" % i)
        plain.check(got[2 + i], dw, dwb, dtype, "dw %d" % i)


def test_backward_into_slices_of_one_gradient():
    """dq and dk written into one fused gradient; what lies between stays."""
    import causal_linear_attention_chunked_b200 as L
    B, N, Hq, Hkv, d = 2, 19, 4, 2, 64
    q, k, wq, wk, g = _case(B * N, Hq, Hkv, d, torch.bfloat16, 5, torch.float32)
    gq, gk = torch.randn(B * N, Hq, d, generator=g).bfloat16(), \
        torch.randn(B * N, Hkv, d, generator=g).bfloat16()
    pos, freq = torch.arange(B * N, dtype=torch.int32), _freq(64)
    fused = torch.full((B * N, (Hq + 2 * Hkv) * d), 7.0, dtype=torch.bfloat16, device="cuda")
    dq = fused[:, :Hq * d].unflatten(-1, (Hq, d))
    dk = fused[:, Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d))
    dev = [t.cuda() for t in (gq, gk, q, k, wq, wk, pos, freq)]
    out = L.qk_norm_rope_bwd(*dev, dq=dq, dk=dk)
    ref = L.qk_norm_rope_bwd(*dev)
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert out[2].dtype == torch.float32
    assert bool((fused[:, (Hq + Hkv) * d:] == 7.0).all())
    none = L.qk_norm_rope_bwd(*dev[:4], None, dev[5], *dev[6:])
    assert none[2] is None and torch.equal(none[3], ref[3])


def test_backward_against_differences():
    """fp32 gradients against central differences of the 64-bit form: the
    differences' own error is O(h^2) = 1e-6 of the third derivative and
    rounding 1e-16 / h, far below the 1e-4 asked."""
    import causal_linear_attention_chunked_b200 as L
    T, H, d, rot = 3, 2, 64, 32
    q, k, wq, wk, g = _case(T, H, 1, d, torch.float32, 6)
    gq, gk = torch.randn(T, H, d, generator=g), torch.randn(T, 1, d, generator=g)
    pos, freq = torch.tensor([3, 70, 1000], dtype=torch.int32), _freq(rot)
    got = L.qk_norm_rope_bwd(*(t.cuda() for t in (gq, gk, q, k, wq, wk, pos, freq)))

    def loss(x, w):
        return float((plain.norm_rope(x, w, pos, freq, 1e-6, False)[0] * gq.double()).sum())

    h = 1e-3
    for idx in [(0, 0, 0), (1, 1, 5), (2, 0, 31), (2, 1, 40), (0, 1, 63)]:
        a, b = q.double(), q.double()
        a[idx] += h
        b[idx] -= h
        num = (loss(a, wq) - loss(b, wq)) / (2 * h)
        assert abs(num - float(got[0][idx])) <= 1e-4 * max(1.0, abs(num))
    for c in (0, 17, 32, 63):
        a, b = wq.double(), wq.double()
        a[c] += h
        b[c] -= h
        num = (loss(q, a) - loss(q, b)) / (2 * h)
        assert abs(num - float(got[2][c])) <= 1e-4 * max(1.0, abs(num))


def test_streams_graphs_and_workspace():
    """Another stream than the current one; a captured call replayed on new
    inputs; a caller's workspace, one too small, and none."""
    import causal_linear_attention_chunked_b200 as L
    from causal_linear_attention_chunked_b200 import _binding as b
    q, k, wq, wk, g = _case(50, 4, 2, 64, torch.bfloat16, 7)
    gq = torch.randn(50, 4, 64, generator=g).bfloat16()
    gk = torch.randn(50, 2, 64, generator=g).bfloat16()
    pos, freq = torch.arange(50, dtype=torch.int32).cuda(), _freq(64).cuda()
    q, k, wq, wk, gq, gk = (t.cuda() for t in (q, k, wq, wk, gq, gk))
    ref = L.qk_norm_rope(q, k, wq, wk, pos, freq)
    refb = L.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, freq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = L.qk_norm_rope(q, k, wq, wk, pos, freq, stream=s)
    gotb = L.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, pos, freq, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got + gotb, ref + refb))
    q2, graph = torch.zeros_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = L.qk_norm_rope(q2, k, wq, wk, pos, freq)
        outb = L.qk_norm_rope_bwd(gq, gk, q2, k, wq, wk, pos, freq)
    for _ in range(2):
        q2.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out + outb, ref + refb))
        q2.zero_()
        graph.replay()
    P = lambda t: ctypes.c_void_p(t.data_ptr())
    need = ctypes.c_size_t()
    assert b.lib.lt_qk_norm_rope_bwd_plan(64, 0, ctypes.byref(need)) == 0
    dq, dk, dwq, dwk = (torch.empty_like(t) for t in (q, k, wq, wk))
    ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    for given, size, st in ((P(ws), need.value, 0), (P(ws), need.value - 1, 1), (None, 0, 0)):
        dwq.zero_()
        assert b.lib.lt_qk_norm_rope_bwd(
            P(gq), P(gk), P(q), P(k), P(wq), P(wk), P(pos), 50, P(freq), 64, 0, P(dq), P(dk),
            P(dwq), P(dwk), 50, 4, 2, 64, 256, 128, 256, 128, 1e-6, given, size,
            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), 1, 1) == st
        torch.cuda.synchronize()
        assert bool((dwq == 0).all()) if st else torch.equal(dwq, refb[2])


def test_feeds_the_linear_attention_pass():
    """Normed and rotated queries and keys go into linear_attn_fwd as they are."""
    import numpy as np
    import causal_linear_attention_chunked_b200 as L
    import oracle
    from parity import row_rel_err, TOL_BF16
    B, N, H, d = 2, 200, 4, 64
    q, k, wq, wk, g = _case(B * N, H, H, d, torch.bfloat16, 8)
    v = torch.randn(B, N, H, d, generator=g).bfloat16()
    q, k = q.view(B, N, H, d).cuda(), k.view(B, N, H, d).cuda()
    pos, freq = torch.arange(N, dtype=torch.int32).cuda(), _freq(64).cuda()
    qr, kr = L.qk_norm_rope(q, k, wq.cuda(), wk.cuda(), pos, freq)
    out = L.linear_attn_fwd(qr, kr, v.cuda())
    ref = oracle.fwd_recurrent(qr.cpu(), kr.cpu(), v, causal=True, eps=1e-6)
    assert row_rel_err(np.asarray(out.float().cpu()), ref) <= TOL_BF16


def test_refusals_on_the_device():
    import causal_linear_attention_chunked_b200 as L
    q = torch.zeros(4, 2, 64, device="cuda")
    with pytest.raises(L.LtError):
        L.qk_norm_rope(q, q, q_out=q)          # in place
    with pytest.raises(ValueError):
        L.qk_norm_rope(q, q.cpu())
    with pytest.raises(ValueError):
        L.qk_norm_rope(q, q, q_out=torch.zeros(4, 2, 63, device="cuda"))
    with pytest.raises(L.LtError):
        L.qk_norm_rope(q, q, eps=0.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [
    (5003, 3, 2, 64, 64, False), (7200, 1, 1, 128, 96, True), (4801, 9, 1, 128, 128, False)])
def test_more_tokens_than_the_device_has_warps(dtype, shape):
    """Warps that go on to further tokens: their rings wrap, and their angles
    change with the token."""
    import causal_linear_attention_chunked_b200 as L
    T, Hq, Hkv, d, rot, il = shape
    q, k, wq, wk, g = _case(T, Hq, Hkv, d, dtype, 9)
    gq = torch.randn(T, Hq, d, generator=g).to(dtype)
    gk = torch.randn(T, Hkv, d, generator=g).to(dtype)
    pos = torch.randint(0, 100000, (T,), generator=g).int()
    freq = _freq(rot)
    dev = [t.cuda() for t in (gq, gk, q, k, wq, wk, pos, freq)]
    _check_fwd([y.cpu() for y in L.qk_norm_rope(*dev[2:], eps=1e-5, interleaved=il)], q, k, wq, wk,
               pos, freq, 1e-5, il)
    got = L.qk_norm_rope_bwd(*dev, eps=1e-5, interleaved=il)
    again = L.qk_norm_rope_bwd(*dev, eps=1e-5, interleaved=il)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for i, (x, w, gr) in enumerate(((q, wq, gq), (k, wk, gk))):
        (dx, dxb), (dw, dwb) = plain.norm_rope_bwd(gr, x, w, pos, freq, 1e-5, il)
        plain.check(got[i], dx, dxb, dtype, "dx %d" % i)
        plain.check(got[2 + i], dw, dwb, dtype, "dw %d" % i)
