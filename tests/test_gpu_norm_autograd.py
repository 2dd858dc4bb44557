"""qk_norm_rope inside a differentiated model: its gradients are those of
qk_norm_rope_bwd, and none is dropped without a word."""
import pytest
import torch

import cache_plain as plain

pytestmark = pytest.mark.gpu
B, N, HQ, HKV, D, ROT = 2, 9, 4, 2, 64, 32


def _case(dtype=torch.bfloat16, grad=True):
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)
    qkv = r(B, N, (HQ + 2 * HKV) * D).requires_grad_(grad)
    wq, wk = r(D).requires_grad_(grad), r(D).requires_grad_(grad)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    freq = torch.rand(ROT // 2, generator=g, device="cuda")
    return qkv, wq, wk, pos, freq, r(B, N, HQ, D), r(B, N, HKV, D)


def _cut(x):
    return (x[..., :HQ * D].unflatten(-1, (HQ, D)),
            x[..., HQ * D:(HQ + HKV) * D].unflatten(-1, (HKV, D)))


def _by_hand(qkv, wq, wk, pos, freq, gq, gk, **kw):
    import causal_linear_attention_chunked_b200 as L
    with torch.no_grad():
        dq, dk, dwq, dwk = L.qk_norm_rope_bwd(gq, gk, *_cut(qkv), wq, wk, pos, freq, **kw)
        full = torch.zeros_like(qkv)
        for part, d in zip(_cut(full), (dq, dk)):
            part.copy_(d)
    return full, dwq, dwk


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_of_a_fused_projection(interleaved):
    import causal_linear_attention_chunked_b200 as L
    qkv, wq, wk, pos, freq, gq, gk = _case()
    kw = dict(eps=1e-5, interleaved=interleaved)
    out = L.qk_norm_rope(*_cut(qkv), wq, wk, pos, freq, **kw)
    with torch.no_grad():
        ref = L.qk_norm_rope(*_cut(qkv), wq, wk, pos, freq, **kw)
    assert all(torch.equal(a, b) and not b.requires_grad for a, b in zip(out, ref))
    got = torch.autograd.grad(out, (qkv, wq, wk), (gq, gk))
    ref = _by_hand(qkv, wq, wk, pos, freq, gq, gk, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_gradients_against_the_formula_differentiated_in_64_bits():
    """fp32, through autograd of the plain form in 64 bits; bounds as for the backward pass."""
    import causal_linear_attention_chunked_b200 as L
    qkv, wq, wk, pos, freq, gq, gk = _case(torch.float32)
    out = L.qk_norm_rope(*_cut(qkv), wq, wk, pos, freq)
    got = torch.autograd.grad(out, (qkv, wq, wk), (gq, gk))
    cpu = [t.detach().cpu() for t in (qkv, wq, wk, pos, freq, gq, gk)]
    x, uq, uk = (t.double().requires_grad_() for t in cpu[:3])
    at = cpu[3].repeat(B)
    outs = [plain.norm_rope(p.reshape(B * N, -1, D), u, at, cpu[4], 1e-6, False)[0]
            for p, u in zip(_cut(x), (uq, uk))]
    ref = torch.autograd.grad(outs, (x, uq, uk), [t.double().reshape(o.shape)
                                                  for t, o in zip(cpu[5:], outs)])
    for i, (p, u, g) in enumerate(zip(_cut(cpu[0]), cpu[1:3], cpu[5:])):
        (_, bx), (_, bw) = plain.norm_rope_bwd(g.reshape(B * N, -1, D), p.reshape(B * N, -1, D), u,
                                               at, cpu[4], 1e-6, False)
        plain.check(_cut(got[0])[i].reshape(bx.shape), _cut(ref[0])[i].reshape(bx.shape), bx,
                    torch.float32, "dx %d" % i)
        plain.check(got[1 + i], ref[1 + i], bw, torch.float32, "dw %d" % i)


def test_some_gradients_wanted_and_some_not():
    """One output used, an upstream gradient that is expanded, inputs that need none,
    a gain for both heads' kinds, no gains."""
    import causal_linear_attention_chunked_b200 as L
    qkv, wq, wk, pos, freq, gq, gk = _case()
    full, dwq, dwk = _by_hand(qkv, wq, wk, pos, freq, torch.zeros_like(gq), torch.ones_like(gk))
    _, ko = L.qk_norm_rope(*_cut(qkv), wq, wk, pos, freq)
    got = torch.autograd.grad(ko.sum(), (qkv, wq, wk))
    assert torch.equal(got[0], full) and not bool(got[1].any()) and torch.equal(got[2], dwk)
    full, dwq, dwk = _by_hand(qkv, wq, wk, pos, freq, gq, gk)
    out = L.qk_norm_rope(*_cut(qkv.detach()), wq, wk.detach(), pos, freq)
    assert torch.equal(torch.autograd.grad(out, wq, (gq, gk))[0], dwq)
    both = torch.autograd.grad(L.qk_norm_rope(*_cut(qkv), wq, wq, pos, freq), wq, (gq, gk))[0]
    a, b = _by_hand(qkv, wq, wq, pos, freq, gq, gk)[1:]
    assert torch.equal(both, a + b)
    none = torch.autograd.grad(L.qk_norm_rope(*_cut(qkv)), qkv, (gq, gk))[0]
    assert torch.equal(none, _by_hand(qkv, None, None, None, None, gq, gk)[0])


def test_gradients_on_another_stream_and_from_a_graph():
    import causal_linear_attention_chunked_b200 as L
    qkv, wq, wk, pos, freq, gq, gk = _case()
    ref = _by_hand(qkv, wq, wk, pos, freq, gq, gk)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = L.qk_norm_rope(*_cut(qkv), wq, wk, pos, freq, stream=side)
    side.synchronize()
    got = torch.autograd.grad(out, (qkv, wq, wk), (gq, gk))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    del out, got
    x = torch.zeros_like(qkv).requires_grad_()
    step = lambda: torch.autograd.grad(L.qk_norm_rope(*_cut(x), wq, wk, pos, freq), (x, wq, wk),
                                       (gq, gk))
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        x.copy_(qkv)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_what_has_no_gradient_says_so():
    import causal_linear_attention_chunked_b200 as L
    qkv, wq, wk, pos, freq, gq, gk = _case()
    q, k = _cut(qkv)
    with pytest.raises(ValueError):
        L.qk_norm_rope(q, k, q_out=torch.empty_like(gq))
    with torch.no_grad():
        L.qk_norm_rope(q, k, q_out=torch.empty_like(gq))
    out = L.qk_norm_rope(q, k, wq, wk, pos, freq.clone().requires_grad_())
    with pytest.raises(RuntimeError, match="inv_freq"):
        torch.autograd.grad(out, qkv, (gq, gk))
    out = L.qk_norm_rope(q, k, wq, wk, pos, freq)
    once = torch.autograd.grad(out, qkv, (gq.requires_grad_(), gk), create_graph=True)[0]
    with pytest.raises(RuntimeError):
        torch.autograd.grad(once.sum(), gq)                     # no second derivative
    c = L.PagedKVCache.empty(1, 16, HKV, D)
    c.k.zero_(), c.v.zero_()
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 5, dtype=torch.int32, device="cuda")
    one = q[:, 0].contiguous()
    out, lse = L.paged_attn_decode(one, c, table, lens, return_lse=True)
    assert torch.equal(out, L.paged_attn_decode(one.detach(), c, table, lens))
    for y in (out, lse, L.paged_attn_decode(one, c, table, lens)):
        with pytest.raises(RuntimeError, match="no backward"):
            y.float().sum().backward(retain_graph=True)
    with pytest.raises(ValueError):
        L.paged_attn_decode(one, c, table, lens, out=torch.empty_like(out))


def test_a_captured_training_step():
    """Forward and backward with accumulation into the leaves' gradients, captured
    after warm-up on a side stream, and replayed on new inputs."""
    import causal_linear_attention_chunked_b200 as L
    qkv, wq, wk, pos, freq, gq, gk = _case()
    ref = _by_hand(qkv, wq, wk, pos, freq, gq, gk)
    x = torch.zeros_like(qkv).requires_grad_()
    leaves = (x, wq, wk)

    def step():
        torch.autograd.backward(L.qk_norm_rope(*_cut(x), wq, wk, pos, freq), (gq, gk))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            for t in leaves:
                t.grad = None
            step()
    torch.cuda.current_stream().wait_stream(side)
    for t in leaves:
        t.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    with torch.no_grad():
        x.copy_(qkv)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t.grad, r) for t, r in zip(leaves, ref))
