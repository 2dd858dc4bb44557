"""Attention of one new token over the paged cache on the GPU against the
64-bit form, and the whole serving step: norm and rotation, write, attend."""
import ctypes

import pytest
import torch

import cache_plain as plain
from test_gpu_kv_cache import _cache, _fill, _pages

pytestmark = pytest.mark.gpu
E4M3, I8 = torch.float8_e4m3fn, torch.int8
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [(BF, BF), (HF, HF), (F32, F32), (BF, E4M3), (BF, I8), (HF, E4M3), (HF, I8), (F32, E4M3),
         (F32, I8)]


def _setup(lens, ps, Hq, Hkv, d, dv, qt, kv, seed, layout="token", extra=1, poison=True):
    """A filled cache, queries, table; what lies past each sequence's end in its
    last page is poisoned with NaN (16-bit and fp32) or NaN scales (8-bit)."""
    g = torch.Generator().manual_seed(seed)
    table, pages = _pages(lens, ps, extra, g)
    c = _cache(pages, ps, Hkv, d, dv, kv, layout)
    _fill(c, g)
    if poison:
        for b, n in enumerate(lens):
            if n % ps:
                p = int(table[b, n // ps])
                for pool, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
                    if scale is not None:
                        scale[p, :, n % ps:] = float("nan")
                    else:
                        pool[p, n % ps:] = float("nan")
    q = torch.randn(len(lens), Hq, d, generator=g).to(qt)
    return c, q, table, torch.tensor(lens, dtype=torch.int32)


def _ref(c, q, table, lens, scale=None, window=0):
    cpu = lambda t: None if t is None else t.cpu()
    return plain.decode(q, cpu(c.k), cpu(c.v), cpu(c.k_scale), cpu(c.v_scale), table, lens,
                        c.page_size, c.d ** -0.5 if scale is None else scale, window)


def _check(got, lse, ref, dtype):
    out, rl, bound, lb = ref
    plain.check(got, out, bound, dtype, "out")
    if lse is not None:
        lse = lse.cpu().double()
        empty = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse), empty)
        assert bool(((lse - rl).abs()[~empty] <= lb[~empty]).all())


@pytest.mark.parametrize("qt,kv", TYPES)
@pytest.mark.parametrize("lens,ps,Hq,Hkv,d,dv,layout", [
    ([1], 1, 1, 1, 64, 64, "token"),
    ([0, 1, 15, 16, 17, 0], 16, 2, 1, 64, 64, "token"),
    ([300, 31, 33, 1], 24, 8, 2, 128, 128, "head"),
    ([777], 16, 8, 8, 64, 64, "token"),
    ([5, 129, 64], 64, 15, 3, 128, 64, "token"),
    ([40, 100], 8, 12, 1, 64, 128, "token"),
    ([70, 3], 128, 40, 2, 128, 128, "pair"),
])
def test_decode(qt, kv, lens, ps, Hq, Hkv, d, dv, layout):
    import causal_linear_attention_chunked_b200 as L
    c, q, table, n = _setup(lens, ps, Hq, Hkv, d, dv, qt, kv, 1, layout)
    got, lse = L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda(), return_lse=True)
    assert L.get_last_device_error() == 0
    _check(got, lse, _ref(c, q, table, n), qt)
    for b, m in enumerate(lens):
        if m == 0:
            assert bool((got[b] == 0).all()) and bool((lse[b] == -float("inf")).all())
    again = L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda())
    assert torch.equal(again, got)


@pytest.mark.parametrize("qt,kv", [(BF, BF), (BF, E4M3), (F32, F32)])
@pytest.mark.parametrize("window", [1, 16, 100, 5000])
def test_window(qt, kv, window):
    import causal_linear_attention_chunked_b200 as L
    c, q, table, n = _setup([700, 0, 99, 101, 1], 16, 4, 2, 64, 64, qt, kv, 2)
    got, lse = L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda(), window=window,
                                   return_lse=True)
    _check(got, lse, _ref(c, q, table, n, window=window), qt)


@pytest.mark.parametrize("qt,kv", [(BF, BF), (BF, E4M3), (HF, I8), (F32, F32)])
def test_long_and_ragged(qt, kv):
    """Pairs shared by many warps, and many pairs per warp."""
    import causal_linear_attention_chunked_b200 as L
    for lens, ps, Hq, Hkv in (([20000, 3, 0, 4097], 64, 4, 1), ([9, 40, 0, 17] * 100, 16, 8, 4)):
        c, q, table, n = _setup(lens, ps, Hq, Hkv, 128, 128, qt, kv, 3)
        got, lse = L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda(), return_lse=True)
        _check(got, lse, _ref(c, q, table, n), qt)


@pytest.mark.parametrize("qt,kv", [(BF, BF), (HF, HF), (BF, E4M3), (BF, I8), (F32, F32)])
def test_growing_scores_and_uneven_values(qt, kv):
    """Scores that rise along the sequence (every tile moves the maximum) and
    value rows of very different size (8-bit scales); a large softmax scale, a
    negative one, and zero (the plain mean)."""
    import causal_linear_attention_chunked_b200 as L
    c, q, table, n = _setup([600, 50], 16, 4, 2, 64, 64, qt, kv, 4, poison=False)
    if kv in (E4M3, I8):
        c.k_scale.mul_(torch.linspace(0.1, 3, c.k_scale.numel(), device="cuda").view_as(c.k_scale))
        c.v_scale.mul_(torch.logspace(-6, 6, c.v_scale.numel(), device="cuda").view_as(c.v_scale))
    else:
        f = torch.linspace(0.1, 3, c.num_pages * 16, device="cuda").view(c.num_pages, 16, 1, 1)
        c.k.copy_((c.k.float() * f).to(kv))
        c.v.copy_((c.v.float() * 10 ** (f - 1.5)).to(kv))
    for scale in (0.125, 1.0, -0.5, 0.0):
        got, lse = L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda(), scale=scale,
                                       return_lse=True)
        _check(got, lse, _ref(c, q, table, n, scale=scale), qt)


def test_small_queries_of_a_wide_type_on_an_8_bit_cache():
    """bf16 queries far outside fp16's range."""
    import causal_linear_attention_chunked_b200 as L
    for f in (1e-30, 1e20):
        c, q, table, n = _setup([100], 16, 4, 2, 64, 64, BF, E4M3, 5)
        q = (q.float() * f).bfloat16()
        got, lse = L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda(), scale=0.125 / f,
                                       return_lse=True)
        _check(got, lse, _ref(c, q, table, n, scale=0.125 / f), BF)


@pytest.mark.parametrize("qt,kv", TYPES)
def test_nan_reaches_its_own_heads_only(qt, kv):
    import causal_linear_attention_chunked_b200 as L
    c, q, table, n = _setup([200, 200], 16, 4, 2, 64, 64, qt, kv, 6)
    ref = L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda())
    p = int(table[1, 3])
    if c.v_scale is not None:
        c.v_scale[p, 1, 2] = float("nan")
    else:
        c.v[p, 2, 1, 7] = float("nan")
    got = L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda())
    assert bool(torch.isnan(got[1, 2:]).any())
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1, :2], ref[1, :2])


def test_bad_lengths_and_pages():
    """A bad length leaves its rows alone; a bad page's tokens take no part;
    both are reported."""
    import causal_linear_attention_chunked_b200 as L
    from causal_linear_attention_chunked_b200 import _binding as b
    c, q, table, n = _setup([64, 48, 32], 16, 4, 2, 64, 64, BF, BF, 7, extra=0)
    ref = L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda())
    for bad in (-1, 65, 2 ** 31 - 1):
        lens = n.clone()
        lens[1] = bad
        out = torch.full((3, 4, 64), 9.0, dtype=BF, device="cuda")
        L.paged_attn_decode(q.cuda(), c, table.cuda(), lens.cuda(), out=out)
        assert L.get_last_device_error() == b.LT_ERR_DEVICE_BAD_SEQLENS
        assert bool((out[1] == 9.0).all())
        assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
    for entry in (-1, c.num_pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 3] = entry                             # the last 16 of 64 tokens
        got = L.paged_attn_decode(q.cuda(), c, t.cuda(), n.cuda())
        assert L.get_last_device_error() == b.LT_ERR_DEVICE_BAD_PAGE
        short = n.clone()
        short[0] = 48
        _check(got, None, _ref(c, q, table, short), BF)
    assert L.get_last_device_error() == 0


def test_pages_of_two_sequences_shared_and_table_slices():
    """A common prefix in shared pages; a table that is a slice of a wider one."""
    import causal_linear_attention_chunked_b200 as L
    c, q, table, n = _setup([64, 64], 16, 4, 2, 64, 64, BF, E4M3, 8, extra=0)
    table[1, :2] = table[0, :2]
    wide = torch.full((2, 40), 10 ** 6, dtype=torch.int32)
    wide[:, 3:3 + table.shape[1]] = table
    got = L.paged_attn_decode(q.cuda(), c, wide.cuda()[:, 3:3 + table.shape[1]], n.cuda())
    assert L.get_last_device_error() == 0
    _check(got, None, _ref(c, q, table, n), BF)


def test_joining_two_parts_by_their_log_sums():
    """Two parts of a sequence, joined outside by lse, are the whole: each
    part's rounding (2^-8) and the weights' stay inside three half steps of the
    larger part."""
    import causal_linear_attention_chunked_b200 as L
    c, q, table, n = _setup([160], 16, 4, 2, 64, 64, F32, F32, 9, extra=0)
    whole, lse = L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda(), return_lse=True)
    parts = [L.paged_attn_decode(q.cuda(), c, t.contiguous().cuda(),
                                 torch.tensor([m], dtype=torch.int32).cuda(), return_lse=True)
             for t, m in ((table[:, :4], 64), (table[:, 4:], 96))]
    l2 = torch.stack([p[1] for p in parts])
    w = torch.softmax(l2, 0)[..., None]
    joined = (torch.stack([p[0] for p in parts]) * w).sum(0)
    _check(joined, torch.logsumexp(l2, 0), tuple(x if i < 2 else 3 * x for i, x in
                                                 enumerate(_ref(c, q, table, n))), F32)
    assert torch.allclose(lse, torch.logsumexp(l2, 0), atol=1e-5)


def test_offsets_past_32_bits():
    """A cache whose pools exceed 2^32 bytes and 2^31 elements: pages at its end."""
    import causal_linear_attention_chunked_b200 as L
    ps, H, d = 256, 8, 128
    pages = 2 ** 31 // (ps * H * d) + 4              # 4.3 GB of bf16 keys, and of values
    c = L.PagedKVCache.empty(pages, ps, H, d)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(300, H, d, generator=g, device="cuda").bfloat16()
    v = torch.randn(300, H, d, generator=g, device="cuda").bfloat16()
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
    slots = torch.cat([torch.arange(256) + (pages - 1) * ps, torch.arange(44) + (pages - 2) * ps])
    L.kv_cache_write(c, k, v, slots.int().cuda())
    cu = torch.tensor([0, 300], dtype=torch.int32).cuda()
    kb, vb = L.kv_cache_read(c, table.cuda(), cu, 300)
    assert torch.equal(kb, k) and torch.equal(vb, v)
    q = torch.randn(1, 16, d, generator=g, device="cuda").bfloat16()
    got = L.paged_attn_decode(q, c, table.cuda(), torch.tensor([300], dtype=torch.int32).cuda())
    small = L.PagedKVCache.empty(2, ps, H, d)
    L.kv_cache_write(small, k, v, torch.arange(300, dtype=torch.int32).cuda())
    ref = L.paged_attn_decode(q, small, torch.tensor([[0, 1]], dtype=torch.int32).cuda(),
                              torch.tensor([300], dtype=torch.int32).cuda())
    assert L.get_last_device_error() == 0
    assert torch.equal(got, ref)


def test_streams_graphs_and_workspaces():
    """Two streams at once, a captured call replayed as its lengths grow, two
    graphs interleaved, a caller's workspace, one too small, and none."""
    import causal_linear_attention_chunked_b200 as L
    from causal_linear_attention_chunked_b200 import _binding as b
    c, q, table, n = _setup([3000, 70, 5], 16, 8, 2, 64, 64, BF, E4M3, 10)
    q, table, n = q.cuda(), table.cuda(), n.cuda()
    ref, rl = L.paged_attn_decode(q, c, table, n, return_lse=True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(10):
        outs.append(L.paged_attn_decode(q, c, table, n, stream=s1))
        outs.append(L.paged_attn_decode(q, c, table, n, stream=s2))
    s1.synchronize()
    s2.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    live = torch.tensor([1, 0, 2], dtype=torch.int32, device="cuda")
    q2 = (q.float() * 0.5).bfloat16()
    ref2 = L.paged_attn_decode(q2, c, table, n)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        oa = L.paged_attn_decode(q, c, table, live)
    with torch.cuda.graph(gb):
        ob = L.paged_attn_decode(q2, c, table, live)
    ga.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, L.paged_attn_decode(q, c, table, live))
    live.copy_(n)
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga.replay()
        with torch.cuda.stream(s2):
            gb.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, ref) and torch.equal(ob, ref2)
    P = lambda t: ctypes.c_void_p(t.data_ptr())
    need = ctypes.c_size_t()
    assert b.lib.lt_paged_attn_decode_plan(8, 2, 64, 64, 1, 3, 0, ctypes.byref(need)) == 0
    ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(ref), torch.empty_like(rl)
    for given, size, st in ((P(ws), need.value, 0), (P(ws), need.value - 1, 1), (None, 0, 0)):
        out.zero_()
        assert b.lib.lt_paged_attn_decode(
            P(q), c._ref, P(table), table.stride(0), table.shape[1], P(n), 3, 8, 0.125, 0, P(out),
            P(lse), given, size, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), 1) == st
        torch.cuda.synchronize()
        assert bool((out == 0).all()) if st else torch.equal(out, ref) and torch.equal(lse, rl)


def test_injected_workspace_failure(monkeypatch):
    from causal_linear_attention_chunked_b200 import _binding as b
    c, q, table, n = _setup([70, 5], 16, 8, 2, 64, 64, BF, BF, 11)
    q, table, n = q.cuda(), table.cuda(), n.cuda()
    out = torch.full((2, 8, 64), 7.0, dtype=BF, device="cuda")
    P = lambda t: ctypes.c_void_p(t.data_ptr())
    monkeypatch.setenv("LT_FAULT_WORKSPACE_ALLOC", "1")
    args = (P(q), c._ref, P(table), table.stride(0), table.shape[1], P(n), 2, 8, 0.125, 0, P(out),
            None, None, 0, None, 1)
    assert b.lib.lt_paged_attn_decode(*args) == b.LT_ERR_CUDA
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())


def test_refusals_on_the_device():
    import causal_linear_attention_chunked_b200 as L
    c, q, table, n = _setup([70, 5], 16, 8, 2, 64, 64, BF, BF, 12)
    q, table, n = q.cuda(), table.cuda(), n.cuda()
    with pytest.raises(L.LtError):
        L.paged_attn_decode(q.half(), c, table, n)
    with pytest.raises(L.LtError):
        L.paged_attn_decode(q[:, :3].contiguous(), c, table, n)
    with pytest.raises(L.LtError):
        L.paged_attn_decode(q, c, table, n, out=q)
    with pytest.raises(L.LtError):
        L.paged_attn_decode(q, c, table, n, window=-1)
    with pytest.raises(ValueError):
        L.paged_attn_decode(q, c, table[:1], n)
    with pytest.raises(TypeError):
        L.paged_attn_decode(q, c, table, n.long())
    with pytest.raises(ValueError):
        L.paged_attn_decode(q[:, :, :32].contiguous(), c, table, n)


@pytest.mark.parametrize("kv", [BF, E4M3, I8])
def test_a_serving_run(kv):
    """A prompt and then single tokens through a layer: norm and rotation of
    slices of the projection, write, attend; every step against softmax
    attention in 64 bits over the rows that the cache holds, and the cache's
    rows against the normed and rotated keys."""
    import causal_linear_attention_chunked_b200 as L
    B, Hq, Hkv, d, ps = 3, 8, 2, 64, 16
    prompt, steps = [37, 1, 16], 20
    g = torch.Generator().manual_seed(13)
    qkv_of = lambda t: torch.randn(t, (Hq + 2 * Hkv) * d, generator=g).to(BF).cuda()
    cut = lambda x: (x[:, :Hq * d].unflatten(-1, (Hq, d)),
                     x[:, Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d)),
                     x[:, (Hq + Hkv) * d:].unflatten(-1, (Hkv, d)))
    wq = (1 + 0.2 * torch.randn(d, generator=g)).to(BF)
    wk = (1 + 0.2 * torch.randn(d, generator=g)).to(BF)
    freq = (10000.0 ** (-torch.arange(d // 2).double() / (d // 2))).float()
    need = [-(-(m + steps) // ps) for m in prompt]
    table, pages = _pages([m * ps for m in need], ps, 0, g)
    c = _cache(pages, ps, Hkv, d, d, kv)
    slot = lambda b, i: int(table[b, i // ps]) * ps + i % ps
    at = [(b, i) for b, m in enumerate(prompt) for i in range(m)]
    keys = {}

    def step(where, x):
        q, k, v = cut(x)
        pos = torch.tensor([i for _, i in where], dtype=torch.int32)
        qr, kr = L.qk_norm_rope(q, k, wq.cuda(), wk.cuda(), pos.cuda(), freq.cuda())
        slots = torch.tensor([slot(*w) for w in where], dtype=torch.int32)
        L.kv_cache_write(c, kr, v, slots.cuda())
        ref, bound = plain.norm_rope(k.cpu(), wk, pos, freq, 1e-6, False)
        plain.check(kr, ref, bound, BF, "keys")
        for t, w in enumerate(where):
            keys[w] = (kr[t].cpu(), v[t].cpu())
        return qr

    step(at, qkv_of(len(at)))
    for s in range(steps):
        where = [(b, m + s) for b, m in enumerate(prompt)]
        qr = step(where, qkv_of(B))
        n = torch.tensor([m + s + 1 for m in prompt], dtype=torch.int32)
        out, lse = L.paged_attn_decode(qr, c, table.cuda(), n.cuda(), return_lse=True)
        _check(out, lse, _ref(c, qr.cpu(), table, n), BF)
    assert L.get_last_device_error() == 0
    for b, m in enumerate(prompt):
        total = m + steps
        K = torch.stack([keys[b, i][0] for i in range(total)])
        got = plain.rows_of(c.k.cpu(), None if c.k_scale is None else c.k_scale.cpu(), table[b],
                            total, ps)
        if kv == BF:
            assert torch.equal(got, K.double())
        else:
            codes, sc = plain.quantise(K, kv)
            assert torch.equal(got, codes.double() * sc.double()[..., None])


@pytest.mark.parametrize("qt,kv", [(BF, E4M3), (HF, I8), (F32, E4M3)])
@pytest.mark.parametrize("lens,ps,Hq,Hkv", [
    ([20000, 3, 0, 4097], 64, 4, 1), ([9, 40, 0, 17] * 100, 16, 8, 4), ([5000, 33, 700], 24, 9, 3),
    ([3000] * 5, 64, 17, 17)])
def test_long_and_ragged_8_bit_rows_of_64(qt, kv, lens, ps, Hq, Hkv):
    """The narrow 8-bit rows, which more warps per block share."""
    import causal_linear_attention_chunked_b200 as L
    c, q, table, n = _setup(lens, ps, Hq, Hkv, 64, 64, qt, kv, 8)
    got, lse = L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda(), return_lse=True)
    assert L.get_last_device_error() == 0
    _check(got, lse, _ref(c, q, table, n), qt)
    assert torch.equal(L.paged_attn_decode(q.cuda(), c, table.cuda(), n.cuda()), got)
