"""Writing into and reading from the paged cache on the GPU: codes and scales
bit for bit against the definition, values read back, skipped and bad slots,
layouts, and what must stay untouched."""
import math

import pytest
import torch

import cache_plain as plain

pytestmark = pytest.mark.gpu
E4M3, I8 = torch.float8_e4m3fn, torch.int8


def _raw(t):
    """Codes as bytes, others as they are (comparable, NaN included)."""
    return t.view(torch.uint8) if t.dtype in (E4M3, I8) else t


def _cache(pages, ps, H, d, dv, dtype, layout="token"):
    """A cache whose rows hold a pattern; layouts: token-major, head-major, and
    keys and values interleaved in one tensor."""
    import causal_linear_attention_chunked_b200 as L
    if layout == "token":
        c = L.PagedKVCache.empty(pages, ps, H, d, dv, dtype)
        k, v = c.k, c.v
    elif layout == "head":
        k = torch.empty(pages, H, ps, d, dtype=dtype, device="cuda").transpose(1, 2)
        v = torch.empty(pages, H, ps, dv, dtype=dtype, device="cuda").transpose(1, 2)
    else:
        both = torch.empty(pages, 2, ps, H, d, dtype=dtype, device="cuda")
        k, v = both[:, 0], both[:, 1]
    ks = vs = None
    if dtype in (E4M3, I8):
        ks = torch.full((pages, H, ps), 0.5, device="cuda")
        vs = torch.full((pages, H, ps), 0.25, device="cuda")
    k.copy_(torch.full((1,), 3.0).to(dtype))
    v.copy_(torch.full((1,), 5.0).to(dtype))
    return L.PagedKVCache(k, v, ks, vs)


def _expect_rows(pool, scale, slots, x, ps, dtype):
    """The pool after the write, by the definition."""
    pool, scale = pool.clone(), None if scale is None else scale.clone()
    if scale is not None:
        codes, sc = plain.quantise(x, dtype)
    else:
        codes, sc = x.to(dtype), None
    for t, s in enumerate(slots.tolist()):
        if s < 0 or s >= pool.shape[0] * ps:
            continue
        pool[s // ps, s % ps] = codes[t]
        if scale is not None:
            scale[s // ps, :, s % ps] = sc[t]
    return pool, scale


@pytest.mark.parametrize("layout", ["token", "head", "pair"])
@pytest.mark.parametrize("src,kv", [
    (torch.bfloat16, E4M3), (torch.bfloat16, I8), (torch.bfloat16, torch.bfloat16),
    (torch.float16, E4M3), (torch.float16, I8), (torch.float16, torch.float16),
    (torch.float32, E4M3), (torch.float32, I8), (torch.float32, torch.float32)])
@pytest.mark.parametrize("shape", [
    # tokens, heads, d, dv, pages, page size
    (1, 1, 64, 64, 1, 1), (5, 3, 128, 64, 4, 16), (70, 8, 64, 128, 9, 24),
    (257, 2, 128, 128, 40, 8)])
def test_write(src, kv, shape, layout):
    import causal_linear_attention_chunked_b200 as L
    T, H, d, dv, pages, ps = shape
    if layout == "pair" and d != dv:
        dv = d
    g = torch.Generator().manual_seed(T)
    c = _cache(pages, ps, H, d, dv, kv, layout)
    k = (torch.randn(T, H, d, generator=g) * torch.rand(T, H, 1, generator=g) * 8).to(src)
    v = torch.randn(T, H, dv, generator=g).to(src)
    k[0, 0] = 0                                     # a row of zeros
    slots = torch.randperm(pages * ps, generator=g)[:T].int()
    if T > 3:
        slots[2] = -1                               # a padding token
    cpu = lambda t: None if t is None else t.cpu()
    want = [_expect_rows(c.k.cpu(), cpu(c.k_scale), slots, k, ps, kv),
            _expect_rows(c.v.cpu(), cpu(c.v_scale), slots, v, ps, kv)]
    L.kv_cache_write(c, k.cuda(), v.cuda(), slots.cuda())
    assert L.get_last_device_error() == 0
    for (pool, scale), got, got_scale in ((want[0], c.k, c.k_scale), (want[1], c.v, c.v_scale)):
        assert torch.equal(_raw(got.cpu().contiguous()), _raw(pool.contiguous()))
        if scale is not None:
            assert torch.equal(got_scale.cpu(), scale)


@pytest.mark.parametrize("kv", [E4M3, I8])
def test_quantisation_error_and_edges(kv):
    """Every value within half a step of its code's spacing times the scale;
    tiny, huge and non-finite rows."""
    import causal_linear_attention_chunked_b200 as L
    g = torch.Generator().manual_seed(3)
    T, H, d = 40, 2, 64
    k = torch.randn(T, H, d, generator=g)
    k[1] *= 1e-37                                   # under the floor of the scale
    k[2] *= 1e36
    k[3] = 2.0 ** -149
    k[4, 0, 5] = float("nan")
    k[5, 1, 6] = -float("inf")
    c = _cache(5, 8, H, d, d, kv)
    L.kv_cache_write(c, k.cuda(), k.cuda(), torch.arange(T, dtype=torch.int32).cuda())
    codes, scale = plain.quantise(k, kv)
    assert torch.equal(_raw(c.k.cpu().flatten(0, 1)), _raw(codes))
    got = c.k_scale.cpu().transpose(1, 2).flatten(0, 1)
    assert torch.equal(torch.isnan(got), torch.isnan(scale))
    assert torch.equal(got[~torch.isnan(got)], scale[~torch.isnan(scale)])
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    back = L.kv_cache_read(c, torch.arange(5, dtype=torch.int32).cuda()[None], cu, T,
                           dtype=torch.float32)[0].cpu()
    bad = torch.isnan(scale)
    assert bool(bad[4, 0]) and bool(bad[5, 1]) and int(bad.sum()) == 2
    assert bool(torch.isnan(back[bad]).all())
    top = k.abs().amax(-1, keepdim=True)
    # half a step: e4m3 2^-4 of the value, at least half the subnormal step 2^-10
    # of the scale; int8 half of the scale; and the roundings of the scale, of
    # the quotient and of the product
    half = 0.5 * scale[..., None].double()
    if kv == E4M3:
        half = torch.maximum(k.abs().double() * 2.0 ** -4, 2.0 ** -10 * scale[..., None].double())
    tol = half * (1 + 2.0 ** -21) + top.double() * 2.0 ** -23 + 2.0 ** -149
    assert bool(((back.double() - k.double()).abs()[~bad] <= tol[~bad]).all())


@pytest.mark.parametrize("kv", [E4M3, I8])
@pytest.mark.parametrize("src,lo,step", [(torch.bfloat16, 128, 1), (torch.float16, 1024, 37)])
def test_every_quotient_of_short_significands(src, lo, step, kv):
    """Codes of every pair of bf16 significands (a row's largest value, another
    value) at 22 differences of exponent, and of a share of fp16's: those of the
    correctly rounded division, although the kernel multiplies."""
    import causal_linear_attention_chunked_b200 as L
    small = torch.arange(lo, 2 * lo, dtype=torch.float32)
    v = torch.cat([small * 2.0 ** -e for e in range(22 if lo == 128 else 12)])
    v = v[torch.arange(0, v.numel(), 1 if lo == 128 else 3)]
    v = torch.cat([v, v.new_zeros(-v.numel() % 127)]).view(-1, 127)
    for top in range(lo, 2 * lo, 16 * step):
        rows = []
        for a in range(top, min(top + 16 * step, 2 * lo), step):
            x = torch.cat([torch.full((v.shape[0], 1), float(a)), torch.clamp(v, max=float(a))], 1)
            rows.append(x / 1024)
        x = torch.cat(rows).to(src)[:, None, :]
        T = x.shape[0]
        c = _cache(-(-T // 64), 64, 1, 128, 128, kv)
        L.kv_cache_write(c, x.cuda(), (-x).cuda(), torch.arange(T, dtype=torch.int32).cuda())
        for y, pool, scale in ((x, c.k, c.k_scale), (-x, c.v, c.v_scale)):
            codes, sc = plain.quantise(y, kv)
            assert torch.equal(_raw(pool.cpu().flatten(0, 1)[:T]), _raw(codes))
            assert torch.equal(scale.cpu().transpose(1, 2).flatten(0, 1)[:T], sc)


def test_bad_slots_are_skipped_and_reported():
    import causal_linear_attention_chunked_b200 as L
    from causal_linear_attention_chunked_b200 import _binding as b
    c = _cache(3, 16, 2, 64, 64, torch.bfloat16)
    before = c.k.clone()
    k = torch.randn(4, 2, 64, device="cuda").bfloat16()
    slots = torch.tensor([48, -2, 2 ** 31 - 1, 5], dtype=torch.int32, device="cuda")
    L.kv_cache_write(c, k, k, slots)
    assert L.get_last_device_error() == b.LT_ERR_DEVICE_BAD_PAGE
    assert L.get_last_device_error() == 0
    assert torch.equal(c.k[0, 5], k[3])
    before[0, 5] = k[3]
    assert torch.equal(c.k, before)


def test_write_takes_slices_of_a_projection():
    import causal_linear_attention_chunked_b200 as L
    B, N, Hq, H, d = 2, 9, 4, 2, 128
    qkv = torch.randn(B, N, (Hq + 2 * H) * d, device="cuda").half()
    k = qkv[..., Hq * d:(Hq + H) * d].unflatten(-1, (H, d))
    v = qkv[..., (Hq + H) * d:].unflatten(-1, (H, d))
    slots = torch.randperm(32, device="cuda")[:B * N].int()
    c, c2 = _cache(2, 16, H, d, d, I8), _cache(2, 16, H, d, d, I8)
    L.kv_cache_write(c, k, v, slots)
    L.kv_cache_write(c2, k.contiguous(), v.contiguous(), slots)
    assert torch.equal(c.k, c2.k) and torch.equal(c.v, c2.v) and torch.equal(c.v_scale, c2.v_scale)


def _pages(lens, ps, extra, g):
    """A block table of shuffled pages (entries past the end: -1)."""
    need = [-(-n // ps) for n in lens]
    order = torch.randperm(max(1, sum(need)), generator=g).int()
    table = torch.full((len(lens), max(1, max(need)) + extra), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, max(1, sum(need))


def _fill(c, g):
    """Random content in every row of a cache."""
    for pool, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x = torch.randn(pool.shape, generator=g)
        if scale is None:
            pool.copy_(x.to(pool.dtype))
        else:
            codes, sc = plain.quantise(x * 3, pool.dtype)
            pool.view(torch.uint8).copy_(codes.view(torch.uint8))
            scale.copy_(sc.transpose(1, 2))


@pytest.mark.parametrize("kv,out", [
    (E4M3, torch.bfloat16), (E4M3, torch.float16), (E4M3, torch.float32), (I8, torch.bfloat16),
    (I8, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
    (torch.float32, torch.float32)])
@pytest.mark.parametrize("lens,ps,H,d,dv,layout", [
    ([1], 1, 1, 64, 64, "token"), ([0, 5, 0, 17, 64, 1, 0], 16, 3, 128, 64, "head"),
    ([100, 3, 257], 24, 2, 64, 128, "token"), ([33] * 9, 8, 8, 128, 128, "pair")])
def test_read(kv, out, lens, ps, H, d, dv, layout):
    import causal_linear_attention_chunked_b200 as L
    g = torch.Generator().manual_seed(len(lens))
    table, pages = _pages(lens, ps, 2, g)
    c = _cache(pages, ps, H, d, dv, kv, layout)
    _fill(c, g)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    N = cu[-1] + 5                                   # rows behind the last sequence
    ko = torch.full((N, H, d), 9.0, dtype=out, device="cuda")
    vo = torch.full((N, H, dv), 9.0, dtype=out, device="cuda")
    L.kv_cache_read(c, table.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), N, dtype=out,
                    k_out=ko, v_out=vo)
    assert L.get_last_device_error() == 0
    for pool, scale, got in ((c.k, c.k_scale, ko), (c.v, c.v_scale, vo)):
        pool, scale = pool.cpu(), None if scale is None else scale.cpu()
        ref = torch.cat([plain.rows_of(pool, scale, table[b], n, ps) for b, n in enumerate(lens)])
        # code x scale in fp32 is the definition: exact in 64 bits, one rounding to fp32
        assert torch.equal(got[:cu[-1]].cpu(), ref.float().to(out))
        assert bool((got[cu[-1]:] == 9.0).all())


def test_read_reports_bad_offsets_and_pages():
    import causal_linear_attention_chunked_b200 as L
    from causal_linear_attention_chunked_b200 import _binding as b
    c = _cache(4, 16, 2, 64, 64, torch.bfloat16)
    table = torch.tensor([[0, 1], [2, 3], [0, 4]], dtype=torch.int32, device="cuda")
    ok = torch.tensor([0, 20, 40, 56], dtype=torch.int32, device="cuda")
    L.kv_cache_read(c, table, ok, 56)
    assert L.get_last_device_error() == 0           # page 4 is not reached by 16 tokens
    for cu, status in (([0, 20, 40, 60], b.LT_ERR_DEVICE_BAD_PAGE),     # page 4 of 4
                       ([0, 40, 20, 56], b.LT_ERR_DEVICE_BAD_SEQLENS),  # not monotone
                       ([0, 33, 40, 56], b.LT_ERR_DEVICE_BAD_SEQLENS),  # over two pages
                       ([4, 20, 40, 56], b.LT_ERR_DEVICE_BAD_SEQLENS),
                       ([0, 20, 40, 70], b.LT_ERR_DEVICE_BAD_SEQLENS)):  # past N
        ko = torch.full((64, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        L.kv_cache_read(c, table, torch.tensor(cu, dtype=torch.int32, device="cuda"), 64,
                        k_out=ko, v_out=torch.empty_like(ko))
        assert L.get_last_device_error() == status, cu
        if status == b.LT_ERR_DEVICE_BAD_PAGE:
            assert bool((ko[56:] == 9.0).all()) and bool((ko[:56] == 3.0).all())


def test_cache_feeds_the_packed_linear_attention_passes():
    """Rows read back are the packed k, v of linear_attn_state: the state of a
    cached prefix."""
    import causal_linear_attention_chunked_b200 as L
    g = torch.Generator().manual_seed(5)
    lens, ps, H, d = [40, 0, 130], 16, 2, 64
    table, pages = _pages(lens, ps, 0, g)
    c = _cache(pages, ps, H, d, d, E4M3)
    _fill(c, g)
    cu = torch.tensor([0, 40, 40, 170], dtype=torch.int32).cuda()
    k, v = L.kv_cache_read(c, table.cuda(), cu, 170)
    S, z = L.linear_attn_state(k, v, cu_seqlens=cu)
    f = torch.nn.functional.elu(k.float()) + 1
    ref = torch.einsum("thd,the->hde", f[40:].double(), v[40:].double())
    assert bool((S[1] == 0).all())
    # bf16 operands: half a step (2^-8) per term, of the terms' sizes
    size = torch.einsum("thd,the->hde", f[40:].double(), v[40:].double().abs())
    assert bool(((S[2].double() - ref).abs() <= 2.0 ** -8 * 1.1 * size).all())


def test_streams_and_graphs():
    import causal_linear_attention_chunked_b200 as L
    g = torch.Generator().manual_seed(6)
    c = _cache(4, 16, 2, 64, 64, E4M3)
    k = torch.randn(10, 2, 64, generator=g).bfloat16().cuda()
    slots = torch.arange(10, dtype=torch.int32).cuda()
    table = torch.tensor([[0]], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 10], dtype=torch.int32).cuda()
    L.kv_cache_write(c, k, k, slots)
    ref = L.kv_cache_read(c, table, cu, 10)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    c2 = _cache(4, 16, 2, 64, 64, E4M3)
    torch.cuda.synchronize()
    L.kv_cache_write(c2, k, k, slots, stream=s)
    got = L.kv_cache_read(c2, table, cu, 10, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    k2, graph = torch.zeros_like(k), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.kv_cache_write(c2, k2, k2, slots)
        out = L.kv_cache_read(c2, table, cu, 10)
    for _ in range(2):
        k2.copy_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], ref[0])
        k2.zero_()
        graph.replay()
    assert math.isfinite(float(out[0].float().sum()))


def test_refusals_on_the_device():
    import causal_linear_attention_chunked_b200 as L
    c = _cache(2, 16, 2, 64, 64, torch.bfloat16)
    k = torch.zeros(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    slots = torch.zeros(3, device="cuda", dtype=torch.int32)
    with pytest.raises(L.LtError):
        L.kv_cache_write(c, k.half(), k.half(), slots)      # not the cache's type
    with pytest.raises(L.LtError):
        L.kv_cache_write(c, c.k.view(-1, 2, 64)[:3], k, slots)  # a row of the pool itself
    with pytest.raises(TypeError):
        L.kv_cache_write(c, k, k, slots.long())
    with pytest.raises(ValueError):
        L.kv_cache_write(c, k[:, :1], k[:, :1], slots)
    with pytest.raises(ValueError):
        L.PagedKVCache(c.k[..., ::2], c.v[..., ::2])
    with pytest.raises(ValueError):
        L.PagedKVCache(c.k.view(torch.int8), c.v.view(torch.int8))
    odd = torch.zeros(2 * 16 * 2 * 64 + 8, device="cuda", dtype=torch.bfloat16)
    shifted = L.PagedKVCache(odd[1:1 + 4096].view(2, 16, 2, 64), c.v)
    with pytest.raises(L.LtError):
        L.kv_cache_write(shifted, k, k, slots)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
def test_strides_of_single_entries_do_not_matter(dtype):
    """One head, one slot per page or one page: torch leaves such a dimension
    any stride, and no address uses it."""
    import causal_linear_attention_chunked_b200 as L
    for pages, ps in ((5, 1), (1, 5)):
        odd = (64 if pages > 1 else 3, 64 if ps > 1 else 7, 1, 1)
        k = torch.zeros(5 * 64, device="cuda").to(dtype).as_strided((pages, ps, 1, 64), odd)
        v = torch.zeros(5 * 64, device="cuda").to(dtype).as_strided((pages, ps, 1, 64), odd)
        s = [torch.ones(pages, 1, ps, device="cuda") if dtype == E4M3 else None for _ in "kv"]
        c = L.PagedKVCache(k, v, *s)
        x = torch.full((5, 1, 64), 2.0, device="cuda").bfloat16()
        x *= torch.arange(1, 6, device="cuda").view(5, 1, 1)
        L.kv_cache_write(c, x, -x, torch.arange(5, dtype=torch.int32, device="cuda"))
        table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
        cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
        kr, vr = L.kv_cache_read(c, table, cu, 5, dtype=torch.bfloat16)
        # each row holds one value m: its scale is m / 448 and its codes 448 (or m
        # itself), whose product rounds back to the bf16 value m
        assert torch.equal(kr, x) and torch.equal(vr, -x)
        out = L.paged_attn_decode(torch.zeros(1, 1, 64, device="cuda").bfloat16(), c, table,
                                  torch.tensor([5], dtype=torch.int32, device="cuda"))
        # equal weights: minus the mean of 2, 4, 6, 8, 10, within fp32 roundings
        # of the five scales and the sum, far below half a step of bf16 at 6
        assert torch.equal(out, torch.full_like(out, -6.0))


@pytest.mark.parametrize("src,kv,T,H,d,dv", [
    (torch.bfloat16, E4M3, 9001, 3, 128, 64), (torch.float16, I8, 9001, 5, 64, 128),
    (torch.float32, E4M3, 7001, 7, 128, 128), (torch.bfloat16, I8, 331, 64, 64, 64)])
def test_write_of_more_rows_than_the_device_takes_at_once(src, kv, T, H, d, dv):
    """Every warp steps through several rows, whose heads and tokens wrap; some
    tokens are skipped."""
    import causal_linear_attention_chunked_b200 as L
    g = torch.Generator().manual_seed(T + H)
    ps = 24
    pages = -(-T // ps) + 1
    c = _cache(pages, ps, H, d, dv, kv)
    k, v = (torch.randn(T, H, w, generator=g).to(src) for w in (d, dv))
    slots = torch.randperm(pages * ps, generator=g)[:T].int()
    slots[::7] = -1
    want = [torch.zeros(0)] * 4
    for i, (pool, scale, x) in enumerate(((c.k, c.k_scale, k), (c.v, c.v_scale, v))):
        rows, sc = _raw(pool.cpu()).flatten(0, 1).clone(), scale.cpu().transpose(1, 2).flatten(0, 1)
        codes, s = plain.quantise(x, kv)
        live = slots >= 0
        rows[slots[live].long()] = _raw(codes)[live]
        sc = sc.clone()
        sc[slots[live].long()] = s[live]
        want[2 * i], want[2 * i + 1] = rows, sc
    L.kv_cache_write(c, k.cuda(), v.cuda(), slots.cuda())
    assert L.get_last_device_error() == 0
    for i, (pool, scale) in enumerate(((c.k, c.k_scale), (c.v, c.v_scale))):
        assert torch.equal(_raw(pool.cpu()).flatten(0, 1), want[2 * i])
        assert torch.equal(scale.cpu().transpose(1, 2).flatten(0, 1), want[2 * i + 1])


def test_8_bit_offsets_past_32_bits():
    """8-bit pools of more than 2^32 bytes: rows written to, read from and
    attended at their end, as in a small cache."""
    import causal_linear_attention_chunked_b200 as L
    ps, H, d, T = 256, 8, 128, 300
    pages = 2 ** 32 // (ps * H * d) + 4
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(T, H, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(1, 16, d, generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    got = []
    for n in (pages, 2):
        c = L.PagedKVCache.empty(n, ps, H, d, dtype=I8)
        table = torch.tensor([[n - 1, n - 2]], dtype=torch.int32).cuda()
        at = torch.arange(T, device="cuda")
        L.kv_cache_write(c, k, v, ((n - 1 - at // ps) * ps + at % ps).int())
        got.append(L.kv_cache_read(c, table, cu, T) +
                   (L.paged_attn_decode(q, c, table, cu[1:]),))
        del c
    assert L.get_last_device_error() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
    # int8: half a step of 1/127 of the row's maximum, bf16's rounding of the
    # product, and the fp32 roundings of scale, quotient and product
    tol = k.float().abs().amax(-1, keepdim=True) * (0.5 / 127 + 2.0 ** -8 + 2.0 ** -21)
    assert bool(((got[0][0].float() - k.float()).abs() <= tol).all())
