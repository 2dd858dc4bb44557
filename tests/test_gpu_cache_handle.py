"""PagedKVCache when its pools are replaced, or their memory moves."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn
PS, H, D = 16, 2, 64


def _step(c, page, seed):
    """Four tokens into the end of `page`, and back: (keys as read, keys)."""
    import causal_linear_attention_chunked_b200 as L
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(4, H, D, generator=g, device="cuda").bfloat16()
    k[..., 0] = 448.0                      # (the scale 1: e4m3 values come back as themselves)
    k = k.to(E4M3).to(BF)
    slots = torch.arange(4, dtype=torch.int32, device="cuda") + page * PS
    L.kv_cache_write(c, k, k, slots)
    table = torch.tensor([[page]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    kr, vr = L.kv_cache_read(c, table, cu, 4)
    out = L.paged_attn_decode(torch.zeros(1, H, D, device="cuda").bfloat16(), c, table, cu[1:])
    assert L.get_last_device_error() == 0
    assert torch.equal(kr, vr) and torch.equal(kr, k)
    # (equal weights: the mean of the four, within its roundings)
    off = (out[0].float() - k.float().mean(0)).abs()
    assert bool((off <= 2.0 ** -8 * k.float().abs().mean(0)).all())


def _parts(c):
    return [t for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]


@pytest.mark.parametrize("dtype", [BF, E4M3])
def test_pools_replaced_by_larger_ones(dtype):
    import causal_linear_attention_chunked_b200 as L
    c = L.PagedKVCache.empty(2, PS, H, D, dtype=dtype)
    for t in _parts(c):
        t.zero_()
    _step(c, 1, 1)
    old = _parts(c)
    kept = [t.clone() for t in old]
    big = L.PagedKVCache.empty(7, PS, H, D, dtype=dtype)
    c.k, c.v = big.k, big.v
    if dtype == E4M3:
        with pytest.raises(ValueError):
            _step(c, 1, 2)                 # the scales are still the small pools'
        c.k_scale, c.v_scale = big.k_scale, big.v_scale
    assert c.num_pages == 7 and c.k is big.k
    _step(c, 6, 2)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(old, kept))
    c.v = big.v[:3]
    with pytest.raises(ValueError):
        _step(c, 1, 3)
    c.v = big.v.half()
    with pytest.raises((TypeError, ValueError)):
        _step(c, 1, 3)


@pytest.mark.parametrize("dtype", [BF, E4M3])
def test_pools_grown_in_place(dtype):
    import causal_linear_attention_chunked_b200 as L
    c = L.PagedKVCache.empty(2, PS, H, D, dtype=dtype)
    _step(c, 1, 4)
    at = c.k.data_ptr()
    for t in _parts(c):
        t.resize_(60000, *t.shape[1:])
    assert c.k.data_ptr() != at and c.num_pages == 60000
    _step(c, 59999, 5)


def test_a_pool_whose_memory_is_exchanged():
    """set_ to other storage under the same tensor objects: rows go to the new one."""
    import causal_linear_attention_chunked_b200 as L
    c = L.PagedKVCache.empty(4, PS, H, D, dtype=BF)
    old = [c.k.clone().zero_(), c.v.clone().zero_()]
    new = [torch.zeros_like(t) for t in old]
    c.k.set_(old[0])
    c.v.set_(old[1])
    _step(c, 3, 6)
    kept = old[0].clone()
    c.k.set_(new[0])
    c.v.set_(new[1])
    _step(c, 2, 7)
    assert torch.equal(old[0], kept) and bool(new[0][2, 0].any())
