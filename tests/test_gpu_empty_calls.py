"""Norm, cache and decode calls that have nothing to do."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn
H, HQ, D, DV = 2, 4, 64, 128
i32 = lambda *x, shape=None: torch.tensor(x, dtype=torch.int32, device="cuda").view(shape or (len(x),))


def _cache(dtype):
    import causal_linear_attention_chunked_b200 as L
    c = L.PagedKVCache.empty(3, 16, H, D, DV, dtype=dtype)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        if t is not None:
            t.zero_()
    return c


@pytest.mark.parametrize("other_stream", [False, True])
@pytest.mark.parametrize("dtype", [BF, E4M3])
def test_cache_calls_of_nothing(dtype, other_stream):
    import causal_linear_attention_chunked_b200 as L
    c = _cache(dtype)
    kw = dict(stream=torch.cuda.Stream()) if other_stream else {}
    z = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")
    L.kv_cache_write(c, z(0, H, D), z(0, H, DV), i32(), **kw)                # no tokens
    L.kv_cache_write(c, z(2, 0, H, D), z(2, 0, H, DV), i32(), **kw)
    assert not any(bool(t.view(torch.uint8).any()) for t in (c.k, c.v))
    # a batch of empty sequences, and one of none
    for table, cu in ((i32(0, 1, shape=(2, 1)), i32(0, 0, 0)), (i32(shape=(0, 1)), i32(0))):
        k, v = L.kv_cache_read(c, table, cu, 0, **kw)
        assert k.shape == (0, H, D) and v.shape == (0, H, DV) and k.dtype == v.dtype == BF
    ko, vo = z(5, H, D) + 9, z(5, H, DV) + 9                                 # rows of nobody
    got = L.kv_cache_read(c, i32(shape=(0, 1)), i32(0), 5, k_out=ko, v_out=vo, **kw)
    assert got[0] is ko and bool((ko == 9).all()) and bool((vo == 9).all())
    for lse in (False, True):
        out = L.paged_attn_decode(z(0, HQ, D), c, i32(shape=(0, 1)), i32(), return_lse=lse, **kw)
        out, l = out if lse else (out, None)
        assert out.shape == (0, HQ, DV) and out.dtype == BF
        assert l is None or (l.shape == (0, HQ) and l.dtype == torch.float32)
    assert L.get_last_device_error() == 0
    with pytest.raises(ValueError):
        L.kv_cache_write(c, z(0, H + 1, D), z(0, H + 1, DV), i32())          # checked all the same
    with pytest.raises(ValueError):
        L.paged_attn_decode(z(0, HQ, DV), c, i32(shape=(0, 1)), i32())


@pytest.mark.parametrize("shape", [(0,), (3, 0)])
def test_norm_of_nothing(shape):
    import causal_linear_attention_chunked_b200 as L
    q = torch.zeros(*shape, HQ, D, dtype=BF, device="cuda")
    k = torch.zeros(*shape, H, D, dtype=BF, device="cuda")
    w = torch.ones(D, device="cuda")
    freq = torch.ones(D // 2, device="cuda")
    qo, ko = L.qk_norm_rope(q, k, w, w, i32(), freq)
    assert qo.shape == q.shape and ko.shape == k.shape
    dq, dk, dqw, dkw = L.qk_norm_rope_bwd(qo, ko, q, k, w, None, i32(), freq)
    assert dq.shape == q.shape and dk.shape == k.shape and dkw is None
    assert dqw.shape == w.shape and not bool(dqw.any())
    assert L.get_last_device_error() == 0
