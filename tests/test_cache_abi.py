"""Host-side refusals of the norm-and-rotation, cache and decode entry points
(none of these calls reaches a CUDA API), their plans, and the binding's own
checks, on the CPU."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x100000)  # never dereferenced: every case fails before that
F2, F3, F4 = (ctypes.c_void_p(0x100000 + (i << 40)) for i in (1, 2, 3))


def _b():
    from causal_linear_attention_chunked_b200 import _binding
    return _binding


NORM = dict(q=FAKE, k=F2, qw=None, kw=None, pos=F3, n_pos=16, freq=F4, rot=64, il=0,
            qo=ctypes.c_void_p(0x700000000000), ko=ctypes.c_void_p(0x710000000000), n=16, Hq=8,
            Hkv=2, d=64, qs=512, ks=128, eps=1e-6, dtype=1, wd=1)


@pytest.mark.parametrize("case,expect", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1),
    (dict(n=0), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=70000, qs=70000 * 64), 1),
    (dict(d=96), 2), (dict(d=32), 2), (dict(rot=60), 2), (dict(rot=72), 2), (dict(rot=-8), 2),
    (dict(pos=None), 1), (dict(freq=None), 1), (dict(n_pos=0), 1), (dict(n_pos=5), 1),
    (dict(il=2), 1), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(qs=504), 1), (dict(qs=511), 1), (dict(ks=129), 1), (dict(qs=1 << 50), 1),
    (dict(dtype=3), 2), (dict(wd=2), 2), (dict(dtype=0, wd=1), 2),
    (dict(q=ctypes.c_void_p(0x100008)), 1), (dict(qw=ctypes.c_void_p(0x100008)), 1),
    (dict(qo=FAKE), 1),                                    # over an input
    (dict(qo=ctypes.c_void_p(0x710000000010)), 1),         # over the other output
    (dict(ko=F3), 1), (dict(n=1 << 40), 1),
])
def test_norm_rope_rejects(case, expect):
    a = dict(NORM, **case)
    st = _b().lib.lt_qk_norm_rope(a["q"], a["k"], a["qw"], a["kw"], a["pos"], a["n_pos"],
                                  a["freq"], a["rot"], a["il"], a["qo"], a["ko"], a["n"], a["Hq"],
                                  a["Hkv"], a["d"], a["qs"], a["ks"], a["eps"], None, a["dtype"],
                                  a["wd"])
    assert st == expect


BWD = dict(NORM, gq=ctypes.c_void_p(0x400000000000), gk=ctypes.c_void_p(0x410000000000),
           dqs=512, dks=128, dqw=None, dkw=None, ws=None, wsb=0)


@pytest.mark.parametrize("case,expect", [
    (dict(gq=None), 1), (dict(gk=None), 1), (dict(qo=None), 1), (dict(d=96), 2),
    (dict(eps=-1.0), 1), (dict(dqs=504), 1), (dict(dks=100), 1), (dict(qo=FAKE), 1),
    (dict(qo=ctypes.c_void_p(0x400000000000)), 1),
    # dq, dk as slices of one gradient: rows that touch, and different strides
    (dict(dqs=640, dks=640, ko=ctypes.c_void_p(0x700000000000 + 511 * 2 - 14)), 1),
    (dict(dqs=640, dks=648, ko=ctypes.c_void_p(0x700000000000 + 512 * 2)), 1),
    (dict(dqw=ctypes.c_void_p(0x700000000002)), 1),
    (dict(dqw=FAKE), 1), (dict(rot=12), 2), (dict(dtype=9), 2),
])
def test_norm_rope_bwd_rejects(case, expect):
    a = dict(BWD, **case)
    st = _b().lib.lt_qk_norm_rope_bwd(a["gq"], a["gk"], a["q"], a["k"], a["qw"], a["kw"], a["pos"],
                                      a["n_pos"], a["freq"], a["rot"], a["il"], a["qo"], a["ko"],
                                      a["dqw"], a["dkw"], a["n"], a["Hq"], a["Hkv"], a["d"],
                                      a["qs"], a["ks"], a["dqs"], a["dks"], a["eps"], a["ws"],
                                      a["wsb"], None, a["dtype"], a["wd"])
    assert st == expect


def _cache(**over):
    """A bf16 cache of 4 pages of 16 tokens, 2 heads of 64; fields replaced by name."""
    f = dict(k=0x500000000000, v=0x510000000000, k_scale=None, v_scale=None,
             k_page_stride=16 * 128, k_slot_stride=128, k_head_stride=64,
             v_page_stride=16 * 128, v_slot_stride=128, v_head_stride=64,
             num_pages=4, page_size=16, H_kv=2, d=64, dv=64, dtype=1)
    f.update(over)
    return _b().KvCacheStruct(*[f[n] for n, _ in _b().KvCacheStruct._fields_])


BAD_CACHES = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=0x500000000008), 1), (dict(num_pages=0), 1),
    (dict(page_size=0), 1), (dict(page_size=65537), 1), (dict(H_kv=0), 1), (dict(d=48), 2),
    (dict(dv=32), 2), (dict(dtype=5), 2), (dict(dtype=-1), 2), (dict(k_slot_stride=32), 1),
    (dict(k_head_stride=60), 1), (dict(v_page_stride=-2048), 1), (dict(v_slot_stride=132), 1),
    (dict(k_page_stride=1 << 60), 1), (dict(k_scale=0x520000000000), 1),
    (dict(dtype=3), 1),                                   # 8 bits without scales
    (dict(dtype=4, k_scale=0x520000000000), 1),
    (dict(num_pages=1 << 30), 1),                         # slots past 32 bits
    (dict(dtype=2), 2), (dict(dtype=0), 2),               # not the tensors' type
]


@pytest.mark.parametrize("over,expect", BAD_CACHES)
def test_every_entry_refuses_a_bad_cache(over, expect):
    lib = _b().lib
    c = ctypes.byref(_cache(**over))
    assert lib.lt_kv_cache_write(c, FAKE, F2, F3, 8, 128, 128, None, 1) == expect
    assert lib.lt_kv_cache_read(c, FAKE, 4, 4, F2, 3, 64, F3, F4, None, 1) == expect
    assert lib.lt_paged_attn_decode(FAKE, c, F2, 4, 4, F3, 3, 8, 0.125, 0, F4, None, None, 0,
                                    None, 1) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(n=0), 1),
    (dict(ks=64), 1), (dict(vs=132), 1), (dict(dtype=4), 2), (dict(dtype=0), 2),
    (dict(k=ctypes.c_void_p(0x500000000100)), 1), (dict(slots=ctypes.c_void_p(0x510000000000)), 1),
    (dict(cache=None), 1), (dict(slots=ctypes.c_void_p(0x100002)), 1),
])
def test_write_rejects(case, expect):
    a = dict(cache=ctypes.byref(_cache()), k=FAKE, v=F2, slots=F3, n=8, ks=128, vs=128, dtype=1)
    a.update(case)
    assert _b().lib.lt_kv_cache_write(a["cache"], a["k"], a["v"], a["slots"], a["n"], a["ks"],
                                      a["vs"], None, a["dtype"]) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(table=None), 1), (dict(cu=None), 1), (dict(ko=None), 1), (dict(vo=None), 1),
    (dict(B=0), 1), (dict(N=0), 1), (dict(pages=0), 1), (dict(stride=3), 1),
    (dict(stride=1 << 50), 1), (dict(dtype=0), 2), (dict(ko=ctypes.c_void_p(0x500000000400)), 1),
    (dict(vo=F3), 1), (dict(ko=F2), 1), (dict(ko=ctypes.c_void_p(0x100008)), 1),
])
def test_read_rejects(case, expect):
    a = dict(table=FAKE, stride=4, pages=4, cu=F2, B=3, N=64, ko=F3, vo=F4, dtype=1)
    a.update(case)
    assert _b().lib.lt_kv_cache_read(ctypes.byref(_cache()), a["table"], a["stride"], a["pages"],
                                     a["cu"], a["B"], a["N"], a["ko"], a["vo"], None,
                                     a["dtype"]) == expect


@pytest.mark.parametrize("case,expect", [
    (dict(q=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(out=None), 1),
    (dict(B=0), 1), (dict(B=70000), 1), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(Hq=70000), 1),
    (dict(pages=0), 1), (dict(stride=3), 1), (dict(window=-1), 1), (dict(scale=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(dtype=5), 2), (dict(dtype=2), 2), (dict(out=FAKE), 1),
    (dict(lse=F4), 1), (dict(lse=F3), 1), (dict(out=ctypes.c_void_p(0x510000000000)), 1),
    (dict(ws=F4, wsb=1 << 20), 1), (dict(ws=FAKE, wsb=1 << 20), 1), (dict(lens=F4), 1),
])
def test_decode_rejects(case, expect):
    a = dict(q=FAKE, table=F2, stride=4, pages=4, lens=F3, B=3, Hq=8, scale=0.125, window=0,
             out=F4, lse=None, ws=None, wsb=0, dtype=1)
    a.update(case)
    assert _b().lib.lt_paged_attn_decode(a["q"], ctypes.byref(_cache()), a["table"], a["stride"],
                                         a["pages"], a["lens"], a["B"], a["Hq"], a["scale"],
                                         a["window"], a["out"], a["lse"], a["ws"], a["wsb"], None,
                                         a["dtype"]) == expect


def test_plans():
    lib = _b().lib
    n = ctypes.c_size_t()
    assert lib.lt_paged_attn_decode_plan(32, 8, 128, 128, 1, 1, 148, ctypes.byref(n)) == 0
    # two pieces of 4 query heads (values, maximum and sum) per warp and per
    # unit, and 16 bytes, per block
    assert n.value == 148 * ((8 + 8) * 2 * 4 * (128 + 2) * 4 + 16)
    assert lib.lt_paged_attn_decode_plan(64, 1, 128, 128, 1, 3, 148, ctypes.byref(n)) == 0
    # 16 query heads per unit at most: four units of one KV head
    assert n.value == 148 * ((8 + 4) * 2 * 16 * (128 + 2) * 4 + 16)
    assert lib.lt_paged_attn_decode_plan(8, 8, 64, 128, 1, 3, 148, ctypes.byref(n)) == 0
    assert n.value == 148 * ((8 + 8) * 2 * 1 * (128 + 2) * 4 + 16)
    for args, st in (((32, 5, 128, 128, 1, 1, 148), 1), ((32, 8, 96, 128, 1, 1, 148), 2),
                     ((32, 8, 128, 128, 1, 2, 148), 2), ((32, 8, 128, 128, 3, 3, 148), 2),
                     ((0, 8, 128, 128, 1, 1, 148), 1)):
        assert lib.lt_paged_attn_decode_plan(*args, ctypes.byref(n)) == st
    assert lib.lt_paged_attn_decode_plan(32, 8, 128, 128, 1, 1, 148, None) == 1
    # one row of sums per block, at most two blocks per SM; tokens do not count
    assert lib.lt_qk_norm_rope_bwd_plan(128, 148, ctypes.byref(n)) == 0
    assert n.value == 2 * 148 * 2 * 128 * 4
    assert lib.lt_qk_norm_rope_bwd_plan(80, 148, ctypes.byref(n)) == 2
    assert lib.lt_qk_norm_rope_bwd_plan(64, 148, None) == 1


def test_token_layouts():
    from causal_linear_attention_chunked_b200.kv_cache import _tokens
    x = torch.zeros(2, 5, 12 * 64)
    assert _tokens(x.unflatten(-1, (12, 64)), "x") == (10, 12, 64, 768)
    q = x[..., :512].unflatten(-1, (8, 64))
    assert _tokens(q, "q") == (10, 8, 64, 768)
    assert _tokens(q[:, 1:2], "q") == (2, 8, 64, 5 * 768)     # one token of each row
    assert _tokens(q[1, 2:4], "q") == (2, 8, 64, 768)
    with pytest.raises(ValueError):
        _tokens(q[:, 1:3], "q")                              # unevenly spaced
    with pytest.raises(ValueError):
        _tokens(q.transpose(1, 2), "q")
    with pytest.raises(ValueError):
        _tokens(q[..., ::2], "q")
    with pytest.raises(ValueError):
        _tokens(x[0], "x")                                   # no heads


def test_binding_refuses_cpu_tensors_and_wrong_types():
    import causal_linear_attention_chunked_b200 as lt
    q, k = torch.zeros(4, 8, 64), torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        lt.qk_norm_rope(q, k)
    with pytest.raises(TypeError):
        lt.qk_norm_rope(q, k.half())
    with pytest.raises(ValueError):
        lt.qk_norm_rope(q, k[:3])
    with pytest.raises(ValueError):
        lt.qk_norm_rope(q, k, positions=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError):
        lt.qk_norm_rope(q, k, positions=torch.zeros(4), inv_freq=torch.zeros(8))
    with pytest.raises(ValueError):
        lt.qk_norm_rope(q, k, positions=torch.zeros(3, dtype=torch.int32), inv_freq=torch.zeros(8))
    with pytest.raises(ValueError):
        lt.qk_norm_rope(q, k, torch.zeros(63))
    pool = torch.zeros(2, 16, 2, 64)
    with pytest.raises(ValueError):
        lt.PagedKVCache(pool, pool)
    with pytest.raises(TypeError):
        lt.PagedKVCache(pool.double(), pool.double())
    with pytest.raises(ValueError):
        lt.PagedKVCache(pool, pool[:1])


def test_limits_of_counts():
    """Counts whose tiles or sequences would pass the kernels' 31-bit indices."""
    lib = _b().lib
    c = ctypes.byref(_cache())
    assert lib.lt_kv_cache_read(c, FAKE, 4, 4, F2, (1 << 30) + 1, 64, F3, F4, None, 1) == 1

    def decode(B, pages, Hq):
        return lib.lt_paged_attn_decode(FAKE, c, F2, pages, pages, F3, B, Hq, 0.125, 0, F4, None,
                                        None, 0, None, 1)
    assert decode(65535, 32768, 2) == 1           # 2^31 - 2^15 tiles of 16 tokens and 65535 more
    assert decode(65535, 17, 65534) == 1          # 2^20 tiles, 65534 heads: over 2^36
    assert _b().lib.lt_status_string(7) != _b().lib.lt_status_string(5)


def test_plan_of_narrow_8_bit_rows():
    """Rows of 64 + 64 bytes: sixteen warps per block, eight under fp32 queries."""
    lib, n = _b().lib, ctypes.c_size_t()
    assert lib.lt_paged_attn_decode_plan(8, 8, 64, 64, 1, 3, 148, ctypes.byref(n)) == 0
    assert n.value == 148 * ((16 + 8) * 2 * 1 * (64 + 2) * 4 + 16)
    assert lib.lt_paged_attn_decode_plan(8, 8, 64, 64, 0, 3, 148, ctypes.byref(n)) == 0
    assert n.value == 148 * ((8 + 8) * 2 * 1 * (64 + 2) * 4 + 16)
