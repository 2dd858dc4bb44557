"""lt_qk_norm_rope_bwd: what its workspace must not be."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
T, HQ, HKV, D = 50, 4, 2, 64


def _tensors():
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    return dict(gq=r(T, HQ, D), gk=r(T, HKV, D), q=r(T, HQ, D), k=r(T, HKV, D), wq=r(D), wk=r(D),
                pos=torch.arange(T, dtype=torch.int32, device="cuda"),
                freq=torch.rand(D // 2, generator=g, device="cuda"))


def _call(a, ws, ws_bytes, gains=True):
    from causal_linear_attention_chunked_b200 import _binding as b
    P = lambda t: t if t is None or isinstance(t, ctypes.c_void_p) else ctypes.c_void_p(t.data_ptr())
    out = [torch.zeros(T, HQ, D, device="cuda").bfloat16(),
           torch.zeros(T, HKV, D, device="cuda").bfloat16(),
           *(torch.zeros(D, device="cuda").bfloat16() if gains else None for _ in "qk")]
    st = b.lib.lt_qk_norm_rope_bwd(
        P(a["gq"]), P(a["gk"]), P(a["q"]), P(a["k"]), P(a["wq"]), P(a["wk"]), P(a["pos"]), T,
        P(a["freq"]), D, 0, *(P(o) for o in out), T, HQ, HKV, D, HQ * D, HKV * D, HQ * D, HKV * D,
        1e-6, P(ws), ws_bytes, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), 1, 1)
    torch.cuda.synchronize()
    return st, out


def _plan():
    from causal_linear_attention_chunked_b200 import _binding as b
    need = ctypes.c_size_t()
    assert b.lib.lt_qk_norm_rope_bwd_plan(D, 0, ctypes.byref(need)) == 0
    return need.value


@pytest.mark.parametrize("name", ["gq", "gk", "q", "k", "wq", "wk", "pos", "freq"])
def test_a_workspace_over_an_input_is_refused(name):
    """Each input in the workspace's last bytes: refused, and nothing written; beside
    it, or under it where no gain's gradient is asked for: taken."""
    a = _tensors()
    need = -(-_plan() // 256) * 256
    x = a[name]
    size = x.numel() * x.element_size()
    room = torch.zeros(need + size, dtype=torch.uint8, device="cuda")
    inside = room[need - 16:need - 16 + size]
    a[name] = inside.view(x.dtype).view(x.shape)
    a[name].copy_(x)
    st, out = _call(a, room, need)
    assert st == 1 and torch.equal(a[name], x) and not any(bool(o.any()) for o in out)
    st, out = _call(a, room, need, gains=False)
    assert st == 0 and torch.equal(a[name], x) and bool(out[0].any())
    beside = room[need:].view(x.dtype).view(x.shape)
    a[name] = beside.copy_(x)
    st, out = _call(a, room, need)
    assert st == 0 and torch.equal(a[name], x)
    ref = _call(_tensors(), None, 0)
    assert ref[0] == 0 and all(torch.equal(p, r) for p, r in zip(out, ref[1]))


def test_host_inputs_are_refused_whatever_the_workspace():
    """An input on the host is refused, also where the workspace, not used
    without gains, has its address."""
    a = _tensors()
    host = torch.zeros(T, HQ, D).bfloat16()
    at = ctypes.c_void_p(-(-host.data_ptr() // 16) * 16)
    for ws in (at, None):
        assert _call(dict(a, q=at), ws, 1 << 20, gains=False)[0] == 1
