"""Norm and rotation: the angle's accuracy in fp32, and few tokens."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
def test_fp32_angles_are_held_in_fp32(interleaved):
    """Rows whose mean square is 1 and whose pairs are (1, 0) come back as the
    cosine and sine themselves.  Correctly rounded ones have errors of at most 2^-25,
    1.5e-8 in the mean square; the fp32 functions are off by a step or so at
    most (2^-23 beside the rounding's) and 1.6 times that in the mean square.  An
    angle rounded to fp32 turns is off by up to 9e-8 by itself."""
    import causal_linear_attention_chunked_b200 as L
    T, d, rot = 4000, 128, 64
    g = torch.Generator().manual_seed(1)
    x = torch.zeros(T, 1, d)
    first = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    second = first + 1 if interleaved else first + rot // 2
    x[..., first] = 1.0                  # 32 ones in the pairs, 32 ones and 16 twos behind them:
    x[..., rot:rot + 32] = 1.0           # 128 in all
    x[..., rot + 32:rot + 48] = 2.0
    pos = torch.randint(0, 200000, (T,), generator=g).int()
    freq = (10000.0 ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / rot)).float()
    # (the smallest eps: the mean plus it rounds to the mean)
    out = L.qk_norm_rope(x.cuda(), x.cuda(), None, None, pos.cuda(), freq.cuda(), eps=1e-30,
                         interleaved=interleaved)
    ang = pos.double()[:, None] * freq.double()
    for y in out:
        y = y[:, 0].cpu().double()
        assert bool((y[:, rot:] == x[:, 0, rot:]).all())
        for got, ref in ((y[:, first], torch.cos(ang)), (y[:, second], torch.sin(ang))):
            err = (got - ref).abs()
            assert float(err.max()) <= 2.0 ** -23 + 2.0 ** -25
            assert float(err.square().mean().sqrt()) <= 1.6 * 1.5e-8


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [200, 600, 790, 1184, 1185])
def test_tokens_whose_heads_several_warps_share(T, dtype):
    """Token counts around the steps of how many warps share a token, both
    directions (32 + 8 heads of 128: several batches each)."""
    import cache_plain as plain
    import causal_linear_attention_chunked_b200 as L
    g = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype)
    q, k, gq, gk = r(T, 32, 128), r(T, 8, 128), r(T, 32, 128), r(T, 8, 128)
    wq, wk = r(128), r(128)
    pos = torch.randint(0, 100000, (T,), generator=g).int()
    freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float()
    dev = [t.cuda() for t in (gq, gk, q, k, wq, wk, pos, freq)]
    out, got = L.qk_norm_rope(*dev[2:]), L.qk_norm_rope_bwd(*dev)
    for i, (x, w, up) in enumerate(((q, wq, gq), (k, wk, gk))):
        plain.check(out[i], *plain.norm_rope(x, w, pos, freq, 1e-6, False), dtype, "out %d" % i)
        (dx, dxb), (dw, dwb) = plain.norm_rope_bwd(up, x, w, pos, freq, 1e-6, False)
        plain.check(got[i], dx, dxb, dtype, "dx %d" % i)
        plain.check(got[2 + i], dw, dwb, dtype, "dw %d" % i)
