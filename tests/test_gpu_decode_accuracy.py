"""Attention of one new token over the paged cache: what its arithmetic must
hold in 32 bits, seen through inputs whose results are known exactly."""
import pytest
import torch

from cache_plain import half_step, smallest
from test_gpu_paged_decode import BF, E4M3, F32, I8, TYPES

pytestmark = pytest.mark.gpu


def _decode(q, K, V, ks, vs, lens, ps, kv, table=None, **kw):
    """(out, lse) of sequences that lie one after another in a cache of pages of
    ps tokens, each from a page of its own on (or by `table`).  K, V [tokens, H,
    w]: values of the cache's type (codes for 8 bits), ks, vs [tokens, H]."""
    import causal_linear_attention_chunked_b200 as L
    if table is None:
        need = [max(1, -(-n // ps)) for n in lens]
        table = torch.zeros(len(lens), max(need), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.arange(at, at + n)
            at += n
    pools = [x.to(kv).view(-1, ps, *x.shape[1:]) for x in (K, V)]
    scales = [None, None]
    if kv in (E4M3, I8):
        scales = [s.float().view(-1, ps, s.shape[1]).transpose(1, 2).contiguous() for s in (ks, vs)]
    c = L.PagedKVCache(*pools, *scales)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = L.paged_attn_decode(q, c, table.cuda(), n, return_lse=True, **kw)
    assert L.get_last_device_error() == 0
    return got


def _codes(shape, kv, g):
    """Random values of the cache's type and, as [..] without the width, scales."""
    x = torch.randn(*shape, generator=g, device="cuda")
    x = torch.clamp(torch.round(40 * x), -127, 127) if kv == I8 else x.to(kv).float()
    return x, torch.rand(shape[:-1], generator=g, device="cuda") + 0.5


@pytest.mark.parametrize("qt,kv", TYPES)
@pytest.mark.parametrize("G,d,dv", [(1, 64, 64), (4, 128, 128), (12, 64, 128)])
def test_one_key_is_its_value_row(qt, kv, G, d, dv):
    """One key: its weight is 1 whatever its score, so a row comes back as it is
    held, and one of 8 bits as code x scale, rounded to fp32 (each half of the
    tensor cores' cut sum at most a step of 2^-23) and then to the output."""
    g = torch.Generator(device="cuda").manual_seed(G)
    B, H = 300, 2
    K, ks = _codes((3 * B, H, d), kv, g)
    V, vs = _codes((3 * B, H, dv), kv, g)
    q = torch.randn(B, G * H, d, generator=g, device="cuda").to(qt)
    if kv == F32:
        V[:3, 0, :4] = torch.tensor([torch.finfo(F32).max, -1.5e38, 2.0 ** -126, 1e-30])
    out, lse = _decode(q, K, V, ks, vs, [3] * B, 3, kv, window=1)
    ref = V[2::3].double() * (vs[2::3].double()[..., None] if kv in (E4M3, I8) else 1)
    ref = ref.repeat_interleave(G, 1)
    tol = half_step(qt) * ref.abs() + 2.0 ** -22 * ref.abs() if kv in (E4M3, I8) else 0
    assert bool(((out.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("qt,kv", TYPES)
@pytest.mark.parametrize("G,d", [(1, 64), (10, 128)])
def test_weights_are_held_in_32_bits(qt, kv, G, d):
    """Three keys of scores 0, -t and -t - e with values 0, 1 and -1: two weights
    that all but cancel, so that their rounding shows under the output's own.
    Each of the two (below 0.9) is off by 2^-22 of itself in the exponential, 2^-22
    in its score's three roundings, 2^-23 in its terms, the sum by 2^-23; over a
    sum of weights of 2.8 that is less than 2^-21."""
    H, B = 8, 250
    t = torch.linspace(0.1, 1.0, H * B, device="cuda").view(B, H)
    t = t if kv in (E4M3, I8) else t.to(kv).float()
    e = 2.0 ** -14
    K = torch.zeros(B, 3, H, d, device="cuda")
    V = torch.zeros(B, 3, H, d, device="cuda")
    V[:, 1], V[:, 2] = 1, -1
    ks = torch.ones(B, 3, H, device="cuda")
    q = torch.zeros(B, G * H, d, device="cuda", dtype=qt)
    q[..., 0] = 1
    if kv in (E4M3, I8):
        K[:, 1:, :, 0] = -1
        ks[:, 1], ks[:, 2] = t, t + e
        lo, hi = ks[:, 1].double(), ks[:, 2].double()
    else:
        q[..., 1] = 1
        K[:, 1:, :, 0] = -t[:, None]
        K[:, 2, :, 1] = -e
        lo, hi = t.double(), t.double() + e
    out, _ = _decode(q, K.flatten(0, 1), V.flatten(0, 1), ks.flatten(0, 1),
                     torch.ones_like(ks).flatten(0, 1), [3] * B, 3, kv, scale=1.0)
    ref = (torch.exp(-lo) - torch.exp(-hi)) / (1 + torch.exp(-lo) + torch.exp(-hi))
    ref = ref.repeat_interleave(G, 1)[..., None].expand(out.shape)
    tol = half_step(qt) * ref + 2.0 ** -21 + smallest(qt)
    assert bool(((out.double() - ref).abs() <= tol).all())


LONG = [
    # lengths, page size, query heads, KV heads, d, dv
    ([20000, 3, 1, 4097], 64, 4, 1, 128, 128), ([19999], 24, 8, 8, 64, 64),
    ([9, 40, 1, 17] * 100, 16, 8, 4, 64, 64), ([5000, 33, 700], 48, 24, 2, 64, 128),
    ([3000] * 5, 128, 17, 17, 128, 64), ([2500, 31], 16, 40, 1, 64, 64)]


@pytest.mark.parametrize("qt,kv", TYPES)
@pytest.mark.parametrize("lens,ps,Hq,H,d,dv", LONG)
def test_every_key_counts_once(qt, kv, lens, ps, Hq, H, d, dv):
    """Queries of zeros weigh every key alike: the log sum is log n (a lost or
    repeated key moves it by 1 / n, 5e-5 at most here), and columns of V that mark
    every so-manieth token, or single ones at the edges of tiles, pages and the
    sequence, come back as their share.  Weights and marks are powers of two and
    their sums whole numbers, so what rounds is the quotient (2 steps) and the
    logarithm (4 of its size in base 2)."""
    need = [max(1, -(-n // ps)) for n in lens]
    V = torch.zeros(sum(need) * ps, H, dv, device="cuda")
    want = torch.zeros(len(lens), dv, dtype=torch.float64, device="cuda")
    cols = torch.arange(dv, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        mark = (j[:, None] % dv == cols) & (cols % 2 == 0)
        edges = [0, n - 1, n - 2, n // 2, 1, 15, 16, 31, 32, 33, ps - 1, ps, 2 * ps, n - ps, 47, 48,
                 n // 3, n // 5, n // 7, n // 148, n // 149 + 1, 1023, 1024, 4095, 4096]
        edges = [x for x in edges if 0 <= x < n][:dv // 2]
        mark[torch.tensor(edges, device="cuda"),
             torch.arange(len(edges), device="cuda") * 2 + 1] = True
        V[at:at + n] = mark[:, None].float()
        want[b] = mark.sum(0).double() / n
        at += need[b] * ps
    ones = torch.ones(V.shape[:2], device="cuda")
    K = torch.ones(V.shape[0], H, d, device="cuda")
    q = torch.zeros(len(lens), Hq, d, device="cuda", dtype=qt)
    out, lse = _decode(q, K, V, ones, ones, lens, ps, kv)
    n = torch.tensor(lens, dtype=torch.float64, device="cuda")[:, None]
    assert bool(((lse.double() - n.log()).abs() <= 2.0 ** -22 * (1 + n.log2())).all())
    ref = want[:, None].expand(out.shape)
    tol = half_step(qt) * ref + 2.0 ** -22 * ref + smallest(qt)
    assert bool(((out.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("kv", [F32, E4M3, I8])
def test_long_sums_are_rounded_not_cut(kv):
    """Means of 16384 positive values: a tile's sum (a few products, each cut at
    2^-23) is added to the rest by rounded additions, so the errors of T tiles do
    not pile up on one side: their mean stays under 2^-21, their size under
    2^-21 + sqrt(T) 2^-24 (T = 1024)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    n, H, d, ps, B = 16384, 8, 64, 64, 148
    V = torch.rand(n, H, d, generator=g, device="cuda") * 0.5 + 0.5
    vs = torch.rand(n, H, generator=g, device="cuda") + 0.5
    if kv == I8:
        V = torch.round(V * 127)
    elif kv == E4M3:
        V = V.to(kv).float()
    lens = [n - b for b in range(B)]
    table = torch.arange(n // ps, dtype=torch.int32)[None].repeat(B, 1)
    q = torch.zeros(B, H, d, device="cuda")
    out, lse = _decode(q, torch.ones_like(V), V, torch.ones_like(vs), vs, lens, ps, kv, table)
    x = V.double() * (vs.double()[..., None] if kv != F32 else 1)
    sums = x.cumsum(0)
    ref = torch.stack([sums[m - 1] / m for m in lens])
    err = (out.double() - ref) / ref
    assert float(err.mean().abs()) <= 2.0 ** -21
    assert float(err.square().mean().sqrt()) <= 2.0 ** -21 + 32 * 2.0 ** -24
    m = torch.tensor(lens, dtype=torch.float64, device="cuda")[:, None]
    assert bool(((lse.double() - m.log()).abs() <= 2.0 ** -22 * (1 + m.log2())).all())


@pytest.mark.parametrize("kv,swap", [(F32, False), (F32, True), (E4M3, False), (I8, False)])
def test_scores_of_fp32_factors_that_cancel(kv, swap):
    """q = (a, -b) over a key (1, 1), or q = (1, -1) over a key (a, b): the score
    is a - b, the last few bits of 24-bit numbers, so every bit of them takes
    part.  The scale, its product and the log sum round: 2^-21 of the value."""
    g = torch.Generator(device="cuda").manual_seed(2)
    B, d = 500, 64
    a = torch.randint(2 ** 23, 2 ** 24 - 200, (B,), generator=g, device="cuda")
    m = torch.randint(1, 100, (B,), generator=g, device="cuda")
    x, y = a.double() * 2.0 ** -23, (a + m).double() * 2.0 ** -23
    q = torch.zeros(B, 1, d, device="cuda")
    K = torch.zeros(B, 1, d, device="cuda")
    if swap:
        q[:, 0, 0], q[:, 0, 1], K[:, 0, 0], K[:, 0, 1] = 1, -1, x.float(), y.float()
    else:
        q[:, 0, 0], q[:, 0, 1], K[:, 0, 0], K[:, 0, 1] = x.float(), -y.float(), 1, 1
    one = torch.ones(B, 1, device="cuda")
    _, lse = _decode(q, K, torch.ones_like(K), one, one, [1] * B, 1, kv, scale=2.0 ** 20)
    ref = -m.double()[:, None] / 8
    assert bool(((lse.double() - ref).abs() <= 2.0 ** -21 * ref.abs()).all())


def test_pieces_of_tiny_weight_and_huge_values_join():
    """Keys whose weight is 2^-127 of the largest, with values of 2^118: 2^-9 of the
    result, whichever block or warp had them.  The score's roundings move that
    share by 127 x 3 x 2^-24, and a piece that mixes both kinds (one of a
    few tiles) holds its weights to 2^-7."""
    n, d = 5000, 64
    K = torch.zeros(n, 1, d, device="cuda")
    V = torch.ones(n, 1, d, device="cuda")
    K[n // 2:, :, 0] = -127
    V[n // 2:] = 2.0 ** 118
    q = torch.zeros(1, 2, d, device="cuda")
    q[..., 0] = 1
    one = torch.ones(n, 1, device="cuda")
    out, _ = _decode(q, K, V, one, one, [n], 8, F32, scale=0.6931471805599453)
    assert bool(((out.double() - 1 - 2.0 ** -9).abs() <= 2.0 ** -20).all())


@pytest.mark.parametrize("qt,kv", [(BF, E4M3), (BF, I8), (F32, E4M3), (F32, I8)])
@pytest.mark.parametrize("exponent", [-126, -110, 100, 106])
def test_value_scales_at_the_ends_of_fp32(qt, kv, exponent):
    """Rows whose scales are the smallest, and large ones whose sum stays inside
    fp32 (6000 x 127 x 2 x 2^106 < 2^127), as the weighted sum of the formula does,
    however many warps and blocks share the sequence.  The sum's
    tiles and pieces and the quotient round: 2^-20; values below fp32's normal
    numbers to half their step, 2^-150."""
    g = torch.Generator(device="cuda").manual_seed(4)
    lens, H, d = [6000, 1, 40], 2, 64
    V, vs = _codes((6048, H, d), kv, g)
    V = V.abs()
    vs = (vs + 0.5) * 2.0 ** exponent
    q = torch.zeros(3, 2 * H, d, device="cuda", dtype=qt)
    out, _ = _decode(q, torch.ones_like(V), V, torch.ones_like(vs), vs, lens, 8, kv)
    x = V.double() * vs.double()[..., None]
    ref = torch.stack([x[:6000].mean(0), x[6000], x[6008:].mean(0)]).repeat_interleave(2, 1)
    tol = (half_step(qt) + 2.0 ** -20) * ref + 2.0 ** -150 + (smallest(qt) if qt == BF else 0)
    assert bool(torch.isfinite(out).all())
    assert bool(((out.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("kv", [BF, torch.float16, F32])
@pytest.mark.parametrize("G,d", [(1, 64), (4, 128), (12, 64)])
def test_keys_of_score_minus_infinity_have_no_weight(kv, G, d):
    """Keys that hold -infinity where the queries are positive: as if they were not
    there.  Their removal only moves other keys to other tiles, so the results
    agree within the roundings of sums (16 terms of 2^-24) and the output's."""
    g = torch.Generator(device="cuda").manual_seed(5)
    lens, H = [700, 30, 17], 2
    n = sum(lens)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(kv)
    q = r(3, G * H, d)
    q[..., 3] = q[..., 3].abs() + 0.5
    K, V = r(n, H, d), r(n, H, d).abs()
    dead = torch.rand(n, generator=g, device="cuda") < 0.3
    dead[700:730] = True                                     # a sequence of such keys alone
    hit = K.clone()
    hit[dead, :, 3] = -float("inf")
    one = torch.ones(n, H, device="cuda")
    out, lse = _decode(q, hit, V, one, one, lens, 1, kv)
    left = [int((~dead[a:b]).sum()) for a, b in ((0, 700), (700, 730), (730, n))]
    # (a page of its own for the sequence that has no key left)
    pad = lambda x: torch.cat([x[:700][~dead[:700]], x[:1], x[730:][~dead[730:]]])
    ref, ref_lse = _decode(q, pad(K), pad(V), pad(one), pad(one), left, 1, kv)
    assert bool((out[1] == 0).all()) and bool((lse[1] == -float("inf")).all())
    keep = [0, 2]
    tol = 2 * half_step(kv) * ref[keep].double().abs() + 2.0 ** -20 + smallest(kv)
    assert bool(((out[keep].double() - ref[keep].double()).abs() <= tol).all())
    assert bool(((lse[keep] - ref_lse[keep]).abs() <= 2.0 ** -20 * (1 + ref_lse[keep].abs())).all())


@pytest.mark.parametrize("qt", [BF, torch.float16])
@pytest.mark.parametrize("kv", [E4M3, I8])
def test_small_query_entries_beside_a_large_one(qt, kv):
    """q = (1, t) over a key (0, c): the score is t c, every bit of t in it, however
    small beside the head's largest entry (down to the type's own 2^-24)."""
    B, d = 300, 64
    t = (torch.logspace(-22, -4, B, base=2.0, device="cuda")).to(qt)
    q = torch.zeros(B, 1, d, device="cuda", dtype=qt)
    q[:, 0, 0], q[:, 0, 1] = 1, t
    K = torch.zeros(B, 1, d, device="cuda")
    K[:, 0, 1] = 64
    one = torch.ones(B, 1, device="cuda")
    _, lse = _decode(q, K, torch.ones_like(K), one, one, [1] * B, 1, kv, scale=2.0 ** 10)
    ref = t.double()[:, None] * 2.0 ** 16
    assert bool(((lse.double() - ref).abs() <= 2.0 ** -21 * ref).all())
