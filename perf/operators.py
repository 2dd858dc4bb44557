"""Measured cases of the softmax-attention serving operators and of the query
and key preparation that feeds them and the linear-attention passes.

Operators (a case's ``op``):

* ``norm_rope``      root-mean-square norm of every query and key head, gain,
                     and the position rotation, in one pass;
* ``norm_rope_bwd``  its backward pass (dq, dk and the gains' gradients);
* ``cache_write``    new keys and values into a paged cache, quantised to
                     8 bits per (token, head) row where the cache holds 8 bits;
* ``cache_read``     a batch of sequences read back from the cache, packed;
* ``decode``         softmax attention of one new token per sequence over the
                     paged cache.

``run`` takes what ``prepare`` returns and computes the operator either in its
plain form (elementary torch operations in 32 bits, angles in 64) or, where
``own`` is true, through this package.  ``exact`` computes it in 64 bits.
Widths and head counts are those of this repository's workloads: 8 heads of
64, and 32 query heads over 8 key heads of 128.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
      "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
QMAX = {"e4m3": 448.0, "int8": 127.0}
EPS = 1e-6
TINY = 2.0 ** -126   # the smallest scale of a quantised row


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the queries and keys of one decode step of a batch of 64
        dict(name="norm_rope_step_b64", op="norm_rope", B=64, N=1, Hq=32, Hkv=8, d=128, rot=128,
             dtype="bf16", interleaved=False, fused=True, start=30000),
        # a prompt batch: slices of the fused q, k, v projection, far positions
        dict(name="norm_rope_prompt_2x16384", op="norm_rope", B=2, N=16384, Hq=32, Hkv=8, d=128,
             rot=128, dtype="bf16", interleaved=False, fused=True, start=100000),
        # training: the sequence length and heads of the grouped-query workload
        dict(name="norm_rope_bwd_2x8192", op="norm_rope_bwd", B=2, N=8192, Hq=32, Hkv=8, d=128,
             rot=128, dtype="bf16", interleaved=False, fused=True, start=0),
        # training, fp32 gradients of a short odd batch; half of the width rotated, in
        # neighbouring pairs
        dict(name="norm_rope_bwd_f32", op="norm_rope_bwd", B=3, N=1023, Hq=8, Hkv=8, d=64, rot=32,
             dtype="f32", interleaved=True, fused=False, start=0),
        # one decode step appends a token to each of 64 sequences
        dict(name="cache_write_step_b64", op="cache_write", T=64, Hkv=8, d=128, dv=128,
             dtype="bf16", kv="e4m3", ps=64, pool=8192, append=True),
        # a prompt batch quantised on its way into the cache
        dict(name="cache_write_prompt_32768", op="cache_write", T=32768, Hkv=8, d=128, dv=128,
             dtype="bf16", kv="e4m3", ps=64, pool=33024, append=False),
        # 64 ragged sequences read back from 8 bits (prefix reuse)
        dict(name="cache_read_64_ragged", op="cache_read", B=64, lo=128, hi=8192, lens=5, Hkv=8,
             d=64, dv=64, dtype="bf16", kv="e4m3", ps=64),
        # one short sequence read back, small pages
        dict(name="cache_read_1_len1001", op="cache_read", B=1, lo=1001, hi=1001, lens=2, Hkv=8,
             d=128, dv=128, dtype="f16", kv="int8", ps=16),
        # a single short conversation: latency
        dict(name="decode_b1_len777", op="decode", B=1, lo=777, hi=777, lens=1, Hq=8, Hkv=8, d=64,
             dv=64, dtype="bf16", kv="bf16", ps=16, window=0, lse=False),
        # a serving batch of 64 ragged sequences
        dict(name="decode_b64_ragged", op="decode", B=64, lo=128, hi=8192, lens=5, Hq=32, Hkv=8,
             d=128, dv=128, dtype="bf16", kv="bf16", ps=64, window=0, lse=False),
        # the same batch over an 8-bit cache
        dict(name="decode_b64_ragged_e4m3", op="decode", B=64, lo=128, hi=8192, lens=5, Hq=32,
             Hkv=8, d=128, dv=128, dtype="bf16", kv="e4m3", ps=64, window=0, lse=False),
        # one long sequence, its logarithm of the sum returned for joining
        dict(name="decode_b1_len65536", op="decode", B=1, lo=65536, hi=65536, lens=3, Hq=32,
             Hkv=8, d=128, dv=128, dtype="bf16", kv="bf16", ps=128, window=0, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "cache_write", "cache_read", "decode",
                     "decode"])
    d = rng.choice([64, 128])
    dv = rng.choice([d, d, 192 - d])
    Hkv = rng.choice([1, 2, 3, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("norm_rope", "norm_rope_bwd"):
        size = {"bf16": 2, "f16": 2, "f32": 4}[dtype]
        passes = 2 if op == "norm_rope" else 3
        most = 6e8 / ((Hq + Hkv) * d * size * passes)
        tokens = _log(rng, 1, min(40000, most))
        B = rng.choice([1, 2, 3, 64]) if tokens >= 64 else 1
        return dict(op=op, B=B, N=max(1, tokens // B), Hq=Hq, Hkv=Hkv, d=d,
                    rot=rng.choice([d, d, d // 2, 16, 0]), dtype=dtype,
                    interleaved=rng.random() < 0.4, fused=rng.random() < 0.5,
                    start=_log(rng, 1, 1000000))
    kv = rng.choice([dtype, "e4m3", "int8"])
    ps = rng.choice([1, 8, 16, 24, 64, 128, 256])
    if op == "cache_write":
        T = _log(rng, 1, 32000)
        return dict(op=op, T=T, Hkv=Hkv, d=d, dv=dv, dtype=dtype, kv=kv, ps=ps,
                    pool=-(-T // ps) * ps + ps * rng.randint(0, 8), append=rng.random() < 0.4)
    if op == "cache_read":
        B = _log(rng, 1, 64)
        hi = _log(rng, 16, min(8192, 250000 // B))
        return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, lens=rng.randint(0, 10 ** 6),
                    Hkv=Hkv, d=d, dv=dv, dtype=dtype, kv=kv, ps=ps)
    B = _log(rng, 1, 128)
    hi = _log(rng, 1, min(65536, 250000 // B))
    if kv == "f32":
        hi = max(1, hi // 2)
    return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, lens=rng.randint(0, 10 ** 6), Hq=Hq,
                Hkv=Hkv, d=d, dv=dv, dtype=dtype, kv=kv, ps=ps,
                window=rng.choice([0, 0, 0, 1, 513]), lse=rng.random() < 0.3)


def _lengths(c):
    """The sequence lengths of a case: part of the case, not of the seed."""
    r = random.Random(c["lens"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]


def _bytes(name):
    return {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1, "int8": 1}[name]


def work(c):
    es = _bytes(c["dtype"])
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        tokens = c["B"] * c["N"]
        rows = tokens * (c["Hq"] + c["Hkv"])
        vals = rows * c["d"]
        small = 4 * tokens + 2 * c["rot"] + 2 * c["d"] * es
        if c["op"] == "norm_rope":
            return {"bytes": 2 * vals * es + small, "flops": 4 * vals + 3 * rows * c["rot"]}
        return {"bytes": 3 * vals * es + small + 2 * c["d"] * es,
                "flops": 11 * vals + 3 * rows * c["rot"]}
    ks = _bytes(c["kv"])
    row = c["d"] + c["dv"]                       # values of one (token, head), keys and values
    scales = 8 if c["kv"] in QMAX else 0
    if c["op"] == "cache_write":
        rows = c["T"] * c["Hkv"]
        return {"bytes": rows * (row * (es + ks) + scales) + 4 * c["T"], "flops": 2 * rows * row}
    lens = _lengths(c)
    if c["op"] == "cache_read":
        rows = sum(lens) * c["Hkv"]
        return {"bytes": rows * (row * (es + ks) + scales), "flops": rows * row}
    keys = sum(min(n, c["window"]) if c["window"] else n for n in lens)
    return {"bytes": keys * c["Hkv"] * (row * ks + scales) + c["B"] * c["Hq"] * row * es,
            "flops": 2 * keys * c["Hq"] * row}


# ---------------------------------------------------------------- inputs
def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _quant(x, kv):
    """Codes and scales of rows x [..., w]: scale = max|x| / qmax, at least 2^-126."""
    x = x.float()
    top = torch.full((), QMAX[kv], device=x.device)
    scale = torch.clamp(x.abs().amax(-1) / top, min=TINY)
    y = x / scale.unsqueeze(-1)
    if kv == "int8":
        return torch.round(y).to(torch.int8), scale
    return y.to(torch.float8_e4m3fn), scale


def _pool(g, c, pages, w):
    """A pool [pages, ps, Hkv, w] that holds earlier tokens, and its scales."""
    x = _randn(g, (pages, c["ps"], c["Hkv"], w), torch.float32)
    if c["kv"] not in QMAX:
        return x.to(DT[c["kv"]]), None
    codes, scale = _quant(x, c["kv"])
    return codes, scale.transpose(1, 2).contiguous()


def _cache(s):
    """The handle that a program keeps for its pools."""
    import causal_linear_attention_chunked_b200 as lt
    return lt.PagedKVCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"c": c}
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        B, N, Hq, Hkv, d, dt = c["B"], c["N"], c["Hq"], c["Hkv"], c["d"], DT[c["dtype"]]
        if c["fused"]:   # queries and keys as slices of one projection's output
            qkv = _randn(g, (B, N, (Hq + 2 * Hkv) * d), dt)
            s["q"] = qkv[..., :Hq * d].unflatten(-1, (Hq, d))
            s["k"] = qkv[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d))
        else:
            s["q"], s["k"] = _randn(g, (B, N, Hq, d), dt), _randn(g, (B, N, Hkv, d), dt)
        s["wq"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        s["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        if N == 1:       # one new token for each sequence, each at its own position
            s["pos"] = torch.randint(0, c["start"] + 1, (B,), generator=g, device="cuda",
                                     dtype=torch.int32)
        else:
            s["pos"] = torch.arange(c["start"], c["start"] + N, device="cuda", dtype=torch.int32)
        half = c["rot"] // 2
        s["freq"] = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64)
                                 / max(1, half))).float()
        if c["op"] == "norm_rope_bwd":
            s["gq"], s["gk"] = _randn(g, (B, N, Hq, d), dt), _randn(g, (B, N, Hkv, d), dt)
        return s
    if c["op"] == "cache_write":
        pages, T = c["pool"] // c["ps"], c["T"]
        s["k_pool"], s["k_scale"] = _pool(g, c, pages, c["d"])
        s["v_pool"], s["v_scale"] = _pool(g, c, pages, c["dv"])
        s["k"] = _randn(g, (T, c["Hkv"], c["d"]), DT[c["dtype"]])
        s["v"] = _randn(g, (T, c["Hkv"], c["dv"]), DT[c["dtype"]])
        if c["append"]:  # anywhere in the pool
            s["slots"] = torch.randperm(pages * c["ps"], generator=g, device="cuda")[:T].int()
        else:            # whole pages in an order of their own
            order = torch.randperm(pages, generator=g, device="cuda")
            at = torch.arange(T, device="cuda")
            s["slots"] = (order[at // c["ps"]] * c["ps"] + at % c["ps"]).int()
    else:
        lens = _lengths(c)
        need = [-(-n // c["ps"]) for n in lens]
        pages = max(1, sum(need))
        s["k_pool"], s["k_scale"] = _pool(g, c, pages, c["d"])
        s["v_pool"], s["v_scale"] = _pool(g, c, pages, c["dv"])
        order = torch.randperm(pages, generator=g, device="cuda").int().cpu()
        table = torch.full((c["B"], max(1, max(need))), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        s["table"] = table.cuda()
        s["total"] = sum(lens)
        if c["op"] == "cache_read":
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        else:
            s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
            s["q"] = _randn(g, (c["B"], c["Hq"], c["d"]), DT[c["dtype"]])
    if own:
        s["cache"] = _cache(s)
    return s


# ------------------------------------------------------------ plain forms
def _angles(s):
    """cos and sin of position x frequency, angles in 64 bits: [1 or B, N, 1, rot / 2]."""
    c = s["c"]
    a = s["pos"].double()[:, None] * s["freq"].double()[None, :]
    a = a.view((c["B"], 1, 1, -1) if c["N"] == 1 else (1, c["N"], 1, -1))
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, rot, interleaved):
    """The rotation of the first rot values of the last axis."""
    if rot == 0:
        return x
    y, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, rest), -1)


def _norm_rope(s):
    c = s["c"]
    cos, sin = _angles(s)
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        out.append(_rotate(y, cos, sin, c["rot"], c["interleaved"]).to(DT[c["dtype"]]))
    return out


def _norm_rope_bwd(s):
    c = s["c"]
    cos, sin = _angles(s)
    dx, dw = [], []
    for x, w, g in ((s["q"], s["wq"], s["gq"]), (s["k"], s["wk"], s["gk"])):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        g = _rotate(g.float(), cos, -sin, c["rot"], c["interleaved"])
        u = g * w.float()
        dx.append((r * u - x * (r ** 3 * (u * x).mean(-1, keepdim=True))).to(DT[c["dtype"]]))
        dw.append((g * x * r).sum((0, 1, 2)).to(DT[c["dtype"]]))
    return dx + dw


def _cache_write(s):
    c = s["c"]
    at = s["slots"].long()
    for x, pool, scale in ((s["k"], s["k_pool"], s["k_scale"]),
                           (s["v"], s["v_pool"], s["v_scale"])):
        rows = pool.view(-1, *pool.shape[2:])
        if scale is None:
            rows[at] = x.to(pool.dtype)
        else:
            codes, sc = _quant(x, c["kv"])
            rows.view(torch.uint8)[at] = codes.view(torch.uint8)
            scale[at // c["ps"], :, at % c["ps"]] = sc
    return [s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"]]


def _gather(pool, scale, table):
    """The rows of every table entry, in 32 bits: [B, pages x ps, Hkv, w]."""
    page = table.long().clamp(min=0)
    x = pool.view(torch.uint8)[page].view(pool.dtype).float() if scale is not None \
        else pool[page].float()
    if scale is not None:
        x = x * scale[page].transpose(2, 3).unsqueeze(-1)
    return x.flatten(1, 2)


def _cache_read(s):
    c = s["c"]
    n = s["cu"][1:] - s["cu"][:-1]
    out = []
    for pool, scale in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])):
        x = _gather(pool, scale, s["table"])
        live = torch.arange(x.shape[1], device="cuda")[None, :] < n[:, None]
        out.append(x[live].to(DT[c["dtype"]]))
    return out


def _decode(s):
    c = s["c"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    K = _gather(s["k_pool"], s["k_scale"], s["table"])
    V = _gather(s["v_pool"], s["v_scale"], s["table"])
    at = torch.arange(K.shape[1], device="cuda")[None, :]
    live = at < s["lens"][:, None]
    if c["window"]:
        live = live & (at >= s["lens"][:, None] - c["window"])
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    x = torch.einsum("bgqd,bjgd->bgqj", q, K) / math.sqrt(d)
    x = torch.where(live[:, None, None, :], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    den = p.sum(-1, keepdim=True)
    V = torch.where(live[:, :, None, None], V, 0.0)
    o = torch.einsum("bgqj,bjgd->bgqd", p, V) / torch.where(den == 0, 1.0, den)
    out = [o.reshape(B, Hq, -1).to(DT[c["dtype"]])]
    if c["lse"]:
        out.append((m + torch.log(den)).reshape(B, Hq))
    return out


PLAIN = {"norm_rope": _norm_rope, "norm_rope_bwd": _norm_rope_bwd, "cache_write": _cache_write,
         "cache_read": _cache_read, "decode": _decode}


# ------------------------------------------------------- the package's calls
def _own(s):
    import causal_linear_attention_chunked_b200 as lt
    c = s["c"]
    if c["op"] == "norm_rope":
        return lt.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"], eps=EPS,
                               interleaved=c["interleaved"])
    if c["op"] == "norm_rope_bwd":
        return lt.qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["pos"],
                                   s["freq"], eps=EPS, interleaved=c["interleaved"])
    if c["op"] == "cache_write":
        lt.kv_cache_write(s["cache"], s["k"], s["v"], s["slots"])
        return [s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"]]
    if c["op"] == "cache_read":
        return lt.kv_cache_read(s["cache"], s["table"], s["cu"], s["total"], dtype=DT[c["dtype"]])
    out = lt.paged_attn_decode(s["q"], s["cache"], s["table"], s["lens"], window=c["window"],
                               return_lse=c["lse"])
    return out if c["lse"] else [out]


def run(s):
    return list(_own(s)) if own else PLAIN[s["c"]["op"]](s)


# ------------------------------------------------------------ 64-bit values
def _turn64(x, s, sign):
    """x with each pair (a, b) of its first rot values as a + ib, times e^(sign i angle)."""
    c = s["c"]
    rot = c["rot"]
    if rot == 0:
        return x
    pos = s["pos"].double().repeat(c["B"]) if c["N"] > 1 else s["pos"].double()
    ang = torch.outer(pos, s["freq"].double()).view(c["B"], c["N"], 1, rot // 2)
    i = torch.arange(rot // 2, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
    z = torch.complex(x[..., ia], x[..., ib]) * torch.polar(torch.ones_like(ang), sign * ang)
    y = x.clone()
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def _e4m3_64(y):
    """The nearest e4m3 value, ties to even, in 64-bit arithmetic."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm_rope":
        out = []
        for x, w in ((s["q"].double(), s["wq"]), (s["k"].double(), s["wk"])):
            y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + EPS)
            out.append(_turn64(y * w.double(), s, 1.0))
        return out
    if c["op"] == "norm_rope_bwd":
        dx, dw = [], []
        for x, w, g in ((s["q"], s["wq"], s["gq"]), (s["k"], s["wk"], s["gk"])):
            x, w, g = x.double(), w.double(), _turn64(g.double(), s, -1.0)
            rms = torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + EPS)
            n = x / rms
            dx.append((g * w - n * ((g * w * n).sum(-1, keepdim=True) / c["d"])) / rms)
            dw.append((g * n).flatten(0, 2).sum(0))
            del x, g, n
        return dx + dw
    if c["op"] == "cache_write":
        out, scales = [], []
        for x, pool, scale in ((s["k"].double(), s["k_pool"], s["k_scale"]),
                               (s["v"].double(), s["v_pool"], s["v_scale"])):
            for_slot = torch.full((pool.shape[0] * pool.shape[1],), -1, device="cuda",
                                  dtype=torch.long)
            for_slot[s["slots"].long()] = torch.arange(c["T"], device="cuda")
            hit = (for_slot >= 0).view(pool.shape[:2])
            old = pool.double()
            if scale is None:
                out.append(torch.where(hit[..., None, None],
                                       x[for_slot.clamp(min=0)].view(old.shape), old))
                scales.append(None)
                continue
            sc = torch.clamp(x.abs().amax(-1) / QMAX[c["kv"]], min=TINY)
            new = sc[for_slot.clamp(min=0)].view(*hit.shape, -1).transpose(1, 2)
            scales.append(torch.where(hit[:, None, :], new, scale.double()))
            if c["kv"] == "int8":
                out.append(None)
                continue
            codes = _e4m3_64(x / sc[..., None])[for_slot.clamp(min=0)].view(old.shape)
            out.append(torch.where(hit[..., None, None], codes, old))
        return out + scales
    out = []
    lens = _lengths(c)
    table = s["table"].cpu()
    rows = [table[b, torch.arange(n) // c["ps"]].long() * c["ps"] + torch.arange(n) % c["ps"]
            for b, n in enumerate(lens)]

    def values(pool, scale, at):
        at = at.cuda()
        x = pool.flatten(0, 1)
        x = x.view(torch.uint8)[at].view(pool.dtype).double() if scale is not None \
            else x[at].double()
        if scale is not None:
            x = x * scale[at // c["ps"], :, at % c["ps"]].double()[..., None]
        return x

    if c["op"] == "cache_read":
        at = torch.cat(rows)
        return [values(s["k_pool"], s["k_scale"], at), values(s["v_pool"], s["v_scale"], at)]
    o = torch.zeros(c["B"], c["Hq"], c["dv"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    G = c["Hq"] // c["Hkv"]
    for b, at in enumerate(rows):
        at = at[-c["window"]:] if c["window"] else at
        if not len(at):
            continue
        K, V = values(s["k_pool"], s["k_scale"], at), values(s["v_pool"], s["v_scale"], at)
        for h in range(c["Hq"]):
            x = K[:, h // G] @ s["q"][b, h].double() * c["d"] ** -0.5
            o[b, h] = torch.softmax(x, 0) @ V[:, h // G]
            lse[b, h] = torch.logsumexp(x, 0)
    return [o, lse] if c["lse"] else [o]
