"""Small, self-checking invocations of the norm, cache and decode kernels for
ncu captures (``profile_cases`` has those of the linear-attention passes).

    python -m causal_linear_attention_chunked_b200.profile_cache_cases CASE

CASE is one of:
  norm         norm and rotation of 8192 tokens of 32 + 8 bf16 heads of 128, slices of
               a fused projection
  norm_bwd     its backward pass
  write        16384 tokens of 8 bf16 heads of 128, keys and values, into e4m3 pages
  read         64 sequences of 128 .. 4096 tokens of 8 heads of 64 back from e4m3 to bf16
  attend       one new token for each of 64 sequences of 128 .. 4096 tokens, 32 query
               over 8 KV heads of 128, bf16 cache
  attend_e4m3  the same over an e4m3 cache
  attend_f32   the same for 32 of the sequences, fp32 queries and cache

Each makes three calls on inputs of more than L2's size and less than 2 GB,
checks the library's device error word after synchronising and prints "ok".
"""
import sys

import torch

from .profile_cases import _lib


def _randn(*shape, dtype=torch.bfloat16, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _norm_inputs(tokens=8192, Hq=32, Hkv=8, d=128):
    qkv = _randn(tokens, (Hq + 2 * Hkv) * d)
    q = qkv[:, :Hq * d].unflatten(-1, (Hq, d))
    k = qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d))
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    freq = 10000.0 ** (-torch.arange(d // 2, device="cuda") / (d // 2))
    return q, k, _randn(d, seed=2), _randn(d, seed=3), pos, freq


def norm():
    x = _norm_inputs()
    for _ in range(3):
        _lib().qk_norm_rope(*x)


def norm_bwd():
    x = _norm_inputs()
    gq, gk = (_randn(*t.shape, seed=4) for t in x[:2])
    for _ in range(3):
        _lib().qk_norm_rope_bwd(gq, gk, *x)


def write(tokens=16384, H=8, d=128, page=64):
    L = _lib()
    c = L.PagedKVCache.empty(tokens // page, page, H, d, dtype=torch.float8_e4m3fn)
    k, v = _randn(tokens, H, d), _randn(tokens, H, d, seed=2)
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(tokens // page, generator=g)[:, None] * page + torch.arange(page)
    slots = slots.flatten().int().cuda()
    for _ in range(3):
        L.kv_cache_write(c, k, v, slots)


def _sequences(B, H, d, dtype, page=64, longest=4096):
    """A cache that holds B sequences, its pages shuffled, their table and lengths."""
    L = _lib()
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(128, longest + 1, (B,), generator=g)
    need = (lens + page - 1) // page
    order = torch.randperm(int(need.sum()), generator=g).int()
    table = torch.full((B, int(need.max())), -1, dtype=torch.int32)
    for b, part in enumerate(order.split(need.tolist())):
        table[b, :part.numel()] = part
    c = L.PagedKVCache.empty(order.numel(), page, H, d, dtype=dtype)
    src = dtype if dtype in (torch.bfloat16, torch.float32) else torch.bfloat16
    slots = torch.arange(order.numel() * page, dtype=torch.int32, device="cuda")
    L.kv_cache_write(c, _randn(slots.numel(), H, d, dtype=src),
                     _randn(slots.numel(), H, d, dtype=src, seed=2), slots)
    return c, table.cuda(), lens.int().cuda()


def read():
    c, table, lens = _sequences(64, 8, 64, torch.float8_e4m3fn)
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0).int()])
    total = int(cu[-1])
    for _ in range(3):
        _lib().kv_cache_read(c, table, cu, total)


def attend(dtype=torch.bfloat16, q_dtype=torch.bfloat16, B=64):
    c, table, lens = _sequences(B, 8, 128, dtype)
    q = _randn(B, 32, 128, dtype=q_dtype)
    for _ in range(3):
        _lib().paged_attn_decode(q, c, table, lens)


def attend_e4m3():
    attend(torch.float8_e4m3fn)


def attend_f32():
    attend(torch.float32, torch.float32, 32)


CASES = {"norm": norm, "norm_bwd": norm_bwd, "write": write, "read": read, "attend": attend,
         "attend_e4m3": attend_e4m3, "attend_f32": attend_f32}


def main(argv):
    if len(argv) != 1 or argv[0] not in CASES:
        raise SystemExit("usage: python -m causal_linear_attention_chunked_b200."
                         "profile_cache_cases {%s}" % ",".join(CASES))
    CASES[argv[0]]()
    torch.cuda.synchronize()
    if _lib().get_last_device_error() != 0:
        raise SystemExit("device error word set")
    print("ok")


if __name__ == "__main__":
    main(sys.argv[1:])
