"""Workspaces of lt_paged_attn_decode over head counts, types and widths (host
arithmetic, on the CPU)."""
import ctypes

import pytest

F32, BF16, F16, E4M3, I8 = 0, 1, 2, 3, 4


@pytest.mark.parametrize("dtype,kv,d,dv,G,heads,warps", [
    # query heads at once and warps per block
    (BF16, E4M3, 64, 64, 8, 8, 16), (BF16, E4M3, 64, 64, 9, 16, 8), (F16, I8, 64, 64, 16, 16, 8),
    (BF16, I8, 64, 64, 40, 16, 8), (F32, E4M3, 64, 64, 8, 8, 8), (F32, I8, 64, 64, 9, 8, 8),
    (BF16, E4M3, 64, 128, 8, 8, 8), (BF16, E4M3, 128, 128, 16, 16, 8),
    (BF16, BF16, 64, 64, 4, 8, 8),
    (F16, F16, 128, 64, 12, 16, 8), (F32, F32, 64, 64, 1, 8, 4), (F32, F32, 128, 128, 20, 8, 4)])
@pytest.mark.parametrize("H_kv", [1, 3])
def test_plan(dtype, kv, d, dv, G, heads, warps, H_kv):
    from causal_linear_attention_chunked_b200 import _binding as b
    n = ctypes.c_size_t()
    assert b.lib.lt_paged_attn_decode_plan(G * H_kv, H_kv, d, dv, dtype, kv, 100,
                                           ctypes.byref(n)) == 0
    unit = min(G, heads)
    units = H_kv * -(-G // heads)
    # two pieces (values, maximum and sum of a unit's heads) per warp and per unit, and
    # 16 bytes, for each of 100 blocks
    assert n.value == 100 * ((warps + units) * 2 * unit * (dv + 2) * 4 + 16)
