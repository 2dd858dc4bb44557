"""Kernelised (linear) attention for NVIDIA B200 (sm_100a).

    O_i = phi(Q_i) S_i / (phi(Q_i) . z_i + eps),  phi(x) = ELU(x) + 1,

causal or non-causal, with grouped-query heads, packed variable-length
sequences, a forward pass that starts from and returns the recurrent state,
and a recurrent decode step.  Next to it, for every kind of attention layer,
the norm and position rotation of queries and keys, and for softmax layers a
paged key-value cache (16-bit, fp32 or quantised to 8 bits) with the attention
of one new token over it.  The computation runs in the CUDA
library ``liblt.so`` behind the C ABI of ``include/lt_linear_attn.h``; this
package is a thin ctypes binding over it (PyTorch supplies device memory and
streams).  ``inputs`` holds the seeded synthetic workloads.

The binding (and with it the library) is loaded on first use of one of the
API names below; a missing library raises ImportError.
"""
_API = ("linear_attn_fwd", "linear_attn_fwd_state", "linear_attn_fwd_plan",
        "linear_attn_decode_step", "linear_attn_state", "linear_attn_state_carry",
        "linear_attn_bwd", "linear_attn_fwd_window",
        "set_schedule",
        "get_last_device_error",
        "linear_attn_fwd_host", "LtError")
_CACHE_API = ("qk_norm_rope", "qk_norm_rope_bwd", "PagedKVCache", "kv_cache_write",
              "kv_cache_read", "paged_attn_decode")


def __getattr__(name):
    if name in _API:
        from . import _binding
        return getattr(_binding, name)
    if name in _CACHE_API:
        from . import kv_cache
        globals()[name] = getattr(kv_cache, name)  # found at once from now on
        return globals()[name]
    raise AttributeError(name)
