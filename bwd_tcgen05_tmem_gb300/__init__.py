"""GB300-native fused causal attention: forward, backward and LSE merge, the
norm and rotation of its queries and keys, and attention over a 4-bit cache.

The compute path is the C-ABI library ``libattn.so`` (hand-written sm_103a
CUDA kernels) declared in ``include/attn.h``; ``bwd_tcgen05_tmem_gb300.attn``
and ``.kv`` (the cache) are thin ctypes bindings over it.  Importing this package loads nothing: the
library is loaded on first use and a missing library raises at that point.
"""
__all__ = ["attn", "kv", "synth", "cp"]
