"""Kimi Delta Attention (KDA) prefill and decode for B200 (sm_100a), the gated
delta rule (one decay per head) and the block norm between such layers.

The compute lives in ``libkda.so`` (hand-written CUDA behind a C ABI, see
``include/kda.h``); ``binding`` marshals arguments to it with ctypes.
The binding is imported lazily so that ``inputs`` (seeded synthetic data)
can be used without touching the CUDA library.
"""
from __future__ import annotations

_CALLS = ("kda_chunk_prefill", "kda_decode_step", "kda_chunk_prefill_workspace_bytes",
          "kda_gdr_chunk_prefill", "kda_gdr_decode", "kda_gdr_backward", "kda_gdr_autograd",
          "kda_block_norm", "kda_block_norm_backward", "kda_block_norm_autograd")
__all__ = ["binding", "inputs", *_CALLS]


def __getattr__(name):
    if name in _CALLS:
        from . import binding
        return getattr(binding, name)
    if name in ("binding", "inputs"):
        import importlib
        return importlib.import_module(f".{name}", __name__)
    raise AttributeError(name)
