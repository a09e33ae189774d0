"""The training-step operators of ``include/ns.h`` in Python.

The operators themselves are functions of the compiled module ``_binding``
(``csrc/python/binding.cpp``), under the C entry points' names; ``operator`` finds
them on first use, so that importing the package loads neither torch nor the
library. The workspace sizes come through ctypes like the rest of the library.

Autograd records nothing of a call: ``examples/moe_distill_step.py`` wraps them in
autograd functions. A call moves the versions of the tensors it writes, so that a
backward pass which saved one of them raises.
"""

from __future__ import annotations

import ctypes
import importlib
import os

from ._lib import NSLibraryMissing, _check, lib

OPERATORS = (
    "ns_qk_norm_rope", "ns_qk_norm_rope_backward",
    "ns_moe_sort", "ns_moe_dispatch", "ns_moe_dispatch_backward", "ns_moe_combine", "ns_moe_combine_backward",
    "ns_distill_topk", "ns_distill_topk_backward",
)


class ns_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("heads", ctypes.c_int32)]


def operator(name: str):
    """The operator of that name (raises NSLibraryMissing if the module was never built)."""
    from .build import BINDING
    if not os.path.exists(BINDING):
        raise NSLibraryMissing(f"{BINDING} not found: build it with `python -m newton_schulz_quintic_amd.build`")
    import torch  # noqa: F401  (the module uses its libraries)
    lib()
    return getattr(importlib.import_module("newton_schulz_quintic_amd._binding"), name)


def ns_qk_norm_rope_workspace_bytes(batch: int, seq: int, head_dim: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ns_qk_norm_rope_workspace_bytes(batch, seq, head_dim, ctypes.byref(n)))
    return n.value


def ns_moe_sort_workspace_bytes(tokens: int, top_k: int, num_experts: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ns_moe_sort_workspace_bytes(tokens, top_k, num_experts, ctypes.byref(n)))
    return n.value


def ns_distill_workspace_bytes(rows: int, vocab: int, top_k: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().ns_distill_workspace_bytes(rows, vocab, top_k, ctypes.byref(n)))
    return n.value
