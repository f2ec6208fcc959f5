"""Binding of the serving operators of libm3.so (include/m3_ops.h), under the
same names.

Native (csrc/ops_binding.cpp, module _ops): it checks shapes, types, devices
and layouts and makes the library's calls.  Tensors are torch tensors of one
GPU; the work goes to `stream`, by default the current stream of that GPU.
Where it is another stream than a tensor's own, the caller orders the two and
keeps the tensor (record_stream), as for any torch call on that stream.
Outputs are the caller's tensors.  What is refused raises M3Error.  There is
no CPU fallback: importing this module fails if _ops is missing.
"""
from __future__ import annotations

from . import m3 as _m3  # noqa: F401  (loads libm3.so)
try:
    from ._ops import (m3_attn_prefix, m3_attn_prefix_workspace, m3_attn_prompt,  # noqa: F401
                       m3_kv_map, m3_kv_store, m3_logit_rules, m3_ops_sync_status)
except ModuleNotFoundError as e:
    raise ImportError("_ops is missing: build it with `python -m autoregressive_audio_token_b200.build`, which says "
                      "what it needs besides libm3.so (no CPU fallback)") from e

EXPORTED = ("m3_kv_map", "m3_kv_store", "m3_attn_prompt", "m3_attn_prefix_workspace",
            "m3_attn_prefix", "m3_logit_rules", "m3_ops_sync_status")
