"""SimSD speculative verification for diffusion LLMs on GB300 (sm_103a).

The hot path -- RoPE-copy + paged KV append, split-KV attention under the
token-level temporal causal mask, split merge, and rejection-sampling
acceptance along the temporal order -- runs in the CUDA kernels of
libsimsd.so behind the C ABI in include/simsd.h; so does the loop over an
8-bit cache (page map, rotary append, attention).  ``binding`` marshals torch
tensors into that ABI; ``staging`` moves host arrays into the device layouts
the ABI expects.  There is no CPU fallback.
"""
from .binding import (SIMSD_ORDER_CAUSAL, SIMSD_ORDER_NODES, SIMSD_ORDER_PAIRED, SimsdError, accept,
                      accept_workspace_size, kvq_append, kvq_verify, kvq_verify_workspace_size,
                      layout, lib, page_map, page_map_workspace_size, prompt_append, read_status,
                      rope, rope_spec, status_string, verify_attn, verify_workspace_size)

__all__ = ["SIMSD_ORDER_CAUSAL", "SIMSD_ORDER_NODES", "SIMSD_ORDER_PAIRED", "SimsdError", "accept",
           "accept_workspace_size", "kvq_append", "kvq_verify", "kvq_verify_workspace_size",
           "layout", "lib", "page_map", "page_map_workspace_size", "prompt_append", "read_status",
           "rope", "rope_spec", "status_string", "verify_attn", "verify_workspace_size"]
