"""GB300-native fused attention backward.

The computation runs in hand-written sm_103a CUDA kernels inside
``libattn_gb300.so`` (C ABI in ``include/attn_bwd.h`` and, for the serving
operators, ``include/attn_cache.h``); this package only
builds and binds it.  PyTorch provides device memory and streams.
"""
from .binding import (AttnError, alloc_workspace, attn_bwd, attn_bwd_host, attn_bwd_host_varlen,
                      attn_fwd,
                      check_device_status, diag_mma, diag_tanh, diag_wait_timeout,
                      host_buffer_size, lib, set_wait_timeout_ns, version, workspace_layout,
                      workspace_size)
from .cache import (alloc_decode_workspace, alloc_evict_workspace, attn_cache_append,
                    attn_cache_evict, attn_decode, attn_rope, decode_workspace_size,
                    evict_workspace_size)
from .cache8 import attn_cache_append8, attn_cache_load8, attn_decode8
from .pages import attn_cache_copy, attn_cache_fork, fork_workspace_size

__all__ = ["AttnError", "alloc_workspace", "attn_bwd", "attn_bwd_host", "attn_bwd_host_varlen",
           "attn_fwd",
           "check_device_status", "diag_mma", "diag_tanh", "diag_wait_timeout",
           "host_buffer_size", "lib", "set_wait_timeout_ns", "version", "workspace_layout",
           "workspace_size", "alloc_decode_workspace", "alloc_evict_workspace",
           "attn_cache_append", "attn_cache_evict", "attn_decode", "attn_rope",
           "decode_workspace_size", "evict_workspace_size", "attn_cache_append8",
           "attn_cache_load8", "attn_decode8", "attn_cache_copy", "attn_cache_fork",
           "fork_workspace_size"]
