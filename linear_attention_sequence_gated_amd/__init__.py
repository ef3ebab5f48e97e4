"""MI355X-native gated delta rule: chunkwise forward, its gradients and single-token decode, and the softmax
attention layers that stand between such layers in a hybrid model.

The compute path is libgdn.so (hand-written HIP kernels for gfx950 behind the C
ABI of include/gdn.h); this package is its thin ctypes binding.
"""
from .gdn import (GDN_BF16, GDN_C64, GDN_CACHE_E4M3, GDN_CACHE_I8, GDN_F32, GDN_NOALLOC_MAX_WORKSPACE, GdnError, chunk_bwd, chunk_fwd, chunk_fwd_prologue,  # noqa: F401
                  fwd_channel_decay, gdn_attn_decode, gdn_attn_decode_workspace_bytes,
                  gdn_attn_prompt, gdn_attn_prompt_bwd, gdn_attn_prompt_bwd_workspace_bytes, gdn_block_tables, gdn_cache_append, gdn_chunk_bwd, gdn_chunk_bwd_workspace_bytes, gdn_chunk_fwd,
                  gdn_chunk_fwd_noalloc, gdn_chunk_fwd_prologue, gdn_chunk_fwd_prologue_workspace_bytes,
                  gdn_chunk_fwd_workspace_bytes, gdn_fwd_channel_decay, gdn_recurrent_step,
                  gdn_status_str, load, recurrent_step)

_ATTN = ("attn_decode", "attn_prompt", "attn_prompt_bwd", "block_tables", "cache_append")


def __getattr__(name):
    """The attention helpers, on first use: they import torch, which the raw entry points do without."""
    if name in _ATTN:
        from . import attn
        globals().update({n: getattr(attn, n) for n in _ATTN})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
