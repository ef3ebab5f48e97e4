"""MI355X-native gated delta rule: chunkwise forward, its gradients and single-token decode, the softmax
attention layers that stand between such layers in a hybrid model, and what stands around a recurrent layer's state
update: norms, short convolutions, and a selective state space scan in the delta rule's place.

The compute path is libgdn.so (hand-written HIP kernels for gfx950 behind the C
ABI of include/gdn.h); this package is its thin ctypes binding.
"""
from .gdn import (GDN_BF16, GDN_C64, GDN_CACHE_E4M3, GDN_CACHE_I8, GDN_F32, GDN_NOALLOC_MAX_WORKSPACE, GdnError, chunk_bwd, chunk_fwd, chunk_fwd_prologue,  # noqa: F401
                  fwd_channel_decay, gdn_attn_decode, gdn_attn_decode_workspace_bytes,
                  gdn_attn_prompt, gdn_attn_prompt_bwd, gdn_attn_prompt_bwd_workspace_bytes, gdn_block_tables, gdn_cache_append, gdn_chunk_bwd, gdn_chunk_bwd_workspace_bytes, gdn_chunk_fwd,
                  gdn_chunk_fwd_noalloc, gdn_chunk_fwd_prologue, gdn_chunk_fwd_prologue_workspace_bytes,
                  gdn_chunk_fwd_workspace_bytes, gdn_fwd_channel_decay, gdn_recurrent_step,
                  gdn_rms_norm, gdn_rms_norm_bwd, gdn_rms_norm_bwd_workspace_bytes, gdn_rms_norm_quant, gdn_short_conv,
                  gdn_short_conv_bwd, gdn_short_conv_bwd_workspace_bytes, gdn_short_conv_step,
                  gdn_ssm_scan, gdn_ssm_scan_bwd, gdn_ssm_scan_bwd_workspace_bytes, gdn_ssm_scan_workspace_bytes, gdn_ssm_step,
                  gdn_status_str, load, recurrent_step)

_ATTN = ("attn_decode", "attn_prompt", "attn_prompt_bwd", "block_tables", "cache_append")
_BLOCK = ("rms_norm", "rms_norm_bwd", "rms_norm_quant", "short_conv", "short_conv_bwd", "short_conv_step",
          "ssm_scan", "ssm_scan_bwd", "ssm_step")


def __getattr__(name):
    """The torch helpers, on first use: they import torch, which the raw entry points do without."""
    for names, module in ((_ATTN, "attn"), (_BLOCK, "block")):
        if name in names:
            from importlib import import_module
            m = import_module("." + module, __name__)
            globals().update({n: getattr(m, n) for n in names})
            return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
