"""Torch helpers of the attention layer's entry points (include/gdn.h): block tables, the 8-bit paged cache, its
single-token read, attention over whole prompts and its gradients.

They check dtypes, shapes, strides and devices, allocate what is not passed in, pass ``data_ptr()`` and the current
HIP stream of the tensors' device (or ``stream``), and raise on a non-OK status.  Rows are [tokens, heads, D] with the heads of a row
side by side; the distance between rows is free, so that q, k and v can be parts of one fused projection.
"""
from __future__ import annotations

import functools

import torch

from . import gdn as raw

_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_FORMATS = {torch.int8: raw.GDN_CACHE_I8, torch.float8_e4m3fn: raw.GDN_CACHE_E4M3}


def _device(t, who):
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{who}: tensors must live on a HIP device")
    return dev


def _dense(t, name, shape, dtype, dev):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev.index or not t.is_contiguous():
        raw._check(t, name, shape, dtype, dev)


def _rows(t, name, shape, dev):
    """Distance between the rows of t [tokens, heads, D], whose rows are dense."""
    tokens, heads, d = shape
    row, head, one = t.stride() if t.dim() == 3 else (0, 0, 0)
    if t.shape != shape or t.dtype is not _BF16 or t.get_device() != dev.index:
        raw._check(t.contiguous(), name, shape, _BF16, dev)
    if d > 1 and one != 1 or heads > 1 and head != d:
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if tokens <= 1:
        return heads * d
    if row < heads * d or row % 8:
        raise ValueError(f"{name}: rows must be a multiple of 8 elements apart and not overlap")
    return row


def _call(dev, fn, *args):
    """fn(*args, the current stream of dev), with dev as the current device.

    Both are asked for by the calls under torch.cuda.current_device() and current_stream(), which take 2 us more to wrap
    the answers."""
    if torch._C._cuda_getDevice() == dev.index:
        s = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            s = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if s != raw.GDN_OK:
        raise raw.GdnError(s)


def _on_stream(f):
    """Adds the argument stream (a hipStream_t as a number; the current stream unless given).  Another stream is made
    the current one for the call, so that what is allocated in it belongs to that stream."""

    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        dev = next(x for x in (*args, *kw.values()) if isinstance(x, torch.Tensor)).device
        if dev.type != "cuda" or stream == torch._C._cuda_getCurrentRawStream(dev.index):
            return f(*args, **kw)
        s = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
        with torch.cuda.stream(s):
            return f(*args, **kw)

    return call


@_on_stream
def block_tables(seq_lens, new_lens, block_table, free_blocks, block_tokens: int, num_blocks: int, tokens: int):
    """Extends block_table [R, width] in place by the blocks that new_lens [R] more tokens need beyond seq_lens [R],
    taken from the front of free_blocks.  All int32.  tokens: the length of the slot map, at least the sum of new_lens
    (what is over is filled with -1).

    Returns (slot_map [tokens], cu_seqlens [R + 1], lens_after [R], used [2]: free blocks taken, requests refused), parts of
    one allocation.
    """
    dev = _device(seq_lens, "block_tables")
    r, width = block_table.shape
    _dense(seq_lens, "seq_lens", (r,), _I32, dev)
    _dense(new_lens, "new_lens", (r,), _I32, dev)
    _dense(block_table, "block_table", (r, width), _I32, dev)
    _dense(free_blocks, "free_blocks", (free_blocks.numel(),), _I32, dev)
    if tokens < 0:
        raise ValueError("block_tables: tokens is negative")
    # one allocation, its parts 16 bytes aligned (four take 1.5 us more)
    a, b = -(r + 1) % 4, -r % 4
    used, _, cu, _, after, _, slot_map = seq_lens.new_empty(4 + r + 1 + a + r + b + tokens).split_with_sizes(
        (2, 2, r + 1, a, r, b, tokens))
    _call(dev, raw.load().gdn_block_tables, seq_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
          free_blocks.data_ptr(), slot_map.data_ptr(), cu.data_ptr(), after.data_ptr(), used.data_ptr(), r, width,
          free_blocks.numel(), block_tokens, num_blocks, tokens)
    return slot_map, cu, after, used


def _cache(k_cache, v_cache, k_scale, v_scale, dev):
    nb, hkv, bt, d = k_cache.shape
    fmt = _FORMATS.get(k_cache.dtype)
    if fmt is None:
        raise TypeError(f"unsupported cache dtype {k_cache.dtype}; use int8 or float8_e4m3fn")
    _dense(k_cache, "k_cache", (nb, hkv, bt, d), k_cache.dtype, dev)
    _dense(v_cache, "v_cache", (nb, hkv, bt, d), k_cache.dtype, dev)
    _dense(k_scale, "k_scale", (nb, hkv), _F32, dev)
    _dense(v_scale, "v_scale", (nb, hkv), _F32, dev)
    return nb, hkv, bt, d, fmt


@_on_stream
def cache_append(k, v, slot_map, k_cache, v_cache, k_scale, v_scale):
    """Writes the rows k, v [T, Hkv, D] bf16 into the cache at slot_map [T] int32 (see block_tables), in place.

    k_cache, v_cache [num_blocks, Hkv, block_tokens, D] int8 or float8_e4m3fn; k_scale, v_scale [num_blocks, Hkv]
    float32: a value is its code times the scale of its block and head.  The tokens of one block follow one another in
    the call with consecutive slots; a token whose slot lies outside the cache is skipped.
    """
    dev = _device(k, "cache_append")
    nb, hkv, bt, d, fmt = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    t = k.shape[0]
    ks, vs = _rows(k, "k", (t, hkv, d), dev), _rows(v, "v", (t, hkv, d), dev)
    _dense(slot_map, "slot_map", (t,), _I32, dev)
    _call(dev, raw.load().gdn_cache_append, k.data_ptr(), v.data_ptr(), slot_map.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), ks, vs, t, hkv, d, bt, nb,
          raw.GDN_BF16, fmt)


@functools.lru_cache(maxsize=1024)
def _decode_workspace(*sizes):
    return raw.gdn_attn_decode_workspace_bytes(*sizes)


@functools.lru_cache(maxsize=1024)
def _bwd_workspace(*sizes):
    return raw.gdn_attn_prompt_bwd_workspace_bytes(*sizes)


@_on_stream
def attn_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, scale: float | None = None, out=None,
                lse=None, workspace=None):
    """Attention of one new token per request, q [R, Hq, D] bf16, over the first seq_lens [R] tokens of its blocks
    block_table [R, width] (int32) in the cache (see cache_append).  scale: 1 / sqrt(D) unless given.

    Returns (out [R, Hq, D] bf16, lse [R, Hq] float32).  The workspace is allocated here unless one of at least
    gdn_attn_decode_workspace_bytes(...) bytes is passed.
    """
    dev = _device(q, "attn_decode")
    nb, hkv, bt, d, fmt = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    r, hq, _ = q.shape
    width = block_table.shape[1]
    qs = _rows(q, "q", (r, hq, d), dev)
    _dense(block_table, "block_table", (r, width), _I32, dev)
    _dense(seq_lens, "seq_lens", (r,), _I32, dev)
    if out is None:
        out = q.new_empty((r, hq, d))
    else:
        _dense(out, "out", (r, hq, d), _BF16, dev)
    if lse is None:
        lse = k_scale.new_empty((r, hq))
    else:
        _dense(lse, "lse", (r, hq), _F32, dev)
    lib = raw.load()
    if workspace is None:
        size = _decode_workspace(r, hq, hkv, d, bt, width)
        workspace = k_scale.new_empty(size // 4) if size else lse
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous on the device of q")
    _call(dev, lib.gdn_attn_decode, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
          v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(),
          d ** -0.5 if scale is None else scale, qs, r, hq, hkv, d, bt, nb, width, raw.GDN_BF16, fmt,
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, lse


def _prompt(q, k, v, cu_seqlens, who):
    dev = _device(q, who)
    t, hq, d = q.shape
    hkv = k.shape[1]
    _dense(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), _I32, dev)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens: needs at least one entry")
    strides = _rows(q, "q", (t, hq, d), dev), _rows(k, "k", (t, hkv, d), dev), _rows(v, "v", (t, hkv, d), dev)
    return dev, t, cu_seqlens.numel() - 1, hq, hkv, d, strides


@_on_stream
def attn_prompt(q, k, v, cu_seqlens, scale: float | None = None, out=None, lse=None):
    """Causal attention over packed prompts: q [T, Hq, D], k, v [T, Hkv, D] bf16, cu_seqlens [R + 1] int32 the offsets
    of the sequences.  scale: 1 / sqrt(D) unless given.

    Returns (out [T, Hq, D] bf16, lse [Hq, T] float32).  Rows in no sequence are not written; outputs that are
    allocated here hold zeros there.
    """
    dev, t, r, hq, hkv, d, strides = _prompt(q, k, v, cu_seqlens, "attn_prompt")
    zero_rest = out is None and lse is None
    if out is None:
        out = q.new_empty((t, hq, d)) if zero_rest else q.new_zeros((t, hq, d))
    else:
        _dense(out, "out", (t, hq, d), _BF16, dev)
    if lse is None:
        lse = q.new_empty((hq, t), dtype=_F32) if zero_rest else q.new_zeros((hq, t), dtype=_F32)
    else:
        _dense(lse, "lse", (hq, t), _F32, dev)
    _call(dev, raw.load().gdn_attn_prompt, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(),
          out.data_ptr(), lse.data_ptr(), d ** -0.5 if scale is None else scale, *strides, t, r, hq, hkv, d,
          raw.GDN_BF16, zero_rest)
    return out, lse


@_on_stream
def attn_prompt_bwd(q, k, v, out, lse, grad_out, cu_seqlens, scale: float | None = None, grad_q=None, grad_k=None,
                    grad_v=None):
    """Gradients of sum(out * grad_out) for attn_prompt's forward, from the out and lse that it returned.

    Returns (grad_q, grad_k, grad_v) bf16, the latter two summed over the query heads that share them.  Passed in, they
    may be parts of one tensor.  Rows in no sequence are not written; gradients that are allocated here hold zeros
    there.  The workspace is allocated here with torch.
    """
    dev, t, r, hq, hkv, d, strides = _prompt(q, k, v, cu_seqlens, "attn_prompt_bwd")
    _dense(out, "out", (t, hq, d), _BF16, dev)
    _dense(lse, "lse", (hq, t), _F32, dev)
    shapes = (t, hq, d), (t, hkv, d), (t, hkv, d)
    grads = (grad_q, grad_k, grad_v)
    zero_rest = all(g is None for g in grads)
    if zero_rest:
        grads = [q.new_empty(s) for s in shapes]
        gstrides = hq * d, hkv * d, hkv * d
    else:
        grads = [q.new_zeros(s) if g is None else g for g, s in zip(grads, shapes)]
        gstrides = [_rows(g, n, s, dev) for g, n, s in zip(grads, ("grad_q", "grad_k", "grad_v"), shapes)]
    gos = _rows(grad_out, "grad_out", (t, hq, d), dev)
    lib = raw.load()
    size = _bwd_workspace(t, hq, hkv, d)
    ws = lse.new_empty(size // 4)
    _call(dev, lib.gdn_attn_prompt_bwd, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
          lse.data_ptr(), grad_out.data_ptr(), cu_seqlens.data_ptr(), *(g.data_ptr() for g in grads),
          d ** -0.5 if scale is None else scale, *strides, gos, *gstrides, t, r, hq, hkv, d, raw.GDN_BF16, zero_rest,
          ws.data_ptr(), size)
    return tuple(grads)
