"""Torch helpers of what stands around a recurrent layer's state update (include/gdn.h): the root-mean-square norm with
the residual's addition, also with an output in 8 bits, the short causal convolution, and the selective state space scan.

They check dtypes, shapes, strides and devices, allocate what is not passed in, pass ``data_ptr()`` and the current
HIP stream of the tensors' device (or ``stream``), and raise on a non-OK status.  Rows are [tokens, channels] with the
channels of a row side by side; the distance between rows is free, so that x can be a part of one fused projection.
"""
from __future__ import annotations

import functools

import torch

from . import gdn as raw
from .attn import _FORMATS, _I32, _call, _dense, _device, _on_stream

_CODES = {torch.bfloat16: raw.GDN_BF16, torch.float32: raw.GDN_F32}


def _types(x, weight, who):
    """The codes of the rows' and the parameters' types."""
    code, wcode = _CODES.get(x.dtype), _CODES.get(weight.dtype)
    if code is None:
        raise TypeError(f"{who}: unsupported dtype {x.dtype}; use bfloat16 or float32")
    if wcode is None or (code == raw.GDN_F32 and wcode != code):
        raise TypeError(f"{who}: parameters must have the rows' dtype or float32, got {weight.dtype}")
    return code, wcode


def _rows(t, name, shape, dtype, dev):
    """Distance between the rows of t [tokens, channels], whose rows are dense."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev.index:
        raw._check(t.contiguous(), name, shape, dtype, dev)
    row, one = t.stride()
    if shape[0] and shape[1] > 1 and one != 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous")
    if shape[0] <= 1:
        return -(-shape[1] // 8) * 8
    if row < shape[1] or row % 8:
        raise ValueError(f"{name}: rows must be a multiple of 8 elements apart and not overlap")
    return row


def _given(t, name, shape, dtype, dev):
    """The address of an optional dense tensor."""
    if t is None:
        return None
    _dense(t, name, shape, dtype, dev)
    return t.data_ptr()


def _norm_inputs(x, weight, residual, who):
    dev = _device(x, who)
    t, c = x.shape
    code, wcode = _types(x, weight, who)
    xs = _rows(x, "x", (t, c), x.dtype, dev)
    _dense(weight, "weight", (c,), weight.dtype, dev)
    rs = 0 if residual is None else _rows(residual, "residual", (t, c), x.dtype, dev)
    return dev, t, c, code, wcode, xs, rs


def _sum_of(x, residual, out):
    """Where the sum goes: x itself without a residual."""
    if residual is None:
        if out is not None:
            raise ValueError("sum_out: there is no sum without a residual")
        return x, None
    t, c = x.shape
    if out is None:
        out = x.new_empty((t, c))
    else:
        _dense(out, "sum_out", (t, c), x.dtype, x.device)
    return out, out.data_ptr()


@_on_stream
def rms_norm(x, weight, residual=None, eps: float = 1e-6, out=None, sum_out=None):
    """Root-mean-square norm of the rows s = x + residual: s weight / sqrt(mean(s^2) + eps).

    x, residual [T, C] bfloat16 or float32, C a multiple of 8; weight [C] of that dtype or float32.  Returns (out [T, C],
    s [T, C], rounded to x's dtype before it is normalised; x itself without a residual).  out and sum_out may be x or
    residual, where their rows lie side by side: sum_out=residual carries the residual on in place.
    """
    dev, t, c, code, wcode, xs, rs = _norm_inputs(x, weight, residual, "rms_norm")
    if out is None:
        out = x.new_empty((t, c))
    else:
        _dense(out, "out", (t, c), x.dtype, dev)
    total, to = _sum_of(x, residual, sum_out)
    _call(dev, raw.load().gdn_rms_norm, x.data_ptr(), raw._ptr(residual), weight.data_ptr(), out.data_ptr(), to, eps, xs, rs,
          t, c, code, wcode)
    return out, total


@_on_stream
def rms_norm_quant(x, weight, residual=None, eps: float = 1e-6, dtype=torch.float8_e4m3fn, block: int = 128, codes=None,
                   scale=None, sum_out=None):
    """rms_norm with an output in 8 bits, for a product in 8 bits: codes [T, C] of dtype (int8 or float8_e4m3fn), and a
    float32 scale for each block of 128 columns [T, C / 128] or, with block = 0, for each row [T, 1].

    Returns (codes, scale, s): a value is its code times its scale.  sum_out: as for rms_norm.
    """
    dev, t, c, code, wcode, xs, rs = _norm_inputs(x, weight, residual, "rms_norm_quant")
    fmt = _FORMATS.get(dtype)
    if fmt is None:
        raise TypeError(f"unsupported dtype {dtype} of the codes; use int8 or float8_e4m3fn")
    if block not in (0, 128) or block and c % block:
        raise ValueError("block: 128 columns, of which a row is a multiple, or 0 for a scale to a row")
    if codes is None:
        codes = x.new_empty((t, c), dtype=dtype)
    else:
        _dense(codes, "codes", (t, c), dtype, dev)
    shape = (t, c // block if block else 1)
    if scale is None:
        scale = x.new_empty(shape, dtype=torch.float32)
    else:
        _dense(scale, "scale", shape, torch.float32, dev)
    total, to = _sum_of(x, residual, sum_out)
    _call(dev, raw.load().gdn_rms_norm_quant, x.data_ptr(), raw._ptr(residual), weight.data_ptr(), codes.data_ptr(),
          scale.data_ptr(), to, eps, xs, rs, t, c, block, code, wcode, fmt)
    return codes, scale, total


@functools.lru_cache(maxsize=1024)
def _norm_workspace(*sizes):
    return raw.gdn_rms_norm_bwd_workspace_bytes(*sizes)


@_on_stream
def rms_norm_bwd(sum, weight, grad_out, eps: float = 1e-6, grad_sum=None):
    """Gradients of sum(out * grad_out) + sum(s * grad_sum) for rms_norm's forward, from the s that it returned.

    Returns (grad_x [T, C], which is the residual's gradient too, grad_weight [C] of the weight's dtype).  The workspace
    is allocated here with torch.
    """
    dev = _device(sum, "rms_norm_bwd")
    t, c = sum.shape
    code, wcode = _types(sum, weight, "rms_norm_bwd")
    ss = _rows(sum, "sum", (t, c), sum.dtype, dev)
    _dense(weight, "weight", (c,), weight.dtype, dev)
    gs = _rows(grad_out, "grad_out", (t, c), sum.dtype, dev)
    gss = 0 if grad_sum is None else _rows(grad_sum, "grad_sum", (t, c), sum.dtype, dev)
    grad_x, grad_weight = sum.new_empty((t, c)), torch.empty_like(weight)
    size = _norm_workspace(t, c, code)
    ws = weight.new_empty(size // 4, dtype=torch.float32)
    _call(dev, raw.load().gdn_rms_norm_bwd, sum.data_ptr(), weight.data_ptr(), grad_out.data_ptr(), raw._ptr(grad_sum),
          grad_x.data_ptr(), grad_weight.data_ptr(), eps, ss, gs, gss, t, c, code, wcode, ws.data_ptr(), size)
    return grad_x, grad_weight


def _conv_inputs(x, weight, bias, who):
    dev = _device(x, who)
    t, c = x.shape
    code, wcode = _types(x, weight, who)
    if weight.dim() != 2:
        raise ValueError("weight: expected [channels, taps]")
    w = weight.shape[1]
    xs = _rows(x, "x", (t, c), x.dtype, dev)
    _dense(weight, "weight", (c, w), weight.dtype, dev)
    return dev, t, c, w, code, wcode, xs, _given(bias, "bias", (c,), weight.dtype, dev)


def _sequences(cu_seqlens, dev):
    _dense(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), _I32, dev)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens: needs at least one entry")
    return cu_seqlens.numel() - 1


@_on_stream
def short_conv(x, weight, cu_seqlens, bias=None, state=None, silu: bool = True, out=None, state_final=None):
    """Depthwise causal convolution over packed sequences, with SiLU: x [T, C] bfloat16 or float32, weight [C, W] with W
    from 2 to 4 (the last tap meets the row itself) and bias [C] of x's dtype or float32, cu_seqlens [R + 1] int32 the
    offsets of the sequences, state [R, W - 1, C] the rows before each (zeros unless given).

    Returns (out [T, C], state_final [R, W - 1, C]), which may not be x and state.  Rows in no sequence are not written; an
    out that is allocated here holds zeros there.
    """
    dev, t, c, w, code, wcode, xs, bp = _conv_inputs(x, weight, bias, "short_conv")
    r = _sequences(cu_seqlens, dev)
    sp = _given(state, "state", (r, w - 1, c), x.dtype, dev)
    zero_rest = out is None
    if out is None:
        out = x.new_empty((t, c))
    else:
        _dense(out, "out", (t, c), x.dtype, dev)
    if state_final is None:
        state_final = x.new_empty((r, w - 1, c))
    else:
        _dense(state_final, "state_final", (r, w - 1, c), x.dtype, dev)
    _call(dev, raw.load().gdn_short_conv, x.data_ptr(), weight.data_ptr(), bp, cu_seqlens.data_ptr(), sp, out.data_ptr(),
          state_final.data_ptr(), xs, t, r, c, w, code, wcode, silu, zero_rest)
    return out, state_final


@functools.lru_cache(maxsize=1024)
def _conv_workspace(*sizes):
    return raw.gdn_short_conv_bwd_workspace_bytes(*sizes)


@_on_stream
def short_conv_bwd(x, weight, grad_out, cu_seqlens, bias=None, state=None, silu: bool = True, grad_state_final=None):
    """Gradients of sum(out * grad_out) + sum(state_final * grad_state_final) for short_conv's forward.

    Returns (grad_x [T, C], zeros in rows of no sequence; grad_weight [C, W]; grad_bias [C] or None without a bias;
    grad_state [R, W - 1, C] or None without a state), each of the dtype of what it is the gradient of.  The workspace is
    allocated here with torch.
    """
    dev, t, c, w, code, wcode, xs, bp = _conv_inputs(x, weight, bias, "short_conv_bwd")
    r = _sequences(cu_seqlens, dev)
    gs = _rows(grad_out, "grad_out", (t, c), x.dtype, dev)
    sp = _given(state, "state", (r, w - 1, c), x.dtype, dev)
    gsp = _given(grad_state_final, "grad_state_final", (r, w - 1, c), x.dtype, dev)
    grad_x, grad_weight = x.new_empty((t, c)), torch.empty_like(weight)
    grad_bias = None if bias is None else torch.empty_like(bias)
    grad_state = None if state is None else torch.empty_like(state)
    size = _conv_workspace(t, c, w)
    ws = x.new_empty(size // 4, dtype=torch.float32)
    _call(dev, raw.load().gdn_short_conv_bwd, x.data_ptr(), weight.data_ptr(), bp, grad_out.data_ptr(),
          cu_seqlens.data_ptr(), sp, gsp, grad_x.data_ptr(), grad_weight.data_ptr(), raw._ptr(grad_bias),
          raw._ptr(grad_state), xs, gs, t, r, c, w, code, wcode, silu, True, ws.data_ptr(), size)
    return grad_x, grad_weight, grad_bias, grad_state


@_on_stream
def short_conv_step(x, weight, state, bias=None, silu: bool = True, out=None):
    """One new row x [R, C] for each of R sequences: returns out [R, C], which may not be x, and moves state [R, W - 1, C] on
    in place."""
    dev, r, c, w, code, wcode, xs, bp = _conv_inputs(x, weight, bias, "short_conv_step")
    _dense(state, "state", (r, w - 1, c), x.dtype, dev)
    if out is None:
        out = x.new_empty((r, c))
    else:
        _dense(out, "out", (r, c), x.dtype, dev)
    _call(dev, raw.load().gdn_short_conv_step, x.data_ptr(), weight.data_ptr(), bp, state.data_ptr(), out.data_ptr(), xs, r,
          c, w, code, wcode, silu)
    return out


def _heads(t, name, shape, dev):
    """Distance between the rows of t [tokens, heads, D] bf16, whose heads lie side by side."""
    if t.shape != shape or t.dtype is not torch.bfloat16 or t.get_device() != dev.index:
        raw._check(t.contiguous(), name, shape, torch.bfloat16, dev)
    n, h, d = shape
    row, head, one = t.stride()
    if n and (d > 1 and one != 1 or h > 1 and head != d):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if n <= 1:
        return h * d
    if row < h * d or row % 8:
        raise ValueError(f"{name}: rows must be a multiple of 8 elements apart and not overlap")
    return row


def _scan_inputs(x, dt, a, B, C, D, dt_bias, who):
    """(device, addresses of the seven inputs, strides, sizes, types)."""
    dev = _device(x, who)
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError(f"{who}: x and B must be [tokens, heads, size]")
    t, h, p = x.shape
    _, g, n = B.shape
    xs, bs, cs = _heads(x, "x", (t, h, p), dev), _heads(B, "B", (t, g, n), dev), _heads(C, "C", (t, g, n), dev)
    dcode, pcode = _CODES.get(dt.dtype), _CODES.get(a.dtype)
    if dcode is None or pcode is None:
        raise TypeError(f"{who}: dt and the parameters must be bfloat16 or float32")
    if dt.shape != (t, h) or dt.get_device() != dev.index:
        raw._check(dt.contiguous(), "dt", (t, h), dt.dtype, dev)
    row, one = dt.stride()
    if t and h > 1 and one != 1:
        raise ValueError("dt: the heads of a row must be contiguous")
    if t > 1 and row < h:
        raise ValueError("dt: rows must not overlap")
    _dense(a, "a", (h,), a.dtype, dev)
    ptrs = (x.data_ptr(), dt.data_ptr(), a.data_ptr(), B.data_ptr(), C.data_ptr(), _given(D, "D", (h,), a.dtype, dev),
            _given(dt_bias, "dt_bias", (h,), a.dtype, dev))
    return dev, ptrs, (xs, row if t > 1 else h, bs, cs), (t, h, p, g, n), (raw.GDN_BF16, dcode, pcode)


@functools.lru_cache(maxsize=1024)
def _scan_workspace(*sizes):
    return raw.gdn_ssm_scan_workspace_bytes(*sizes)


@_on_stream
def ssm_scan(x, dt, a, B, C, cu_seqlens, D=None, dt_bias=None, S0=None, out=None, S_final=None):
    """Selective state space scan over packed sequences: with d = softplus(dt + dt_bias), per head

        S_t = exp(a d_t) S_{t-1} + d_t B_t x_t^T,    out_t = S_t^T C_t + D x_t.

    x [T, H, P] bf16 and B, C [T, G, N] bf16 (P, N 64 or 128; head h reads group h // (H / G)), each of which may be a part
    of wider rows; dt [T, H] bf16 or float32; a (negative), D, dt_bias [H] bf16 or float32, one dtype; cu_seqlens [R + 1]
    int32 the offsets of the sequences; S0 [R, H, N, P] float32 the states before (zeros unless given).

    Returns (out [T, H, P] bf16, S_final [R, H, N, P] float32), which may not be x and S0.  Rows in no sequence are not
    written; an out that is allocated here holds zeros there.  The workspace is allocated here with torch.
    """
    dev, ptrs, strides, (t, h, p, g, n), types = _scan_inputs(x, dt, a, B, C, D, dt_bias, "ssm_scan")
    r = _sequences(cu_seqlens, dev)
    sp = _given(S0, "S0", (r, h, n, p), torch.float32, dev)
    zero_rest = out is None
    if out is None:
        out = x.new_empty((t, h, p))
    else:
        _dense(out, "out", (t, h, p), torch.bfloat16, dev)
    if S_final is None:
        S_final = x.new_empty((r, h, n, p), dtype=torch.float32)
    else:
        _dense(S_final, "S_final", (r, h, n, p), torch.float32, dev)
    size = _scan_workspace(t, h, p, g, n)
    ws = S_final.new_empty(size // 4) if size else None
    _call(dev, raw.load().gdn_ssm_scan, *ptrs, cu_seqlens.data_ptr(), sp, out.data_ptr(), S_final.data_ptr(), *strides, t, r,
          h, p, g, n, *types, zero_rest, raw._ptr(ws), size)
    return out, S_final


@functools.lru_cache(maxsize=1024)
def _scan_bwd_workspace(*sizes):
    return raw.gdn_ssm_scan_bwd_workspace_bytes(*sizes)


@_on_stream
def ssm_scan_bwd(x, dt, a, B, C, grad_out, cu_seqlens, D=None, dt_bias=None, S0=None, grad_S_final=None, grad_x=None,
                 grad_B=None, grad_C=None):
    """Gradients of sum(out * grad_out) + sum(S_final * grad_S_final) for ssm_scan's forward, which is computed again.

    Returns (grad_x [T, H, P], grad_dt [T, H], grad_a [H], grad_B, grad_C [T, G, N], grad_D [H] or None without D,
    grad_dt_bias [H] or None without dt_bias, grad_S0 [R, H, N, P] or None without S0), each of the dtype of what it is the
    gradient of; grad_B and grad_C are summed over the heads that share them.  grad_x, grad_B and grad_C may be passed in,
    as parts of one tensor; rows in no sequence are not written then, and hold zeros in gradients that are allocated here.
    The workspace is allocated here with torch.
    """
    dev, ptrs, strides, (t, h, p, g, n), types = _scan_inputs(x, dt, a, B, C, D, dt_bias, "ssm_scan_bwd")
    r = _sequences(cu_seqlens, dev)
    gs = _heads(grad_out, "grad_out", (t, h, p), dev)
    sp = _given(S0, "S0", (r, h, n, p), torch.float32, dev)
    gsp = _given(grad_S_final, "grad_S_final", (r, h, n, p), torch.float32, dev)
    zero_rest = grad_x is None and grad_B is None and grad_C is None
    rows, gstrides = [], []
    for v, name, shape in ((grad_x, "grad_x", (t, h, p)), (grad_B, "grad_B", (t, g, n)), (grad_C, "grad_C", (t, g, n))):
        rows.append((x.new_empty if zero_rest else x.new_zeros)(shape) if v is None else v)
        gstrides.append(shape[1] * shape[2] if v is None else _heads(v, name, shape, dev))
    grad_dt = dt.new_empty((t, h)) if zero_rest else dt.new_zeros((t, h))
    grad_a = torch.empty_like(a)
    grad_D, grad_bias, grad_S0 = (None if v is None else torch.empty_like(v) for v in (D, dt_bias, S0))
    size = _scan_bwd_workspace(t, r, h, p, g, n)
    ws = x.new_empty(size // 2)
    _call(dev, raw.load().gdn_ssm_scan_bwd, *ptrs, grad_out.data_ptr(), cu_seqlens.data_ptr(), sp, gsp, rows[0].data_ptr(),
          grad_dt.data_ptr(), grad_a.data_ptr(), rows[1].data_ptr(), rows[2].data_ptr(), raw._ptr(grad_D), raw._ptr(grad_bias),
          raw._ptr(grad_S0), *strides, gs, *gstrides, t, r, h, p, g, n, *types, zero_rest, ws.data_ptr(), size)
    return rows[0], grad_dt, grad_a, rows[1], rows[2], grad_D, grad_bias, grad_S0


@_on_stream
def ssm_step(x, dt, a, B, C, S, D=None, dt_bias=None, out=None):
    """One token for each of R sequences of ssm_scan: x [R, H, P], dt [R, H], B, C [R, G, N], in place on S [R, H, N, P]
    float32.  Returns out [R, H, P] bf16, which may not be x."""
    dev, ptrs, strides, (r, h, p, g, n), types = _scan_inputs(x, dt, a, B, C, D, dt_bias, "ssm_step")
    _dense(S, "S", (r, h, n, p), torch.float32, dev)
    if out is None:
        out = x.new_empty((r, h, p))
    else:
        _dense(out, "out", (r, h, p), torch.bfloat16, dev)
    _call(dev, raw.load().gdn_ssm_step, *ptrs, S.data_ptr(), out.data_ptr(), *strides, r, h, p, g, n, *types)
    return out
