"""Refusals of the entry points around a recurrent layer (norm, short convolution, state space scan), on the CPU: no call
here reaches a kernel (each fails validation or has nothing to do)."""
import pytest

import linear_attention_sequence_gated_amd as gdn
from linear_attention_sequence_gated_amd import gdn as raw

A = 0x10000  # a 16-byte aligned fake address; validation rejects before any use
NAN = float("nan")


def each(names, value, status):
    return [(dict([(n, value)]), status) for n in names]


TYPES = [(dict(dtype=7), raw.GDN_ERR_DTYPE), (dict(weight_dtype=-1), raw.GDN_ERR_DTYPE),
         (dict(dtype=raw.GDN_C64), raw.GDN_ERR_UNSUPPORTED), (dict(weight_dtype=raw.GDN_C64), raw.GDN_ERR_UNSUPPORTED),
         (dict(dtype=raw.GDN_F32, weight_dtype=raw.GDN_BF16), raw.GDN_ERR_UNSUPPORTED)]
NORM = TYPES + [(dict(T=-1), raw.GDN_ERR_SHAPE), (dict(T=1 << 24), raw.GDN_ERR_SHAPE), (dict(C=0), raw.GDN_ERR_SHAPE),
                (dict(eps=NAN), raw.GDN_ERR_SHAPE), (dict(eps=-1e-6), raw.GDN_ERR_SHAPE), (dict(eps=float("inf")), raw.GDN_ERR_SHAPE)]


def norm(**kw):
    args = dict(x=A, residual=A, weight=A, out=A, sum=A, eps=1e-6, x_stride=256, residual_stride=256, T=4, C=256,
                dtype=raw.GDN_BF16, weight_dtype=raw.GDN_BF16, stream=None)
    args.update(kw)
    return gdn.gdn_rms_norm(**args)


@pytest.mark.parametrize("kw,status", NORM + [
    (dict(C=252, x_stride=256), raw.GDN_ERR_UNSUPPORTED), (dict(C=16392, x_stride=16392, residual_stride=16392), raw.GDN_ERR_UNSUPPORTED),
    (dict(x_stride=248), raw.GDN_ERR_SHAPE), (dict(x_stride=260), raw.GDN_ERR_SHAPE), (dict(residual_stride=248), raw.GDN_ERR_SHAPE),
    (dict(x_stride=1 << 32), raw.GDN_ERR_SHAPE),
    *each(("x", "weight", "out", "sum"), None, raw.GDN_ERR_NULL),
    *each(("x", "residual", "weight", "out", "sum"), A + 8, raw.GDN_ERR_ALIGN)])
def test_norm_argument_errors(kw, status):
    assert norm(**kw) == status


def test_norm_of_nothing_is_noop():
    assert norm(T=0, x=None, residual=None, weight=None, out=None, sum=None) == raw.GDN_OK


def quant(**kw):
    args = dict(x=A, residual=A, weight=A, codes=A, scale=A, sum=A, eps=1e-6, x_stride=256, residual_stride=256, T=4,
                C=256, block=128, dtype=raw.GDN_BF16, weight_dtype=raw.GDN_BF16, format=raw.GDN_CACHE_E4M3, stream=None)
    args.update(kw)
    return gdn.gdn_rms_norm_quant(**args)


@pytest.mark.parametrize("kw,status", NORM + [
    (dict(format=2), raw.GDN_ERR_DTYPE), (dict(format=-1), raw.GDN_ERR_DTYPE), (dict(block=-1), raw.GDN_ERR_SHAPE),
    (dict(block=64), raw.GDN_ERR_UNSUPPORTED), (dict(C=192), raw.GDN_ERR_UNSUPPORTED),
    *each(("x", "weight", "codes", "scale", "sum"), None, raw.GDN_ERR_NULL),
    *each(("x", "residual", "weight", "codes", "scale", "sum"), A + 4, raw.GDN_ERR_ALIGN)])
def test_quant_argument_errors(kw, status):
    assert quant(**kw) == status


def norm_bwd(**kw):
    args = dict(sum=A, weight=A, grad_out=A, grad_sum=A, grad_x=A, grad_weight=A, eps=1e-6, sum_stride=256,
                grad_out_stride=256, grad_sum_stride=256, T=4, C=256, dtype=raw.GDN_BF16, weight_dtype=raw.GDN_BF16,
                workspace=A, workspace_bytes=1 << 40, stream=None)
    args.update(kw)
    return gdn.gdn_rms_norm_bwd(**args)


@pytest.mark.parametrize("kw,status", NORM + [
    (dict(sum_stride=248), raw.GDN_ERR_SHAPE), (dict(grad_out_stride=260), raw.GDN_ERR_SHAPE), (dict(grad_sum_stride=0), raw.GDN_ERR_SHAPE),
    *each(("sum", "weight", "grad_out", "grad_x", "grad_weight"), None, raw.GDN_ERR_NULL),
    *each(("sum", "weight", "grad_out", "grad_sum", "grad_x", "grad_weight", "workspace"), A + 8, raw.GDN_ERR_ALIGN),
    (dict(workspace=None), raw.GDN_ERR_WORKSPACE), (dict(workspace_bytes=0), raw.GDN_ERR_WORKSPACE)])
def test_norm_bwd_argument_errors(kw, status):
    assert norm_bwd(**kw) == status


def test_norm_bwd_workspace():
    need = gdn.gdn_rms_norm_bwd_workspace_bytes(4, 256, raw.GDN_BF16)
    assert need > 0 and norm_bwd(workspace_bytes=need - 1) == raw.GDN_ERR_WORKSPACE
    assert gdn.gdn_rms_norm_bwd_workspace_bytes(0, 256, raw.GDN_BF16) == 0
    assert gdn.gdn_rms_norm_bwd_workspace_bytes(4, 252, raw.GDN_BF16) == 0  # unsupported arguments
    assert gdn.gdn_rms_norm_bwd_workspace_bytes(4, 256, raw.GDN_C64) == 0


CONV = TYPES + [(dict(C=0), raw.GDN_ERR_SHAPE), (dict(W=0), raw.GDN_ERR_SHAPE), (dict(R=-1), raw.GDN_ERR_SHAPE),
                (dict(R=1 << 20), raw.GDN_ERR_SHAPE), (dict(W=1), raw.GDN_ERR_UNSUPPORTED), (dict(W=5), raw.GDN_ERR_UNSUPPORTED),
                (dict(C=60, x_stride=64), raw.GDN_ERR_UNSUPPORTED), (dict(C=65544, x_stride=65544), raw.GDN_ERR_UNSUPPORTED),
                (dict(x_stride=56), raw.GDN_ERR_SHAPE), (dict(x_stride=68), raw.GDN_ERR_SHAPE)]


def conv(**kw):
    args = dict(x=A, weight=A, bias=A, cu_seqlens=A, state=A, out=A, state_final=A, x_stride=64, T=9, R=2, C=64, W=4,
                dtype=raw.GDN_BF16, weight_dtype=raw.GDN_BF16, silu=1, zero_rest=1, stream=None)
    args.update(kw)
    return gdn.gdn_short_conv(**args)


@pytest.mark.parametrize("kw,status", CONV + [
    (dict(T=-1), raw.GDN_ERR_SHAPE), (dict(T=1 << 28), raw.GDN_ERR_SHAPE), (dict(T=1 << 27, C=1024, x_stride=1024), raw.GDN_ERR_SHAPE),
    (dict(R=1 << 19, C=8192, x_stride=8192), raw.GDN_ERR_SHAPE),
    *each(("x", "weight", "cu_seqlens", "out"), None, raw.GDN_ERR_NULL),
    *each(("x", "weight", "bias", "cu_seqlens", "state", "out", "state_final"), A + 8, raw.GDN_ERR_ALIGN)])
def test_conv_argument_errors(kw, status):
    assert conv(**kw) == status


def test_conv_of_nothing_is_noop():
    none = dict(x=None, weight=None, bias=None, cu_seqlens=None, state=None, out=None)
    assert conv(T=0, R=0, **none) == raw.GDN_OK
    assert conv(T=0, state_final=None, **none) == raw.GDN_OK


def conv_bwd(**kw):
    args = dict(x=A, weight=A, bias=A, grad_out=A, cu_seqlens=A, state=A, grad_state_final=A, grad_x=A, grad_weight=A,
                grad_bias=A, grad_state=A, x_stride=64, grad_out_stride=64, T=9, R=2, C=64, W=4, dtype=raw.GDN_BF16,
                weight_dtype=raw.GDN_BF16, silu=1, zero_rest=1, workspace=A, workspace_bytes=1 << 40, stream=None)
    args.update(kw)
    return gdn.gdn_short_conv_bwd(**args)


@pytest.mark.parametrize("kw,status", CONV + [
    (dict(T=-1), raw.GDN_ERR_SHAPE), (dict(grad_out_stride=56), raw.GDN_ERR_SHAPE),
    *each(("x", "weight", "grad_out", "cu_seqlens", "grad_x", "grad_weight"), None, raw.GDN_ERR_NULL),
    *each(("x", "weight", "bias", "grad_out", "cu_seqlens", "state", "grad_state_final", "grad_x", "grad_weight", "grad_bias",
           "grad_state", "workspace"), A + 8, raw.GDN_ERR_ALIGN),
    (dict(workspace=None), raw.GDN_ERR_WORKSPACE), (dict(workspace_bytes=0), raw.GDN_ERR_WORKSPACE)])
def test_conv_bwd_argument_errors(kw, status):
    assert conv_bwd(**kw) == status


def test_conv_bwd_workspace():
    need = gdn.gdn_short_conv_bwd_workspace_bytes(9, 64, 4)
    assert need == 64 * 5 * 4 and conv_bwd(workspace_bytes=need - 1) == raw.GDN_ERR_WORKSPACE
    assert gdn.gdn_short_conv_bwd_workspace_bytes(0, 64, 4) == 0
    assert gdn.gdn_short_conv_bwd_workspace_bytes(9, 64, 5) == 0  # unsupported arguments


def conv_step(**kw):
    args = dict(x=A, weight=A, bias=A, state=A, out=A, x_stride=64, R=2, C=64, W=4, dtype=raw.GDN_BF16,
                weight_dtype=raw.GDN_BF16, silu=1, stream=None)
    args.update(kw)
    return gdn.gdn_short_conv_step(**args)


@pytest.mark.parametrize("kw,status", CONV + [
    *each(("x", "weight", "state", "out"), None, raw.GDN_ERR_NULL),
    *each(("x", "weight", "bias", "state", "out"), A + 8, raw.GDN_ERR_ALIGN)])
def test_conv_step_argument_errors(kw, status):
    assert conv_step(**kw) == status


def test_conv_step_of_nothing_is_noop():
    assert conv_step(R=0, x=None, weight=None, state=None, out=None) == raw.GDN_OK


def test_helpers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    x, w, cu = torch.zeros(4, 64), torch.ones(64), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.rms_norm(x, w)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.rms_norm_quant(x, w)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.rms_norm_bwd(x, w, x)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.short_conv(x, torch.zeros(64, 4), cu)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.short_conv_bwd(x, torch.zeros(64, 4), x, cu)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.short_conv_step(x, torch.zeros(64, 4), torch.zeros(4, 3, 64))


# ------------------------------------------------------------------------ scan
SCAN = [(dict(dtype=7), raw.GDN_ERR_DTYPE), (dict(dt_dtype=-1), raw.GDN_ERR_DTYPE), (dict(param_dtype=9), raw.GDN_ERR_DTYPE),
        (dict(dtype=raw.GDN_F32), raw.GDN_ERR_UNSUPPORTED), (dict(dt_dtype=raw.GDN_C64), raw.GDN_ERR_UNSUPPORTED),
        (dict(param_dtype=raw.GDN_C64), raw.GDN_ERR_UNSUPPORTED), (dict(R=-1), raw.GDN_ERR_SHAPE), (dict(R=1 << 20), raw.GDN_ERR_SHAPE),
        (dict(H=0), raw.GDN_ERR_SHAPE), (dict(P=0), raw.GDN_ERR_SHAPE), (dict(G=0), raw.GDN_ERR_SHAPE), (dict(N=0), raw.GDN_ERR_SHAPE),
        (dict(G=3), raw.GDN_ERR_SHAPE), (dict(H=1 << 16, x_stride=1 << 23), raw.GDN_ERR_SHAPE), (dict(R=1 << 19, H=8), raw.GDN_ERR_SHAPE),
        (dict(P=32), raw.GDN_ERR_UNSUPPORTED), (dict(P=192), raw.GDN_ERR_UNSUPPORTED), (dict(N=16), raw.GDN_ERR_UNSUPPORTED),
        (dict(N=256), raw.GDN_ERR_UNSUPPORTED), (dict(x_stride=248), raw.GDN_ERR_SHAPE), (dict(x_stride=260), raw.GDN_ERR_SHAPE),
        (dict(B_stride=120), raw.GDN_ERR_SHAPE), (dict(C_stride=132), raw.GDN_ERR_SHAPE), (dict(dt_stride=3), raw.GDN_ERR_SHAPE)]


def scan(**kw):
    args = dict(x=A, dt=A + 2, a=A + 2, B=A, C=A, D=A, dt_bias=A, cu_seqlens=A, S0=A, out=A, S_final=A, x_stride=256, dt_stride=4,
                B_stride=128, C_stride=128, T=9, R=2, H=4, P=64, G=2, N=64, dtype=raw.GDN_BF16, dt_dtype=raw.GDN_BF16,
                param_dtype=raw.GDN_BF16, zero_rest=1, workspace=A, workspace_bytes=1 << 40, stream=None)
    args.update(kw)
    return gdn.gdn_ssm_scan(**args)


@pytest.mark.parametrize("kw,status", SCAN + [
    (dict(T=-1), raw.GDN_ERR_SHAPE), (dict(T=1 << 26), raw.GDN_ERR_SHAPE), (dict(x_stride=1 << 24), raw.GDN_ERR_SHAPE),
    (dict(T=1 << 25, H=64, x_stride=4096, dt_stride=64), raw.GDN_ERR_SHAPE),
    *each(("x", "dt", "a", "B", "C", "cu_seqlens", "out"), None, raw.GDN_ERR_NULL),
    *each(("x", "B", "C", "cu_seqlens", "S0", "out", "S_final", "workspace"), A + 8, raw.GDN_ERR_ALIGN),
    *each(("dt", "a", "D", "dt_bias"), A + 1, raw.GDN_ERR_ALIGN), (dict(dt_dtype=raw.GDN_F32), raw.GDN_ERR_ALIGN),
    (dict(T=1000, workspace=None), raw.GDN_ERR_WORKSPACE), (dict(T=1000, workspace_bytes=0), raw.GDN_ERR_WORKSPACE)])
def test_scan_argument_errors(kw, status):
    assert scan(**kw) == status


def test_scan_of_nothing_is_noop():
    none = dict(x=None, dt=None, a=None, B=None, C=None, cu_seqlens=None, out=None, S0=None, workspace=None)
    assert scan(T=0, R=0, **none) == raw.GDN_OK
    assert scan(T=0, S_final=None, **none) == raw.GDN_OK


def test_scan_workspace():
    need = gdn.gdn_ssm_scan_workspace_bytes(1000, 4, 64, 2, 64)  # four segments of 256 rows: three borders
    assert need == 3 * 4 * (64 * 64 + 1) * 4 and scan(T=1000, workspace_bytes=need - 1) == raw.GDN_ERR_WORKSPACE
    assert gdn.gdn_ssm_scan_workspace_bytes(256, 4, 64, 2, 64) == 0  # one segment
    assert gdn.gdn_ssm_scan_workspace_bytes(1000, 4, 96, 2, 64) == 0  # unsupported arguments


def scan_bwd(**kw):
    args = dict(x=A, dt=A + 2, a=A, B=A, C=A, D=A, dt_bias=A, grad_out=A, cu_seqlens=A, S0=A, grad_S_final=A, grad_x=A, grad_dt=A,
                grad_a=A, grad_B=A, grad_C=A, grad_D=A, grad_dt_bias=A, grad_S0=A, x_stride=256, dt_stride=4, B_stride=128,
                C_stride=128, grad_out_stride=256, grad_x_stride=256, grad_B_stride=128, grad_C_stride=128, T=9, R=2, H=4, P=64,
                G=2, N=64, dtype=raw.GDN_BF16, dt_dtype=raw.GDN_BF16, param_dtype=raw.GDN_BF16, zero_rest=1, workspace=A,
                workspace_bytes=1 << 60, stream=None)
    args.update(kw)
    return gdn.gdn_ssm_scan_bwd(**args)


@pytest.mark.parametrize("kw,status", SCAN + [
    (dict(T=-1), raw.GDN_ERR_SHAPE), (dict(T=1 << 26), raw.GDN_ERR_SHAPE), (dict(grad_out_stride=248), raw.GDN_ERR_SHAPE),
    (dict(grad_x_stride=252), raw.GDN_ERR_SHAPE), (dict(grad_B_stride=64), raw.GDN_ERR_SHAPE), (dict(grad_C_stride=1 << 24), raw.GDN_ERR_SHAPE),
    *each(("x", "dt", "a", "B", "C", "grad_out", "cu_seqlens", "grad_x", "grad_dt", "grad_a", "grad_B", "grad_C"), None, raw.GDN_ERR_NULL),
    *each(("x", "B", "C", "grad_out", "cu_seqlens", "S0", "grad_S_final", "grad_x", "grad_dt", "grad_B", "grad_C", "grad_S0", "workspace"),
          A + 8, raw.GDN_ERR_ALIGN),
    *each(("dt", "a", "D", "dt_bias", "grad_a", "grad_D", "grad_dt_bias"), A + 1, raw.GDN_ERR_ALIGN),
    (dict(workspace=None), raw.GDN_ERR_WORKSPACE), (dict(workspace_bytes=0), raw.GDN_ERR_WORKSPACE)])
def test_scan_bwd_argument_errors(kw, status):
    assert scan_bwd(**kw) == status


def test_scan_bwd_workspace():
    need = gdn.gdn_ssm_scan_bwd_workspace_bytes(9, 2, 4, 64, 2, 64)
    # two states for each of 1 + 2 pieces at most, three sums a head, gB and gC of both heads of a group apart
    states, heads, shares = 3 * 4 * 64 * 64 * 2, 256, 2 * 2 * 9 * 2 * 64 * 4
    assert need == 2 * states + heads + shares and scan_bwd(workspace_bytes=need - 1) == raw.GDN_ERR_WORKSPACE
    assert gdn.gdn_ssm_scan_bwd_workspace_bytes(9, 2, 4, 64, 2, 32) == 0  # unsupported arguments


def step(**kw):
    args = dict(x=A, dt=A + 2, a=A, B=A, C=A, D=A, dt_bias=A, S=A, out=A, x_stride=256, dt_stride=4, B_stride=128, C_stride=128,
                R=2, H=4, P=64, G=2, N=64, dtype=raw.GDN_BF16, dt_dtype=raw.GDN_BF16, param_dtype=raw.GDN_BF16, stream=None)
    args.update(kw)
    return gdn.gdn_ssm_step(**args)


@pytest.mark.parametrize("kw,status", SCAN + [
    *each(("x", "dt", "a", "B", "C", "S", "out"), None, raw.GDN_ERR_NULL), *each(("x", "B", "C", "S", "out"), A + 8, raw.GDN_ERR_ALIGN),
    *each(("dt", "a", "D", "dt_bias"), A + 1, raw.GDN_ERR_ALIGN)])
def test_step_argument_errors(kw, status):
    assert step(**kw) == status


def test_step_of_nothing_is_noop():
    assert step(R=0, x=None, dt=None, a=None, B=None, C=None, S=None, out=None) == raw.GDN_OK


def test_scan_helpers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    x, dt, a, B = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 2), torch.zeros(2), torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.ssm_scan(x, dt, a, B, B, cu)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.ssm_scan_bwd(x, dt, a, B, B, x, cu)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.ssm_step(x, dt, a, B, B, torch.zeros(4, 2, 64, 64))


OTHER = A + 0x10000


@pytest.mark.parametrize("call,apart,pairs", [
    (conv, ("out", "state_final"), [("x", "out"), ("state", "state_final")]),
    (conv_bwd, ("grad_x", "grad_state"), [("x", "grad_x"), ("grad_out", "grad_x"), ("state", "grad_state"), ("grad_state_final", "grad_state")]),
    (scan, ("out", "S_final"), [("x", "out"), ("S0", "S_final")]),
    (scan_bwd, ("grad_x", "grad_B", "grad_C", "grad_S0"), [("x", "grad_x"), ("grad_out", "grad_x"), ("B", "grad_B"), ("C", "grad_C"),
                                                           ("S0", "grad_S0"), ("grad_S_final", "grad_S0")])])
def test_results_in_place_of_what_is_read_are_refused(call, apart, pairs):
    for read, written in pairs:
        kw = {k: OTHER + 0x1000 * i for i, k in enumerate(apart)}
        kw[read] = kw[written]
        assert call(**kw) == raw.GDN_ERR_UNSUPPORTED, (read, written)
