"""Results in place of what is read, of the entry points around a recurrent layer: which are refused (on the CPU; no call here
reaches a kernel), and what those that are not give (on the GPU)."""
import pytest

import linear_attention_sequence_gated_amd as gdn
from linear_attention_sequence_gated_amd import gdn as raw
from test_block_abi import A, conv, conv_bwd, conv_step, norm, norm_bwd, quant, scan, scan_bwd, step

FAR = [A + 0x100000 * i for i in range(1, 24)]


def apart(call, names, **kw):
    """call with every buffer of its own, but for those that kw gives by the name of another."""
    at = dict(zip(names, FAR))
    return call(**{**at, **{k: at.get(v, v) for k, v in kw.items()}})


NORM = ("x", "residual", "weight", "out", "sum")
QUANT = ("x", "residual", "weight", "codes", "scale", "sum")
BWD = ("sum", "weight", "grad_out", "grad_sum", "grad_x", "grad_weight", "workspace")


@pytest.mark.parametrize("call,names,kw", [
    (norm, NORM, dict(out="x", x_stride=264)), (norm, NORM, dict(out="residual", residual_stride=264)),
    (norm, NORM, dict(sum="x", x_stride=512)), (norm, NORM, dict(sum="residual", residual_stride=512)), (norm, NORM, dict(sum="out")),
    (quant, QUANT, dict(codes="x")), (quant, QUANT, dict(codes="residual")), (quant, QUANT, dict(codes="sum")), (quant, QUANT, dict(scale="x")),
    (quant, QUANT, dict(scale="residual")), (quant, QUANT, dict(sum="x", x_stride=264)), (quant, QUANT, dict(sum="residual", residual_stride=264)),
    (norm_bwd, BWD, dict(grad_x="sum", sum_stride=264)), (norm_bwd, BWD, dict(grad_x="grad_out", grad_out_stride=264)),
    (norm_bwd, BWD, dict(grad_x="grad_sum", grad_sum_stride=264))])
def test_norm_in_place_of_other_rows_is_refused(call, names, kw):
    assert apart(call, names, **kw) == raw.GDN_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("t,c", [(1, 64), (37, 512), (1500, 768), (33, 1024), (300, 2048), (9, 4096), (5, 8192), (3, 16384)])
def test_norm_in_place_gives_the_same(t, c, dtype, wdtype):
    """The sum in place of the residual (or x), the output in place of either: bit for bit what apart gives."""
    from gpu_util import note, torch_dev
    torch = torch_dev()
    note(f"norm in place {t}x{c} {dtype}")
    kinds = {"bf16": torch.bfloat16, "f32": torch.float32}
    make = lambda *shape: torch.randn(*shape, device="cuda").to(kinds[dtype])  # noqa: E731
    x, r, w = make(t, c), make(t, c), torch.rand(c, device="cuda") + 0.5
    y, s = gdn.rms_norm(x, w, r)
    one = lambda: (x.clone(), r.clone())  # noqa: E731
    a, b = one()
    y2, s2 = gdn.rms_norm(a, w, b, sum_out=b)
    assert s2 is b and torch.equal(y2, y) and torch.equal(b, s) and torch.equal(a, x)
    a, b = one()
    gdn.rms_norm(a, w, b, out=a, sum_out=b)
    assert torch.equal(a, y) and torch.equal(b, s)
    a, b = one()
    gdn.rms_norm(a, w, b, out=b, sum_out=a)
    assert torch.equal(b, y) and torch.equal(a, s)
    a, b = one()
    assert torch.equal(gdn.rms_norm(a, w, out=a)[0], gdn.rms_norm(x, w)[0])
    for dt, block in ((torch.float8_e4m3fn, 128 if c % 128 == 0 else 0), (torch.int8, 0)):
        want = gdn.rms_norm_quant(x, w, r, dtype=dt, block=block)
        a, b = one()
        got = gdn.rms_norm_quant(a, w, b, dtype=dt, block=block, sum_out=b)
        assert all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(got, want)) and torch.equal(b, s)
    g, h = make(t, c), make(t, c)
    gx, gw = gdn.rms_norm_bwd(s, w, g, grad_sum=h)
    code, wcode = (raw.GDN_BF16 if dtype == "bf16" else raw.GDN_F32), raw.GDN_F32
    size = gdn.gdn_rms_norm_bwd_workspace_bytes(t, c, code)
    for at in range(3):
        rows = [s.clone(), g.clone(), h.clone()]
        got_w, ws = torch.empty_like(w), torch.empty(size, dtype=torch.uint8, device="cuda")
        assert gdn.gdn_rms_norm_bwd(rows[0].data_ptr(), w.data_ptr(), rows[1].data_ptr(), rows[2].data_ptr(), rows[at].data_ptr(),
                                    got_w.data_ptr(), 1e-6, c, c, c, t, c, code, wcode, ws.data_ptr(), size,
                                    torch.cuda.current_stream().cuda_stream) == raw.GDN_OK
        torch.cuda.synchronize()
        assert torch.equal(rows[at], gx) and torch.equal(got_w, gw)
        assert all(torch.equal(u, v) for i, (u, v) in enumerate(zip(rows, (s, g, h))) if i != at)


CONV_STEP = ("x", "weight", "bias", "state", "out")
STEP = ("x", "dt", "a", "B", "C", "D", "dt_bias", "S", "out")
SCAN = ("x", "dt", "a", "B", "C", "D", "dt_bias", "cu_seqlens", "S0", "out", "S_final", "workspace")
SCAN_BWD = ("x", "dt", "a", "B", "C", "D", "dt_bias", "grad_out", "cu_seqlens", "S0", "grad_S_final", "grad_x", "grad_dt", "grad_a", "grad_B",
            "grad_C", "grad_D", "grad_dt_bias", "grad_S0", "workspace")
CONV = ("x", "weight", "bias", "cu_seqlens", "state", "out", "state_final")
CONV_BWD = ("x", "weight", "bias", "grad_out", "cu_seqlens", "state", "grad_state_final", "grad_x", "grad_weight", "grad_bias", "grad_state",
            "workspace")


@pytest.mark.parametrize("call,names,reads,writes", [
    (conv, CONV, ("x", "state"), ("out", "state_final")), (conv_bwd, CONV_BWD, ("x", "grad_out", "state", "grad_state_final"), ("grad_x", "grad_state")),
    (conv_step, CONV_STEP, ("x", "state"), ("out",)), (conv_step, CONV_STEP, ("x",), ("state",)),
    (scan, SCAN, ("x", "dt", "B", "C", "S0"), ("out", "S_final")),
    (scan_bwd, SCAN_BWD, ("x", "dt", "B", "C", "grad_out", "S0", "grad_S_final"), ("grad_x", "grad_dt", "grad_B", "grad_C", "grad_S0")),
    (step, STEP, ("x", "dt", "B", "C", "S"), ("out",)), (step, STEP, ("x", "dt", "B", "C"), ("S",))])
def test_results_in_place_of_any_rows_or_states_are_refused(call, names, reads, writes):
    for read in reads:
        for written in writes:
            assert apart(call, names, **{written: read}) == raw.GDN_ERR_UNSUPPORTED, (read, written)


def test_nothing_read_is_nothing_in_place():
    """Without rows (sequences), the addresses of rows (states) say nothing."""
    at = dict(zip(SCAN, FAR))
    assert scan(**{**at, "T": 0, "R": 0, "x": A, "out": A}) == raw.GDN_OK
    assert conv(**{**dict(zip(CONV, FAR)), "T": 0, "R": 0, "x": A, "out": A}) == raw.GDN_OK
