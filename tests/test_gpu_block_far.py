"""Rows as far apart as the entry points around a recurrent layer take them, and states of more than 4 GiB: bit for bit what
the same rows give side by side."""
import pytest

from gpu_util import note, torch_dev

pytestmark = pytest.mark.gpu


def far(torch, rows, stride):
    """The same rows, `stride` elements apart."""
    wide = torch.empty((rows.shape[0] - 1) * stride + rows[0].numel(), device="cuda", dtype=rows.dtype)
    out = wide.as_strided(rows.shape, (stride, *rows[0].contiguous().stride()))
    out.copy_(rows)
    return out


def make(torch, *shape, dtype=None):
    return torch.randn(*shape, device="cuda").to(dtype or torch.bfloat16)


@pytest.mark.parametrize("h,p,g,n", [(3, 64, 1, 128), (2, 128, 1, 64), (5, 64, 1, 64)])
def test_scan_rows_far_apart(h, p, g, n):
    """Strides of x, B and C next to 2^24, of dt past 2^25; pieces of 64 rows and of a few."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"scan far h{h} p{p} g{g} n{n}")
    t, step = 133, (1 << 24) - 8
    cu = torch.tensor([0, 130, 133], dtype=torch.int32, device="cuda")
    x, B, C, go, dt = make(torch, t, h, p), make(torch, t, g, n), make(torch, t, g, n), make(torch, t, h, p), make(torch, t, h)
    a, D, bias, S0 = -torch.rand(h, device="cuda") - 1, make(torch, h, dtype=torch.float32), make(torch, h, dtype=torch.float32), make(torch, 2, h, n, p, dtype=torch.float32)
    more = dict(D=D, dt_bias=bias, S0=S0)
    want = gdn.ssm_scan(x, dt, a, B, C, cu, **more)
    grads = gdn.ssm_scan_bwd(x, dt, a, B, C, go, cu, **more, grad_S_final=S0)
    fx, fB, fC = (far(torch, v, step) for v in (x, B, C))
    fdt = far(torch, dt, (1 << 25) + 1)
    got = gdn.ssm_scan(fx, fdt, a, fB, fC, cu, **more)
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    fgo, gx, gB, gC = (far(torch, v, step) for v in (go, torch.zeros_like(x), torch.zeros_like(B), torch.zeros_like(C)))
    got = gdn.ssm_scan_bwd(fx, fdt, a, fB, fC, fgo, cu, **more, grad_S_final=S0, grad_x=gx, grad_B=gB, grad_C=gC)
    assert all(torch.equal(u, v) for u, v in zip(got, grads))
    S, S2 = S0.clone(), S0.clone()
    y = gdn.ssm_step(x[:2], dt[:2], a, B[:2], C[:2], S, D=D, dt_bias=bias)
    y2 = gdn.ssm_step(fx[:2], fdt[:2], a, fB[:2], fC[:2], S2, D=D, dt_bias=bias)
    assert torch.equal(y, y2) and torch.equal(S, S2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_and_convolution_rows_far_apart(dtype):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"norm and convolution far {dtype}")
    kind = torch.bfloat16 if dtype == "bf16" else torch.float32
    t, c, step = 4, 520, (1 << 31) + 8
    x, r, g = (make(torch, t, c, dtype=kind) for _ in range(3))
    w, w4, cu = make(torch, c, dtype=torch.float32), make(torch, c, 4, dtype=torch.float32), torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    fx, fg = far(torch, x, step), far(torch, g, step)
    for u, v in ((gdn.rms_norm(x, w, r), gdn.rms_norm(fx, w, r)), (gdn.rms_norm(r, w, x), gdn.rms_norm(r, w, fx)),
                 (gdn.rms_norm_bwd(x, w, g, grad_sum=r), gdn.rms_norm_bwd(fx, w, fg, grad_sum=r)),
                 (gdn.short_conv(x, w4, cu), gdn.short_conv(fx, w4, cu)),
                 (gdn.short_conv_bwd(x, w4, g, cu)[:2], gdn.short_conv_bwd(fx, w4, fg, cu)[:2])):
        assert all(torch.equal(a, b) for a, b in zip(u, v))
    st, st2 = (torch.zeros(t, 3, c, device="cuda", dtype=kind) for _ in range(2))
    assert torch.equal(gdn.short_conv_step(x, w4, st), gdn.short_conv_step(fx, w4, st2)) and torch.equal(st, st2)


def test_states_past_4_GiB():
    """6000 sequences of one row, whose states take 4.7 GB: the scan's are the step's, and the last ones' gradients those of a call
    of their own."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note("states past 4 GiB")
    r, h, p, n = 6000, 24, 64, 128
    args = make(torch, r, h, p), make(torch, r, h), -torch.rand(h, device="cuda") - 1, make(torch, r, 1, n), make(torch, r, 1, n)
    S0 = make(torch, r, h, n, p, dtype=torch.float32)
    cu = torch.arange(r + 1, dtype=torch.int32, device="cuda")
    out, last = gdn.ssm_scan(*args, cu, S0=S0)
    S = S0.clone()
    y = gdn.ssm_step(*args, S)
    # each piece is one row: two ways to the same, within float32's and the outputs' rounding
    assert all((last[i:i + 500] - S[i:i + 500]).norm() <= 2e-6 * S[i:i + 500].norm() for i in range(0, r, 500))
    assert (out.float() - y.float()).norm() <= 4e-3 * y.float().norm()
    del S, y
    go = make(torch, r, h, p)
    grads = gdn.ssm_scan_bwd(*args, go, cu, S0=S0, grad_S_final=S0)
    few = [v if v.dim() == 1 else v[-3:] for v in args]
    some = gdn.ssm_scan_bwd(*few, go[-3:], cu[:4], S0=S0[-3:], grad_S_final=S0[-3:])
    for k in (0, 1, 3, 4, 7):
        assert (grads[k][-3:].float() - some[k].float()).norm() <= 4e-3 * some[k].float().norm(), k
    assert (grads[7][-3:] - some[7]).norm() <= 2e-6 * some[7].norm()
