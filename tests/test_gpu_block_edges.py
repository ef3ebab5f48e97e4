"""Edges of the entry points around a recurrent layer: steps and decays of all sizes with their gradients, offsets that lead
outside with every result between guards, and the statuses behind refusals.  Tolerances of the scan: test_gpu_scan.py; of the
convolution: test_gpu_block.py."""
import numpy as np
import pytest

from gpu_util import down, note, torch_dev
from oracle import block as ref
from test_gpu_block import CHAIN, TERM, U, near
from test_gpu_scan import Case, check, check_gradients

pytestmark = pytest.mark.gpu


def normal(torch, seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).cuda()


# ------------------------------------------------------------ steps of all sizes
STEPS = {"none to hundreds": [-200.0, -30.0, 0.0, 300.0], "small": [-30.0, -12.0, -8.0, -4.0], "one decay in a row": [-3.0, -3.0, -3.0, 100.0]}


@pytest.mark.parametrize("kind", STEPS)
@pytest.mark.parametrize("n,p", [(64, 64), (128, 64), (64, 128)])
def test_gradients_with_steps_of_all_sizes(kind, n, p):
    """Element by element and in norm, as for ordinary steps: a decay that forgets all leaves terms of zero, and a weight behind
    strong decays is off by at most 13 roundings of 2^-24 of their sum E in the piece (six additions for each of two sums, and
    log d_j - G_j), 9 E 2^-24 of itself, which the room has (16 E)."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"steps of all sizes: {kind} n{n} p{p}")
    t, h = 200, 4
    c = Case(torch, [0, 150, t], t, h, p, 1, n, dt="f32", param="f32")
    at = np.random.default_rng(8).integers(0, 4, (t, h)) if kind == "one decay in a row" else np.arange(t * h).reshape(t, h) * 7 % 4
    c.dt = torch.tensor(STEPS[kind], device="cuda")[torch.from_numpy(at).cuda()].contiguous()
    c.bias.zero_()
    c.x = (c.x / 64).contiguous()
    out, last = gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
    check(c, out, last, 5)
    go, gl = normal(torch, 1, t, h, p).to(torch.bfloat16), normal(torch, 2, 2, h, n, p)
    got = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0, grad_S_final=gl)
    check_gradients(c, got, down(go).astype(np.float64), down(gl).astype(np.float64))


def test_weights_behind_strong_decays():
    """Rows of small steps behind forty that forget all: out within what rounding leaves in norm."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note("weights behind strong decays")
    t, h = 128, 4
    c = Case(torch, [0, t], t, h, 64, 1, 128, dt="f32", param="f32", slow=True)
    c.dt = torch.where(torch.arange(t, device="cuda")[:, None] % 64 < 40, 500.0, 0.0).expand(t, h).contiguous()
    out, last = gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
    ins, S0 = c.numbers()
    want, want_last = ref.ssm_scan(*ins, c.cu, S0)
    for lo in (40, 104):
        rows = slice(lo, lo + 24)
        rel = np.linalg.norm(down(out)[rows] - want[rows]) / np.linalg.norm(want[rows])
        print(f"[parity] rows {lo}..: norm {rel:.2e}", flush=True)
        assert rel <= 4e-3
    rel = np.linalg.norm(down(last) - want_last) / np.linalg.norm(want_last)
    print(f"[parity] S: norm {rel:.2e}", flush=True)
    assert rel <= 2e-6


@pytest.mark.parametrize("log2_keep", [-1.0, -100.0, -125.5, -130.0, -159.0, -161.0, -1000.0])
def test_what_a_large_state_keeps(log2_keep):
    """A decay is a float32 number, which ends at 2^-126: a state of any size is off by at most that much of itself, and by the
    exponent's roundings (log2 e, its product with a, softplus to four, the product with it: 7 2^-24 of the exponent, 0.7 of that
    as a factor)."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"large state, log2 of its decay {log2_keep}")
    h = 2
    c = Case(torch, [0, 1], 1, h, 64, 1, 64, dt="f32", param="f32")
    c.x, c.dt = torch.zeros_like(c.x), torch.full((1, h), 1.0, device="cuda")
    c.bias.zero_()
    d = float(np.log1p(np.e))
    c.a = torch.full((h,), log2_keep * float(np.log(2)) / d, device="cuda")
    c.S0 *= 2.0 ** 100
    _, last = gdn.ssm_scan(*c.args(), c.offsets, dt_bias=c.bias, S0=c.S0)
    S = c.S0.clone()
    gdn.ssm_step(*c.args(), S, dt_bias=c.bias)
    keep = np.exp(down(c.a).astype(np.float64)[0] * d)
    S0 = down(c.S0).astype(np.float64)
    for got in (last, S):
        assert (np.abs(down(got) - keep * S0) <= np.abs(S0) * (2.0 ** -126 + keep * (8 + 5 * abs(log2_keep)) * U)).all()


# --------------------------------------------------------- offsets that lead outside
class Guarded:
    """Tensors with as much again before and behind them, whose values have to stay."""

    def __init__(self, torch):
        self.torch, self.all = torch, []

    def make(self, shape, dtype):
        n = int(np.prod(shape))
        pad = -(-n // 8) * 8 + 64
        whole = self.torch.full((2 * pad + n,), 5.0, device="cuda", dtype=dtype)
        self.all.append((whole, pad, n))
        return whole[pad:pad + n].view(shape)

    def stayed(self):
        return all(bool((w[:pad] == 5).all()) and bool((w[pad + n:] == 5).all()) for w, pad, n in self.all)


ASCENDING = [[-5, 3, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1], [40, 50, 60], [-9, -9, -3, 8, 20, 22, 23]]
OTHERS = [[9, 2, 30], [0, 2 ** 31 - 1, 5], [30, -7, 12, 3]]


@pytest.mark.parametrize("cu", ASCENDING + OTHERS)
@pytest.mark.parametrize("w", [2, 4])
def test_conv_offsets_that_lead_outside(cu, w):
    """Ascending ones are clamped to the rows; whatever they are, nothing is written outside the results."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    raw = gdn.gdn
    note(f"conv offsets {cu} w{w}")
    t, c, r, f32 = 21, 72, len(cu) - 1, torch.float32
    x, wt, b, st, g, gl = (normal(torch, i, *s) for i, s in enumerate(((t, c), (c, w), (c,), (r, w - 1, c), (t, c), (r, w - 1, c))))
    offs = torch.tensor(cu, dtype=torch.int32, device="cuda")
    guard = Guarded(torch)
    out, last = guard.make((t, c), f32), guard.make((r, w - 1, c), f32)
    gdn.short_conv(x, wt, offs, bias=b, state=st, out=out, state_final=last)
    grads = [guard.make(s, f32) for s in ((t, c), (c, w), (c,), (r, w - 1, c))]
    size = gdn.gdn_short_conv_bwd_workspace_bytes(t, c, w)
    ws = guard.make((size // 4,), f32)
    assert gdn.gdn_short_conv_bwd(x.data_ptr(), wt.data_ptr(), b.data_ptr(), g.data_ptr(), offs.data_ptr(), st.data_ptr(), gl.data_ptr(),
                                  *(v.data_ptr() for v in grads), c, c, t, r, c, w, raw.GDN_F32, raw.GDN_F32, 1, 1, ws.data_ptr(), size,
                                  torch.cuda.current_stream().cuda_stream) == raw.GDN_OK
    torch.cuda.synchronize()
    assert guard.stayed()
    if cu in OTHERS:
        return
    xn, wn, bn, sn, gn, gln = (down(v).astype(np.float64) for v in (x, wt, b, st, g, gl))
    want, want_last, size_p = ref.short_conv(xn, wn, bn, cu, sn)
    inside = np.zeros(t, bool)
    for _, lo, hi in ref._sequences(cu, t):
        inside[lo:hi] = True
    # an error of p moves silu(p) by at most 1.1 of it
    near("out", down(out)[inside], want[inside], "f32", 1.1 * (CHAIN + TERM) * U * size_p[inside])
    assert (down(out)[~inside] == 5).all() and (down(last) == want_last).all()
    grads64, sizes = ref.short_conv_bwd(xn, wn, bn, cu, gn, sn, gln)
    # silu' follows p, with a slope of 1/2 at most: what p is off by, of the largest p
    slope = (8 + TERM) * U * (1 + size_p.max(initial=0.0))
    most, cols = np.abs(gn).max(), np.abs(gn).sum(0).max()
    extra = (slope * most * w * np.abs(wn).max(), slope * 2 * cols * max(np.abs(xn).max(), np.abs(sn).max()), slope * 2 * cols,
             slope * most * w * np.abs(wn).max())
    for name, got, want, size, more in zip(("x", "weight", "bias", "state"), grads, grads64, sizes, extra):
        near(name, down(got), want, "f32", (CHAIN + TERM) * U * 1.1 * size + more)


@pytest.mark.parametrize("cu", [[-5, 30, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1], [400, 500, 600], [90, 20, 300], [0, 2 ** 31 - 1, 5]])
@pytest.mark.parametrize("n", [64, 128])
def test_scan_offsets_that_lead_outside(cu, n):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    raw = gdn.gdn
    note(f"scan offsets {cu} n{n}")
    t, h, p, g, r, bf, f32 = 300, 4, 64, 2, len(cu) - 1, torch.bfloat16, torch.float32
    c = Case(torch, cu, t, h, p, g, n, param="f32")
    guard = Guarded(torch)
    out, last = guard.make((t, h, p), bf), guard.make((r, h, n, p), f32)
    gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0, out=out, S_final=last)
    go, gl = normal(torch, 1, t, h, p).to(bf), normal(torch, 2, r, h, n, p)
    grads = [guard.make(*s) for s in (((t, h, p), bf), ((t, h), bf), ((h,), f32), ((t, g, n), bf), ((t, g, n), bf), ((h,), f32), ((h,), f32),
                                      ((r, h, n, p), f32))]
    size = gdn.gdn_ssm_scan_bwd_workspace_bytes(t, r, h, p, g, n)
    ws = guard.make((size // 4,), f32)
    ptr = lambda v: v.data_ptr()  # noqa: E731
    assert gdn.gdn_ssm_scan_bwd(*map(ptr, (*c.args(), c.D, c.bias, go, c.offsets, c.S0, gl, *grads)), c.x.stride(0), c.dt.stride(0),
                                c.B.stride(0), c.C.stride(0), h * p, h * p, g * n, g * n, t, r, h, p, g, n, raw.GDN_BF16, raw.GDN_BF16,
                                raw.GDN_F32, 1, ptr(ws), size, torch.cuda.current_stream().cuda_stream) == raw.GDN_OK
    torch.cuda.synchronize()
    assert guard.stayed()
    if sorted(cu) != cu:
        return
    inside = np.zeros(t, bool)
    for _, lo, hi in ref._sequences(cu, t):
        inside[lo:hi] = True
    assert (down(out)[~inside] == 5).all()
    out[torch.from_numpy(~inside).cuda()] = 0
    check(c, out, last, 2 + t // 64)
    check_gradients(c, grads, down(go).astype(np.float64), down(gl).astype(np.float64))


# --------------------------------------------------------------------- statuses
def test_refusals_have_their_status():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    raw = gdn.gdn
    x, w, cu = torch.randn(8, 64, device="cuda"), torch.randn(64, device="cuda"), torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    wide = torch.randn(1, 16392, device="cuda")
    for call, status in ((lambda: gdn.rms_norm(x[:1, :60].contiguous(), w[:60].contiguous()), raw.GDN_ERR_UNSUPPORTED),
                         (lambda: gdn.rms_norm(wide, wide[0]), raw.GDN_ERR_UNSUPPORTED),
                         (lambda: gdn.rms_norm(x, w, eps=float("nan")), raw.GDN_ERR_SHAPE),
                         (lambda: gdn.rms_norm_quant(x, w, block=0, eps=-1.0), raw.GDN_ERR_SHAPE),
                         (lambda: gdn.rms_norm_bwd(x, w, x.clone(), eps=float("inf")), raw.GDN_ERR_SHAPE),
                         (lambda: gdn.short_conv(x, torch.randn(64, 5, device="cuda"), cu), raw.GDN_ERR_UNSUPPORTED),
                         (lambda: gdn.short_conv(x, torch.randn(64, 1, device="cuda"), cu), raw.GDN_ERR_UNSUPPORTED),
                         (lambda: gdn.short_conv(x, torch.randn(64, 4, device="cuda"), cu, out=x), raw.GDN_ERR_UNSUPPORTED),
                         (lambda: gdn.short_conv_step(x, torch.randn(64, 4, device="cuda"), torch.randn(8, 3, 64, device="cuda"), out=x),
                          raw.GDN_ERR_UNSUPPORTED),
                         (lambda: gdn.rms_norm(x[:, :32], w[:32], out=x.view(-1)[:256].view(8, 32)), raw.GDN_ERR_UNSUPPORTED)):
        with pytest.raises(gdn.GdnError) as e:
            call()
        assert e.value.status == status
