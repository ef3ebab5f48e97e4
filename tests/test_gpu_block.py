"""The norm and the short convolution on the GPU against their fp64 references, element by element.

Tolerances.  A result is rounded once, to nearest: half a step, EPS of itself.  Before that, float32 arithmetic: n
additions one after the other leave n 2^-24 of the sum of the terms' magnitudes.  A sum over a row's channels has chains of
at most 128 (a lane's values, the lanes of a wave, four waves); a sum over rows of at most CHAIN = 256 (rows to a wave,
waves to a workgroup, shares to a thread, threads to a column), at the sizes here.  A term has at most 16 roundings of
2^-24 of its own (products, the square root, a quotient, 2^x and its argument)."""
import numpy as np
import pytest

from gpu_util import down, note, torch_dev
from oracle import block as ref

pytestmark = pytest.mark.gpu

EPS = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U, TERM, CHAIN, TINY = 2.0 ** -24, 16, 256, 1e-30


def near(name, got, want, dtype, slack):
    """|got - want| <= EPS |want| + slack (1 + EPS), at every element."""
    got = got.astype(np.float64)
    assert got.shape == want.shape and np.isfinite(got).all(), name
    room = EPS[dtype] * np.abs(want) + slack * (1 + EPS[dtype]) + TINY
    worst = float((np.abs(got - want) / room).max(initial=0.0))
    print(f"[parity] {name}: worst {worst:.3f} of its room", flush=True)
    assert worst <= 1.0, (name, worst)


class Inputs:
    """Seeded tensors on the device, and the numbers that they hold."""

    def __init__(self, torch, seed):
        self.torch, self.rng = torch, np.random.default_rng(seed)

    def make(self, shape, dtype, scale=1.0, pad=0, mean=0.0):
        x = self.torch.from_numpy((mean + scale * self.rng.standard_normal((*shape[:-1], shape[-1] + pad))).astype(np.float32))
        t = x.to(self.torch.bfloat16 if dtype == "bf16" else self.torch.float32).cuda()
        t = t[..., pad:] if pad else t
        return t, down(t).astype(np.float64)


def host(t):
    return None if t is None else down(t)


# ------------------------------------------------------------------------ norm
SIZES = [(1, 8), (3, 64), (5, 72), (33, 512), (7, 520), (130, 768), (9, 1024), (6, 1032), (40, 2048), (5, 2056), (3, 4096),
         (2, 5000), (2, 8192), (3, 16384)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("t,c", SIZES)
def test_norm_and_its_gradients(t, c, dtype, wdtype):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    for residual in (False, True):
        note(f"norm {t}x{c} {dtype}/{wdtype} residual={residual}")
        make = Inputs(torch, t * c + residual).make
        x, xn = make((t, c), dtype, pad=8)
        w, wn = make((c,), wdtype, 0.2, mean=1.0)
        r = make((t, c), dtype, 3.0)[0] if residual else None
        out, s = gdn.rms_norm(x, w, r, eps=1e-5)
        if residual:
            assert torch.equal(s, (x.float() + r.float()).to(x.dtype))
        else:
            assert s is x
        sn = down(s).astype(np.float64)
        want, rstd = ref.rms_norm(sn, wn, 1e-5)
        near("out", down(out), want, dtype, (128 + TERM) * U * np.abs(want))
        g, gn = make((t, c), dtype, pad=16)
        h, hn = make((t, c), dtype)
        for extra in (None, h):
            gx, gw = gdn.rms_norm_bwd(s, w, g, eps=1e-5, grad_sum=extra)
            a, b, size = ref.rms_norm_bwd(sn, wn, 1e-5, gn, None if extra is None else hn)
            n = sn * rstd
            terms = rstd * (np.abs(wn * gn) + np.abs(n) * np.abs(wn * gn * n).mean(1, keepdims=True)) + (0 if extra is None else np.abs(hn))
            near("grad_x", down(gx), a, dtype, (128 + TERM) * U * terms)
            near("grad_weight", down(gw), b, wdtype, (CHAIN + TERM + 128) * U * size)


@pytest.mark.parametrize("t,c", [(1024, 1024), (1025, 1024), (1500, 520), (1300, 2048)])
def test_norm_of_many_rows(t, c):
    """Rows enough for one wave to each, and a few less."""
    test_norm_and_its_gradients(t, c, "bf16", "bf16")


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("t,c,block", [(1, 8, 0), (5, 72, 0), (33, 768, 0), (3, 2056, 0), (3, 16384, 0), (1, 128, 128), (9, 384, 128),
                                       (40, 2048, 128), (6, 2176, 128), (3, 4096, 128), (2, 16384, 128)])
def test_norm_in_8_bits(t, c, block, dtype, wdtype, kind):
    """Codes are rounded from y / scale, to half a step: 1/2 (int8), or 2^-4 of itself, 2^-10 where that is more (e4m3).
    y / scale is off by the norm's own error and its roundings, of itself."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"quant {t}x{c} block {block} {dtype} {kind}")
    make = Inputs(torch, t + c).make
    x, _ = make((t, c), dtype, pad=8)
    r, _ = make((t, c), dtype)
    x[0] = 0
    r[0] = 0  # a row of zeros
    w, wn = make((c,), wdtype, 0.3, mean=1.0)
    tt = torch.int8 if kind == "int8" else torch.float8_e4m3fn
    codes, scale, s = gdn.rms_norm_quant(x, w, r, dtype=tt, block=block)
    assert torch.equal(s, (x.float() + r.float()).to(x.dtype)) and codes.dtype is tt
    y, _ = ref.rms_norm(down(s).astype(np.float64), wn, 1e-6)
    sc, want = ref.quantise(y, block, kind)
    near("scale", down(scale), sc, "f32", (128 + TERM) * U * sc)
    got = codes.float().cpu().numpy().astype(np.float64)
    half = 0.5 if kind == "int8" else np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10)
    assert (np.abs(got - want) <= half + 2 * (128 + TERM) * U * np.abs(want) + TINY).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_norm_of_values_that_are_not_finite(kind):
    """They reach their own row (block of a scale) alone, and as NaN."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    x = torch.randn(6, 256, device="cuda", dtype=torch.float32)
    w = torch.ones(256, device="cuda")
    clean, _ = gdn.rms_norm(x, w)
    x[1, 7], x[3, 200], x[4, 0] = float("nan"), float("inf"), float("-inf")
    out, _ = gdn.rms_norm(x, w)
    bad = torch.tensor([1, 3, 4], device="cuda")
    fine = torch.tensor([0, 2, 5], device="cuda")
    assert torch.equal(out[fine], clean[fine]) and torch.isnan(out[bad]).any(1).all()
    tt = torch.int8 if kind == "int8" else torch.float8_e4m3fn
    codes, scale, _ = gdn.rms_norm_quant(x, w, dtype=tt)
    value = (codes.float().view(6, 2, 128) * scale[..., None]).view(6, 256)
    assert torch.isfinite(value[fine]).all() and torch.isnan(value[bad]).any(1).all()
    assert (torch.isnan(out) <= torch.isnan(value)).all()
    w[5] = float("inf")  # an infinite value beside finite ones
    codes, scale, _ = gdn.rms_norm_quant(x[fine], w, dtype=tt)
    value = codes.float().view(3, 2, 128) * scale[..., None]
    assert torch.isnan(value[:, 0]).all() and torch.isfinite(value[:, 1]).all()


# ----------------------------------------------------------------- convolution
def offsets(torch, cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


RUNS = [("one row", [0, 1], 1), ("short", [0, 2, 3, 3, 7], 7), ("empty", [0, 0, 0], 0), ("no sequences", [0], 5),
        ("rows outside", [3, 40, 41, 90], 101), ("a run's ends", [0, 32, 64, 127, 128, 130, 256, 257], 257), ("long", [0, 1500, 1501, 2600], 2600),
        ("singles", list(range(700)), 699), ("many short", list(range(0, 1800, 3)), 1797)]


@pytest.mark.parametrize("name,cu,t", RUNS, ids=[r[0] for r in RUNS])
@pytest.mark.parametrize("dtype,wdtype,c,w,act", [("bf16", "bf16", 8, 4, True), ("bf16", "f32", 520, 4, True), ("bf16", "bf16", 1024, 3, True),
                                                  ("f32", "f32", 72, 4, True), ("f32", "f32", 264, 2, True), ("bf16", "bf16", 256, 2, False)])
def test_conv_and_its_gradients(name, cu, t, dtype, wdtype, c, w, act):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    R = len(cu) - 1
    make = Inputs(torch, c + t).make
    x, xn = make((t, c), dtype, pad=24)
    wt, wn = make((c, w), wdtype, 0.5)
    b, bn = make((c,), wdtype)
    st, sn = make((R, w - 1, c), dtype)
    g, gn = make((t, c), dtype, pad=8)
    gl, gln = make((R, w - 1, c), dtype)
    cut = offsets(torch, cu)
    inside = np.zeros(t, bool)
    for lo, hi in zip(cu, cu[1:]):
        inside[lo:hi] = True
    for full in (True, False):
        note(f"conv {name} t{t} c{c} w{w} {dtype}/{wdtype} state={full}")
        bias, state, last_g = (b, st, gl) if full else (None, None, None)
        out, last = gdn.short_conv(x, wt, cut, bias=bias, state=state, silu=act)
        want, want_last, size = ref.short_conv(xn, wn, bn if full else np.zeros(c), cu, sn if full else None, act)
        near("out", down(out), want, dtype, (8 + TERM) * U * 1.1 * size)  # 1.1: the largest slope of silu
        assert np.array_equal(down(last).astype(np.float64), want_last)
        assert not down(out)[~inside].any()
        got = gdn.short_conv_bwd(x, wt, g, cut, bias=bias, state=state, silu=act, grad_state_final=last_g)
        grads, sizes = ref.short_conv_bwd(xn, wn, bn if full else np.zeros(c), cu, gn, sn if full else None, gln if full else None, act)
        # silu' follows p, with a slope of 1/2 at most: what p is off by, of the largest p
        slope = (8 + TERM) * U * (1 + size.max(initial=0.0)) if act else 0.0
        for k, (what, kind) in enumerate((("grad_x", dtype), ("grad_weight", wdtype), ("grad_bias", wdtype), ("grad_state", dtype))):
            if not full and k >= 2:
                assert got[k] is None
                continue
            chain = CHAIN if k in (1, 2) else 8
            weight = np.abs(wn).max() if k in (0, 3) else 1.0
            extra = slope * np.abs(gn).max(initial=0.0) * (w * weight if k in (0, 3) else 1.0)
            if k == 1:
                extra = slope * 2 * np.abs(gn).sum(0).max(initial=0.0) * max(np.abs(xn).max(initial=0.0), np.abs(sn).max(initial=0.0))
            elif k == 2:
                extra = slope * 2 * np.abs(gn).sum(0).max(initial=0.0)
            near(what, down(got[k]), grads[k], kind, (chain + TERM) * U * 1.1 * sizes[k] + extra)


def test_conv_leaves_the_rest_of_given_outputs():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    x, w = torch.randn(20, 64, device="cuda"), torch.randn(64, 4, device="cuda")
    out = torch.full((20, 64), 7.0, device="cuda")
    gdn.short_conv(x, w, offsets(torch, [4, 9, 15]), out=out)
    assert (out[:4] == 7).all() and (out[15:] == 7).all() and (out[4:15] != 7).any(1).all()


@pytest.mark.parametrize("cu", [[-5, 3, 2 ** 31 - 1], [9, 2, 30], [-2 ** 31, 2 ** 31 - 1], [40, 50, 60]])
def test_conv_with_offsets_that_lead_outside(cu):
    """Nothing outside the buffers is read or written; rows before the first bad offset keep their results."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"conv offsets {cu}")
    t, c, R = 21, 64, len(cu) - 1
    big = torch.full((t + 2 * t, c), 5.0, device="cuda")
    x, w = torch.randn(t, c, device="cuda"), torch.randn(c, 4, device="cuda")
    st = torch.randn(R, 3, c, device="cuda")
    out = big[t:2 * t]
    gdn.short_conv(x, w, offsets(torch, cu), state=st, out=out)
    gdn.short_conv_bwd(x, w, x, offsets(torch, cu), state=st, grad_state_final=st)
    torch.cuda.synchronize()
    assert (big[:t] == 5).all() and (big[2 * t:] == 5).all()


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("r,c,w,act", [(1, 8, 4, True), (3, 72, 2, True), (7, 520, 3, False), (256, 1792, 4, True), (5, 4096, 4, True)])
def test_conv_step_follows_the_prompt(r, c, w, act, dtype, wdtype):
    """Steps give what the convolution of the whole sequences gives, bit for bit: the same sums in the same order."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"conv step r{r} c{c} w{w} {dtype}/{wdtype}")
    make = Inputs(torch, r + c).make
    steps = 6
    x, _ = make((r, steps, c), dtype)
    wt, _ = make((c, w), wdtype, 0.5)
    b, _ = make((c,), wdtype)
    state, _ = make((r, w - 1, c), dtype)
    flat = x.reshape(r * steps, c)
    want, last = gdn.short_conv(flat, wt, offsets(torch, [i * steps for i in range(r + 1)]), bias=b, state=state, silu=act)
    for i in range(steps):
        out = gdn.short_conv_step(x[:, i], wt, state, bias=b, silu=act)
        assert torch.equal(out, want.view(r, steps, c)[:, i])
    assert torch.equal(state, last)


def test_prompt_in_pieces_is_the_whole_prompt():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    x, w = torch.randn(50, 128, device="cuda", dtype=torch.bfloat16), torch.randn(128, 4, device="cuda")
    whole, last = gdn.short_conv(x, w, offsets(torch, [0, 50]))
    state, got = None, []
    for lo, hi in ((0, 1), (1, 3), (3, 3), (3, 30), (30, 50)):
        o, state = gdn.short_conv(x[lo:hi], w, offsets(torch, [0, hi - lo]), state=state)
        got.append(o)
    assert torch.equal(torch.cat(got), whole) and torch.equal(state, last)


def test_refusals():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    x, w, cu = torch.randn(8, 64, device="cuda"), torch.randn(64, device="cuda"), offsets(torch, [0, 8])
    w4, half = torch.randn(64, 4, device="cuda"), torch.float16
    for call in (lambda: gdn.rms_norm(x.to(half), w), lambda: gdn.rms_norm(x, w.to(torch.bfloat16)), lambda: gdn.rms_norm(x, w, x.to(torch.bfloat16)),
                 lambda: gdn.rms_norm_quant(x, w, dtype=torch.float32), lambda: gdn.short_conv(x, w4, cu.long()),
                 lambda: gdn.short_conv(x, w4, cu, bias=w.to(torch.bfloat16))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: gdn.rms_norm(x, w[:32]), lambda: gdn.rms_norm(x, w, x[:4]), lambda: gdn.rms_norm(x.t(), w[:8]),
                 lambda: gdn.rms_norm_quant(x, w, block=64), lambda: gdn.rms_norm_quant(x, w, block=128), lambda: gdn.rms_norm(x, w, sum_out=x),
                 lambda: gdn.rms_norm(torch.randn(8, 68, device="cuda")[:, 4:], w), lambda: gdn.rms_norm_bwd(x, w, x[:, :32]),
                 lambda: gdn.short_conv(x, w, cu), lambda: gdn.short_conv(x, w4.t().contiguous(), cu), lambda: gdn.short_conv(x, w4, cu[:0]),
                 lambda: gdn.short_conv(x, w4, cu, state=x), lambda: gdn.short_conv(x, w4.cpu(), cu),
                 lambda: gdn.short_conv_step(x, w4, torch.randn(7, 3, 64, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: gdn.rms_norm(x[:, :60].contiguous(), w[:60].contiguous()), gdn.gdn.GDN_ERR_SHAPE),
                         (lambda: gdn.rms_norm(x, w, eps=float("nan")), gdn.gdn.GDN_ERR_SHAPE),
                         (lambda: gdn.short_conv(x, torch.randn(64, 5, device="cuda"), cu), gdn.gdn.GDN_ERR_UNSUPPORTED)):
        with pytest.raises((gdn.GdnError, ValueError)):
            call()
