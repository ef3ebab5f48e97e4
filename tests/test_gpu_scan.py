"""The selective state space scan on the GPU against its fp64 reference.

Tolerances, element by element, relative to SIZE: what the same recurrence gives for the inputs' magnitudes, so the sum of
the magnitudes of a result's terms.
  out  Each term is rounded to bf16 once (its weight, or the state that it is part of): 2^-8 of SIZE; float32 sums of N + 64
       terms and their weights' exponents, (N + 128) 2^-24 and 16 2^-24 of the largest sum of decays in a piece; then the
       result to bf16, 2^-8 of itself.
  S    A term is kept to 2^-25, and each piece's sum of 64 and the decays' exponents to (64 + 64 E) 2^-24, where E is
       the largest sum of decays in a piece (up to the 160 where what it multiplies is gone); the products with a piece's
       decay add 2 2^-24 a piece.
A second, normwise bound tells random rounding from a wrong row: independent errors of at most half a bf16 step are, in the
root of their mean square, 2^-8 / sqrt(3) of the values; two of them (term and result) 3.2e-3; 4e-3 is asked."""
import numpy as np
import pytest

from gpu_util import down, note, torch_dev
from oracle import block as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


class Case:
    """Seeded inputs on the device (strided as parts of projections), and the numbers that they hold."""

    def __init__(self, torch, cu, t, h, p, g, n, seed=0, dt="bf16", param="bf16", state=True, spread=1.0, slow=False):
        import numpy as np
        self.torch, self.cu, self.shape = torch, cu, (t, h, p, g, n)
        rng = np.random.default_rng([seed, t, h])
        types = {"bf16": torch.bfloat16, "f32": torch.float32}

        def make(shape, kind="bf16", f=None):
            v = rng.standard_normal(shape) if f is None else f
            return torch.from_numpy(np.asarray(v, np.float32)).to(types[kind]).cuda()

        rows = make((t, h * p + 2 * g * n + 8))
        self.x = rows[:, 8:8 + h * p].view(t, h, p)
        self.B = rows[:, 8 + h * p:8 + h * p + g * n].view(t, g, n)
        self.C = rows[:, 8 + h * p + g * n:].view(t, g, n)
        self.dt = make((t, h + 3), dt, spread * rng.standard_normal((t, h + 3)))[:, 3:]
        step = np.exp(rng.uniform(np.log(1e-3), np.log(1e-2 if slow else 1e-1), h))
        self.bias = make(h, param, np.log(np.expm1(step)))
        self.a = make(h, param, -rng.uniform(1, 2 if slow else 16, h))
        self.D = make(h, param)
        self.S0 = make((len(cu) - 1, h, n, p), "f32") if state else None
        self.offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.names = ("x", "dt", "a", "B", "C")

    def args(self):
        return [getattr(self, k) for k in self.names]

    def numbers(self):
        f = lambda t: None if t is None else down(t).astype(np.float64)  # noqa: E731
        return [f(v) for v in (*self.args(), self.D, self.bias)], f(self.S0)

    def exponents(self):
        """The largest sum of log2 decays over a piece of 64 rows, at most."""
        (x, dt, a, B, C, D, bias), _ = self.numbers()
        g = np.minimum(-a * ref.softplus(dt + bias) * 1.4427, 160.0)
        return float(max((g[i:i + 64].sum(0).max() for i in range(0, len(g), 32)), default=0.0))


def check(c, out, last, pieces):
    ins, S0 = c.numbers()
    x, dt, a, B, C, D, bias = ins
    t, h, p, g, n = c.shape
    want, want_last = ref.ssm_scan(*ins, c.cu, S0)
    size, size_last = ref.ssm_scan(np.abs(x), dt, a, np.abs(B), np.abs(C), np.abs(D), bias, c.cu, None if S0 is None else np.abs(S0))
    E = c.exponents()
    got, got_last = down(out).astype(np.float64), down(last).astype(np.float64)
    assert np.isfinite(got).all() and np.isfinite(got_last).all()
    room = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + (n + 128 + 16 * E) * U) * 1.01 * size + 1e-30
    room_last = (64 + 64 * min(E, 160) + 2 * pieces) * U * size_last + 1e-30
    worst = np.abs(got - want).max(initial=0) and float((np.abs(got - want) / room).max())
    worst_last = float((np.abs(got_last - want_last) / room_last).max(initial=0))
    norm = np.linalg.norm(want)
    rel = np.linalg.norm(got - want) / norm if norm else 0.0
    nl = np.linalg.norm(want_last)
    print(f"[parity] out {worst:.3f} of its room, norm {rel:.2e}; S {worst_last:.3f}, norm {np.linalg.norm(got_last - want_last) / max(nl, 1e-300):.2e}", flush=True)
    assert worst <= 1 and worst_last <= 1 and rel <= 4e-3


SHAPES = [(2, 64, 1, 64), (3, 64, 1, 128), (4, 64, 2, 128), (6, 64, 2, 64), (2, 128, 1, 128), (3, 128, 3, 64), (1, 64, 1, 128)]
RUNS = [("one row", [0, 1], 1), ("a piece", [0, 64], 64), ("short", [0, 2, 3, 3, 7], 7), ("odd", [0, 131], 131), ("empty", [0, 0, 0], 0),
        ("no sequences", [0], 5), ("rows outside", [3, 40, 41, 90], 101), ("ends", [0, 63, 64, 127, 128, 130, 193], 193), ("ragged", [0, 300, 301, 517], 517),
        ("singles", list(range(70)), 69)]


@pytest.mark.parametrize("name,cu,t", RUNS, ids=[r[0] for r in RUNS])
@pytest.mark.parametrize("h,p,g,n", SHAPES)
def test_scan(name, cu, t, h, p, g, n):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    for state in (True, False):
        note(f"scan {name} t{t} h{h} p{p} g{g} n{n} state={state}")
        c = Case(torch, cu, t, h, p, g, n, state=state, dt="bf16" if state else "f32", param="f32" if state else "bf16")
        out, last = gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
        check(c, out, last, 2 + t // 64)
        inside = np.zeros(t, bool)
        for lo, hi in zip(cu, cu[1:]):
            inside[lo:hi] = True
        assert not down(out)[~inside].any()


@pytest.mark.parametrize("dt,param", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("r,h,p,g,n", [(1, 1, 64, 1, 64), (3, 6, 64, 3, 128), (5, 4, 128, 2, 64), (40, 24, 64, 1, 128), (2, 5, 128, 1, 128)])
def test_step(r, h, p, g, n, dt, param):
    """out is rounded once; a state's element takes one product and one sum, the sum over N elements N + 8."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"step r{r} h{h} p{p} g{g} n{n} {dt} {param}")
    cu = list(range(r + 1))
    c = Case(torch, cu, r, h, p, g, n, dt=dt, param=param)
    ins, S0 = c.numbers()
    want, want_last = ref.ssm_scan(*ins, cu, S0)
    x, d, a, B, C, D, bias = ins
    size, size_last = ref.ssm_scan(np.abs(x), d, a, np.abs(B), np.abs(C), np.abs(D), bias, cu, np.abs(S0))
    S = c.S0.clone()
    out = gdn.ssm_step(*c.args(), S, D=c.D, dt_bias=c.bias)
    assert (np.abs(down(out) - want) <= 2.0 ** -8 * np.abs(want) + 1.01 * (n + 24 + c.exponents()) * U * size).all()
    assert (np.abs(down(S) - want_last) <= (16 + c.exponents()) * U * size_last).all()


def test_steps_follow_the_prompt():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    r, steps = 3, 70
    cu = [i * steps for i in range(r + 1)]
    c = Case(torch, cu, r * steps, 4, 64, 2, 128)
    want, last = gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
    S, rows = c.S0.clone(), torch.arange(r, device="cuda") * steps
    got = torch.empty_like(want)
    for i in range(steps):
        got[rows + i] = gdn.ssm_step(*(v if k == "a" else v[rows + i] for k, v in zip(c.names, c.args())), S, D=c.D, dt_bias=c.bias)
    assert (S - last).norm() <= 2e-6 * last.norm()
    assert (got.float() - want.float()).norm() <= 4e-3 * want.float().norm()


def test_prompt_in_pieces_is_the_whole_prompt():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    c = Case(torch, [0, 400], 400, 3, 64, 1, 64, state=False, slow=True)
    whole, last = gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias)
    S, got = None, []
    for lo, hi in ((0, 1), (1, 130), (130, 130), (130, 400)):
        part = [v if k == "a" else v[lo:hi] for k, v in zip(c.names, c.args())]
        o, S = gdn.ssm_scan(*part, torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"), D=c.D, dt_bias=c.bias, S0=S)
        got.append(o)
    assert (S - last).norm() <= 2e-6 * last.norm()
    assert (torch.cat(got).float() - whole.float()).norm() <= 4e-3 * whole.float().norm()


# ------------------------------------------------------------------- gradients
def gradients(c, g, gl):
    """The oracle's gradients, and what its recurrence gives for the inputs' magnitudes, whose terms add up."""
    (x, dt, a, B, C, D, bias), S0 = c.numbers()
    want = ref.ssm_scan_bwd(x, dt, a, B, C, D, bias, c.cu, g, S0, gl)
    m = lambda v: None if v is None else np.abs(v)  # noqa: E731
    size = ref.ssm_scan_bwd(m(x), dt, -np.abs(a), m(B), m(C), m(D), bias, c.cu, m(g), m(S0), m(gl))
    # of dt and what is summed from it: direct terms and those by the decay have opposite signs there (a < 0)
    x, B, C, g, S0, gl = m(x), m(B), m(C), m(g), m(S0), m(gl)
    up = ref.ssm_scan_bwd(x, dt, a, B, C, 0 * D, bias, c.cu, g, S0, gl)
    z = dt + bias
    d, sig = ref.softplus(z), 1 / (1 + np.exp(-z))
    rep = x.shape[1] // B.shape[1]
    by_x = (up[0] * x).sum(2)  # what d_t multiplies, times d_t: x_t . gx_t
    direct = by_x / np.maximum(d, 1e-300)
    by_a = np.abs(up[1] / sig - direct)  # a gg_t
    size[1] = (direct + by_a) * sig
    size[6] = size[1].sum(0)
    size[2] = (by_a / np.abs(a) * d).sum(0)
    return want, size


NAMES = ("x", "dt", "a", "B", "C", "D", "bias", "S0")


def check_gradients(c, got, g, gl):
    """Element by element: a term has a weight or a state rounded to bf16, 2^-8 of it, and for C and B the sum over heads
    none more; dt's terms have a state rounded in one factor and its gradient in the other at most, 2 2^-8 (the products
    <Z, S>).  The result is rounded to its type.  S0 is a state (see above).  Normwise: as for out, 4e-3; the parameters'
    gradients, whose terms cancel, of their terms' size.  dt's terms have random signs here, so that its norm is of the order
    of the root of their squares' sum, and their independent errors, 2^-8 / sqrt(3) in each of two factors and the result,
    leave 3.9e-3 of that; three times as much is asked, since a decay takes some terms from the norm.  The normwise
    bounds are asked of 64 rows and more: in one row, the terms of two heads may cancel by chance."""
    want, size = gradients(c, g, gl)
    E = c.exponents()
    T = c.shape[0]
    for k, name in enumerate(NAMES):
        if got[k] is None:
            continue
        v = down(got[k]).astype(np.float64)
        assert v.shape == want[k].shape and np.isfinite(v).all(), name
        half = 2.0 ** -8 if got[k].dtype.itemsize == 2 else U
        term = {"S0": 0.0, "D": 0.0, "dt": 2.0 ** -7, "a": 2.0 ** -7, "bias": 2.0 ** -7}.get(name, 2.0 ** -8)
        chain = 64 + 64 * min(E, 160) + 2 * (T // 64 + 2) if name == "S0" else 384 + 16 * E + T / 64
        room = half * np.abs(want[k]) + (term + chain * U) * 1.02 * size[k] + 1e-30
        worst = float((np.abs(v - want[k]) / room).max(initial=0))
        norm = np.linalg.norm(want[k])
        rel = np.linalg.norm(v - want[k]) / norm if norm else 0.0
        of_size = np.linalg.norm(v - want[k]) / max(np.linalg.norm(size[k]), 1e-300)
        print(f"[parity] {name}: {worst:.3f} of its room, norm {rel:.2e}, of its terms {of_size:.2e}", flush=True)
        assert worst <= 1, (name, worst)
        if T >= 64:
            assert (rel if name in ("x", "B", "C", "S0") else of_size) <= 4e-3, (name, rel)
            assert name != "dt" or rel <= 1.2e-2, (name, rel)


@pytest.mark.parametrize("name,cu,t", RUNS, ids=[r[0] for r in RUNS])
@pytest.mark.parametrize("h,p,g,n", SHAPES)
def test_scan_gradients(name, cu, t, h, p, g, n):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    for state in (True, False):
        note(f"scan gradients {name} t{t} h{h} p{p} g{g} n{n} state={state}")
        c = Case(torch, cu, t, h, p, g, n, state=state, dt="bf16" if state else "f32", param="f32" if state else "bf16")
        seeded = torch.Generator(device="cuda").manual_seed(t + h)
        go = torch.randn(t, h * p + 8, generator=seeded, device="cuda").to(torch.bfloat16)[:, :h * p].view(t, h, p)
        gl = torch.randn(len(cu) - 1, h, n, p, generator=seeded, device="cuda") if state else None
        got = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0, grad_S_final=gl)
        check_gradients(c, got, down(go).astype(np.float64), None if gl is None else down(gl).astype(np.float64))
        inside = np.zeros(t, bool)
        for lo, hi in zip(cu, cu[1:]):
            inside[lo:hi] = True
        assert not any(down(got[k])[~inside].any() for k in (0, 1, 3, 4))


# --------------------------------------------------------------- larger forms
@pytest.mark.parametrize("name,cu,h,p,g,n", [
    ("four strips to a workgroup, segments", [0, 700, 701, 1200], 128, 64, 1, 64),
    ("many segments of one sequence, joined by a launch", [0, 2300], 1, 64, 1, 64),
    ("a segment's end is a sequence's", [0, 256, 512, 512, 700, 1024], 2, 64, 1, 128),
    ("more offsets than LDS holds", [min(i, 555) for i in range(601)], 2, 64, 1, 64),
    ("groups of five strips", [0, 90, 300], 10, 64, 2, 64),
    ("many groups", [0, 100], 40, 64, 40, 64)])
def test_scan_forms(name, cu, h, p, g, n):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"scan {name}")
    c = Case(torch, cu, cu[-1], h, p, g, n, slow=True)
    out, last = gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
    check(c, out, last, 2 + cu[-1] // 64)


@pytest.mark.parametrize("name,cu,h,p,g,n", [
    ("many segments", [0, 1100, 1101, 1400], 2, 64, 1, 64), ("sequences as segments", [0, 512, 1024], 1, 64, 1, 64),
    ("more heads than one run takes", [0, 70], 70, 64, 1, 64), ("more offsets than LDS holds", list(range(0, 560, 4)), 2, 64, 1, 64),
    ("wide heads of one group", [0, 100, 200], 5, 128, 1, 128)])
def test_scan_gradients_of_forms(name, cu, h, p, g, n):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"scan gradients {name}")
    t = cu[-1]
    c = Case(torch, cu, t, h, p, g, n, slow=True)
    go = torch.from_numpy(np.random.default_rng(1).standard_normal((t, h, p)).astype(np.float32)).to(torch.bfloat16).cuda()
    gl = torch.from_numpy(np.random.default_rng(2).standard_normal((len(cu) - 1, h, n, p)).astype(np.float32)).cuda()
    got = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0, grad_S_final=gl)
    check_gradients(c, got, down(go).astype(np.float64), down(gl).astype(np.float64))
    again = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0, grad_S_final=gl)
    assert all(torch.equal(u, v) for u, v in zip(got, again))  # sums in a fixed order


# ------------------------------------------------------------------- extremes
def test_steps_of_all_sizes():
    """Steps from none to hundreds: decays that forget everything at once, and states that stay for good."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    t, h = 200, 4
    c = Case(torch, [0, 150, t], t, h, 64, 1, 64, dt="f32", param="f32")
    c.dt = torch.tensor([-200.0, -30.0, 0.0, 300.0], device="cuda")[torch.arange(t * h, device="cuda").view(t, h) * 7 % 4].contiguous()
    c.bias.zero_()
    c.x = (c.x / 64).contiguous()
    out, last = gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
    check(c, out, last, 5)
    go = torch.randn(t, h, 64, device="cuda").to(torch.bfloat16)
    got = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
    assert all(torch.isfinite(v).all() for v in got)
    S = c.S0.clone()
    one = [v if k == "a" else v[:2] for k, v in zip(c.names, c.args())]
    assert torch.isfinite(gdn.ssm_step(*one, S, D=c.D, dt_bias=c.bias)).all() and torch.isfinite(S).all()


def test_a_step_of_zero_has_the_slope_of_softplus():
    """softplus'(0) = 1/2: dt and bias that cancel."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    c = Case(torch, [0, 80], 80, 2, 64, 1, 64, dt="f32", param="f32")
    c.dt = (-c.bias).expand(80, 2).contiguous()
    go = torch.from_numpy(np.random.default_rng(4).standard_normal((80, 2, 64)).astype(np.float32)).to(torch.bfloat16).cuda()
    got = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
    check_gradients(c, got, down(go).astype(np.float64), None)


def test_without_the_optional_parts():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    c = Case(torch, [0, 100], 100, 3, 64, 1, 64, state=False)
    zero = torch.zeros_like(c.D)
    out, last = gdn.ssm_scan(*c.args(), c.offsets)
    want, want_last = gdn.ssm_scan(*c.args(), c.offsets, D=zero, dt_bias=zero, S0=torch.zeros_like(last))
    assert torch.equal(out, want) and torch.equal(last, want_last)
    go = torch.randn_like(out)
    got = gdn.ssm_scan_bwd(*c.args(), go, c.offsets)
    want = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, D=zero, dt_bias=zero)
    assert all(torch.equal(u, v) for u, v in zip(got[:5], want[:5])) and got[5:] == (None, None, None)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_sequence(bad):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    cu, t = [0, 100, 130, 400], 400
    c = Case(torch, cu, t, 4, 64, 2, 128)
    go = torch.randn(t, 4, 64, device="cuda").to(torch.bfloat16)
    run = lambda: (*gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0),  # noqa: E731
                   gdn.ssm_scan_bwd(*c.args(), go, c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0))
    out, last, grads = run()
    for name in ("x", "B", "C", "dt"):
        v = getattr(c, name)
        kept = v.clone()
        v[110] = bad
        out2, last2, grads2 = run()
        v[110] = kept[110]
        rest = torch.tensor([i for i in range(t) if not 100 <= i < 130], device="cuda")
        assert torch.equal(out2[rest], out[rest]) and torch.equal(last2[[0, 2]], last[[0, 2]]), name
        assert all(torch.equal(grads2[k][rest], grads[k][rest]) for k in (0, 1, 3, 4)) and torch.equal(grads2[7][[0, 2]], grads[7][[0, 2]]), name


@pytest.mark.parametrize("cu", [[-5, 30, 2 ** 31 - 1], [90, 20, 300], [-2 ** 31, 2 ** 31 - 1], [400, 500, 600], [0, 2 ** 31 - 1, 5]])
def test_offsets_that_lead_outside(cu):
    """Nothing outside the buffers is read or written."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"scan offsets {cu}")
    t, h, R = 300, 2, len(cu) - 1
    c = Case(torch, cu, t, h, 64, 1, 64)
    big = torch.full((3 * t, h, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0, out=big[t:2 * t])
    gx = torch.full((3 * t, h, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    gb = torch.full((3 * t, 2, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    gdn.ssm_scan_bwd(*c.args(), c.x.contiguous(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0, grad_S_final=c.S0, grad_x=gx[t:2 * t],
                     grad_B=gb[t:2 * t, :1], grad_C=gb[t:2 * t, 1:])
    torch.cuda.synchronize()
    for v in (big, gx, gb):
        assert (v[:t] == 5).all() and (v[2 * t:] == 5).all()


def test_given_outputs():
    """Gradients as parts of one tensor; what stands in rows of no sequence, and behind the parts, stays."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    t, h, g, n = 90, 4, 2, 64
    c = Case(torch, [10, 50, 80], t, h, 64, g, n)
    go = torch.randn(t, h, 64, device="cuda").to(torch.bfloat16)
    more = dict(D=c.D, dt_bias=c.bias, S0=c.S0)
    want = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, **more)
    rows = torch.full((t, h * 64 + 2 * g * n + 16), 3.0, device="cuda", dtype=torch.bfloat16)
    gx, gB, gC = rows[:, :h * 64].view(t, h, 64), rows[:, h * 64:h * 64 + g * n].view(t, g, n), rows[:, h * 64 + g * n:-16].view(t, g, n)
    got = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, **more, grad_x=gx, grad_B=gB, grad_C=gC)
    assert got[0] is gx and all(torch.equal(u[10:80], v[10:80]) for u, v in zip(got[:5], want[:5]) if u.dim() > 1)
    assert (rows[:10] == 3).all() and (rows[80:] == 3).all() and (rows[:, -16:] == 3).all()
    out = torch.full((t, h, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    last = torch.empty_like(c.S0)
    a, b = gdn.ssm_scan(*c.args(), c.offsets, **more, out=out, S_final=last)
    w, wl = gdn.ssm_scan(*c.args(), c.offsets, **more)
    assert a is out and b is last and torch.equal(out[10:80], w[10:80]) and torch.equal(last, wl)
    assert (out[:10] == 3).all() and (out[80:] == 3).all()


def test_refusals():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    c = Case(torch, [0, 20], 20, 4, 64, 2, 64)
    x, dt, a, B, C = c.args()
    with pytest.raises(TypeError):
        gdn.ssm_scan(x.float(), dt, a, B, C, c.offsets)
    with pytest.raises(TypeError):
        gdn.ssm_scan(x, dt.to(torch.float16), a, B, C, c.offsets)
    with pytest.raises(TypeError):
        gdn.ssm_scan(x, dt, a, B, C, c.offsets, D=c.D.float())
    with pytest.raises(TypeError):
        gdn.ssm_scan(x, dt, a, B, C, c.offsets, S0=c.S0.to(torch.bfloat16))
    for call in (lambda: gdn.ssm_scan(x, dt, a, B, C[:, :1], c.offsets), lambda: gdn.ssm_scan(x, dt[:, :2], a, B, C, c.offsets),
                 lambda: gdn.ssm_scan(x, dt, a[:2], B, C, c.offsets), lambda: gdn.ssm_scan(x.transpose(0, 1), dt, a, B, C, c.offsets),
                 lambda: gdn.ssm_scan(x, dt, a, B, C, c.offsets[:0]), lambda: gdn.ssm_scan(x, dt, a, B, C, c.offsets, S0=c.S0[:, :2]),
                 lambda: gdn.ssm_scan(x, dt.t().contiguous().t(), a, B, C, c.offsets),
                 lambda: gdn.ssm_scan_bwd(x, dt, a, B, C, x[:, :2], c.offsets), lambda: gdn.ssm_step(x, dt, a, B, C, c.S0)):
        with pytest.raises(ValueError):
            call()
    for h, g, n, status in ((3, 2, 64, gdn.gdn.GDN_ERR_SHAPE), (4, 2, 48, gdn.gdn.GDN_ERR_UNSUPPORTED)):
        z = torch.zeros(20, g, n, device="cuda", dtype=torch.bfloat16)
        with pytest.raises(gdn.GdnError) as e:
            gdn.ssm_scan(x[:, :h].contiguous(), dt[:, :h].contiguous(), a[:h].contiguous(), z, z, c.offsets)
        assert e.value.status == status


@pytest.mark.parametrize("name", ["dt", "a", "dt_bias"])
def test_nan_is_not_hidden(name):
    """A step or a rate that is NaN gives NaN from its row on, in the scan and in the step."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    c = Case(torch, [0, 100], 100, 2, 64, 1, 64, dt="f32", param="f32")
    if name == "dt":
        c.dt[40, 1] = float("nan")
    else:
        (c.a if name == "a" else c.bias)[1] = float("nan")
    out, last = gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
    assert torch.isnan(out[40:, 1]).all() and torch.isnan(last[:, 1]).all() and torch.isfinite(out[:, 0]).all() and torch.isfinite(last[:, 0]).all()
    S = c.S0.clone()
    one = [v if k == "a" else v[40:41] for k, v in zip(c.names, c.args())]
    y = gdn.ssm_step(*one, S, D=c.D, dt_bias=c.bias)
    assert torch.isnan(y[:, 1]).all() and torch.isnan(S[:, 1]).all() and torch.isfinite(y[:, 0]).all() and torch.isfinite(S[:, 0]).all()


@pytest.mark.parametrize("p,n", [(64, 64), (64, 128), (128, 128)])
def test_a_padded_batch(p, n):
    """Many sequences without rows, among the others and behind them: their states pass through, gradients back."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    cu = [0, 300] + [300] * 40 + [700, 701] + [701] * 90
    c = Case(torch, cu, 720, 4, p, 2, n, slow=True)
    lengths = np.diff(cu)
    empty = torch.from_numpy(np.flatnonzero(lengths == 0)).cuda()
    out, last = gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
    assert torch.equal(last[empty], c.S0[empty])
    check(c, out, last, 2 + 720 // 64)
    assert (gdn.ssm_scan(*c.args(), c.offsets)[1][empty] == 0).all()
    go = torch.from_numpy(np.random.default_rng(6).standard_normal((720, 4, p)).astype(np.float32)).to(torch.bfloat16).cuda()
    gl = torch.from_numpy(np.random.default_rng(7).standard_normal(tuple(c.S0.shape)).astype(np.float32)).cuda()
    got = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0, grad_S_final=gl)
    assert torch.equal(got[7][empty], gl[empty])
    check_gradients(c, got, down(go).astype(np.float64), down(gl).astype(np.float64))
