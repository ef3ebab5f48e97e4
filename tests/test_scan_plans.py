"""The cuts of the scan's work that the GPU's tests ask for by name, against the sizes of the library's workspaces, and
that every form that a launch can choose is among them."""
import random

import numpy as np
import pytest

import linear_attention_sequence_gated_amd as gdn
import scan_plans as plans
from oracle import block as ref

SIZES = [(8 * 2048, 8, 24, 64, 1), (16384, 1, 32, 128, 4), (131, 1, 24, 64, 1), (7000, 13, 16, 128, 4), (0, 3, 4, 64, 2)]


def some():
    rng = random.Random(5)
    for _ in range(3000):
        g = rng.choice([1, 1, 2, 4, 16, 65, 128])
        r = rng.choice([1, 2, 6, 8, 100])
        t = rng.choice([rng.randrange(0, 300), rng.randrange(0, 20000), r * 64 * rng.randrange(1, 40)])
        yield t, r, g * rng.choice([1, 2, 3, 5, 24, 64, 70]), rng.choice([64, 128]), g


@pytest.mark.parametrize("n", [64, 128])
def test_cuts_are_those_of_the_library(n):
    for t, r, h, p, g in [*SIZES, *some()]:
        assert gdn.gdn_ssm_scan_workspace_bytes(t, h, p, g, n) == plans.forward_bytes(t, h, p, g, n), (t, h, p, g)
        assert gdn.gdn_ssm_scan_bwd_workspace_bytes(t, r, h, p, g, n) == plans.backward_bytes(t, r, h, p, g, n), (t, r, h, p, g)


@pytest.mark.parametrize("form", plans.FORWARD, ids=lambda f: f.name)
def test_forward_takes_the_form(form):
    got = plans.forward(*form.sizes)
    assert {k: getattr(got, k) for k in form.want} == form.want


@pytest.mark.parametrize("form", plans.BACKWARD, ids=lambda f: f.name)
def test_gradients_take_the_form(form):
    got = plans.backward(*form.sizes)
    assert {k: getattr(got, k) for k in form.want} == form.want


def test_every_form_is_there():
    fwd = [(f, plans.forward(*f.sizes)) for f in plans.FORWARD]
    for n in (64, 128):
        here = [c for f, c in fwd if f.n == n]
        assert {c.last for c in here if c.ns == 4} >= {1, 2, 3} and {c.nseg > 1 for c in here if c.ns == 4} == {True, False}
        assert any(c.joined for c in here if c.ns == 4) and any(c.joined for c in here if c.ns == 2)
    bwd = [(f, plans.backward(*f.sizes)) for f in plans.BACKWARD]
    for n in (64, 128):
        for p in (64, 128):
            assert any(c.heads >= 3 or p == 128 and c.heads >= 2 for f, c in bwd if (f.n, f.p) == (n, p)), (n, p)
        here = [(f, c) for f, c in bwd if f.n == n]
        assert any(c.runs > 1 and c.last < c.heads > 1 for _, c in here) and any(c.whole for _, c in here)
        assert {f.state for f, c in here if c.nseg > 1} == {True, False}
    assert max(c.heads for _, c in bwd) == plans.MOST_HEADS


@pytest.mark.parametrize("wrong", ["none", "rate", "step", "piece", "state", "head"])
def test_the_rooms_of_parameters_gradients_tell_mistakes(wrong):
    """Mistakes of the kind that a loop over heads can make, planted in the reference: each leaves the room, none stays."""
    rng = np.random.default_rng(3)
    t, h, p, n, cu = 70, 4, 16, 16, (0, 20, 70)
    x, B, C, g = (rng.standard_normal(v) for v in ((t, h, p), (t, 1, n), (t, 1, n), (t, h, p)))
    dt, a, D = rng.standard_normal((t, h)), -rng.uniform(1, 2, h), rng.standard_normal(h)
    bias, S0 = np.log(np.expm1(np.exp(rng.uniform(np.log(1e-3), np.log(1e-2), h)))), rng.standard_normal((2, h, n, p))
    ins = x, dt, a, B, C, D, bias
    rooms = plans.parameter_gradients(ins, cu, g, S0, None)
    turned = lambda v, axis=0: np.roll(v, 1, axis)  # noqa: E731
    if wrong == "rate":
        ins = x, dt, turned(a), B, C, D, bias
    elif wrong == "step":
        ins = x, turned(dt, 1), a, B, C, D, bias
    elif wrong == "state":
        S0 = turned(S0, 1)
    got = ref.ssm_scan_bwd(*ins, cu, g, S0)
    ga, gb = (turned(got[2]), turned(got[6])) if wrong == "head" else (got[2], got[6])
    if wrong == "piece":  # the last one's sums in place of all
        x, dt, a, B, C, D, bias = ins
        got = ref.ssm_scan_bwd(x[20:], dt[20:], a, B[20:], C[20:], D, bias, (0, 50), g[20:], S0[1:])
        ga, gb = got[2], got[6]
    out = [(np.abs(v - w) > room).any() for v, (w, room) in zip((ga, gb), rooms)]
    assert out == [wrong != "none"] * 2, wrong
