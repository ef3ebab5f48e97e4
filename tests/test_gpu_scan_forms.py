"""The forms of the scan's kernels that a launch can choose (scan_plans.py), each run once against the fp64 reference.

A form needs many workgroups, so many groups of heads; these are `distinct` ones over and over.  The reference is computed of
those, and every other group's results have to be theirs bit for bit: groups never meet, and a workgroup's arithmetic does not
depend on which one it is.  Tolerances: those of test_gpu_scan.py."""
import numpy as np
import pytest

import scan_plans as plans
from gpu_util import down, note, torch_dev
from test_gpu_scan import Case, check, check_gradients

pytestmark = pytest.mark.gpu


class Tiled:
    """A form's call: `few`, the distinct groups, and what the call is given."""

    def __init__(self, torch, form):
        self.form, self.torch = form, torch
        t = form.cu[-1]
        self.few = c = Case(torch, list(form.cu), t, form.heads * form.distinct, form.p, form.distinct, form.n, seed=11, state=form.state,
                            dt="f32" if form.state else "bf16", param="f32", slow=True)
        self.group = torch.arange(form.groups, device="cuda") % form.distinct
        self.head = (self.group[:, None] * form.heads + torch.arange(form.heads, device="cuda")).flatten()
        self.x, self.B, self.C = c.x[:, self.head], c.B[:, self.group], c.C[:, self.group]
        self.dt, self.a, self.D, self.bias = c.dt[:, self.head], c.a[self.head], c.D[self.head], c.bias[self.head]
        self.S0 = None if c.S0 is None else c.S0[:, self.head]
        self.args = self.x, self.dt, self.a, self.B, self.C
        self.more = dict(D=self.D, dt_bias=self.bias, S0=self.S0)

    def distinct(self, v, axis, by):
        """The results of the distinct groups, of v along axis; all others' are the same."""
        n = self.form.distinct * (self.form.heads if by is self.head else 1)
        few = v.narrow(axis, 0, n)
        assert self.torch.equal(few.index_select(axis, by), v)
        return few


@pytest.mark.parametrize("form", plans.FORWARD, ids=lambda f: f.name)
def test_scan_takes_every_form(form):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"scan form {form.name}")
    assert plans.forward(*form.sizes).nseg == form.want["nseg"]
    c = Tiled(torch, form)
    out, last = gdn.ssm_scan(*c.args, c.few.offsets, **c.more)
    check(c.few, c.distinct(out, 1, c.head), c.distinct(last, 1, c.head), 2 + form.cu[-1] // 64)
    again, last2 = gdn.ssm_scan(*c.args, c.few.offsets, **c.more)
    assert torch.equal(out, again) and torch.equal(last, last2)


@pytest.mark.parametrize("form", plans.BACKWARD, ids=lambda f: f.name)
def test_gradients_take_every_form(form):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"scan gradients form {form.name}")
    c = Tiled(torch, form)
    few, t = c.few, form.cu[-1]
    rng = np.random.default_rng([1, t, form.heads])
    make = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()  # noqa: E731
    go = make(t, few.shape[1], form.p).to(torch.bfloat16)
    gl = make(len(form.cu) - 1, few.shape[1], form.n, form.p) if form.state else None
    got = gdn.ssm_scan_bwd(*c.args, go[:, c.head], few.offsets, **c.more, grad_S_final=None if gl is None else gl[:, c.head])
    # x, dt, a, B, C, D, bias, S0
    axes = ((1, c.head), (1, c.head), (0, c.head), (1, c.group), (1, c.group), (0, c.head), (0, c.head), (1, c.head))
    small = [None if v is None else c.distinct(v, *ax) for v, ax in zip(got, axes)]
    check_gradients(few, small, down(go).astype(np.float64), None if gl is None else down(gl).astype(np.float64))
    ins, S0 = few.numbers()
    for name, v, (want, room) in zip(("a", "bias"), (small[2], small[6]),
                                     plans.parameter_gradients(ins, form.cu, down(go).astype(np.float64), S0,
                                                               None if gl is None else down(gl).astype(np.float64))):
        worst = float((np.abs(down(v) - want) / room).max())
        print(f"[parity] {name} of its rows' terms: {worst:.3f} of its room", flush=True)
        assert worst <= 1, name
