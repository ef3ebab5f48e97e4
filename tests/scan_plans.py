"""How the scan and its gradients cut their work (csrc/ssm_scan.hip and csrc/ssm_scan_bwd.hip, `cut` and `plan`), written
again, so that a test can ask for a form of the kernels by name; test_scan_plans.py holds it against the sizes of the
workspaces that the library asks for."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from oracle import block as ref

Q, MOST_HEADS, CUS = 64, 64, 256


def up(a, b):
    return -(-a // b)


@dataclass(frozen=True)
class Cut:
    ns: int  # strips to a workgroup
    last: int  # strips of a group's last workgroup
    nseg: int
    joined: bool  # by a launch of its own


def forward(T, R, H, P, G):
    strips = H // G * (P // 64)
    for ns in (4, 2):
        sets = G * up(strips, ns)
        per = max(up(up(T, Q), max(CUS // sets, 1)), 4)
        nseg = up(T, per * Q) if T > per * Q else 1
        if ns == 2 or (strips > 2 and sets * nseg >= 128):
            break
    return Cut(ns, strips - (up(strips, ns) - 1) * ns, nseg, nseg > 1 and T > 8 * per * Q * max(R, 1))


def forward_bytes(T, H, P, G, N):
    return (forward(T, 1, H, P, G).nseg - 1) * H * (P // 64) * (N * 64 + 1) * 4


@dataclass(frozen=True)
class Plan:
    nseg: int
    whole: bool  # segments are whole sequences, were these alike
    runs: int  # of heads of a group
    heads: int  # to a run
    last: int  # to a group's last run


def backward(T, R, H, P, G):
    strips, spp, blocks = H * (P // 64), P // 64, up(T, Q)
    want = max(192 // strips, 1)
    per, whole = up(blocks, want), False
    if want > 1 and R > 1 and T % R == 0 and T // R % Q == 0 and per * Q <= 2 * (T // R) and T // R <= 2 * per * Q:
        per, whole = T // R // Q, T // R // Q >= 4 and T // R // Q != max(per, 4)
    per = max(per, 4)
    heads = H // G
    best = None
    few = up(heads, MOST_HEADS)
    for n in range(few, min(heads, few + 1023) + 1):
        length = up(heads, n)
        if up(heads, length) != n:
            continue
        cost = up(blocks * G * n, CUS) * (length * spp + 2)
        if best is None or cost < best[0]:
            best = cost, n, length
    _, runs, length = best
    return Plan(up(T, per * Q) if T > per * Q else 1, whole, runs, length, heads - (runs - 1) * length)


def backward_bytes(T, R, H, P, G, N):
    p = backward(T, R, H, P, G)
    strips, blocks = H * (P // 64), up(T, Q)
    room = lambda x: up(x, 256) * 256  # noqa: E731
    shares = 2 * p.runs * T * G * N * 4 if p.runs > 1 else 0
    return 2 * room((p.nseg - 1) * strips * (N * 64 + 1) * 4) + 2 * room((blocks + R) * strips * N * 64 * 2) + room(blocks * H * 12) + shares


@dataclass(frozen=True)
class Form:
    """A call that takes a form of the kernels: `distinct` groups of `heads` heads each, tiled to `groups` of them."""
    name: str
    cu: tuple
    heads: int
    groups: int
    p: int
    n: int
    want: dict
    distinct: int = 2
    state: bool = True

    @property
    def sizes(self):  # T, R, H, P, G
        return self.cu[-1], len(self.cu) - 1, self.heads * self.groups, self.p, self.groups


def parameter_gradients(ins, cu, g, S0, g_last):
    """((grad_a, room), (grad_dt_bias, room)), each [H]: sums over rows, and how far off they may be.

    The rows' terms are d_t gg_t and gz_t (the gradient of dt).  Those of dt are within 1.2e-2 of their norm (test_gpu_scan.py
    derives 3.9e-3 for independent roundings and asks for three times that).  The share of <Z, S> is one number for the
    64 rows of a piece, so that its error is too: a sum over rows is off by at most sqrt(64) times the root of its terms'
    squares' errors where pieces are independent of each other; 0.1 of the root of the terms' squares."""
    x, dt, a, B, C, D, bias = ins
    want = ref.ssm_scan_bwd(x, dt, a, B, C, D, bias, cu, g, S0, g_last)
    z = dt + bias
    d, sig = ref.softplus(z), 1 / (1 + np.exp(-z))
    inside = np.zeros((len(x), 1), bool)
    for _, lo, hi in ref._sequences(cu, len(x)):
        inside[lo:hi] = True
    direct = ((want[0] - np.where(inside[..., None], D[:, None] * g, 0.0)) * x).sum(2)  # d_t B_t . (Z x_t)
    by_row = (want[1] / sig * d - direct) / a  # d_t gg_t
    assert np.allclose(by_row.sum(0), want[2], rtol=1e-6, atol=1e-9 * np.abs(by_row).sum(0).max(initial=0))
    return tuple((w, 0.1 * np.sqrt((t * t).sum(0)) + 2.0 ** -8 * np.abs(w)) for w, t in ((want[2], by_row), (want[6], want[1])))


# Forms of the forward.  Sequences cross the borders of segments, begin and end at them and within them.
FORWARD = [
    Form("four strips, last workgroup with one", (0, 130, 131, 131, 300), 5, 32, 64, 128, dict(ns=4, last=1, nseg=2, joined=False)),
    Form("four strips, last workgroup with two, wide heads", (0, 255, 300), 3, 32, 128, 128, dict(ns=4, last=2, nseg=2, joined=False)),
    Form("four strips, last workgroup with three", (0, 70, 300), 7, 32, 64, 128, dict(ns=4, last=3, nseg=2, joined=False)),
    Form("four strips, last workgroup with one, N = 64", (0, 1, 300), 5, 32, 64, 64, dict(ns=4, last=1, nseg=2, joined=False)),
    Form("four strips, last workgroup with two, N = 64, wide heads", (0, 256, 300), 3, 32, 128, 64, dict(ns=4, last=2, nseg=2, joined=False)),
    Form("four strips, last workgroup with three, N = 64, no state", (0, 299, 300), 7, 32, 64, 64, dict(ns=4, last=3, nseg=2, joined=False), state=False),
    Form("four strips, whole workgroups, many segments", (0, 600, 640, 700, 1300), 8, 16, 64, 128, dict(ns=4, last=4, nseg=6, joined=False)),
    Form("four strips, one segment", (0, 3, 70), 4, 128, 64, 128, dict(ns=4, last=4, nseg=1, joined=False)),
    Form("four strips, one segment, last workgroup with two", (0, 70), 3, 64, 128, 64, dict(ns=4, last=2, nseg=1, joined=False)),
    Form("four strips, joined by a launch", (0, 2350), 3, 17, 64, 128, dict(ns=4, last=3, nseg=10, joined=True)),
    Form("four strips, joined by a launch, wide heads", (0, 2350), 2, 16, 128, 128, dict(ns=4, last=4, nseg=10, joined=True), state=False),
    Form("four strips, joined by a launch, N = 64", (0, 2350), 3, 17, 64, 64, dict(ns=4, last=3, nseg=10, joined=True)),
    Form("two strips, joined by a launch, wide heads", (0, 2300), 1, 1, 128, 128, dict(ns=2, last=2, nseg=9, joined=True), distinct=1),
    Form("two strips, joined by a launch, last workgroup with one", (0, 2300), 3, 1, 64, 64, dict(ns=2, last=1, nseg=9, joined=True), distinct=1),
    Form("two strips, segments, wide heads", (0, 100, 700, 900), 3, 2, 128, 128, dict(ns=2, last=2, nseg=4, joined=False)),
]

# Forms of the gradients.  Blocks of 64 rows with pieces of one, two and more sequences.
BACKWARD = [
    Form("three heads to a run", (0, 20, 70), 3, 65, 64, 64, dict(nseg=1, runs=1, heads=3)),
    Form("three heads to a run, N = 128", (0, 20, 20, 29, 70), 3, 65, 64, 128, dict(nseg=1, runs=1, heads=3)),
    Form("three wide heads to a run", (0, 20, 70), 3, 65, 128, 64, dict(nseg=1, runs=1, heads=3)),
    Form("three wide heads to a run, N = 128", (0, 66, 70), 3, 65, 128, 128, dict(nseg=1, runs=1, heads=3)),
    Form("four heads to a run", (0, 33, 70), 4, 70, 64, 128, dict(nseg=1, runs=1, heads=4)),
    Form("twenty-three heads to a run, N = 128", (0, 20, 70), 23, 128, 64, 128, dict(nseg=1, runs=1, heads=23)),
    Form("runs of three heads and of two", (0, 20, 70), 5, 44, 64, 64, dict(nseg=1, runs=2, heads=3, last=2)),
    Form("runs of three heads and of two, N = 128, no state", (0, 65, 70), 5, 44, 64, 128, dict(nseg=1, runs=2, heads=3, last=2), state=False),
    Form("runs of two wide heads and of one, N = 128", (0, 20, 70), 3, 44, 128, 128, dict(nseg=1, runs=2, heads=2, last=1)),
    Form("runs of two wide heads and of one", (0, 64, 70), 3, 44, 128, 64, dict(nseg=1, runs=2, heads=2, last=1)),
    Form("all heads that a run can have", (0, 2, 5), 64, 256, 64, 64, dict(nseg=1, runs=1, heads=64), distinct=1, state=False),
    Form("more heads than a run can have", (0, 2, 5), 65, 128, 64, 64, dict(nseg=1, runs=2, heads=33, last=32), distinct=1, state=False),
    Form("several heads to a run, segments", (0, 100, 420, 520), 3, 23, 64, 128, dict(nseg=2, heads=3)),
    Form("wide heads, segments, no state", (0, 300, 520), 2, 24, 128, 64, dict(nseg=2, heads=2), state=False),
    Form("segments, N = 128, no state", (0, 1100, 1101, 1400), 2, 1, 64, 128, dict(nseg=6), distinct=1, state=False),
    Form("segments, wide heads, N = 128", (0, 700, 701, 1000), 1, 2, 128, 128, dict(nseg=4)),
    Form("sequences of one length as segments", tuple(range(0, 1921, 320)), 2, 12, 64, 64, dict(nseg=6, whole=True)),
    Form("sequences of one length as segments, N = 128, no state", tuple(range(0, 1921, 320)), 1, 23, 64, 128, dict(nseg=6, whole=True), state=False),
    Form("as many rows as if of one length", (0, 100, 700, 701, 1300, 1300, 1920), 2, 12, 64, 64, dict(nseg=6, whole=True)),
]
