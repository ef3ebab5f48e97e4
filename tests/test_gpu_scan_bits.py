"""What the scan keeps of its terms before the one rounding of its results: the output, wherever it comes from, and the gradients of
sequences of one piece, whose every term is a weight of rows.

Element by element a term is off by 2^-16 of itself (two bf16 parts of a number leave 2^-17, for weights and for a decay's float32
exponent at the sizes here) and the sums of N + 128 terms by as many 2^-24; the result by half a step, 2^-8 of itself.  In norm the
one rounding leaves at most 2^-8 / sqrt(3); with a second one of each term it would be 2.4e-3 and more."""
import numpy as np
import pytest

from gpu_util import down, note, torch_dev
from oracle import block as ref
from test_gpu_scan import Case, gradients

pytestmark = pytest.mark.gpu

U, ONCE = 2.0 ** -24, 2.0 ** -8 / np.sqrt(3.0)


def once(name, got, want, size, chain):
    """got is want rounded once, of terms whose magnitudes add up to size."""
    got = down(got).astype(np.float64)
    room = 2.0 ** -8 * np.abs(want) + (2.0 ** -16 + chain * U) * 1.02 * size + 1e-30
    worst = float((np.abs(got - want) / room).max(initial=0.0))
    rel = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-300)
    print(f"[parity] {name}: {worst:.3f} of its room, norm {rel:.2e}", flush=True)
    assert worst <= 1 and rel <= ONCE, (name, worst, rel)


@pytest.mark.parametrize("h,p,g,n", [(4, 64, 1, 64), (3, 64, 1, 128), (2, 128, 1, 64), (5, 128, 1, 128), (128, 64, 16, 128), (96, 128, 32, 64)])
@pytest.mark.parametrize("kind", ["rows", "state", "both"])
def test_output_is_rounded_once(kind, h, p, g, n):
    """From the rows, from the state that a sequence begins with, from both; pieces of 64 rows and of a few."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"scan bits {kind} h{h} p{p} g{g} n{n}")
    cu = [0, 130, 131, 300]
    c = Case(torch, cu, 300, h, p, g, n, seed=3, dt="f32", param="f32", state=kind != "rows", slow=True)
    if kind == "state":
        c.S0 *= 64
        c.D *= 0
    out, _ = gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
    (x, dt, a, B, C, D, bias), S0 = c.numbers()
    want, _ = ref.ssm_scan(x, dt, a, B, C, D, bias, cu, S0)
    size, _ = ref.ssm_scan(np.abs(x), dt, a, np.abs(B), np.abs(C), np.abs(D), bias, cu, None if S0 is None else np.abs(S0))
    once("out", out, want, size, n + 128 + 16 * c.exponents())


@pytest.mark.parametrize("h,p,g,n", [(8, 64, 1, 64), (6, 64, 2, 128), (4, 128, 1, 64), (5, 128, 1, 128), (24, 64, 1, 128), (195, 64, 65, 64), (220, 128, 44, 64)])
@pytest.mark.parametrize("cu", [[0, 1, 2, 3], [0, 20, 64, 70], [0, 64, 100]])
def test_gradients_of_a_piece_are_rounded_once(cu, h, p, g, n):
    """x, B and C, those summed over the heads of a group, which may cancel."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"scan gradients' bits {cu} h{h} p{p} g{g} n{n}")
    t = cu[-1]
    c = Case(torch, cu, t, h, p, g, n, seed=5, dt="f32", param="f32", state=False, slow=True)
    go = torch.from_numpy(np.random.default_rng(h).standard_normal((t, h, p)).astype(np.float32)).to(torch.bfloat16).cuda()
    got = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, D=c.D, dt_bias=c.bias)
    want, size = gradients(c, down(go).astype(np.float64), None)
    for k, name in ((0, "x"), (3, "B"), (4, "C")):
        once(name, got[k], want[k], size[k], 384 + 16 * c.exponents())
