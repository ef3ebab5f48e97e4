"""Padded batches with few rows: the states of sequences without rows pass through the scan, and their gradients back, bit
for bit and in the time that their bytes take."""
import numpy as np
import pytest

from gpu_util import note, torch_dev
from test_gpu_scan import Case, check

pytestmark = pytest.mark.gpu


def time_us(torch, fn):
    """The least of five times of four calls."""
    fn()
    best = float("inf")
    for _ in range(5):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(4):
            fn()
        end.record()
        end.synchronize()
        best = min(best, start.elapsed_time(end) / 4 * 1e3)
    return best


@pytest.mark.parametrize("t,cu", [(0, [0] * 41), (1, [0] * 20 + [1] * 21), (70, [3] * 5 + [40] * 30 + [70]), (70, [0, 70] + [70] * 600),
                                  (300, [0] * 3 + [300] * 3), (700, [0, 300] + [300] * 20 + [700] * 20), (90, [10, 10]), (64, [0] * 2 + [64] * 2)])
@pytest.mark.parametrize("h,p,g,n", [(2, 64, 1, 64), (3, 64, 1, 128), (5, 128, 5, 64)])
def test_states_pass_through(t, cu, h, p, g, n):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"padded t{t} r{len(cu) - 1} h{h} p{p} g{g} n{n}")
    c = Case(torch, cu, t, h, p, g, n, slow=True)
    empty = torch.from_numpy(np.diff(cu) == 0).cuda()
    out, last = gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias, S0=c.S0)
    assert torch.equal(last[empty], c.S0[empty])
    check(c, out, last, 2 + t // 64)
    assert (gdn.ssm_scan(*c.args(), c.offsets, D=c.D, dt_bias=c.bias)[1][empty] == 0).all()
    go, gl = torch.randn(t, h, p, device="cuda").to(torch.bfloat16), torch.randn_like(c.S0)
    more = dict(D=c.D, dt_bias=c.bias, S0=c.S0)
    got = gdn.ssm_scan_bwd(*c.args(), go, c.offsets, **more, grad_S_final=gl)
    assert torch.equal(got[7][empty], gl[empty])
    assert (gdn.ssm_scan_bwd(*c.args(), go, c.offsets, **more)[7][empty] == 0).all()
    # the others' results are those of a batch without these
    rest = torch.from_numpy(np.flatnonzero(np.diff(cu))).cuda()
    if len(rest):
        few = torch.tensor([cu[int(i)] for i in rest] + [cu[int(rest[-1]) + 1]], dtype=torch.int32, device="cuda")
        out2, last2 = gdn.ssm_scan(*c.args(), few, D=c.D, dt_bias=c.bias, S0=c.S0[rest])
        got2 = gdn.ssm_scan_bwd(*c.args(), go, few, D=c.D, dt_bias=c.bias, S0=c.S0[rest], grad_S_final=gl[rest])
        assert torch.equal(out, out2) and torch.equal(last[rest], last2) and torch.equal(got[0], got2[0]) and torch.equal(got[7][rest], got2[7])


@pytest.mark.parametrize("t", [0, 1, 131, 2048])
def test_few_rows_take_as_long_as_the_states(t):
    """256 sequences, one with rows, 24 heads of 64, N = 128: the states' copy (75 us) and the rows' own time are a bound that
    leaves three copies; dealt to the workgroups of the rows alone, 131 rows took 970 us, and 600 for the gradients."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"padded time t{t}")
    r, h, p, n = 256, 24, 64, 128
    make = lambda *shape: torch.randn(*shape, device="cuda").to(torch.bfloat16)  # noqa: E731
    args = make(t, h, p), make(t, h), -torch.rand(h, device="cuda") - 1, make(t, 1, n), make(t, 1, n)
    one, all_ = (torch.tensor([0] + [t] * k, dtype=torch.int32, device="cuda") for k in (1, r))
    S0, go = torch.randn(r, h, n, p, device="cuda"), make(t, h, p)
    into = torch.empty_like(S0)
    copy = time_us(torch, lambda: into.copy_(S0))
    for name, call in (("scan", lambda cu, k: gdn.ssm_scan(*args, cu, S0=S0[:k])),
                       ("gradients", lambda cu, k: gdn.ssm_scan_bwd(*args, go, cu, S0=S0[:k], grad_S_final=S0[:k]))):
        alone, padded = time_us(torch, lambda: call(one, 1)), time_us(torch, lambda: call(all_, r))
        print(f"[time] {name}: {alone:.1f} us for one sequence, {padded:.1f} with {r - 1} without rows, their copy {copy:.1f}", flush=True)
        assert padded <= alone + 3 * copy, name
