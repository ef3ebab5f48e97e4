"""Gradients of attention over packed prompts on the GPU against the 64-bit oracle's, and against differences.

Tolerances, element by element, with u = 2^-8 (half a bf16 step).  dv: every weight p is rounded to bf16 once and the
sum once, u (sum p |do| + |dv|).  delta is summed from the rounded output, so it errs by u sum |do o|; ds = p (dp -
delta) errs by p u sum |do o| and, rounded once where it enters dk, by u |ds| more; for dq it enters in two parts, 2^-16 |ds|,
which float32's share covers.  It reaches dq and dk through |k| and |q|; these are rounded once.
float32 exponents and sums add 2^-12 of the same sums with |dp| + |delta| in place of |dp - delta| (scores here are below
2^6, so exponents err by less than 2^-17; sums of 700 terms by less than 2^-14).
"""
import numpy as np
import pytest

from gpu_util import note, torch_dev
from oracle import attention as ref
from test_gpu_attn_prompt import BEHIND, RAGGED, RANKED, cu_of, host, make, offsets, padded, ranked  # noqa: F401

pytestmark = pytest.mark.gpu
U, F = 2.0 ** -8, 2.0 ** -12


def bounds(q, k, v, do, cu, scale, grads):
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    tq, tk, tv = (np.abs(x) * U + 1e-30 for x in grads)
    for a, b in zip(cu[:-1], cu[1:]):
        for h in range(Hq if b > a else 0):
            s = q[a:b, h] @ k[a:b, h // G].T * scale
            s = np.where(np.tril(np.ones_like(s, dtype=bool)), s, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o, dp = p @ v[a:b, h // G], do[a:b, h] @ v[a:b, h // G].T
            delta, off = (do[a:b, h] * o).sum(1, keepdims=True), np.abs(do[a:b, h] * o).sum(1, keepdims=True)
            e = abs(scale) * p * (U * off + F * (np.abs(dp) + np.abs(delta)))
            tq[a:b, h] += e @ np.abs(k[a:b, h // G])
            tk[a:b, h // G] += (e + abs(scale) * p * U * np.abs(dp - delta)).T @ np.abs(q[a:b, h])
            tv[a:b, h // G] += (U + F) * p.T @ np.abs(do[a:b, h])
    return tq, tk, tv


def check(torch, q, k, v, cu, scale=None, do=None, seed=0, into=None):
    import linear_attention_sequence_gated_amd as gdn
    T, Hq, D = q.shape
    H = k.shape[1]
    if do is None:
        do = torch.from_numpy(np.random.default_rng(seed + 99).standard_normal((T, Hq, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    c = cu_of(torch, cu)
    out, lse = gdn.attn_prompt(q, k, v, c, scale)
    grads = into or [torch.full((T, n, D), 7.0, dtype=torch.bfloat16, device="cuda") for n in (Hq, H, H)]
    got = gdn.attn_prompt_bwd(q, k, v, out, lse, do, c, scale, *grads)
    torch.cuda.synchronize()
    x = [np.nan_to_num(y, nan=0, posinf=0, neginf=0) for y in host(q, k, v, do)]
    scale = D ** -0.5 if scale is None else scale
    want = ref.prompt(x[0], x[1], x[2], cu, scale, x[3])[2:]
    tol = bounds(*x, cu, scale, want)
    inside = np.zeros(T, bool)
    for a, b in zip(cu[:-1], cu[1:]):
        inside[a:b] = True
    worst = []
    for g, w, t in zip(host(*got), want, tol):
        assert np.all(g[~inside] == 7), "rows of no sequence are left as they were"
        worst.append((np.abs(g - w) / t)[inside].max(initial=0))
    print("worst share of the tolerance: dq %.2f dk %.2f dv %.2f" % tuple(worst))
    assert max(worst) <= 1
    return got


@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300, 513, 700])
@pytest.mark.parametrize("Hq,H,D", [(2, 2, 64), (2, 1, 128)])
def test_one_prompt(L, Hq, H, D):
    torch = torch_dev()
    note(f"bwd L{L} Hq{Hq} H{H} D{D}")
    check(torch, *make(torch, np.random.default_rng(L), L, Hq, H, D), offsets([L]))


@pytest.mark.parametrize("lens", RAGGED.values(), ids=RAGGED.keys())
@pytest.mark.parametrize("Hq,H,D,fused", [(3, 1, 64, True), (4, 4, 64, False), (4, 2, 128, True), (8, 1, 128, False)])
def test_packed_prompts(lens, Hq, H, D, fused):
    torch = torch_dev()
    note(f"bwd packed {len(lens)} sequences Hq{Hq} H{H} D{D}")
    check(torch, *make(torch, np.random.default_rng(len(lens)), sum(lens), Hq, H, D, fused), offsets(lens))


@pytest.mark.parametrize("lens", RANKED.values(), ids=RANKED.keys())
@pytest.mark.parametrize("H,D", [(16, 64), (4, 64), (16, 128), (4, 128)])
def test_tiles_taken_by_length(lens, H, D):
    """Rows and keys: four key heads are shared out by query heads, so that there are as many workgroups."""
    torch = torch_dev()
    cu = offsets(lens, 37)
    T = int(cu[-1]) + 150
    assert ranked(T, len(lens), 16) and ranked(T, len(lens) + 260, 16)
    note(f"bwd by length {len(lens)} sequences H{H} D{D}")
    check(torch, *make(torch, np.random.default_rng(len(lens)), T, 16, H, D), cu)


@pytest.mark.parametrize("R,most", [(511, 9), (512, 9), (1400, 4)])
@pytest.mark.parametrize("Hq,H,D", [(4, 4, 64), (4, 1, 64), (2, 2, 128), (4, 1, 128)])
def test_more_sequences_than_a_window(R, most, Hq, H, D):
    """More offsets than are looked up at once, for dq, for dk and dv, and for the sums of shared heads."""
    torch = torch_dev()
    lens = np.random.default_rng(R).integers(0, most + 1, R)
    lens[R // 2] = 150
    note(f"bwd {R} sequences Hq{Hq} H{H} D{D}")
    check(torch, *make(torch, np.random.default_rng(R + D), int(lens.sum()), Hq, H, D), offsets(lens))


def test_gradients_into_one_projection():
    """q, k, v and their gradients as parts of fused tensors; grad_out with room between its rows."""
    torch = torch_dev()
    rng = np.random.default_rng(5)
    lens, Hq, H, D = [40, 100, 3], 4, 2, 64
    q, k, v = make(torch, rng, sum(lens), Hq, H, D)
    wide = torch.from_numpy(rng.standard_normal((sum(lens), 2 * Hq, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    d = torch.full((sum(lens), Hq + 2 * H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    note("bwd into one projection")
    check(torch, q, k, v, offsets(lens), do=wide[:, Hq:], into=list(d.split([Hq, H, H], 1)))


@pytest.mark.parametrize("D", [64, 128])
def test_rows_outside_may_hold_anything(D):
    torch = torch_dev()
    lens, rng = [70, 30, 90], np.random.default_rng(6)
    cu = offsets(lens, before=9)
    T = cu[-1] + 60
    q, k, v = make(torch, rng, T, 2, 1, D)
    do = torch.from_numpy(rng.standard_normal((T, 2, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    for x in (q, k, v, do):
        x[:9], x[cu[-1]:] = float("nan"), float("inf")
    note(f"bwd outside D{D}")
    good = check(torch, q, k, v, cu, do=do)
    # a neighbour that is not finite changes nothing elsewhere, and shows in its own gradients
    import linear_attention_sequence_gated_amd as gdn
    for bad in range(4):
        x = [t.clone() for t in (q, k, v, do)]
        x[bad][cu[1] + 12] = float("nan")
        c = cu_of(torch, cu)
        out, lse = gdn.attn_prompt(*x[:3], c)
        got = gdn.attn_prompt_bwd(*x[:3], out, lse, x[3], c)
        keep = np.r_[cu[0]:cu[1], cu[2]:cu[3]]
        for a, b in zip(got, good):
            assert torch.equal(a[keep], b[keep])
        # dv = sum p do does not contain v
        assert all(g[cu[1]:cu[2]].isnan().any() for g in (got[:2] if bad == 2 else got))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("first,end", BEHIND)
def test_waves_behind_the_last_key(first, end, D):
    """Waves of a tile that no sequence reaches any more: their rows' gradients are zeros, whatever rows outside hold."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    T = -(-end // 128) * 128 + 70
    q, k, v = make(torch, np.random.default_rng(end), T, 4, 2, D, fused=False)
    do = torch.from_numpy(np.random.default_rng(end + 1).standard_normal((T, 4, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    cu = np.array([first, end])
    note(f"bwd behind {first} {end} D{D}")
    good = check(torch, q, k, v, cu, do=do)
    outside, c = np.r_[0:first, end:T], cu_of(torch, cu)
    for bad in ("nan", "inf"):
        for x in (q, k, v, do):
            x[outside] = float(bad)
        out, lse = gdn.attn_prompt(q, k, v, c)
        for a, b in zip(gdn.attn_prompt_bwd(q, k, v, out, lse, do, c), good):
            assert (a[outside] == 0).all() and torch.equal(a[first:end], b[first:end])


def reached(lens, bad, Hq, H):
    """Where results cannot be finite, given where q, k, v and do are not: by the formulas, every row for itself."""
    q, k, v, do = bad
    G, cu = Hq // H, offsets(lens)
    out, dq, dk, dv = (np.zeros_like(x) for x in (q, q, k, v))
    for a, b in zip(cu[:-1], cu[1:]):
        for h in range(Hq):
            kv = h // G
            keys = np.logical_or.accumulate(k[a:b, kv].any(1))  # a key that row i sees is not finite
            values = np.logical_or.accumulate(v[a:b, kv], 0)
            weights = q[a:b, h].any(1) | keys  # the row's scores, its lse
            out[a:b, h] = weights[:, None] | values
            scores = weights | do[a:b, h].any(1) | values.any(1)  # the gradients of the row's scores
            dq[a:b, h] = scores[:, None]
            dk[a:b, kv] |= np.logical_or.accumulate(scores[::-1])[::-1][:, None]
            dv[a:b, kv] |= np.logical_or.accumulate((weights[:, None] | do[a:b, h])[::-1], 0)[::-1]
    return out, dq, dk, dv


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(4, 2), (3, 3)])
@pytest.mark.parametrize("lens", [[300, 5, 400, 200], [900], [130, 640, 1, 129]])
def test_values_that_are_not_finite_reach_what_the_formulas_say(lens, Hq, H, D):
    """A value that is not finite in one tensor, at rows of every part of a tile, in a column: results that depend on it
    are not finite, through however many tiles, and the others are bit for bit what they were."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    rng = np.random.default_rng(len(lens) + D)
    T = sum(lens)
    good = [t.contiguous() for t in make(torch, rng, T, Hq, H, D, fused=False)]
    good.append(torch.from_numpy(rng.standard_normal((T, Hq, D)).astype(np.float32)).to(torch.bfloat16).cuda())
    c = cu_of(torch, offsets(lens))

    def run(x):
        out, lse = gdn.attn_prompt(*x[:3], c)
        return [out, *gdn.attn_prompt_bwd(*x[:3], out, lse, x[3], c)]

    want = run(good)
    for which, value in [(0, "nan"), (1, "nan"), (2, "nan"), (2, "inf"), (2, "-inf"), (3, "nan"), (3, "inf")]:
        for rows in ([T // 2], [0], [T - 1], [127, 128], [31, 300], [5, T - 40]):
            x, bad = [t.clone() for t in good], [np.zeros(tuple(t.shape), bool) for t in good]
            for row in rows:
                h, d = rng.integers(x[which].shape[1]), rng.integers(D)
                x[which][row, h, d], bad[which][row, h, d] = float(value), True
            note(f"bwd not finite {lens} Hq{Hq} H{H} D{D}: {which} {value} {rows}")
            for name, got, clean, no in zip(("out", "dq", "dk", "dv"), run(x), want, reached(lens, bad, Hq, H)):
                assert np.array_equal(~got.isfinite().cpu().numpy(), no), name
                no = torch.from_numpy(no).cuda()
                assert torch.equal(got.masked_fill(no, 0), clean.masked_fill(no, 0)), name


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[4096], [2050, 2046]])
def test_a_step_that_diverged_is_no_slower_by_orders(lens, D):
    """All of one tensor not finite: the forward and the gradients stay within ten times their usual time (rows that every
    lane looked through by itself took 600 times as long)."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    T, c = sum(lens), cu_of(torch, offsets(lens))
    good = [t.contiguous() for t in make(torch, np.random.default_rng(3), T, 8, 2, D, fused=False)]
    good.append(torch.ones(T, 8, D, dtype=torch.bfloat16, device="cuda"))

    def time(x):
        best = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            out, lse = gdn.attn_prompt(*x[:3], c)
            gdn.attn_prompt_bwd(*x[:3], out, lse, x[3], c)
            b.record()
            torch.cuda.synchronize()
            best.append(a.elapsed_time(b))
        return min(best)

    usual = time(good)
    for which in range(4):
        x = list(good)
        x[which] = torch.full_like(x[which], float("nan"))
        note(f"bwd diverged {lens} D{D}: {which}")
        took = time(x)
        print("%.3f ms, usually %.3f" % (took, usual))
        assert took <= 10 * usual


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (-0.2, 1.0), (1.0, 2.0), (1e-3, 30.0)])
def test_scales(D, scale, size):
    torch = torch_dev()
    note(f"bwd scale {scale} size {size} D{D}")
    check(torch, *make(torch, np.random.default_rng(7), 300, 2, 2, D, size=size), offsets([150, 150]), scale)


def test_same_gradients_every_time():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    q, k, v = make(torch, np.random.default_rng(8), 900, 8, 2, 64)
    c, do = cu_of(torch, [0, 400, 900]), torch.ones(900, 8, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = gdn.attn_prompt(q, k, v, c)
    a, b = (gdn.attn_prompt_bwd(q, k, v, out, lse, do, c) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_against_differences():
    """Along random directions, sum grad . direction against a central difference of the oracle's forward."""
    torch = torch_dev()
    lens, D = [50, 90], 64
    q, k, v = make(torch, np.random.default_rng(9), sum(lens), 4, 2, D)
    cu = offsets(lens)
    note("bwd differences")
    got = host(*check(torch, q, k, v, cu, seed=1))
    do = np.random.default_rng(1 + 99).standard_normal((sum(lens), 4, D)).astype(np.float32)
    do = torch.from_numpy(do).to(torch.bfloat16).float().numpy().astype(np.float64)
    x = host(q, k, v)
    want = ref.prompt(*x, cu, D ** -0.5, do)[2:]
    tol = bounds(*x, do, cu, D ** -0.5, want)
    for i in range(3):
        for seed in range(3):
            d = np.random.default_rng(seed).standard_normal(x[i].shape)
            ends = []
            for eps in (1e-5, -1e-5):
                y = list(x)
                y[i] = y[i] + eps * d
                ends.append((ref.prompt(*y, cu, D ** -0.5)[0] * do).sum())
            diff = (ends[0] - ends[1]) / 2e-5
            assert abs((got[i] * d).sum() - diff) <= (tol[i] * np.abs(d)).sum() + 1e-4 * abs(diff) + 1e-3


@pytest.mark.parametrize("cu", [[-5, 40, 30, 100000, 2 ** 31 - 1], [100, 50, 0], [-2 ** 31, -1, 2 ** 31 - 1], [7], [64, 64, 64]])
def test_offsets_out_of_order(cu):
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    q, k, v = make(torch, np.random.default_rng(9), 200, 2, 1, 64)
    c = cu_of(torch, cu)
    note(f"bwd offsets {cu}")
    out, lse = gdn.attn_prompt(q, k, v, c)
    gdn.attn_prompt_bwd(q, k, v, out, lse, out, c)
    torch.cuda.synchronize()
