"""Causal attention over packed prompts on the GPU against the 64-bit oracle.

Tolerances of the forward, element by element: a weight is rounded to bf16 once (2^-8 relative, its exponent errs by far
less), so a result is off by at most 2^-8 of the weighted sum of |v|, and by 2^-8 of itself when it is rounded.  lse:
float32 sums of D exact products, 2^-19 of (largest sum |q k| + 1 + |lse|) covers D = 128 additions of half an ulp each.
"""
import numpy as np
import pytest

from gpu_util import note, torch_dev
from oracle import attention as ref
from test_gpu_attn_cache import ints

pytestmark = pytest.mark.gpu
PAD = [False]


@pytest.fixture(params=[False, True], ids=["as given", "padded"], autouse=True)
def padded(request):
    """With many sequences of no rows behind the others: few rows to a sequence choose the other tiles."""
    PAD[0] = request.param
    yield
    PAD[0] = False


def cu_of(torch, cu):
    return ints(torch, np.concatenate([cu, np.repeat(cu[-1:], 260)]) if PAD[0] else cu)


def make(torch, rng, T, Hq, H, D, fused=True, size=1.0):
    """(q, k, v) bf16 on the GPU, parts of one projection or dense."""
    x = torch.from_numpy((size * rng.standard_normal((T, Hq + 2 * H, D))).astype(np.float32)).to(torch.bfloat16).cuda()
    parts = x.split([Hq, H, H], 1)
    return parts if fused else [p.contiguous() for p in parts]


def host(*ts):
    return [t.float().cpu().numpy().astype(np.float64) for t in ts]


def check_forward(torch, q, k, v, cu, scale=None):
    import linear_attention_sequence_gated_amd as gdn
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, T), 7.0, device="cuda")
    gdn.attn_prompt(q, k, v, cu_of(torch, cu), scale, out=out, lse=lse)
    torch.cuda.synchronize()
    scale = D ** -0.5 if scale is None else scale
    qs, ks, vs = host(q, k, v)
    want, wlse = ref.prompt(qs, ks, vs, cu, scale)
    weighted, _ = ref.prompt(qs, ks, np.abs(vs), cu, scale)
    inside = np.zeros(T, bool)
    for a, b in zip(cu[:-1], cu[1:]):
        inside[a:b] = True
    got, glse = host(out)[0], lse.cpu().numpy().astype(np.float64)
    assert np.all(got[~inside] == 7) and np.all(glse[:, ~inside] == 7), "rows of no sequence are left as they were"
    tol = 2.0 ** -8 * (np.abs(want) + weighted) + 1e-30
    size = abs(scale) * np.abs(qs[inside]).sum(2).max() * np.abs(ks[inside]).max()
    eo = (np.abs(got - want) / tol)[inside].max(initial=0)
    el = (np.abs(glse - wlse) / (2.0 ** -19 * (size + 1 + np.abs(wlse))))[:, inside].max(initial=0)
    print("worst share of the tolerance: out %.2f lse %.2f" % (eo, el))
    assert eo <= 1 and el <= 1
    return out, lse


def offsets(lens, before=0):
    return np.concatenate([[0], np.cumsum(lens)]) + before


@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300, 513, 700])
@pytest.mark.parametrize("Hq,H,D", [(2, 2, 64), (2, 1, 128)])
def test_one_prompt(L, Hq, H, D):
    torch = torch_dev()
    note(f"prompt L{L} Hq{Hq} H{H} D{D}")
    check_forward(torch, *make(torch, np.random.default_rng(L), L, Hq, H, D), offsets([L]))


RAGGED = {
    "mixed": [5, 0, 130, 1, 1, 64, 63, 200, 0, 0, 33, 257, 2],
    "tiny": [1] * 150 + [0] * 20 + [2, 3] * 30 + [16] * 10,
    "empty ends": [0, 0, 100, 0, 0, 0, 28, 0],
    "long then short": [600, 1, 7, 300],
}


@pytest.mark.parametrize("lens", RAGGED.values(), ids=RAGGED.keys())
@pytest.mark.parametrize("Hq,H,D,fused", [(3, 1, 64, True), (4, 4, 64, False), (4, 2, 128, True), (8, 1, 128, False)])
def test_packed_prompts(lens, Hq, H, D, fused):
    torch = torch_dev()
    note(f"packed {len(lens)} sequences Hq{Hq} H{H} D{D}")
    check_forward(torch, *make(torch, np.random.default_rng(len(lens)), sum(lens), Hq, H, D, fused), offsets(lens))


RANKED = {
    "equal": [350] * 13,
    "ragged": [1201, 0, 700, 3, 0, 512, 640, 1, 900, 128, 127, 129, 261],
    "one long": [1900] + [5, 200, 64, 0, 131] * 7,
    "many": [17, 40, 3, 128, 0, 60] * 19,
}


def ranked(T, R, heads):
    """Whether tiles of 128 rows are taken by their length: several sequences, more workgroups than run at once."""
    tiles = -(-T // 128)
    mean = T // R
    return 1 < R < 512 and tiles <= 256 and tiles * heads > 512 and T * heads * (600 + mean) >= 108000 * mean


@pytest.mark.parametrize("lens", RANKED.values(), ids=RANKED.keys())
@pytest.mark.parametrize("H,D", [(16, 64), (4, 128)])
def test_tiles_taken_by_length(lens, H, D):
    """Every tile is taken once, whatever the lengths: ties, empty sequences, rows outside, tiles no multiple of four."""
    torch = torch_dev()
    cu = offsets(lens, 37)
    T = int(cu[-1]) + 150
    assert ranked(T, len(lens), 16) and ranked(T, len(lens) + 260, 16)
    note(f"by length {len(lens)} sequences H{H} D{D}")
    check_forward(torch, *make(torch, np.random.default_rng(len(lens)), T, 16, H, D), cu)


def test_thousands_of_sequences():
    torch = torch_dev()
    lens = np.random.default_rng(1).integers(0, 4, 5000)
    note("5000 sequences")
    check_forward(torch, *make(torch, np.random.default_rng(2), int(lens.sum()), 1, 1, 64), offsets(lens))


@pytest.mark.parametrize("lens", [[300, 300, 300, 300], [1, 511, 64, 65, 0, 600], [1200], [1000, 31, 33, 100]])
def test_tiles_with_keys_in_halves(lens):
    """Work and chains of tiles in between: the form that halves the keys; rows outside, and values there that are not finite."""
    torch = torch_dev()
    heads = {4: 24, 6: 17, 1: 40}[len(lens)]
    cu = offsets(lens, 7)
    T = int(cu[-1]) + 9
    mean = T // len(lens)
    assert 62000 * mean <= T * heads * (600 + mean) < 108000 * mean
    q, k, v = make(torch, np.random.default_rng(len(lens)), T, heads, 1, 128)
    note(f"halves {lens}")
    out, lse = check_forward(torch, q, k, v, cu)
    v[:7], v[-9:], k[:7], k[-9:] = float("inf"), float("nan"), float("nan"), float("nan")
    again, lse2 = check_forward(torch, q, k, v, cu)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    row = int(cu[0] + cu[1]) // 2  # a row of the first sequence: those before it and those of the others do not see it
    v[row, 0, 3] = float("-inf")
    bad = check_nothing_else(torch, q, k, v, cu, out)
    assert torch.equal(bad[row:int(cu[1]), :, 3], torch.full_like(bad[row:int(cu[1]), :, 3], float("-inf")))


def check_nothing_else(torch, q, k, v, cu, good):
    """The forward's output, which is the given one but for column 3 of the first sequence."""
    import linear_attention_sequence_gated_amd as gdn
    out = torch.full_like(good, 7.0)
    lse = torch.full((q.shape[1], q.shape[0]), 7.0, device="cuda")
    gdn.attn_prompt(q, k, v, cu_of(torch, cu), out=out, lse=lse)
    a, b = out.clone(), good.clone()
    a[cu[0]:cu[1], :, 3] = b[cu[0]:cu[1], :, 3] = 0
    assert torch.equal(a, b)
    return out


@pytest.mark.parametrize("D", [64, 128])
def test_rows_outside_and_what_they_hold(D):
    """Rows before the first and behind the last sequence hold NaN and infinities; so may a sequence's own later rows
    and its neighbours, without a trace in the rows that do not attend to them."""
    torch = torch_dev()
    rng = np.random.default_rng(3)
    lens = [70, 30, 90]
    cu = offsets(lens, before=11)
    T = cu[-1] + 25
    q, k, v = make(torch, rng, T, 2, 1, D)
    for x, bad in ((q, "nan"), (k, "inf"), (v, "nan")):
        x[:11], x[cu[-1]:] = float(bad), -float(bad)
    note(f"outside D{D}")
    out, lse = check_forward(torch, q, k, v, cu)
    # a whole neighbouring sequence, and one row late in the first
    for x in (k, v):
        x[cu[1]:cu[2]] = float("nan")
    v[cu[0] + 50, 0, 3], v[cu[0] + 60, 0, 4], k[cu[0] + 65] = float("inf"), -float("inf"), float("nan")
    import linear_attention_sequence_gated_amd as gdn
    out2, lse2 = gdn.attn_prompt(q, k, v, cu_of(torch, cu))
    keep = np.r_[cu[0]:cu[0] + 50, cu[2]:cu[3]]
    assert torch.equal(out2[keep], out[keep]) and torch.equal(lse2[:, keep], lse[:, keep])
    assert out2[cu[1]:cu[2]].isnan().all()
    late = out2[cu[0] + 50:cu[0] + 60].float()
    assert (late[..., 3] == float("inf")).all() and late[..., 4].isfinite().all()
    late = out2[cu[0] + 60:cu[0] + 65].float()
    assert (late[..., 3] == float("inf")).all() and (late[..., 4] == -float("inf")).all()
    assert out2[cu[0] + 65:cu[1]].isnan().all()
    v[cu[0] + 62, 1 - 1, 3] = float("nan")
    out3, _ = gdn.attn_prompt(q, k, v, cu_of(torch, cu))
    assert out3[cu[0] + 62:cu[0] + 65, :, 3].isnan().all() and torch.equal(out3[cu[0]:cu[0] + 62], out2[cu[0]:cu[0] + 62])


BEHIND = [(0, 129), (5, 133), (5, 135), (0, 140), (1, 161), (100, 290), (0, 1), (3, 5)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("first,end", BEHIND)
def test_waves_behind_the_last_key(first, end, D):
    """Waves of a tile that no sequence reaches any more: their rows are zeros, whatever rows outside hold."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    T = -(-end // 128) * 128 + 70
    q, k, v = make(torch, np.random.default_rng(end), T, 4, 2, D, fused=False)
    cu = np.array([first, end])
    note(f"behind {first} {end} D{D}")
    good, glse = check_forward(torch, q, k, v, cu)
    outside = np.r_[0:first, end:T]
    for bad in ("nan", "inf"):
        for x in (q, k, v):
            x[outside] = float(bad)
        out, lse = gdn.attn_prompt(q, k, v, cu_of(torch, cu))
        assert (out[outside] == 0).all() and (lse[:, outside] == 0).all()
        assert torch.equal(out[first:end], good[first:end]) and torch.equal(lse[:, first:end], glse[:, first:end])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (-0.2, 1.0), (1.0, 3.0), (1e-3, 30.0), (30.0, 0.2)])
def test_scales(D, scale, size):
    """Uniform weights, turned signs, weights on one key, large numbers: the running maximum moves often or never."""
    torch = torch_dev()
    note(f"scale {scale} size {size} D{D}")
    check_forward(torch, *make(torch, np.random.default_rng(7), 400, 2, 2, D, size=size), offsets([150, 250]), scale)


def test_growing_scores():
    """Every key beats those before it: the maximum moves in every tile."""
    torch = torch_dev()
    q, k, v = make(torch, np.random.default_rng(8), 520, 1, 1, 64)
    q[:] = 1.0
    k[:] = (torch.arange(520, device="cuda") / 16).view(-1, 1, 1)
    note("growing")
    check_forward(torch, q, k, v, offsets([520]))
    k[:] = -k
    check_forward(torch, q, k, v, offsets([520]))


@pytest.mark.parametrize("D", [64, 128])
def test_equal_scores_at_the_end_of_their_range(D):
    """-2^29 and 2^29: exponents have no fraction left, but equal scores have equal weights."""
    torch = torch_dev()
    q, k, v = make(torch, np.random.default_rng(9), 200, 1, 1, D, fused=False)
    note(f"equal scores D{D}")
    for sign in (-1, 1):
        q[:], k[:] = 2.0 ** 13, sign * 2.0 ** 13
        check_forward(torch, q, k, v, offsets([140, 60]), 8.0 / D)


@pytest.mark.parametrize("cu", [[-5, 40, 30, 100000, 2 ** 31 - 1], [100, 50, 0], [-2 ** 31, -1, 2 ** 31 - 1], [7], [64, 64, 64]])
def test_offsets_out_of_order(cu):
    """Offsets that are no offsets lead to no access outside the buffers, and only to rows' results that mean nothing."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    q, k, v = make(torch, np.random.default_rng(9), 200, 2, 1, 64)
    note(f"offsets {cu}")
    gdn.attn_prompt(q, k, v, cu_of(torch, cu))
    torch.cuda.synchronize()
