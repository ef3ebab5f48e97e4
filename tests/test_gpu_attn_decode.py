"""Single-token attention over the 8-bit cache on the GPU against the 64-bit oracle.

Tolerances, element by element.  Codes and scales are exact on both sides.  A weight is rounded to fp16 once (2^-11
relative); its exponent is a float32 number of size |s|, so exp errs by about |s| 2^-22, under 2^-13 for the scores here
(|s| < 100): together under 2^-10 of the weighted sum of |v|.  The result is rounded to bf16 once: 2^-8 of its value.
The scores are float32 sums of D exact products, and lse is a logarithm of float32 sums: 2^-19 of (sum |q k| + 1 +
|lse|) covers D = 128 additions that err half an ulp each, in the order the matrix core takes them.
"""
import numpy as np
import pytest

from gpu_util import note, torch_dev
from oracle import attention as ref
from test_gpu_attn_cache import ints, make_cache, values

pytestmark = pytest.mark.gpu
WIDE = [False]  # whether tables have room for many more tokens than their requests have


@pytest.fixture(params=[False, True], ids=["narrow", "wide"], autouse=True)
def wide(request):
    """Both ways to deal out the work: by the width of the table no request is long, or some could be."""
    WIDE[0] = request.param
    yield
    WIDE[0] = False



def make(torch, rng, lens, Hq, H, D, bt, kind, extra_width=0, spread=1.0):
    lens = np.asarray(lens, np.int64)
    blocks = -(-np.maximum(lens, 0) // bt)
    nb = int(blocks.sum()) + 2
    ids = rng.permutation(nb)
    extra_width += 65 * 128 // bt if WIDE[0] else 0
    table = np.full((len(lens), max(1, int(blocks.max(initial=0))) + extra_width), -1)
    at = 0
    for r, b in enumerate(blocks):
        table[r, :b] = ids[at:at + b]
        at += b
    kc, ks = make_cache(torch, rng, nb, H, bt, D, kind)
    vc, vs = make_cache(torch, rng, nb, H, bt, D, kind)
    vs *= torch.from_numpy(np.exp(spread * rng.standard_normal(tuple(vs.shape))).astype(np.float32))
    q = torch.from_numpy(rng.standard_normal((len(lens), Hq, D)).astype(np.float32)).to(torch.bfloat16)
    return q, kc, vc, ks, vs, table, lens


def bounds(q, kv, vv, ks, vs, table, lens, scale, out, lse):
    """(out's, lse's) tolerance from |v| weighted and |q||k| summed."""
    nb = kv.shape[0]
    weighted, _ = ref.decode(q, kv, np.abs(vv), ks, vs, table, lens, scale)
    R, Hq, _ = q.shape
    size = np.zeros((R, Hq))
    for r in range(R):
        ids = [int(b) for b in table[r, :-(-max(0, int(lens[r])) // kv.shape[2])] if 0 <= b < nb]
        for h in range(Hq if ids else 0):
            g = h * kv.shape[1] // Hq
            size[r, h] = (np.abs(kv[ids, g]) * ks[ids, g][:, None, None] @ np.abs(q[r, h])).max() * scale
    return 2.0 ** -8 * np.abs(out) + 2.0 ** -10 * weighted + 1e-30, 2.0 ** -19 * (size + 1 + np.abs(np.where(np.isfinite(lse), lse, 0)))


def check(torch, q, kc, vc, ks, vs, table, lens, scale=None, qdev=None):
    import linear_attention_sequence_gated_amd as gdn
    D = q.shape[-1]
    args = [ints(torch, table), ints(torch, np.minimum(lens, 2 ** 31 - 1))]
    out, lse = gdn.attn_decode(q.cuda() if qdev is None else qdev, kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), *args, scale)
    torch.cuda.synchronize()
    scale = D ** -0.5 if scale is None else scale
    x = (q.float().numpy().astype(np.float64), values(kc), values(vc), ks.numpy(), vs.numpy(), table, lens, scale)
    want, wlse = ref.decode(*x)
    to, tl = bounds(x[0], x[1], x[2], *x[3:], want, wlse)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.array_equal(np.isneginf(lse), np.isneginf(wlse))
    eo = np.abs(out - want) / to
    some = np.isfinite(wlse)
    el = np.abs(lse[some] - wlse[some]) / tl[some]
    print("worst share of the tolerance: out %.2f lse %.2f" % (eo.max(initial=0), el.max(initial=0)))
    assert eo.max(initial=0) <= 1 and el.max(initial=0) <= 1
    return out, lse


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 65, 127, 128, 129, 200, 0, 511, 640]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("bt", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,H,D", [(4, 4, 64), (6, 2, 64), (8, 1, 128), (16, 1, 64), (12, 4, 128)])
def test_decode_ragged(Hq, H, D, bt, kind):
    torch = torch_dev()
    note(f"decode Hq{Hq} H{H} D{D} bt{bt} {kind}")
    check(torch, *make(torch, np.random.default_rng(Hq + D + bt), LENS, Hq, H, D, bt, kind))


@pytest.mark.parametrize("Hq,H", [(17, 1), (40, 2), (64, 2)])
def test_decode_more_query_heads_than_columns(Hq, H):
    torch = torch_dev()
    note(f"decode Hq{Hq} H{H}")
    check(torch, *make(torch, np.random.default_rng(Hq), [0, 5, 130, 300], Hq, H, 64, 32, "int8"))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,D", [([1], 64), ([9000], 64), ([40000], 128), ([20011, 3, 0, 5000], 128)])
def test_decode_long_and_few(lens, D, kind):
    """One request over many workgroups, whose shares begin and end inside it."""
    torch = torch_dev()
    note(f"decode long {lens} D{D} {kind}")
    check(torch, *make(torch, np.random.default_rng(len(lens)), lens, 2, 1, D, 64, kind))


def test_decode_many_requests():
    """More requests than threads find them, runs of empty ones between, several requests to a workgroup."""
    torch = torch_dev()
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 300, 1500)
    lens[100:400] = 0
    lens[-70:] = 0
    note("decode many")
    check(torch, *make(torch, rng, lens, 2, 1, 64, 16, "e4m3"))


@pytest.mark.parametrize("D,H", [(64, 3), (128, 2)])
@pytest.mark.parametrize("R", [70, 300, 800])
def test_decode_shares_that_begin_and_end_anywhere(R, D, H):
    """Lengths around whole units of 128 tokens, many more units than workgroups and about as many: shares that begin
    or end with a request's first unit, its last, or between two requests."""
    torch = torch_dev()
    rng = np.random.default_rng(R + D)
    lens = rng.choice([0, 1, 127, 128, 129, 256, 257, 900], R)
    note(f"decode shares R{R} D{D}")
    check(torch, *make(torch, rng, lens, 2 * H, H, D, 128, "int8"))


def forms(R, H, longest):
    """Whether one workgroup takes all of a request and key head (there is nothing to join) for tables of `longest`."""
    import linear_attention_sequence_gated_amd as gdn
    return gdn.gdn_attn_decode_workspace_bytes(R, 2 * H, H, 64, 16, -(-longest // 16)) == 0


@pytest.mark.parametrize("D,kind", [(64, "int8"), (128, "e4m3")])
@pytest.mark.parametrize("R,H,longest", [(60, 4, 4000), (63, 4, 4500), (64, 4, 4600), (65, 4, 2500), (126, 2, 3400), (1030, 1, 5200), (40, 9, 2900)])
def test_decode_long_requests_in_one_workgroup(R, H, longest, D, kind):
    """Long requests that one workgroup takes each, many of them: a few of the longest among short ones."""
    torch = torch_dev()
    rng = np.random.default_rng(R + longest)
    lens = rng.choice([0, 1, 33, 128, 300, 511], R)
    lens[rng.permutation(R)[:5]] = [longest, longest - 1, longest - 15, longest // 2 + 7, 1025]
    note(f"decode whole R{R} H{H} {longest} D{D} {kind}")
    assert forms(R, H, longest)
    check(torch, *make(torch, rng, lens, 2 * H, H, D, 16, kind))


def test_decode_many_requests_of_many_heads():
    """More query heads to a key head than columns, the last group in part, more rows than ends of shares."""
    torch = torch_dev()
    rng = np.random.default_rng(4)
    note("decode many heads")
    check(torch, *make(torch, rng, rng.choice([0, 3, 128, 300, 700], 500), 46, 2, 64, 64, "e4m3"))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_decode_ignores_what_lies_behind(kind):
    """Bits behind a request's last token, unused blocks and their scales may be anything, NaN codes included."""
    torch = torch_dev()
    rng = np.random.default_rng(4)
    q, kc, vc, ks, vs, table, lens = make(torch, rng, [5, 16, 77, 0, 130], 4, 2, 64, 32, kind, extra_width=3)
    a, b = kc.view(torch.int8), vc.view(torch.int8)
    used = np.zeros(len(kc), bool)
    for r, n in enumerate(lens):
        for i in range(-(-n // 32)):
            used[table[r, i]] = True
            a[table[r, i], :, max(0, n - 32 * i):] = 0x7f
            b[table[r, i], :, max(0, n - 32 * i):] = 0x7f
    a[~used], b[~used] = -1, 0x7f
    ks[torch.from_numpy(~used)], vs[torch.from_numpy(~used)] = float("nan"), float("inf")
    table[table < 0] = rng.choice([-1, 10 ** 9, 2 ** 31 - 1, -2 ** 31], (table < 0).sum())
    note(f"decode behind {kind}")
    import linear_attention_sequence_gated_amd as gdn
    out, lse = gdn.attn_decode(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), ints(torch, table), ints(torch, lens))
    clean = [torch.where(torch.from_numpy(used).view(-1, 1, 1, 1), x.float(), 0).nan_to_num(0) for x in (kc, vc)]
    want, wlse = ref.decode(q.float().numpy(), *(x.numpy() for x in clean), ks.nan_to_num(1).numpy(),
                            torch.where(torch.isinf(vs), 1, vs).numpy(), table, lens, 64 ** -0.5)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isfinite(out).all() and np.array_equal(np.isneginf(lse), np.isneginf(wlse))
    assert np.abs(out - want).max() <= 2.0 ** -8 * np.abs(want).max() * 2
    assert np.all(out[3] == 0)


def test_decode_blocks_outside_the_cache_and_lengths_past_the_table():
    """A block that does not exist is left out; a length past the table's width ends there; negative ones are empty."""
    torch = torch_dev()
    rng = np.random.default_rng(6)
    q, kc, vc, ks, vs, table, lens = make(torch, rng, [100, 64, 200, 16, 16], 4, 2, 128, 16, "int8")
    table[0, 2], table[0, 6], table[2, 0], table[3, 0] = -1, len(kc), 2 ** 31 - 1, -2 ** 31
    lens[2], lens[4] = 2 ** 31 - 1, -5
    note("decode bad blocks")
    out, lse = check(torch, q, kc, vc, ks, vs, table, lens)
    assert np.isneginf(lse[3]).all() and np.all(out[4] == 0)


def test_decode_strided_queries_scale_and_large_numbers():
    torch = torch_dev()
    rng = np.random.default_rng(8)
    for size in (1e-30, 1.0, 1e4):
        q, kc, vc, ks, vs, table, lens = make(torch, rng, [3, 50, 257], 6, 3, 64, 64, "e4m3", spread=8.0)
        q = (q.float() * size).to(torch.bfloat16)
        wide = torch.zeros(3, 12, 64, dtype=torch.bfloat16)
        wide[:, 6:] = q
        note(f"decode strided {size}")
        check(torch, q, kc, vc, ks, vs, table, lens, scale=0.3 / size, qdev=wide.cuda()[:, 6:])


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.125, -0.4, 1e-30])
def test_decode_scales_of_scores(scale, kind):
    """Uniform weights, turned signs; a scale of nearly nothing."""
    torch = torch_dev()
    note(f"decode scale {scale} {kind}")
    check(torch, *make(torch, np.random.default_rng(9), [1, 40, 0, 700, 2100], 4, 2, 64, 32, kind), scale=scale)


def test_decode_blocks_of_zeros_beside_others():
    """A block of zeros has the smallest scale, 2^-100: its tokens still count in the denominator."""
    torch = torch_dev()
    q, kc, vc, ks, vs, table, lens = make(torch, np.random.default_rng(10), [64, 48, 16], 2, 1, 64, 16, "int8")
    for x, s in ((kc, ks), (vc, vs)):
        x[table[0, 0]], s[table[0, 0]] = 0, 2.0 ** -100
        x[table[1, 1]], s[table[1, 1]] = 0, 2.0 ** -100
        x[table[2, 0]], s[table[2, 0]] = 0, 2.0 ** -100
    note("decode zeros")
    check(torch, q, kc, vc, ks, vs, table, lens)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gap", [8.0, 12.0, 16.0, 19.5])
def test_decode_one_token_far_above_the_others(gap, D, kind):
    """One token's score lies far above those of the others, which are equal, and its value is zero: the output is that
    of the others, whose weights are small numbers (down to e^-19.5 of the largest)."""
    torch = torch_dev()
    q, kc, vc, ks, vs, table, lens = make(torch, np.random.default_rng(15), [20, 300, 2000, 2000], 4, 2, D, 32, kind)
    most = 127 if kind == "int8" else 448
    q[:], ks[:] = 1.0, 1.0
    kc.view(torch.int8)[:] = 0
    for r, at in enumerate((0, 299, 1000, 0)):
        kc[table[r, at // 32], :, at % 32] = torch.full((D,), float(most)).to(kc.dtype)
        vc.view(torch.int8)[table[r, at // 32], :, at % 32] = 0
    note(f"decode far above {gap} D{D} {kind}")
    check(torch, q, kc, vc, ks, vs, table, lens, scale=gap / (most * D))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("power", [-126, -118, -100, -60, 60, 100, 120])
def test_decode_scales_at_the_ends_of_their_range(power, kind):
    """All values' scales next to the smallest or largest that there are: the denominator's sums stay numbers.

    lse is that of any other scales; it is put together from numbers as large as log2 of the scale (below 2^7) plus
    scores and lengths (2^6), which err by half an ulp, 2^-18, where they are added: 2^-15 covers eight such.  Where
    neither they nor their products leave the range of normal bf16 numbers, outputs are those of scales of one, moved."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    q, kc, vc, ks, vs, table, lens = make(torch, np.random.default_rng(14), [1, 30, 700, 9000], 4, 2, 64, 64, kind)
    vs[:] = 1.0
    rest = ints(torch, table), ints(torch, lens)
    x = (q.float().numpy().astype(np.float64), values(kc), values(vc), ks.numpy(), vs.numpy(), table, lens, 64 ** -0.5)
    want, wlse = ref.decode(*x)
    to, tl = bounds(*x, want, wlse)
    note(f"decode scales of 2^{power} {kind}")
    out, lse = gdn.attn_decode(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), torch.full_like(vs, 2.0 ** power).cuda(), *rest)
    assert (np.abs(lse.cpu().numpy() - wlse) <= tl + 2.0 ** -15).all()
    if abs(power) <= 100:
        assert (np.abs(np.ldexp(out.double().cpu().numpy(), -power) - want) <= to).all()


@pytest.mark.parametrize("lens", [[40], [5000, 40, 0]])
def test_decode_queries_that_are_not_finite(lens):
    """A head whose query is not finite gets NaN, and no other head does; a request without tokens gets zeros even so."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    q, kc, vc, ks, vs, table, lens = make(torch, np.random.default_rng(12), lens, 4, 2, 64, 16, "int8")
    dev = [x.cuda() for x in (kc, vc, ks, vs)] + [ints(torch, table), ints(torch, lens)]
    good, _ = gdn.attn_decode(q.cuda(), *dev)
    for bad in (float("nan"), float("inf")):
        x = q.clone()
        x[:, 2, 7] = bad
        out, lse = gdn.attn_decode(x.cuda(), *dev)
        some = torch.from_numpy(lens > 0)
        assert out[some][:, 2].isnan().all() and lse[some][:, 2].isnan().all()
        assert torch.equal(out[:, [0, 1, 3]], good[:, [0, 1, 3]]) and (out[~some] == 0).all()
