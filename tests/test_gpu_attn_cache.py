"""Block tables and the 8-bit cache's write side on the GPU against the oracle: every whole number, code and scale
equal, since each is defined bit by bit."""
import numpy as np
import pytest

from gpu_util import note, torch_dev
from oracle import attention as ref

pytestmark = pytest.mark.gpu


def ints(torch, x, dev="cuda"):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(dev)


def make_requests(rng, R, bt, longest, prompts):
    held = rng.integers(0, longest + 1, R)
    new = np.ones(R, np.int64)
    for r in rng.permutation(R)[:prompts]:
        held[r], new[r] = 0, rng.integers(0, longest + 1)
    return held, new


def make_table(rng, held, new, bt, spare=3):
    blocks = -(-held // bt)
    need = -(-(held + new) // bt)
    total = int(need.sum()) + spare
    ids = rng.permutation(total)
    table = np.full((len(held), max(1, int(need.max(initial=0)))), -7)
    at = 0
    for r, b in enumerate(blocks):
        table[r, :b] = ids[at:at + b]
        at += b
    return table, ids[at:], total


def run_tables(torch, held, new, table, free, bt, nb, T):
    import linear_attention_sequence_gated_amd as gdn
    t = ints(torch, table)
    got = gdn.block_tables(ints(torch, held), ints(torch, new), t, ints(torch, free), bt, nb, T)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (t, *got)]


@pytest.mark.parametrize("R,bt,longest,prompts,pad", [
    (1, 16, 0, 0, 0), (1, 16, 15, 1, 3), (1, 64, 1, 0, 5), (5, 32, 100, 2, 0), (16, 16, 64, 0, 1), (17, 128, 300, 5, 2),
    (64, 16, 33, 64, 700), (255, 64, 500, 3, 0), (257, 32, 129, 20, 1), (1000, 16, 400, 10, 300), (4095, 16, 90, 9, 3), (4097, 32, 90, 9, 3), (9001, 16, 40, 3, 0)])
def test_tables(R, bt, longest, prompts, pad):
    torch = torch_dev()
    rng = np.random.default_rng(R + bt)
    held, new = make_requests(rng, R, bt, longest, prompts)
    table, free, nb = make_table(rng, held, new, bt)
    T = int(new.sum()) + pad
    note(f"tables R{R} bt{bt} T{T}")
    got = run_tables(torch, held, new, table, free, bt, nb, T)
    for name, a, b in zip(("table", "slots", "cu", "after", "used"), got, ref.block_tables(held, new, table, free, bt, nb, T)):
        assert np.array_equal(a, b), name


@pytest.mark.parametrize("what", ["free list short", "slot map short", "table narrow", "negative", "huge", "bad ids", "nothing"])
def test_tables_that_cannot_be_served(what):
    """Requests that do not fit are refused one by one, the others served; nothing outside the buffers is touched."""
    torch = torch_dev()
    rng = np.random.default_rng(3)
    held, new = make_requests(rng, 40, 16, 100, 4)
    table, free, nb = make_table(rng, held, new, 16)
    T = int(new.sum())
    if what == "free list short":
        free = free[:len(free) // 2]
    elif what == "slot map short":
        T = T // 2
    elif what == "table narrow":
        table = np.ascontiguousarray(table[:, :4])
    elif what == "negative":
        held[5], new[7], held[11], new[11] = -3, -1, -2 ** 31, -2 ** 31
    elif what == "huge":
        held[5], new[6], new[7], held[7] = 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1
    elif what == "bad ids":
        free = np.where(rng.random(len(free)) < 0.5, free, rng.choice([-1, nb, 2 ** 31 - 1], len(free)))
    else:
        free, nb = free[:0], 0
    note(f"tables {what}")
    got = run_tables(torch, held, new, table, free, 16, nb, T)
    for name, a, b in zip(("table", "slots", "cu", "after", "used"), got, ref.block_tables(held, new, table, free, 16, nb, T)):
        assert np.array_equal(a, b), name


def test_tables_without_requests():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    slots, cu, after, used = gdn.block_tables(none, none, none.view(0, 0), none, 16, 0, 5)
    assert slots.tolist() == [-1] * 5 and cu.tolist() == [0] and after.numel() == 0 and used.tolist() == [0, 0]


# ------------------------------------------------------------------- append
def make_cache(torch, rng, nb, H, bt, D, kind):
    """Random codes (tensor on the GPU, values in float64) and scales."""
    if kind == "int8":
        c = torch.from_numpy(rng.integers(-127, 128, (nb, H, bt, D)).astype(np.int8))
    else:
        c = torch.from_numpy(np.clip(rng.standard_normal((nb, H, bt, D)) * 120, -448, 448).astype(np.float32)).to(torch.float8_e4m3fn)
    scale = torch.from_numpy((0.002 + 0.03 * rng.random((nb, H))).astype(np.float32))
    return c, scale


def values(c):
    return c.cpu().float().numpy().astype(np.float64)


def run_append(torch, k, v, slots, kc, vc, ks, vs):
    import linear_attention_sequence_gated_amd as gdn
    dev = [x.cuda() for x in (kc, vc, ks, vs)]
    gdn.cache_append(k, v, ints(torch, slots), *dev)
    torch.cuda.synchronize()
    return dev


def check_append(torch, rng, x, slots, nb, H, bt, D, kind, caches=None):
    kc, ks = make_cache(torch, rng, nb, H, bt, D, kind)
    vc, vs = make_cache(torch, rng, nb, H, bt, D, kind)
    kv = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()  # [T, 2H, D], a fused projection's parts
    got = run_append(torch, kv[:, :H], kv[:, H:], slots, kc, vc, ks, vs)
    xs = kv.float().cpu().numpy()
    for name, new, c, s, gc, gs in (("k", xs[:, :H], kc, ks, got[0], got[2]), ("v", xs[:, H:], vc, vs, got[1], got[3])):
        want, scale = ref.cache_append(new, slots, values(c), s.numpy(), kind)
        assert np.array_equal(gs.cpu().numpy(), scale), name
        assert np.array_equal(values(gc), want), name


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("bt,D", [(16, 64), (16, 128), (32, 64), (32, 128), (64, 64), (64, 128), (128, 64), (128, 128)])
def test_append_prompts_and_single_tokens(bt, D, kind):
    """A step of prompts and single tokens together, through the tables: ragged lengths, blocks with older rows."""
    torch = torch_dev()
    rng = np.random.default_rng(bt + D)
    held, new = make_requests(rng, 37, bt, 3 * bt + 5, 9)
    table, free, nb = make_table(rng, held, new, bt)
    T = int(new.sum()) + 7
    _, slots, *_ = ref.block_tables(held, new, table, free, bt, nb, T)
    note(f"append bt{bt} D{D} {kind} T{T}")
    x = rng.standard_normal((T, 6, D)) * rng.choice([0.05, 1.0, 30.0], (T, 6, 1))
    check_append(torch, rng, x, slots, nb, 3, bt, D, kind)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_append_many_tokens(kind):
    """More tokens than are looked at one by one: runs that begin anywhere in a window and end in a later one."""
    torch = torch_dev()
    rng = np.random.default_rng(11)
    new = np.array([0, 1, 700, 31, 33, 1500, 64, 2, 15, 16, 17, 300] + [1] * 100)
    held = np.concatenate([np.zeros(12, np.int64), rng.integers(0, 200, 100)])
    table, free, nb = make_table(rng, held, new, 64)
    T = int(new.sum()) + 40
    _, slots, *_ = ref.block_tables(held, new, table, free, 64, nb, T)
    note(f"append many {kind} T{T}")
    check_append(torch, rng, rng.standard_normal((T, 2, 64)), slots, nb, 1, 64, 64, kind)


@pytest.mark.parametrize("T,H", [(5000, 1), (6000, 3), (9000, 8)])
def test_append_runs_of_whole_blocks(T, H):
    """Blocks of 128 tokens whose rows begin anywhere among the slots that a workgroup looks at."""
    torch = torch_dev()
    rng = np.random.default_rng(T)
    new, held = [], []
    while sum(new) < T:
        new.append(int(rng.choice([1, 2, 5, 127, 128, 129, 256, 300])))
        held.append(int(rng.choice([0, 0, 1, 63, 64, 127])))
    new, held = np.array(new), np.array(held)
    table, free, nb = make_table(rng, held, new, 128)
    _, slots, *_ = ref.block_tables(held, new, table, free, 128, nb, int(new.sum()))
    note(f"append whole blocks T{T} H{H}")
    check_append(torch, rng, rng.standard_normal((int(new.sum()), 2 * H, 64)), slots, nb, H, 128, 64, "int8")


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_append_edges(kind):
    """Zeros, the smallest and largest numbers, infinities and NaN; slots outside the cache; a full block; ties."""
    torch = torch_dev()
    rng = np.random.default_rng(5)
    T, H, D, bt, nb = 48, 1, 64, 16, 8
    x = rng.standard_normal((T, 2 * H, D))
    x[0:16] = 0
    x[16:20] = 1e-39
    x[20, 0, 3], x[21, 1, 4], x[22, 0, 0] = np.inf, -np.inf, np.nan
    x[32] = np.linspace(-127, 127, D)
    x[33, :, :] = 0.5 * np.arange(D)
    slots = np.concatenate([np.arange(16), 64 + np.arange(16), [96, 97, 98, -1, -5, nb * bt, 2 ** 31 - 1, -2 ** 31], 40 + np.arange(8)])
    note(f"append edges {kind}")
    check_append(torch, rng, x, slots, nb, H, bt, D, kind)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_append_token_by_token(kind):
    """A block filled one token at a time with growing values: the scale grows, and the older codes move each time."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    rng = np.random.default_rng(9)
    kc, ks = make_cache(torch, rng, 2, 2, 16, 64, kind)
    vc, vs = make_cache(torch, rng, 2, 2, 16, 64, kind)
    dev = [c.cuda() for c in (kc, vc, ks, vs)]
    want = [(values(kc), ks.numpy()), (values(vc), vs.numpy())]
    for t in range(16):
        x = rng.standard_normal((1, 4, 64)) * (1.3 ** t)
        kv = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
        gdn.cache_append(kv[:, :2], kv[:, 2:], ints(torch, [16 + t]), *dev)
        xs = kv.float().cpu().numpy()
        want = [ref.cache_append(xs[:, 2 * i:2 * i + 2], [16 + t], *want[i], kind) for i in range(2)]
    for i in range(2):
        assert np.array_equal(values(dev[i]), want[i][0]) and np.array_equal(dev[2 + i].cpu().numpy(), want[i][1])
