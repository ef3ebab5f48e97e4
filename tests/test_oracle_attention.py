"""The attention oracle against facts that do not depend on it: gradients against differences, one key's value returned,
uniform weights, the cache's codes against torch's own 8-bit floats, tables of a step by hand."""
import numpy as np
import pytest

from oracle import attention as ref


def test_gradients_against_differences():
    rng = np.random.default_rng(0)
    q, k, v, do = (rng.standard_normal(s) for s in ((9, 4, 5), (9, 2, 5), (9, 2, 5), (9, 4, 5)))
    cu, scale = [1, 4, 4, 8], 0.7
    grads = ref.prompt(q, k, v, cu, scale, do)[2:]
    for i in range(3):
        for _ in range(20):
            at = tuple(rng.integers(0, n) for n in grads[i].shape)
            f = []
            for eps in (1e-6, -1e-6):
                x = [q.copy(), k.copy(), v.copy()]
                x[i][at] += eps
                f.append((ref.prompt(*x, cu, scale)[0] * do).sum())
            assert abs((f[0] - f[1]) / 2e-6 - grads[i][at]) < 1e-7


def test_first_row_and_uniform_weights():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal((6, 2, 4)) for _ in range(3))
    out, lse = ref.prompt(q, k, v, [0, 6], 0.0)
    assert np.allclose(out, np.cumsum(v, 0) / np.arange(1, 7)[:, None, None]) and np.allclose(lse, np.log(np.arange(1, 7)))
    out, lse = ref.prompt(q, k, v, [0, 6], 0.5)
    assert np.allclose(out[0], v[0]) and np.allclose(lse[:, 0], 0.5 * (q[0] * k[0]).sum(1))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_codes(kind):
    torch = pytest.importorskip("torch")
    y = np.concatenate([np.linspace(-460, 460, 4001), np.geomspace(1e-5, 1, 500)]).astype(np.float32)
    y = np.concatenate([y, np.arange(-130, 130, 0.5, dtype=np.float32)])
    t = torch.from_numpy(y)
    want = t.clamp(-127, 127).round() if kind == "int8" else t.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    assert np.array_equal(ref.to_code(y, kind), want.double().numpy())


def test_decode_is_the_last_row_of_a_prompt():
    rng = np.random.default_rng(2)
    kc, vc = rng.integers(-127, 128, (4, 2, 16, 8)), rng.integers(-127, 128, (4, 2, 16, 8))
    ks, vs = rng.random((4, 2)).astype(np.float32) * 0.02, rng.random((4, 2)).astype(np.float32) * 0.02
    table, n = np.array([[2, 0, 3]]), 37
    q = rng.standard_normal((1, 4, 8))
    k = np.concatenate([kc[b].transpose(1, 0, 2) * ks[b][None, :, None] for b in table[0]])[:n]
    v = np.concatenate([vc[b].transpose(1, 0, 2) * vs[b][None, :, None] for b in table[0]])[:n]
    out, lse = ref.decode(q, kc, vc, ks, vs, table, [n], 0.3)
    po, pl = ref.prompt(np.repeat(q, n, 0), k, v, [0, n], 0.3)
    assert np.allclose(out[0], po[-1]) and np.allclose(lse[0], pl[:, -1])


def test_tables_by_hand():
    # 17 tokens held (2 blocks of 16) and 16 more: one block; an empty request with 3 new tokens: one block
    table, slots, cu, after, used = ref.block_tables([17, 0], [16, 3], [[5, 6, -1], [-1, -1, -1]], [9, 4, 2], 16, 10, 21)
    assert table.tolist() == [[5, 6, 9], [4, -1, -1]]
    assert slots.tolist() == [6 * 16 + i for i in range(1, 16)] + [9 * 16] + [64, 65, 66, -1, -1]
    assert cu.tolist() == [0, 16, 19] and after.tolist() == [33, 3] and used.tolist() == [2, 0]


def test_append_by_hand():
    cache, scale = np.zeros((1, 1, 16, 2)), np.array([[9.0]], np.float32)
    cache, scale = ref.cache_append(np.array([[[1.27, -0.635]]]), [0], cache, scale, "int8")
    assert cache[0, 0, 0].tolist() == [127, -64] and abs(scale[0, 0] - 0.01) < 1e-9  # a first row: the old scale does not count
    cache, scale = ref.cache_append(np.array([[[2.54, 0.0]]]), [1], cache, scale, "int8")
    assert cache[0, 0, :2].tolist() == [[64, -32], [127, 0]] and abs(scale[0, 0] - 0.02) < 1e-9
