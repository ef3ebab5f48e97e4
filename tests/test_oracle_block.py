"""The references of the norm and the short convolution against differences and against a hand-worked case."""
import numpy as np
import pytest

from oracle import block as ref


def numeric(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + step
        up = f()
        x[i] = old - step
        g[i] = (up - f()) / (2 * step)
        x[i] = old
    return g


def test_norm_of_a_hand_worked_row():
    y, rstd = ref.rms_norm(np.array([[3.0, 4.0, 0.0, 0.0]]), np.array([1.0, 2.0, 1.0, 1.0]), 0.0)
    assert np.allclose(y, [[1.2, 3.2, 0, 0]]) and np.isclose(rstd, 0.4)


def test_conv_of_a_hand_worked_column():
    x = np.array([[1.0], [2.0], [3.0], [5.0]])
    out, last, _ = ref.short_conv(x, np.array([[10.0, 1.0]]), np.array([0.5]), [0, 3, 3, 4], np.array([[[7.0]], [[8.0]], [[9.0]]]), act=False)
    assert out[:, 0].tolist() == [71.5, 12.5, 23.5, 95.5] and last[:, 0, 0].tolist() == [3.0, 8.0, 5.0]


def test_norm_gradients_are_differences():
    rng = np.random.default_rng(0)
    s, w, g, h = (rng.standard_normal(n) for n in ((3, 8), 8, (3, 8), (3, 8)))

    def loss():
        return (ref.rms_norm(s, w, 1e-3)[0] * g + s * h).sum()

    gs, gw, _ = ref.rms_norm_bwd(s, w, 1e-3, g, h)
    assert np.allclose(gs, numeric(loss, s), atol=1e-7) and np.allclose(gw, numeric(loss, w), atol=1e-7)


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_gradients_are_differences(W, act):
    rng = np.random.default_rng(W)
    cu, C = [0, 5, 5, 6, 8], 3  # lengths from none to longer than the taps
    x, w, b, g = (rng.standard_normal(n) for n in ((9, C), (C, W), C, (9, C)))
    st, gl = rng.standard_normal((4, W - 1, C)), rng.standard_normal((4, W - 1, C))

    def loss():
        out, last, _ = ref.short_conv(x, w, b, cu, st, act)
        return (out * g).sum() + (last * gl).sum()

    got, _ = ref.short_conv_bwd(x, w, b, cu, g, st, gl, act)
    for a, v in zip(got, (x, w, b, st)):
        assert np.allclose(a, numeric(loss, v), atol=1e-7)


def test_scan_of_a_hand_worked_column():
    """One head, one state, one channel; softplus(0) = ln 2, so that a = -1 halves the state."""
    one = np.ones((3, 1, 1))
    x, dt = np.array([1.0, 2.0, 4.0]).reshape(3, 1, 1), np.zeros((3, 1))
    out, last = ref.ssm_scan(x, dt, np.array([-1.0]), one, 2 * one, np.array([10.0]), np.zeros(1), [0, 0, 2, 3], np.full((3, 1, 1, 1), 8.0))
    d = np.log(2.0)
    S = [4 + d, (4 + d) / 2 + 2 * d, 4 + 4 * d]
    assert np.allclose(out[:, 0, 0], [2 * S[0] + 10, 2 * S[1] + 20, 2 * S[2] + 40])
    assert np.allclose(last.reshape(-1), [8, S[1], S[2]])


def test_scan_gradients_are_differences():
    rng = np.random.default_rng(5)
    H, P, G, N, T, cu = 4, 2, 2, 3, 9, [1, 5, 5, 6, 8]
    x, dt, B, C, g = (rng.standard_normal(s) for s in ((T, H, P), (T, H), (T, G, N), (T, G, N), (T, H, P)))
    a, D, bias = -np.exp(rng.standard_normal(H)), rng.standard_normal(H), rng.standard_normal(H)
    S0, gl = rng.standard_normal((4, H, N, P)), rng.standard_normal((4, H, N, P))

    def loss():
        out, last = ref.ssm_scan(x, dt, a, B, C, D, bias, cu, S0)
        return (out * g).sum() + (last * gl).sum()

    got = ref.ssm_scan_bwd(x, dt, a, B, C, D, bias, cu, g, S0, gl)
    for v, w in zip(got, (x, dt, a, B, C, D, bias, S0)):
        assert np.allclose(v, numeric(loss, w), atol=2e-7)
