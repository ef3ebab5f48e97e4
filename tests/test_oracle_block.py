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
