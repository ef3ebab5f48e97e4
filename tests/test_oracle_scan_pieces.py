"""The scan's recurrence against its form by pieces of rows, and its gradients against theirs, as csrc/ssm_scan.hip and
csrc/ssm_scan_bwd.hip write them down, in 64 bits."""
import numpy as np
import pytest

from oracle import block as ref


def by_pieces(x, dt, a, B, C, D, bias, cu, Q, S0, g, gl):
    """(out, S_final, gradients in the order of ref.ssm_scan_bwd): one head after the other, pieces of up to Q rows."""
    T, H, P = x.shape
    G, N, R = B.shape[1], B.shape[2], len(cu) - 1
    out, last = np.zeros((T, H, P)), np.zeros((R, H, N, P))
    z = dt + bias
    d, sig = ref.softplus(z), 1 / (1 + np.exp(-z))
    gx, gz, gB, gC, gS0 = np.zeros_like(x), np.zeros_like(dt), np.zeros_like(B), np.zeros_like(C), np.zeros((R, H, N, P))
    ga, gD, gbias = np.zeros(H), np.zeros(H), np.zeros(H)
    for h in range(H):
        k = h // (H // G)
        for r in range(R):
            pieces = [(i, min(i + Q, cu[r + 1])) for i in range(cu[r], cu[r + 1], Q)]
            states = [S0[r, h]]
            for lo, hi in pieces:
                S, X, Bp, Cp, dp = states[-1], x[lo:hi, h], B[lo:hi, k], C[lo:hi, k], d[lo:hi, h]
                Gs = np.cumsum(a[h] * dp)
                L = np.tril(np.exp(Gs[:, None] - Gs[None])) * dp
                out[lo:hi, h] = ((Cp @ Bp.T) * L) @ X + np.exp(Gs)[:, None] * (Cp @ S) + D[h] * X
                states.append(np.exp(Gs[-1]) * S + (Bp * (np.exp(Gs[-1] - Gs) * dp)[:, None]).T @ X)
            last[r, h] = states[-1]
            Z = gl[r, h]
            for (lo, hi), S in zip(reversed(pieces), reversed(states[:-1])):
                X, Bp, Cp, dp, hp = x[lo:hi, h], B[lo:hi, k], C[lo:hi, k], d[lo:hi, h], g[lo:hi, h]
                Gs = np.cumsum(a[h] * dp)
                L, w, n = np.tril(np.exp(Gs[:, None] - Gs[None])) * dp, np.exp(Gs[-1] - Gs) * dp, hi - lo
                M, W = (Cp @ Bp.T) * L, (hp @ X.T) * L
                E = (hp @ X.T) * M
                gx[lo:hi, h] = M.T @ hp + w[:, None] * (Bp @ Z) + D[h] * hp
                up, behind = np.exp(Gs)[:, None] * (hp @ S.T), w[:, None] * (X @ Z.T)
                gC[lo:hi, k] += W @ Bp + up
                gB[lo:hi, k] += W.T @ Cp + behind
                Rr, Qq = (Cp * up).sum(1), (Bp * behind).sum(1)
                gg = np.array([E[t:, :t].sum() + Rr[t:].sum() + Qq[:t].sum() for t in range(n)]) + np.exp(Gs[-1]) * (Z * S).sum()
                gz[lo:hi, h] = (a[h] * gg + (E.sum(0) + Qq) / dp) * sig[lo:hi, h]
                ga[h] += (gg * dp).sum()
                gD[h] += (hp * X).sum()
                Z = np.exp(Gs[-1]) * Z + (Cp * np.exp(Gs)[:, None]).T @ hp
            gS0[r, h] = Z
    gbias = gz.sum(0)
    return out, last, [gx, gz, ga, gB, gC, gD, gbias, gS0]


@pytest.mark.parametrize("Q", [1, 4, 64])
@pytest.mark.parametrize("h,g", [(2, 1), (4, 2)])
def test_pieces_are_the_recurrence(Q, h, g):
    rng = np.random.default_rng([Q, h])
    t, p, n, cu = 30, 5, 6, [0, 9, 9, 30]
    x, B, C, go = (rng.standard_normal(s) for s in ((t, h, p), (t, g, n), (t, g, n), (t, h, p)))
    dt, a, D, bias = rng.standard_normal((t, h)), -rng.uniform(0.1, 3, h), rng.standard_normal(h), rng.standard_normal(h)
    S0, gl = rng.standard_normal((3, h, n, p)), rng.standard_normal((3, h, n, p))
    out, last, grads = by_pieces(x, dt, a, B, C, D, bias, cu, Q, S0, go, gl)
    want, want_last = ref.ssm_scan(x, dt, a, B, C, D, bias, cu, S0)
    assert np.allclose(out, want, rtol=1e-10, atol=1e-12) and np.allclose(last, want_last, rtol=1e-10, atol=1e-12)
    for u, v in zip(grads, ref.ssm_scan_bwd(x, dt, a, B, C, D, bias, cu, go, S0, gl)):
        assert np.allclose(u, v, rtol=1e-9, atol=1e-11)
