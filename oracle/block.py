"""fp64 references of what stands around a recurrent layer's state update, from the definitions in include/gdn.h: the
root-mean-square norm with the residual's addition and an 8-bit output, the short causal convolution over packed
sequences, and the selective state space scan.  numpy only; everything is computed in float64 from the stored inputs."""
from __future__ import annotations

import numpy as np

from .attention import MOST

SMALLEST_SCALE = 2.0 ** -100


def rms_norm(s, weight, eps):
    """s [T, C] (the sum, already rounded): (out, rstd [T, 1])."""
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    return s * rstd * weight, rstd


def rms_norm_bwd(s, weight, eps, g, h=None):
    """(grad_x, grad_weight, sum over rows of the absolute terms of grad_weight)."""
    _, rstd = rms_norm(s, weight, eps)
    n = s * rstd
    wg = g * weight
    gs = (wg - n * (wg * n).mean(1, keepdims=True)) * rstd
    return gs if h is None else gs + h, (g * n).sum(0), np.abs(g * n).sum(0)


def quantise(y, block, fmt):
    """Scales [T, C / block or 1] and the values y / scale that codes are rounded from, of magnitude MOST[fmt] at most."""
    t, c = y.shape
    parts = y.reshape(t, -1, block or c)
    scale = np.maximum(np.abs(parts).max(2) / MOST[fmt], SMALLEST_SCALE)
    return scale, np.clip((parts / scale[..., None]).reshape(t, c), -MOST[fmt], MOST[fmt])


def _sequences(cu, T):
    """(sequence, first row, row behind the last) as the entry points clamp them."""
    for r in range(len(cu) - 1):
        b = min(max(int(cu[r]), 0), T)
        yield r, b, min(max(int(cu[r + 1]), b), T)


def silu(p):
    return p / (1.0 + np.exp(-p))


def silu_slope(p):
    s = 1.0 / (1.0 + np.exp(-p))
    return s * (1.0 + p * (1.0 - s))


def short_conv(x, weight, bias, cu, state=None, act=True):
    """(out [T, C] with zeros in rows of no sequence, state_final, size: sums of the absolute terms of p)."""
    T, C = x.shape
    W, R = weight.shape[1], len(cu) - 1
    out, size = np.zeros((T, C)), np.zeros((T, C))
    last = np.zeros((R, W - 1, C))
    for r, b, e in _sequences(cu, T):
        z = np.concatenate([np.zeros((W - 1, C)) if state is None else state[r], x[b:e]])
        last[r] = z[e - b:]
        p, a = np.zeros((e - b, C)) + bias, np.zeros((e - b, C)) + np.abs(bias)
        for j in range(W):
            p += weight[:, j] * z[j:j + e - b]
            a += np.abs(weight[:, j] * z[j:j + e - b])
        out[b:e], size[b:e] = silu(p) if act else p, a
    return out, last, size


def short_conv_bwd(x, weight, bias, cu, g, state=None, g_last=None, act=True):
    """(grad_x, grad_weight, grad_bias, grad_state) and, in the same places, the sums of their terms' magnitudes."""
    T, C = x.shape
    W, R = weight.shape[1], len(cu) - 1
    got = [np.zeros((T, C)), np.zeros((C, W)), np.zeros(C), np.zeros((R, W - 1, C))]
    size = [np.zeros_like(v) for v in got]
    for r, b, e in _sequences(cu, T):
        n = e - b
        z = np.concatenate([np.zeros((W - 1, C)) if state is None else state[r], x[b:e]])
        p = bias + sum(weight[:, j] * z[j:j + n] for j in range(W)) if n else np.zeros((0, C))
        q = g[b:e] * silu_slope(p) if act else g[b:e]
        gz, az = np.zeros_like(z), np.zeros_like(z)
        if g_last is not None:
            gz[n:], az[n:] = g_last[r], np.abs(g_last[r])
        for j in range(W):
            gz[j:j + n] += q * weight[:, j]
            az[j:j + n] += np.abs(q * weight[:, j])
            got[1][:, j] += (q * z[j:j + n]).sum(0)
            size[1][:, j] += np.abs(q * z[j:j + n]).sum(0)
        got[2] += q.sum(0)
        size[2] += np.abs(q).sum(0)
        got[0][b:e], got[3][r], size[0][b:e], size[3][r] = gz[W - 1:], gz[:W - 1], az[W - 1:], az[:W - 1]
    return got, size


def softplus(z):
    return np.where(z > 30, z, np.log1p(np.exp(np.minimum(z, 30.0))))


def ssm_scan(x, dt, a, B, C, D, bias, cu, S0=None):
    """Token after token.  x [T, H, P], dt [T, H], B, C [T, G, N]; D, bias [H].  Returns (out, S_final [R, H, N, P])."""
    T, H, P = x.shape
    rep, N, R = H // B.shape[1], B.shape[2], len(cu) - 1
    Bh, Ch = np.repeat(B, rep, 1), np.repeat(C, rep, 1)
    d = softplus(dt + bias)
    keep = np.exp(a * d)
    out, last = np.zeros((T, H, P)), np.zeros((R, H, N, P))
    for r, b, e in _sequences(cu, T):
        S = np.zeros((H, N, P)) if S0 is None else S0[r].copy()
        for t in range(b, e):
            S = keep[t][:, None, None] * S + (d[t][:, None] * Bh[t])[:, :, None] * x[t][:, None]
            out[t] = np.einsum("hn,hnp->hp", Ch[t], S) + D[:, None] * x[t]
        last[r] = S
    return out, last


def ssm_scan_bwd(x, dt, a, B, C, D, bias, cu, g, S0=None, g_last=None):
    """Gradients of sum(out * g) + sum(S_final * g_last), in the order x, dt, a, B, C, D, bias, S0."""
    T, H, P = x.shape
    G, N, R = B.shape[1], B.shape[2], len(cu) - 1
    rep = H // G
    Bh, Ch = np.repeat(B, rep, 1), np.repeat(C, rep, 1)
    z = dt + bias
    d = softplus(z)
    keep = np.exp(a * d)
    gx, gd, ga, gB, gC = np.zeros_like(x), np.zeros_like(dt), np.zeros(H), np.zeros_like(Bh), np.zeros_like(Ch)
    gS0 = np.zeros((R, H, N, P))
    gx += D[:, None] * g
    for r, b, e in _sequences(cu, T):
        S = [np.zeros((H, N, P)) if S0 is None else S0[r]]
        for t in range(b, e):
            S.append(keep[t][:, None, None] * S[-1] + (d[t][:, None] * Bh[t])[:, :, None] * x[t][:, None])
        gS = np.zeros((H, N, P)) if g_last is None else g_last[r].copy()
        for t in range(e - 1, b - 1, -1):
            new, old = S[t - b + 1], S[t - b]
            gC[t] = np.einsum("hnp,hp->hn", new, g[t])
            gS = gS + Ch[t][:, :, None] * g[t][:, None]
            bx = np.einsum("hnp,hp->hn", gS, x[t])
            gB[t] = d[t][:, None] * bx
            gx[t] += d[t][:, None] * np.einsum("hn,hnp->hp", Bh[t], gS)
            gk = (gS * old).sum((1, 2)) * keep[t]
            gd[t] = a * gk + (Bh[t] * bx).sum(1)
            ga += d[t] * gk
            gS = keep[t][:, None, None] * gS
        gS0[r] = gS
    gz = gd / (1.0 + np.exp(-z))
    inside = np.zeros(T, bool)
    for _, b, e in _sequences(cu, T):
        inside[b:e] = True
    gx[~inside] = 0
    g = np.where(inside[:, None, None], g, 0.0)
    return [gx, gz, ga, gB.reshape(T, G, rep, N).sum(2), gC.reshape(T, G, rep, N).sum(2), (g * x).sum((0, 2)), gz.sum(0), gS0]
