"""Oracle of the attention layer, in 64 bits on the CPU: request by request and token by token where that is readable,
sharing no code with the GPU path.  Codes and scales of the cache follow their definition in include/gdn.h: scales,
reciprocals and ratios are float32, and what is rounded to a code is a float32 product.
"""
from __future__ import annotations

import numpy as np

MOST = {"int8": 127.0, "e4m3": 448.0}
F = np.float32


def block_tables(seq_lens, new_lens, table, free, bt, num_blocks, T):
    """(table, slot_map, cu, after, used) for int arrays; the inputs are not changed."""
    table, slots = np.array(table, np.int64), np.full(T, -1, np.int64)
    R, width = table.shape
    cu, after, off, used, refused, at = [0], [], 0, 0, 0, 0
    for r in range(R):
        n, m = int(seq_lens[r]), int(new_lens[r])
        have, need = -(-n // bt), -(-(n + m) // bt)
        valid = n >= 0 and m >= 0 and need <= width and n + m < 2 ** 31
        want = need - have if valid else 0
        m = max(m, 0)
        if valid and at + m <= T and (want == 0 or off + want <= len(free)):
            for i in range(want):
                table[r, have + i] = free[off + i]
            for i in range(m):
                b = table[r, (n + i) // bt]
                slots[at + i] = b * bt + (n + i) % bt if 0 <= b < num_blocks else -1
            after.append(n + m)
            used = max(used, off + want) if want else used
        else:
            refused += 1
            after.append(n)
        off += want
        at += m
        cu.append(min(at, T))
    return table, slots, np.array(cu), np.array(after, np.int64), np.array([used, refused])


def to_code(y, kind):
    """Round-to-nearest-even codes, as the values they are, of float32 numbers y; NaN becomes 0."""
    y = np.where(np.isnan(y), F(0), y.astype(F)).astype(np.float64)
    y = np.clip(y, -MOST[kind], MOST[kind])
    if kind == "int8":
        return np.rint(y)
    e = np.frexp(np.abs(y))[1] - 1  # |y| in [2^e, 2^(e+1)); below 2^-6 the step stays 2^-9
    step = np.ldexp(1.0, np.maximum(e, -6) - 3)
    return np.rint(y / step) * step


def cache_append(x, slots, cache, scale, kind):
    """x [T, H, D] float, cache [NB, H, bt, D] code values, scale [NB, H] float32: the new (cache, scale)."""
    cache, scale = np.array(cache, np.float64), np.array(scale, F)
    nb, _, bt, _ = cache.shape
    runs = {}
    for t, s in enumerate(slots):
        if 0 <= s < nb * bt:
            runs.setdefault(int(s) // bt, []).append((int(s) % bt, t))
    for b, toks in runs.items():
        first, ts = toks[0][0], [t for _, t in toks]
        rows = x[ts].astype(np.float64)  # [n, H, D]
        a = np.where(np.isnan(rows), 0.0, np.abs(rows)).max((0, 2))
        a = np.minimum(a, float(F(3.38953139e38))).astype(F)
        old = scale[b] if first else np.zeros_like(scale[b])
        s = np.maximum(np.maximum(a * F(1.0 / MOST[kind]), old), F(2.0 ** -100)).astype(F)
        if first:
            cache[b, :, :first] = to_code(cache[b, :, :first].astype(F) * (old / s)[:, None, None], kind)
        with np.errstate(invalid="ignore", over="ignore"):
            y = rows.astype(F) * (F(1) / s)[None, :, None]
        cache[b, :, first:first + len(ts)] = to_code(y, kind).transpose(1, 0, 2)
        scale[b] = s
    return cache, scale


def decode(q, k_cache, v_cache, k_scale, v_scale, table, lens, scale):
    """q [R, Hq, D]; caches as code values.  (out [R, Hq, D], lse [R, Hq])."""
    R, Hq, D = q.shape
    nb, H, bt, _ = k_cache.shape
    out, lse = np.zeros((R, Hq, D)), np.full((R, Hq), -np.inf)
    for r in range(R):
        n = max(0, min(int(lens[r]), table.shape[1] * bt))
        cols = [(int(table[r, p // bt]), p % bt) for p in range(n)]
        cols = [(b, o) for b, o in cols if 0 <= b < nb]
        if not cols:
            continue
        b, o = np.array(cols).T
        for h in range(Hq):
            g = h * H // Hq
            k = k_cache[b, g, o].astype(np.float64) * k_scale[b, g].astype(np.float64)[:, None]
            v = v_cache[b, g, o].astype(np.float64) * v_scale[b, g].astype(np.float64)[:, None]
            s = (k @ q[r, h].astype(np.float64)) * scale
            m = s.max()
            p = np.exp(s - m)
            out[r, h], lse[r, h] = p @ v / p.sum(), m + np.log(p.sum())
    return out, lse


def prompt(q, k, v, cu, scale, grad_out=None):
    """q [T, Hq, D], k, v [T, H, D]: (out, lse [Hq, T]) and, with grad_out, (dq, dk, dv) too.  Rows of no sequence stay 0."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = np.zeros_like(q), np.zeros((Hq, T))
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for a, b in zip(cu[:-1], cu[1:]):
        for h in range(Hq if b > a else 0):
            s = q[a:b, h] @ k[a:b, h // G].T * scale
            s = np.where(np.tril(np.ones_like(s, dtype=bool)), s, -np.inf)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            z = p.sum(1, keepdims=True)
            p, lse[h, a:b] = p / z, (m + np.log(z))[:, 0]
            out[a:b, h] = p @ v[a:b, h // G]
            if grad_out is not None:
                do = np.asarray(grad_out[a:b, h], np.float64)
                dp = do @ v[a:b, h // G].T
                ds = p * (dp - (do * out[a:b, h]).sum(1, keepdims=True)) * scale
                dq[a:b, h] = ds @ k[a:b, h // G]
                dk[a:b, h // G] += ds.T @ q[a:b, h]
                dv[a:b, h // G] += p.T @ do
    return (out, lse) if grad_out is None else (out, lse, dq, dk, dv)
