"""Cases for the attention layers that stand between gated delta-rule layers in a hybrid model: causal attention over
packed prompts and its gradients, the 8-bit paged cache (write and single-token read), and the block tables that both
are addressed by.  `run` computes them in plain torch operations, or, where `own` is set, with the package's kernels.

Lengths of a ragged batch are a function of the case alone; every value comes from the seed."""
import math

import numpy as np
import torch

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")

own = False

SMALLEST_SCALE = 2.0 ** -100  # a block of zeros keeps a finite reciprocal


def listed():
    return [
        # one short prompt of the 12-head d = 64 layer, grouped heads: the time to the first token of a short request
        dict(name="prompt_short", op="prompt", n=1, longest=131, ragged=False, hq=12, hkv=4, d=64, fused=True),
        # the attention layer beside the 8 x 2048 x 12 x 64 delta layer, grouped heads, from a fused projection
        dict(name="prompt_layer", op="prompt", n=8, longest=2048, ragged=False, hq=12, hkv=4, d=64, fused=True),
        # 16k context at 16 heads of 128
        dict(name="prompt_long", op="prompt", n=1, longest=16384, ragged=False, hq=16, hkv=4, d=128, fused=False),
        # a training step of the 8 x 2048 layer: forward and gradients, one key head per query head
        dict(name="train_layer", op="train", n=8, longest=2048, ragged=False, hq=12, hkv=12, d=64, fused=True),
        # documents of many lengths packed into one training row, grouped heads
        dict(name="train_ragged", op="train", n=13, longest=1201, ragged=True, hq=16, hkv=4, d=128, fused=False),
        # one request's next token
        dict(name="decode_one", op="decode", n=1, longest=777, ragged=False, hq=12, hkv=4, d=64, bt=16, kind="int8"),
        # a serving batch of many lengths
        dict(name="decode_batch", op="decode", n=64, longest=4099, ragged=True, hq=16, hkv=4, d=128, bt=64, kind="e4m3"),
        # few requests with a long context
        dict(name="decode_long", op="decode", n=4, longest=65521, ragged=False, hq=16, hkv=4, d=128, bt=64, kind="int8"),
        # packed prompts' keys and values into the cache, a key head per query head
        dict(name="append_prompt", op="append", n=9, longest=2500, ragged=True, decode=False, hkv=16, d=128, bt=64, kind="int8"),
        # one new token for each request of a decoding batch, most of them into blocks that hold older tokens
        dict(name="append_decode", op="append", n=256, longest=1, ragged=False, decode=True, hkv=4, d=64, bt=32, kind="e4m3"),
        # a step's tables: decoding requests and a few prompts together
        dict(name="tables_mixed", op="tables", n=700, longest=9000, ragged=True, bt=64, prompts=5),
        # a large batch's tables
        dict(name="tables_large", op="tables", n=4096, longest=5000, ragged=True, bt=16, prompts=40),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "train", "decode", "decode", "append", "tables"])
    hq, hkv, d = rng.choice([(12, 12, 64), (12, 4, 64), (16, 4, 64), (8, 1, 64), (16, 4, 128), (16, 16, 128), (16, 2, 128), (6, 3, 128)])
    ragged, fused = rng.random() < 0.6, rng.random() < 0.5
    kind = rng.choice(["int8", "e4m3"])
    if op in ("prompt", "train"):
        total = _log(rng, 64, 8000 if op == "train" else 14000)
        n = _log(rng, 1, max(1, total // 16))
        return dict(op=op, n=n, longest=max(1, total // n), ragged=ragged, hq=hq, hkv=hkv, d=d, fused=fused)
    if op == "decode":
        total = _log(rng, 128, 250000 if hkv <= 4 else 60000)
        n = _log(rng, 1, max(1, min(512, total // 32)))
        return dict(op=op, n=n, longest=max(1, total // n), ragged=ragged, hq=hq, hkv=hkv, d=d, bt=rng.choice([16, 32, 64, 128]), kind=kind)
    if op == "append":
        bt = rng.choice([16, 32, 64, 128])
        if rng.random() < 0.5:
            return dict(op=op, n=_log(rng, 1, 700), longest=1, ragged=False, decode=True, hkv=hkv, d=d, bt=bt, kind=kind)
        total = _log(rng, 64, 11000)
        n = _log(rng, 1, max(1, total // 16))
        return dict(op=op, n=n, longest=max(1, total // n), ragged=ragged, decode=False, hkv=hkv, d=d, bt=bt, kind=kind)
    n = _log(rng, 1, 4000)
    return dict(op=op, n=n, longest=_log(rng, 8, 5000), ragged=True, bt=rng.choice([16, 32, 64, 128]), prompts=rng.randrange(0, min(n, 40) + 1))


def lengths(case):
    """Tokens of each sequence: a function of the case, so that work() knows them."""
    n, longest = case["n"], case["longest"]
    if not case["ragged"]:
        return np.full(n, longest, dtype=np.int64)
    got = np.random.default_rng([n, longest]).integers(0, longest + 1, n)
    got[n // 2] = 0
    got[0] = longest
    return got


def _step(case):
    """tables: tokens held and new of each request."""
    held = lengths(case)
    new = np.ones(case["n"], dtype=np.int64)
    at = np.random.default_rng([case["n"], 7]).permutation(case["n"])[: case["prompts"]]
    new[at], held[at] = held[at] // 2 + 1, 0
    return held, new


def _blocks(tokens, bt):
    return (tokens + bt - 1) // bt


def work(case):
    op = case["op"]
    if op in ("prompt", "train"):
        n = lengths(case).astype(float)
        t, pairs = n.sum(), (n * (n + 1) / 2).sum()
        rows = t * case["d"] * (case["hq"] + case["hkv"])  # q and out or k and v, in elements of two tensors
        if op == "prompt":
            return {"bytes": 4 * rows + 4 * t * case["hq"], "flops": 4 * case["d"] * case["hq"] * pairs}
        return {"bytes": 4 * rows + 2 * t * case["d"] * case["hq"] + 4 * rows, "flops": 14 * case["d"] * case["hq"] * pairs}
    if op == "decode":
        n = lengths(case).astype(float)
        b = 2 * n.sum() * case["hkv"] * case["d"] + 8 * _blocks(n, case["bt"]).sum() * case["hkv"]
        return {"bytes": b + case["n"] * case["hq"] * (4 * case["d"] + 4), "flops": 4 * n.sum() * case["hq"] * case["d"]}
    if op == "append":
        t = float(lengths(case).sum())
        return {"bytes": 6 * t * case["hkv"] * case["d"] + 4 * t, "flops": 6 * t * case["hkv"] * case["d"]}
    held, new = _step(case)
    taken = float((_blocks(held + new, case["bt"]) - _blocks(held, case["bt"])).sum())
    return {"bytes": 8 * taken + 4.0 * new.sum() + 16 * case["n"], "flops": 0}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]
    st = {"case": case}

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(torch.bfloat16)

    def ints(x):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)

    if op in ("prompt", "train"):
        n, hq, hkv, d = lengths(case), case["hq"], case["hkv"], case["d"]
        t = int(n.sum())
        qkv = normal(t, hq + 2 * hkv, d)
        st["q"], st["k"], st["v"] = (x if case["fused"] else x.contiguous() for x in qkv.split([hq, hkv, hkv], dim=1))
        st["cu"] = ints(np.concatenate([[0], np.cumsum(n)]))
        st["scale"] = 1.0 / math.sqrt(d)
        if op == "train":
            st["grad_out"] = normal(t, hq, d)
        return st
    bt = case["bt"]
    if op == "tables":
        held, new = _step(case)
        own_blocks = _blocks(held, bt)
        width = int(_blocks(held + new, bt).max())
        total = int(_blocks(held + new, bt).sum()) + 17
        ids = rng.permutation(total)
        table = np.full((case["n"], width), -1)
        at = np.arange(width)[None] < own_blocks[:, None]
        table[at] = ids[: int(own_blocks.sum())]
        st["held"], st["new"], st["table"], st["free"] = ints(held), ints(new), ints(table), ints(ids[int(own_blocks.sum()):])
        st["tokens"], st["blocks"] = int(new.sum()), total
        return st
    hkv, d = case["hkv"], case["d"]
    if op == "decode":
        n = lengths(case)
        nb = _blocks(n, bt)
        total, width = int(nb.sum()) + 3, max(1, int(nb.max()))
        table = np.full((case["n"], width), -1)
        table[np.arange(width)[None] < nb[:, None]] = rng.permutation(total)[: int(nb.sum())]
        st["table"], st["lens"] = ints(table), ints(n)
        st["q"] = normal(case["n"], case["hq"], d)
        st["scale"] = 1.0 / math.sqrt(d)
    else:
        n = lengths(case)
        held = np.random.default_rng([case["n"], bt]).integers(0, 4 * bt, case["n"]) if case["decode"] else np.zeros(case["n"], dtype=np.int64)
        nb = _blocks(held + n, bt)
        total = int(nb.sum()) + 3
        ids, base = rng.permutation(total), np.concatenate([[0], np.cumsum(nb)])
        row = np.repeat(np.arange(case["n"]), n)
        pos = np.arange(int(n.sum())) - np.repeat(np.cumsum(n) - n, n) + held[row]
        st["slots"] = ints(ids[base[row] + pos // bt] * bt + pos % bt)
        kv = normal(int(n.sum()), 2 * hkv, d)
        st["k"], st["v"] = kv.split([hkv, hkv], dim=1)
    for x in ("k", "v"):
        codes = torch.randn(total, hkv, bt, d, generator=g, device=DEV)
        if case["kind"] == "int8":
            st[x + "_cache"] = (codes * 32).round_().clamp_(-127, 127).to(torch.int8)
        else:
            st[x + "_cache"] = (codes * 110).clamp_(-448, 448).to(torch.float8_e4m3fn)
        unit = 1 / 32 if case["kind"] == "int8" else 1 / 110
        st[x + "_scale"] = unit * (0.6 + 0.6 * torch.rand(total, hkv, generator=g, device=DEV))
    return st


# ---------------------------------------------------------------- plain forms
def _scores(q, k, cu, scale):
    t, hkv, g = q.shape[0], k.shape[1], q.shape[1] // k.shape[1]
    at = torch.arange(t, device=q.device)
    seq = torch.searchsorted(cu.long(), at, right=True)
    unseen = (seq[:, None] != seq[None]) | (at[None] > at[:, None])
    s = torch.matmul(_heads(q, g), k.float().permute(1, 2, 0).contiguous()).view(hkv, g, t, t)
    return s.mul_(scale).masked_fill_(unseen, -math.inf)


def _heads(x, g):
    """[t, hkv * g, d] -> [hkv, g * t, d] in 32 bits."""
    t, h, d = x.shape
    return x.float().view(t, h // g, g, d).permute(1, 2, 0, 3).reshape(h // g, g * t, d)


def _rows(x, g):
    """[hkv, g * t, d] -> [t, hkv * g, d]."""
    hkv, n, d = x.shape
    return x.view(hkv, g, n // g, d).permute(2, 0, 1, 3).reshape(n // g, hkv * g, d)


def _plain_prompt(st):
    q, k, v, g = st["q"], st["k"], st["v"], st["q"].shape[1] // st["k"].shape[1]
    p = _scores(q, k, st["cu"], st["scale"])
    m = p.amax(-1, keepdim=True)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    hkv, t = k.shape[1], k.shape[0]
    o = torch.matmul(p.view(hkv, g * t, t), v.float().permute(1, 0, 2).contiguous()) / l.view(hkv, g * t, 1)
    return _rows(o, g), (m + l.log()).view(hkv * g, t)


def _plain_train(st):
    q, k, v, g = st["q"], st["k"], st["v"], st["q"].shape[1] // st["k"].shape[1]
    hkv, t = k.shape[1], k.shape[0]
    out, lse = _plain_prompt(st)
    p = _scores(q, k, st["cu"], st["scale"]).sub_(lse.view(hkv, g, t, 1)).exp_().view(hkv, g * t, t)
    do, kf = _heads(st["grad_out"], g), k.float().permute(1, 0, 2).contiguous()
    dv = torch.matmul(p.transpose(1, 2), do)
    ds = torch.matmul(do, v.float().permute(1, 2, 0).contiguous())
    ds = ds.sub_((do * _heads(out, g)).sum(-1, keepdim=True)).mul_(p).mul_(st["scale"])
    dq = _rows(torch.matmul(ds, kf), g)
    dk = torch.matmul(ds.transpose(1, 2), _heads(q, g))
    return [out, lse, dq, dk.permute(1, 0, 2), dv.permute(1, 0, 2)]


def _plain_decode(st):
    q, table = st["q"].float(), st["table"].long().clamp(min=0)
    r, hq, d = q.shape
    hkv, bt = st["k_cache"].shape[1:3]

    def gather(cache, scale):
        x = cache[table].float() * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(r, hkv, -1, d)

    k, v = gather(st["k_cache"], st["k_scale"]), gather(st["v_cache"], st["v_scale"])
    seen = (torch.arange(k.shape[2], device=q.device)[None] < st["lens"][:, None])[:, None, None]
    v = torch.where(seen.view(r, 1, -1, 1), v, 0.0)
    s = torch.matmul(q.view(r, hkv, hq // hkv, d), k.transpose(2, 3)) * st["scale"]
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.clamp(min=-3e38))
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, torch.matmul(p, v) / l, 0.0)
    return [o.view(r, hq, d), (m + l.log()).view(r, hq)]


def _plain_append(st):
    slots, bt = st["slots"].long(), st["case"]["bt"]
    blk, pos = slots // bt, slots % bt
    out = []
    for x in ("k", "v"):
        cache, scale, new = st[x + "_cache"], st[x + "_scale"], st[x].float()
        nb, hkv = scale.shape
        most = 127.0 if cache.dtype == torch.int8 else 448.0
        top = torch.zeros_like(scale).scatter_reduce_(0, blk[:, None].expand(-1, hkv), new.abs().amax(-1), "amax")
        first = torch.full((nb,), bt, device=slots.device).scatter_reduce_(0, blk, pos, "amin")
        touched = torch.zeros(nb, dtype=torch.bool, device=slots.device).index_fill_(0, blk, True)
        older = torch.where((first > 0)[:, None], scale, 0.0)
        s = torch.maximum(older, top * (1.0 / most)).clamp(min=SMALLEST_SCALE)
        kept = (torch.arange(bt, device=slots.device)[None] < first[:, None]) & touched[:, None]
        ratio = torch.where(kept[:, None], (older / s)[..., None], 1.0)[..., None]
        moved = cache.float() * ratio
        fresh = new * (1.0 / s)[blk][..., None]
        if cache.dtype == torch.int8:
            moved, fresh = moved.round_(), fresh.round_()
        cache.copy_(moved.clamp_(-most, most).to(cache.dtype))
        cache.view(torch.int8)[blk, :, pos] = fresh.clamp_(-most, most).to(cache.dtype).view(torch.int8)
        scale.copy_(torch.where(touched[:, None], s, scale))
        out += [cache, scale]
    return out


def _plain_tables(st):
    held, new, table, free, bt = st["held"].long(), st["new"].long(), st["table"], st["free"], st["case"]["bt"]
    dev, (n, width) = held.device, table.shape
    have, need = (held + bt - 1) // bt, (held + new + bt - 1) // bt
    off = torch.cumsum(need - have, 0) - (need - have)
    col = torch.arange(width, device=dev)[None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    at = (off[:, None] + col - have[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[at], table)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(new, 0)])
    t = torch.arange(st["tokens"], device=dev)
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = held[r] + t - cu[r]
    slots = table[r, pos // bt].long() * bt + pos % bt
    used = torch.stack([(need - have).sum(), torch.zeros((), dtype=torch.long, device=dev)])
    return [table, slots.int(), cu.int(), (held + new).int(), used.int()]


def run(st):
    op = st["case"]["op"]
    if own:
        import linear_attention_sequence_gated_amd as gdn
        if op == "prompt":
            return list(gdn.attn_prompt(st["q"], st["k"], st["v"], st["cu"], st["scale"]))
        if op == "train":
            out, lse = gdn.attn_prompt(st["q"], st["k"], st["v"], st["cu"], st["scale"])
            return [out, lse, *gdn.attn_prompt_bwd(st["q"], st["k"], st["v"], out, lse, st["grad_out"], st["cu"], st["scale"])]
        if op == "decode":
            return list(gdn.attn_decode(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["table"], st["lens"], st["scale"]))
        if op == "append":
            gdn.cache_append(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
            return [st["k_cache"], st["k_scale"], st["v_cache"], st["v_scale"]]
        slots, cu, after, used = gdn.block_tables(st["held"], st["new"], st["table"], st["free"], st["case"]["bt"], st["blocks"], st["tokens"])
        return [st["table"], slots, cu, after, used]
    if op == "prompt":
        out, lse = _plain_prompt(st)
        return [out.to(torch.bfloat16), lse]
    if op == "train":
        out, lse, dq, dk, dv = _plain_train(st)
        return [out.to(torch.bfloat16), lse, dq.to(torch.bfloat16), dk.to(torch.bfloat16), dv.to(torch.bfloat16)]
    if op == "decode":
        out, lse = _plain_decode(st)
        return [out.to(torch.bfloat16), lse]
    return _plain_append(st) if op == "append" else _plain_tables(st)


# ---------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None
    st = prepare(case, seed)
    return {"prompt": _exact_prompt, "train": _exact_prompt, "decode": _exact_decode, "append": _exact_append}[op](st)


def _exact_prompt(st):
    train = "grad_out" in st
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    t, hq, d = q.shape
    g = hq // k.shape[1]
    out, lse = torch.zeros_like(q), torch.zeros(hq, t, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    cu = st["cu"].tolist()
    for a, b in zip(cu, cu[1:]):
        for h in range(hq if b > a else 0):
            qs, ks, vs = q[a:b, h], k[a:b, h // g], v[a:b, h // g]
            s = (qs @ ks.T) * st["scale"]
            s += torch.triu(torch.full_like(s, -math.inf), 1)
            lse[h, a:b] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[h, a:b, None])
            del s
            out[a:b, h] = p @ vs
            if train:
                do = st["grad_out"][a:b, h].double()
                dv[a:b, h // g] += p.T @ do
                dp = do @ vs.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True))
                dq[a:b, h] = st["scale"] * (ds @ ks)
                dk[a:b, h // g] += st["scale"] * (ds.T @ qs)
    return [out, lse, dq, dk, dv] if train else [out, lse]


def _exact_decode(st):
    q = st["q"].double()
    r, hq, d = q.shape
    hkv, bt = st["k_cache"].shape[1:3]
    out = torch.zeros(r, hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((r, hq), -math.inf, dtype=torch.float64, device=q.device)
    for i, n in enumerate(st["lens"].tolist()):
        if not n:
            continue
        ids = st["table"][i, : -(-n // bt)].long()
        blocks = (st[x + "_cache"][ids].double() * st[x + "_scale"][ids].double()[..., None, None] for x in ("k", "v"))
        k, v = (x.permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n] for x in blocks)
        s = (q[i].view(hkv, -1, 1, d) * k[:, None]).sum(-1) * st["scale"]
        lse[i] = torch.logsumexp(s, -1).view(-1)
        out[i] = torch.matmul(torch.softmax(s, -1), v).view(hq, d)
    return [out, lse]


def _exact_append(st):
    """By definition the scales, their reciprocals and ratios, and the number that is rounded to a code are 32-bit numbers: a value at half
    the block's largest falls between two codes, and the rounding of the product decides."""
    slots, bt = st["slots"].cpu().numpy().astype(np.int64), st["case"]["bt"]
    answer = []
    for x in ("k", "v"):
        cache = st[x + "_cache"].float().cpu().numpy().astype(np.float64)
        scale, new = st[x + "_scale"].cpu().numpy().copy(), st[x].float().cpu().numpy().astype(np.float64)
        whole = st[x + "_cache"].dtype == torch.int8
        most = 127.0 if whole else 448.0

        def code(y):
            y = y.astype(np.float32).astype(np.float64)
            if whole:
                return np.clip(np.rint(y), -most, most)
            y = np.clip(y, -most, most)
            step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 1e-300))), -6) - 3)
            return np.rint(y / step) * step

        cut = np.flatnonzero(np.diff(slots // bt, prepend=-1))
        for a, b in zip(cut, np.append(cut[1:], len(slots))):
            blk, first = slots[a] // bt, slots[a] % bt
            old = scale[blk] if first else np.zeros_like(scale[blk])
            s = np.maximum(old, np.abs(new[a:b]).max((0, 2)).astype(np.float32) * np.float32(1 / most))
            s = np.maximum(s, np.float32(SMALLEST_SCALE)).astype(np.float32)
            ratio = (old / s).astype(np.float32).astype(np.float64)
            cache[blk, :, :first] = code(cache[blk, :, :first] * ratio[:, None, None])
            cache[blk, :, first:first + b - a] = code(new[a:b].transpose(1, 0, 2) * (np.float32(1) / s).astype(np.float64)[:, None, None])
            scale[blk] = s
        answer += [cache, scale.astype(np.float64)]
    return answer
