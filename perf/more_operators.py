"""Cases for what stands around a recurrent layer's state update in a hybrid model: the root-mean-square norm with the
residual's addition (also with an output in 8 bits), the short causal convolution, and the selective state space scan,
each for packed prompts, for training and for single tokens.  `run` computes them in plain torch operations, or, where
`own` is set, with the package's kernels.

Lengths of a ragged batch are a function of the case alone; every value comes from the seed."""
import math

import numpy as np
import torch

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")

own = False

CHUNK = 64  # of the plain scan
SMALLEST_SCALE = 2.0 ** -100
EPS = 1e-6


def listed():
    return [
        # the norm before the projection of a few requests' next tokens, 12 heads of 64 wide
        dict(name="norm_tokens", op="norm_quant", t=6, c=768, dtype="bf16", block=128, kind="e4m3", residual=True),
        # a prefill batch's norm with 8-bit rows for the projection, 16 heads of 128 wide
        dict(name="norm_quant", op="norm_quant", t=9869, c=2048, dtype="bf16", block=128, kind="e4m3", residual=True),
        # a training step of the 8 x 2048 x 12 x 64 layer's norm, forward and gradients
        dict(name="norm_train", op="norm_train", t=16384, c=768, dtype="bf16", residual=True),
        # prompts of many lengths through the convolution of x, B and C together
        dict(name="conv_prompt", op="conv_prompt", n=9, longest=2500, ragged=True, c=1792, w=4, dtype="bf16", silu=True, carried=False),
        # the convolution of q, k and v of the 8 x 2048 x 12 x 64 layer, forward and gradients
        dict(name="conv_train", op="conv_train", n=8, longest=2048, ragged=False, c=2304, w=4, dtype="bf16", silu=True),
        # one new token for each request of a decoding batch
        dict(name="conv_tokens", op="conv_step", n=256, c=1792, w=4, dtype="bf16", silu=True),
        # one short prompt: the time to the first token
        dict(name="scan_short", op="scan", n=1, longest=131, ragged=False, h=24, p=64, g=1, s=128, carried=False),
        # the state space layer of the 8 x 2048 x 12 x 64 model, inner width twice the model's
        dict(name="scan_layer", op="scan", n=8, longest=2048, ragged=False, h=24, p=64, g=1, s=128, carried=False),
        # 16k context, heads of 128 in groups, going on from a state
        dict(name="scan_long", op="scan", n=1, longest=16384, ragged=False, h=32, p=128, g=4, s=128, carried=True),
        # a training step of the 8 x 2048 layer, forward and gradients
        dict(name="scan_train", op="scan_train", n=8, longest=2048, ragged=False, h=24, p=64, g=1, s=128),
        # documents of many lengths packed into one training row
        dict(name="scan_train_ragged", op="scan_train", n=13, longest=1201, ragged=True, h=16, p=128, g=4, s=64),
        # one new token for each request of a decoding batch
        dict(name="scan_tokens", op="scan_step", n=256, h=24, p=64, g=1, s=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_quant", "norm_train", "conv_prompt", "conv_train", "conv_step", "scan", "scan", "scan_train", "scan_step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("norm"):
        c = 8 * _log(rng, 8, 1024)
        t = _log(rng, 1, max(1, 12000000 // c))
        if op == "norm_train":
            return dict(op=op, t=t, c=c, dtype=dtype, residual=rng.random() < 0.7)
        block = 128 if c % 128 == 0 and rng.random() < 0.7 else 0
        return dict(op=op, t=t, c=c, dtype=dtype, block=block, kind=rng.choice(["e4m3", "e4m3", "int8"]), residual=rng.random() < 0.7)
    if op.startswith("conv"):
        c, w, silu = 8 * _log(rng, 8, 640), rng.choice([2, 3, 4, 4]), rng.random() < 0.8
        if op == "conv_step":
            return dict(op=op, n=_log(rng, 1, 512), c=c, w=w, dtype=dtype, silu=silu)
        total = _log(rng, 16, 20000000 // c)
        n = _log(rng, 1, max(1, total // 8))
        return dict(op=op, n=n, longest=max(1, total // n), ragged=rng.random() < 0.6, c=c, w=w, dtype=dtype, silu=silu, carried=rng.random() < 0.3)
    h, p, g = rng.choice([(24, 64, 1), (24, 64, 1), (7, 64, 1), (16, 64, 4), (6, 64, 3), (16, 128, 4), (5, 128, 1), (8, 128, 8)])
    s = rng.choice([64, 128, 128])
    if op == "scan_step":
        return dict(op=op, n=_log(rng, 1, 5000000 // (h * p * s)), h=h, p=p, g=g, s=s)
    total = _log(rng, 64, 9000 if op == "scan_train" else 14000)
    n = _log(rng, 1, max(1, min(64, total // 16)))
    return dict(op=op, n=n, longest=max(1, total // n), ragged=rng.random() < 0.6, h=h, p=p, g=g, s=s, carried=op == "scan" and rng.random() < 0.4)


def lengths(case):
    """Tokens of each sequence: a function of the case, so that work() knows them."""
    n, longest = case["n"], case["longest"]
    if not case["ragged"]:
        return np.full(n, longest, dtype=np.int64)
    got = np.random.default_rng([n, longest]).integers(0, longest + 1, n)
    got[n // 2] = 0
    got[0] = longest
    return got


def work(case):
    op = case["op"]
    size = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if op.startswith("norm"):
        e = float(case["t"] * case["c"])
        rows = size * e
        if op == "norm_quant":  # x and the residual in, the sum and the codes out
            scales = 4.0 * case["t"] * (case["c"] // case["block"] if case["block"] else 1)
            return {"bytes": rows * (3 if case["residual"] else 1) + e + scales + size * case["c"], "flops": 6 * e}
        # forward: x and the residual in, the sum and the output out; gradients: the sum, those of output and sum in, one out
        return {"bytes": rows * ((4 + 4) if case["residual"] else (2 + 3)) + 2.0 * size * case["c"], "flops": 14 * e}
    if op.startswith("conv"):
        c, w = case["c"], case["w"]
        if op == "conv_step":
            return {"bytes": size * case["n"] * c * (2.0 + 2 * (w - 1)) + size * c * (w + 1), "flops": case["n"] * c * (2.0 * w + 4)}
        e, states = float(lengths(case).sum()) * c, float(case["n"] * (w - 1) * c)
        if op == "conv_prompt":
            return {"bytes": size * (2 * e + states * (2 if case["carried"] else 1) + c * (w + 1)), "flops": e * (2 * w + 4)}
        return {"bytes": size * (5 * e + 2 * c * (w + 1)), "flops": e * (8 * w + 14)}
    h, p, g, s = (case[x] for x in "hpgs")
    if op == "scan_step":
        n = case["n"]
        return {"bytes": 8.0 * n * h * p * s + 2 * n * (2 * h * p + 2 * g * s + h), "flops": 5.0 * n * h * p * s}
    t = float(lengths(case).sum())
    rows, states = 2 * t * (2 * h * p + 2 * g * s + h), 4.0 * case["n"] * h * p * s
    if op == "scan":
        return {"bytes": rows + states * (2 if case["carried"] else 1), "flops": 4 * t * h * p * s}
    return {"bytes": 2 * t * (5 * h * p + 6 * g * s + 3 * h), "flops": 14 * t * h * p * s}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    dt = torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device=DEV) * (hi - lo) + lo

    if op.startswith("norm"):
        t, c = case["t"], case["c"]
        st["x"], st["weight"] = normal(t, c), (1.0 + 0.2 * normal(c, dtype=torch.float32)).to(dt)
        st["residual"] = normal(t, c, scale=3.0) if case["residual"] else None
        if op == "norm_train":
            st["grad_out"] = normal(t, c)
            st["grad_sum"] = normal(t, c) if case["residual"] else None
        return st
    if op != "conv_step" and op != "scan_step":
        n = lengths(case)
        st["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(DEV)
        t = int(n.sum())
    else:
        t = case["n"]
    if op.startswith("conv"):
        c, w = case["c"], case["w"]
        # the projection's columns before those of the convolution hold the gate
        st["x"] = normal(t, c + 64)[:, 64:]
        st["weight"], st["bias"] = normal(c, w, scale=w ** -0.5), normal(c, scale=0.1)
        if op == "conv_step" or case.get("carried"):
            st["state"] = normal(case["n"], w - 1, c)
        if op == "conv_train":
            st["grad_out"] = normal(t, c)
        return st
    h, p, groups, s = (case[x] for x in "hpgs")
    # x, B and C as one convolution leaves them
    rows = normal(t, h * p + 2 * groups * s)
    x, b, c = rows.split([h * p, groups * s, groups * s], dim=1)
    st["x"], st["b"], st["c"] = x.view(t, h, p), b.view(t, groups, s), c.view(t, groups, s)
    st["dt"] = normal(t, h)
    # steps from 1/1000 to 1/10, decay rates from 1 to 16, as such layers begin
    step = torch.exp(uniform(h, lo=math.log(1e-3), hi=math.log(1e-1)))
    st["dt_bias"] = torch.log(torch.expm1(step)).to(dt)
    st["a"], st["d"] = (-uniform(h, lo=1.0, hi=16.0)).to(dt), normal(h, scale=0.2)
    if op == "scan_step" or case.get("carried"):
        st["state"] = normal(case["n"], h, s, p, dtype=torch.float32)
    if op == "scan_train":
        st["grad_out"] = normal(t, h, p)
    return st


# ------------------------------------------------------------- plain forms
def _plain_norm(st):
    x, w = st["x"], st["weight"].float()
    total = x if st["residual"] is None else (x.float() + st["residual"].float()).to(x.dtype)
    f = total.float()
    rstd = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    return total, f, rstd, f * rstd * w


def _plain_norm_quant(st):
    total, _, _, y = _plain_norm(st)
    t, c = y.shape
    block = st["case"]["block"] or c
    most = 127.0 if st["case"]["kind"] == "int8" else 448.0
    parts = y.view(t, c // block, block)
    scale = (parts.abs().amax(-1) * (1.0 / most)).clamp(min=SMALLEST_SCALE)
    q = (parts * (1.0 / scale)[..., None]).clamp(-most, most).view(t, c)
    codes = q.round().to(torch.int8) if st["case"]["kind"] == "int8" else q.to(torch.float8_e4m3fn)
    return _values(st, codes, scale) + [scale, total]


def _values(st, codes, scale):
    """8-bit floats as they are, whole numbers as what they stand for."""
    if codes.dtype != torch.int8:
        return [codes]
    t, c = codes.shape
    return [(codes.view(t, scale.shape[1], -1).float() * scale[..., None]).view(t, c)]


def _plain_norm_train(st):
    total, f, rstd, y = _plain_norm(st)
    dt, w, g = total.dtype, st["weight"].float(), st["grad_out"].float()
    wg = w * g
    gs = rstd * wg - f * rstd.pow(3) * (wg * f).mean(-1, keepdim=True)
    if st["grad_sum"] is not None:
        gs = gs + st["grad_sum"].float()
    return [y.to(dt), total, gs.to(dt), (g * f * rstd).sum(0).to(dt)]


def _places(cu, n, width):
    """[n, width]: the rows that the sequences' tokens stand in, and whether they are there."""
    at = cu[:-1, None].long() + torch.arange(width, device=cu.device)[None]
    there = at < cu[1:, None]
    return at, there


def _taps(st):
    """x and what the convolution sees behind it: [rows, w, c] in 32 bits."""
    x, cu, w = st["x"].float(), st["cu"].long(), st["case"]["w"]
    t, c = x.shape
    rows = torch.arange(t, device=x.device)
    seq = torch.searchsorted(cu[1:].contiguous(), rows, right=True)
    pos = rows - cu[seq]
    back = torch.arange(1 - w, 1, device=x.device)
    inside = (pos[:, None] + back[None]) >= 0
    got = torch.where(inside[..., None], x[(rows[:, None] + back[None]).clamp(min=0)], 0.0)
    if st.get("state") is not None:
        slot = (pos[:, None] + back[None] + w - 1).clamp(max=w - 2)
        got = torch.where(inside[..., None], got, st["state"].float()[seq[:, None], slot])
    return got, inside, rows[:, None] + back[None]


def _last(st):
    """The last w - 1 inputs of each sequence."""
    x, cu, w = st["x"], st["cu"].long(), st["case"]["w"]
    back = torch.arange(1 - w, 0, device=x.device)
    n = cu[1:] - cu[:-1]
    at = cu[1:, None] + back[None]
    inside = n[:, None] + back[None] >= 0
    got = torch.where(inside[..., None], x[at.clamp(min=0, max=max(0, x.shape[0] - 1))], 0.0)
    if st.get("state") is not None:
        slot = (n[:, None] + back[None] + w - 1).clamp(max=w - 2)
        got = torch.where(inside[..., None], got, torch.gather(st["state"], 1, slot[..., None].expand(-1, -1, x.shape[1])))
    return got.to(x.dtype)


def _plain_conv(st):
    got, _, _ = _taps(st)
    p = (got * st["weight"].float().t()[None]).sum(1) + st["bias"].float()
    y = p * torch.sigmoid(p) if st["case"]["silu"] else p
    return [y.to(st["x"].dtype), _last(st)]


def _plain_conv_train(st):
    got, inside, at = _taps(st)
    dt, wt = st["x"].dtype, st["weight"].float().t()
    p = (got * wt[None]).sum(1) + st["bias"].float()
    sig = torch.sigmoid(p)
    y = p * sig if st["case"]["silu"] else p
    gp = st["grad_out"].float()
    if st["case"]["silu"]:
        gp = gp * (sig * (1.0 + p * (1.0 - sig)))
    gw, gb = (got * gp[:, None]).sum(0).t(), gp.sum(0)
    back = torch.where(inside[..., None], gp[:, None] * wt[None], 0.0)  # what goes to the row `at`
    rows, w = torch.arange(gp.shape[0], device=gp.device)[:, None], wt.shape[0]
    ahead = (rows + (w - 1 - torch.arange(w, device=gp.device))[None]).clamp(max=gp.shape[0] - 1)
    tap = torch.arange(w, device=gp.device)[None].expand_as(ahead)
    fits = at[ahead, tap] == rows
    gx = torch.where(fits[..., None], back[ahead, tap], 0.0).sum(1)
    return [y.to(dt), gx.to(dt), gw.to(dt).contiguous(), gb.to(dt)]


def _plain_conv_step(st):
    x, state = st["x"], st["state"]
    got = torch.cat([state, x[:, None]], 1).float()
    p = (got * st["weight"].float().t()[None]).sum(1) + st["bias"].float()
    y = p * torch.sigmoid(p) if st["case"]["silu"] else p
    state.copy_(got[:, 1:].to(state.dtype))
    return [y.to(x.dtype), state]


def _softplus(z):
    return torch.where(z > 20.0, z, torch.log1p(torch.exp(z.clamp(max=20.0))))  # its gradient at 0 is 1/2


def _plain_scan(st, x, dt, a, b, c, d, bias):
    """(y [t, h, p], final states [n, h, s, p]) in 32 bits: chunks within, and chunks with each other, as products."""
    case = st["case"]
    n, h, p, g, s = case["n"], case["h"], case["p"], case["g"], case["s"]
    nc = -(-case["longest"] // CHUNK)
    at, there = _places(st["cu"], n, nc * CHUNK)
    at = at.clamp(max=x.shape[0] - 1)
    delta = torch.where(there[..., None], _softplus(dt[at] + bias), 0.0).view(n, nc, CHUNK, h).permute(0, 1, 3, 2)  # n, nc, h, Q
    xs = torch.where(there[..., None, None], x[at], 0.0).view(n, nc, CHUNK, h, p).permute(0, 1, 3, 2, 4)
    bs, cs = (torch.where(there[..., None, None], y[at], 0.0).view(n, nc, CHUNK, g, s).permute(0, 1, 3, 2, 4) for y in (b, c))
    run = torch.cumsum(delta * a[:, None], -1)  # n, nc, h, Q
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp(torch.where(lower, run[..., :, None] - run[..., None, :], -math.inf))
    cb = torch.matmul(cs, bs.transpose(-1, -2)).repeat_interleave(h // g, 2)
    y = torch.matmul(cb * decay * delta[..., None, :], xs)
    left = torch.exp(run[..., -1:] - run) * delta
    bh, ch = bs.repeat_interleave(h // g, 2), cs.repeat_interleave(h // g, 2)
    local = torch.matmul((bh * left[..., None]).transpose(-1, -2), xs)  # n, nc, h, s, p
    whole = torch.cumsum(run[..., -1], 1)  # n, nc, h
    first = torch.zeros(n, h, s, p, device=x.device) if st.get("state") is None else st["state"].float()
    local = torch.cat([first[:, None], local], 1)
    whole = torch.cat([torch.zeros_like(whole[:, :1]), whole], 1).permute(0, 2, 1)  # n, h, nc + 1
    lower = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=x.device).tril()
    carry = torch.exp(torch.where(lower, whole[..., :, None] - whole[..., None, :], -math.inf))
    states = torch.matmul(carry, local.permute(0, 2, 1, 3, 4).reshape(n, h, nc + 1, s * p)).view(n, h, nc + 1, s, p)
    y = y + torch.exp(run)[..., None] * torch.matmul(ch, states[:, :, :-1].transpose(1, 2))
    y = (y + d[:, None, None] * xs).permute(0, 1, 3, 2, 4).reshape(n, nc * CHUNK, h, p)
    return y[there], states[:, :, -1]


def _plain_scan_train(st):
    names = ("x", "dt", "a", "b", "c", "d", "dt_bias")
    with torch.enable_grad():
        ins = [st[k].float().detach().requires_grad_(True) for k in names]
        y, _ = _plain_scan(st, *ins)
        grads = torch.autograd.grad(y, ins, st["grad_out"].float())
    return [y.detach().to(torch.bfloat16)] + [v.to(torch.bfloat16) for v in grads]


def _plain_scan_step(st):
    case, state = st["case"], st["state"]
    rep = case["h"] // case["g"]
    b, c = (st[k].float().repeat_interleave(rep, 1) for k in "bc")
    x = st["x"].float()
    delta = _softplus(st["dt"].float() + st["dt_bias"].float())
    keep = torch.exp(delta * st["a"].float())
    state.mul_(keep[..., None, None]).add_((delta[..., None] * b)[..., None] * x[:, :, None])
    y = (state * c[..., None]).sum(2) + st["d"].float()[:, None] * x
    return [y.to(torch.bfloat16), state]


def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st)
    if op == "norm_quant":
        return _plain_norm_quant(st)
    if op == "norm_train":
        return _plain_norm_train(st)
    if op == "conv_prompt":
        return _plain_conv(st)
    if op == "conv_train":
        return _plain_conv_train(st)
    if op == "conv_step":
        return _plain_conv_step(st)
    if op == "scan":
        y, last = _plain_scan(st, *(st[k].float() for k in ("x", "dt", "a", "b", "c", "d", "dt_bias")))
        return [y.to(torch.bfloat16), last]
    return _plain_scan_train(st) if op == "scan_train" else _plain_scan_step(st)


def _own(st):
    import linear_attention_sequence_gated_amd as gdn
    case, op = st["case"], st["case"]["op"]
    if op == "norm_quant":
        kind = torch.int8 if case["kind"] == "int8" else torch.float8_e4m3fn
        codes, scale, total = gdn.rms_norm_quant(st["x"], st["weight"], st["residual"], eps=EPS, dtype=kind, block=case["block"])
        return _values(st, codes, scale) + [scale, total]
    if op == "norm_train":
        y, total = gdn.rms_norm(st["x"], st["weight"], st["residual"], eps=EPS)
        return [y, total, *gdn.rms_norm_bwd(total, st["weight"], st["grad_out"], eps=EPS, grad_sum=st["grad_sum"])]
    if op == "conv_prompt":
        return list(gdn.short_conv(st["x"], st["weight"], st["cu"], bias=st["bias"], state=st.get("state"), silu=case["silu"]))
    if op == "conv_train":
        y, _ = gdn.short_conv(st["x"], st["weight"], st["cu"], bias=st["bias"], state=st.get("state"), silu=case["silu"])
        gx, gw, gb, _ = gdn.short_conv_bwd(st["x"], st["weight"], st["grad_out"], st["cu"], bias=st["bias"], state=st.get("state"), silu=case["silu"])
        return [y, gx, gw, gb]
    if op == "conv_step":
        return [gdn.short_conv_step(st["x"], st["weight"], st["state"], bias=st["bias"], silu=case["silu"]), st["state"]]
    args = st["x"], st["dt"], st["a"], st["b"], st["c"]
    more = dict(D=st["d"], dt_bias=st["dt_bias"])
    if op == "scan":
        return list(gdn.ssm_scan(*args, st["cu"], S0=st.get("state"), **more))
    if op == "scan_train":
        y, _ = gdn.ssm_scan(*args, st["cu"], **more)
        gx, gdt, ga, gb, gc, gd, gbias, _ = gdn.ssm_scan_bwd(*args, st["grad_out"], st["cu"], **more)
        return [y, gx, gdt, ga, gb, gc, gd, gbias]
    return [gdn.ssm_step(*args, st["state"], **more), st["state"]]


# ---------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        return _exact_norm(st)
    if op.startswith("conv"):
        return _exact_conv(st)
    return _exact_scan(st)


def _exact_norm(st):
    case, x, w = st["case"], st["x"], st["weight"].double()
    total = x if st["residual"] is None else (x.double() + st["residual"].double()).to(x.dtype)  # the sum is a number of the rows' type
    s = total.double()
    root = torch.sqrt(s.square().sum(-1, keepdim=True) / s.shape[1] + EPS)
    y = s / root * w
    if case["op"] == "norm_train":
        g = st["grad_out"].double()
        n = s / root
        gn = g * w
        gs = (gn - n * (gn * n).sum(-1, keepdim=True) / s.shape[1]) / root
        if st["grad_sum"] is not None:
            gs = gs + st["grad_sum"].double()
        return [y, s, gs, (g * n).sum(0)]
    t, c = y.shape
    most = 127.0 if case["kind"] == "int8" else 448.0
    parts = y.reshape(t, -1, case["block"] or c)
    scale = (parts.abs().amax(-1) / most).clamp(min=SMALLEST_SCALE)
    q = (parts / scale[..., None]).clamp(-most, most)
    if case["kind"] == "int8":
        return [(q.round() * scale[..., None]).view(t, c), scale, s]
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=1e-300))).clamp(min=-6) - 3)
    return [(torch.round(q / step) * step).view(t, c), scale, s]


def _exact_conv(st):
    """Sequence after sequence, by the sum itself."""
    case = st["case"]
    w, c, op = case["w"], case["c"], case["op"]
    x, wt, bias = st["x"].double(), st["weight"].double(), st["bias"].double()
    cu = list(range(case["n"] + 1)) if op == "conv_step" else st["cu"].tolist()
    y, last = torch.zeros_like(x), torch.zeros(case["n"], w - 1, c, dtype=torch.float64, device=x.device)
    gx, gw, gb = torch.zeros_like(x), torch.zeros_like(wt), torch.zeros_like(bias)
    for i, (lo, hi) in enumerate(zip(cu, cu[1:])):
        n = hi - lo
        seen = torch.zeros(w - 1 + n, c, dtype=torch.float64, device=x.device)
        if st.get("state") is not None:
            seen[:w - 1] = st["state"][i].double()
        seen[w - 1:] = x[lo:hi]
        last[i] = seen[n:]
        if not n:
            continue
        p = bias + sum(wt[:, j] * seen[j:j + n] for j in range(w))
        y[lo:hi] = p / (1 + torch.exp(-p)) if case["silu"] else p
        if op == "conv_train":
            g = st["grad_out"][lo:hi].double()
            if case["silu"]:
                e = torch.exp(-p)
                g = g * (1 / (1 + e) + p * e / (1 + e).square())
            gs = torch.zeros_like(seen)
            for j in range(w):
                gs[j:j + n] += g * wt[:, j]
                gw[:, j] += (g * seen[j:j + n]).sum(0)
            gb += g.sum(0)
            gx[lo:hi] = gs[w - 1:]
    return [y, gx, gw, gb] if op == "conv_train" else [y, last]


def _exact_scan(st):
    """Token after token, every sequence at once; the gradients by the same recurrence backwards."""
    case, train = st["case"], st["case"]["op"] == "scan_train"
    n, h, p, s, rep = case["n"], case["h"], case["p"], case["s"], case["h"] // case["g"]
    x, a, d = st["x"].double(), st["a"].double(), st["d"].double()
    z = st["dt"].double() + st["dt_bias"].double()
    delta = torch.where(z > 30, z, torch.log1p(torch.exp(z.clamp(max=30))))
    b, c = (st[k].double().repeat_interleave(rep, 1) for k in "bc")
    lens = np.ones(n, dtype=np.int64) if case["op"] == "scan_step" else lengths(case)
    start = np.concatenate([[0], np.cumsum(lens)])[:-1]
    order = np.argsort(-lens, kind="stable")  # the sequences that go on are the first ones
    lens, start = lens[order], start[order]
    place = torch.from_numpy(order).to(x.device)
    state = torch.zeros(n, h, s, p, dtype=torch.float64, device=x.device)
    if st.get("state") is not None:
        state = st["state"][place].double()
    y, before, at = torch.zeros_like(x), [], []
    begin = torch.from_numpy(start).to(x.device)
    for i in range(int(lens.max())):
        m = int((lens > i).sum())
        r = begin[:m] + i
        at.append(r)
        old = state[:m]
        if train:
            before.append(old.clone())
        new = torch.exp(a * delta[r])[..., None, None] * old + (delta[r][..., None] * b[r])[..., None] * x[r][:, :, None]
        y[r] = torch.matmul(c[r][:, :, None], new)[:, :, 0] + d[:, None] * x[r]
        state[:m] = new
    if not train:
        last = torch.empty_like(state)
        last[place] = state
        return [y, last]
    gy = st["grad_out"].double()
    gx, gdelta, gb, gc, ga = torch.zeros_like(x), torch.zeros_like(delta), torch.zeros_like(b), torch.zeros_like(c), torch.zeros_like(a)
    gs = torch.zeros_like(state)
    for r, old in zip(reversed(at), reversed(before)):
        m = len(r)
        keep = torch.exp(a * delta[r])
        new = keep[..., None, None] * old + (delta[r][..., None] * b[r])[..., None] * x[r][:, :, None]
        gc[r] = torch.matmul(new, gy[r][..., None])[..., 0]
        g = gs[:m] + c[r][..., None] * gy[r][:, :, None]
        gbx = torch.matmul(g, x[r][..., None])[..., 0]  # [m, h, s]
        gb[r] = delta[r][..., None] * gbx
        gx[r] = delta[r][..., None] * torch.matmul(b[r][:, :, None], g)[:, :, 0] + d[:, None] * gy[r]
        gkeep = (g * old).sum((2, 3)) * keep
        gdelta[r] = a * gkeep + (b[r] * gbx).sum(-1)
        ga += (delta[r] * gkeep).sum(0)
        gs[:m] = keep[..., None, None] * g
    gz = gdelta * torch.sigmoid(z)
    t = x.shape[0]
    return [y, gx, gz, ga, gb.view(t, -1, rep, s).sum(2), gc.view(t, -1, rep, s).sum(2), (gy * x).sum((0, 2)), gz.sum(0)]
