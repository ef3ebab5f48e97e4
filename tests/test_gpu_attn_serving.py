"""The attention layer's operators together, as a server and a trainer use them: a step's tables, the cache's write, the
prompts and the single tokens; captured and replayed; on other streams; with buffers that the caller keeps."""
import numpy as np
import pytest

from gpu_util import note, torch_dev
from oracle import attention as ref
from test_gpu_attn_cache import ints, values

pytestmark = pytest.mark.gpu
HQ, H, D, BT = 6, 2, 64, 16


class Server:
    """Requests with growing contexts: projections are random, the keys and values of every token are kept in 64 bits."""

    def __init__(self, torch, kind, requests, blocks, width, seed=0):
        self.torch, self.kind, self.rng = torch, kind, np.random.default_rng(seed)
        dt = torch.int8 if kind == "int8" else torch.float8_e4m3fn
        self.kc, self.vc = (torch.zeros(blocks, H, BT, D, dtype=torch.int8, device="cuda").view(dt) for _ in range(2))
        self.ks, self.vs = (torch.zeros(blocks, H, device="cuda") for _ in range(2))
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.free = ints(torch, self.rng.permutation(blocks))
        self.history = [[] for _ in range(requests)]
        self.blocks = blocks

    def project(self, tokens):
        x = torch_random(self.torch, self.rng, tokens)
        return x, x.split([HQ, H, H], 1)

    def step(self, new, pad=0):
        """One step of new[r] tokens each: (prompt attention's outputs, slots, offsets)."""
        import linear_attention_sequence_gated_amd as gdn
        torch = self.torch
        total = int(sum(new)) + pad
        x, (q, k, v) = self.project(total)
        slots, cu, after, used = gdn.block_tables(self.lens, ints(torch, new), self.table, self.free, BT, self.blocks, total)
        gdn.cache_append(k, v, slots, self.kc, self.vc, self.ks, self.vs)
        taken, refused = used.tolist()
        assert refused == 0
        self.free, self.lens = self.free[taken:].clone(), after
        kv = x.float().cpu().numpy().astype(np.float64)
        at = 0
        for r, m in enumerate(new):
            self.history[r] += [(kv[t, HQ:HQ + H], kv[t, HQ + H:]) for t in range(at, at + m)]
            at += m
        return q, k, v, cu

    def oracle(self, r, q):
        """Attention of q [Hq, D] over request r's tokens as they were before the cache rounded them."""
        k, v = (np.stack([t[i] for t in self.history[r]]) for i in (0, 1))
        out, lse = ref.prompt(np.repeat(q[None], len(k), 0), k, v, [0, len(k)], D ** -0.5)
        return out[-1], lse[:, -1]


def torch_random(torch, rng, tokens):
    return torch.from_numpy(rng.standard_normal((tokens, HQ + 2 * H, D)).astype(np.float32)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_serving_loop(kind):
    """Prompts of several requests, then single tokens with a new prompt joining: the read over the cache agrees with
    the oracle on what the cache holds (to the read's own rounding), and with attention over the unrounded tokens to the
    cache's: a code is off by half a step at most, 1/254 of a block's largest value (int8) or 2^-4 of the value (e4m3)."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    note(f"serving {kind}")
    s = Server(torch, kind, requests=5, blocks=60, width=12)
    q, k, v, cu = s.step([37, 1, 16, 0, 100], pad=3)
    out, lse = gdn.attn_prompt(q, k, v, cu)
    host = [x.float().cpu().numpy().astype(np.float64) for x in (q, k, v)]
    want, _ = ref.prompt(*host, cu.tolist(), D ** -0.5)
    weighted, _ = ref.prompt(host[0], host[1], np.abs(host[2]), cu.tolist(), D ** -0.5)
    assert np.all(np.abs(out.float().cpu().numpy() - want) <= 2.0 ** -8 * (np.abs(want) + weighted) + 1e-30)
    for i in range(20):
        new = [1, 1, 1, 25 if i == 7 else int(i > 7), 1]
        q, k, v, cu = s.step(new)
        last = [int(c) - 1 for c in cu.tolist()[1:]]  # each request's newest token asks (one without tokens: any)
        qd = q[[max(t, 0) for t in last]].contiguous()
        out, lse = gdn.attn_decode(qd, s.kc, s.vc, s.ks, s.vs, s.table, s.lens)
        caches = values(s.kc), values(s.vc), s.ks.cpu().numpy(), s.vs.cpu().numpy(), s.table.cpu().numpy(), s.lens.tolist()
        qh = qd.float().cpu().numpy()
        want, wlse = ref.decode(qh, *caches, D ** -0.5)
        weighted, _ = ref.decode(qh, caches[0], np.abs(caches[1]), *caches[2:], D ** -0.5)
        got = out.float().cpu().numpy()
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * weighted + 1e-30)
        some = [r for r in range(5) if s.history[r]]
        assert np.allclose(lse.cpu().numpy()[some], wlse[some], atol=1e-4)
        for r in some:
            full, _ = s.oracle(r, qh[r].astype(np.float64))
            kv = np.stack([np.stack(t) for t in s.history[r]])  # [n, 2, H, D]
            # errors of the scores move the weights by a factor e^(2 d); those of the values add to the result
            half = 4.5 / 254 if kind == "int8" else 2.0 ** -4  # int8: blocks whose largest value is under 4.5
            d = D ** -0.5 * np.abs(qh[r]).sum(1).max() * half * (1 if kind == "int8" else np.abs(kv[:, 0]).max())
            bound = (np.exp(2 * d) - 1) * np.abs(kv[:, 1]).max() + half * (1 if kind == "int8" else np.abs(kv[:, 1]).max()) + 0.02
            assert np.abs(got[r] - full).max() <= bound
            rms = np.sqrt(((got[r] - full) ** 2).mean() / (full ** 2).mean())
            assert rms < (0.05 if kind == "int8" else 0.12), rms
    assert (out[3] != 0).any()


def test_decode_step_captured():
    """A step captured once (tables, write, read) and replayed with other lengths, tokens and free lists, the eager step
    and other work in between: every replay equals the eager step bit for bit."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    R, width, nb = 7, 20, 200
    x = torch.zeros(R, HQ + 2 * H, D, dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split([HQ, H, H], 1)
    lens, new = (torch.zeros(R, dtype=torch.int32, device="cuda") for _ in range(2))
    table, free = torch.full((R, width), -1, dtype=torch.int32, device="cuda"), torch.zeros(nb, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(nb, H, BT, D, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(nb, H, device="cuda") for _ in range(2))

    def step():
        slots, cu, after, used = gdn.block_tables(lens, new, table, free, BT, nb, R)
        gdn.cache_append(k, v, slots, kc, vc, ks, vs)
        out, lse = gdn.attn_decode(q, kc, vc, ks, vs, table, after)
        return out, lse, after, used

    def fill(seed):
        g = np.random.default_rng(seed)
        n = g.integers(0, width * BT - 1, R)
        n[seed % R] = 0
        blocks = -(-n // BT)
        ids, t, at = g.permutation(nb), np.full((R, width), -1), 0
        for r, b in enumerate(blocks):
            t[r, :b] = ids[at:at + b]
            at += b
        lens.copy_(ints(torch, n))
        new.copy_(ints(torch, g.integers(0, 2, R)))
        table.copy_(ints(torch, t))
        free.copy_(ints(torch, np.concatenate([ids[at:], np.zeros(at)])))
        x.copy_(torch_random(torch, g, R))
        for c, sc in ((kc, ks), (vc, vs)):
            c.copy_(torch.from_numpy(g.integers(-127, 128, c.shape).astype(np.int8)))
            sc.copy_(torch.from_numpy((0.01 + 0.02 * g.random(sc.shape)).astype(np.float32)))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    fill(0)
    graph = torch.cuda.CUDAGraph()
    note("capture a decode step")
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(1, 6):
        fill(seed)
        eager = [t.clone() for t in (*step(), table, kc, vc, ks, vs)]
        torch.cuda.synchronize()
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (*captured, table, kc, vc, ks, vs)):
            assert torch.equal(a, b), seed


def test_training_pass_captured():
    """Forward and gradients captured once and replayed with other data and other offsets."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    T = 300
    x, do = (torch.zeros(T, n, D, dtype=torch.bfloat16, device="cuda") for n in (HQ + 2 * H, HQ))
    q, k, v = x.split([HQ, H, H], 1)
    cu = torch.zeros(5, dtype=torch.int32, device="cuda")

    def step():
        out, lse = gdn.attn_prompt(q, k, v, cu)
        return out, lse, *gdn.attn_prompt_bwd(q, k, v, out, lse, do, cu)

    def fill(seed):
        g = np.random.default_rng(seed)
        x.copy_(torch_random(torch, g, T))
        do.copy_(torch_random(torch, g, T)[:, :HQ])
        cu.copy_(ints(torch, np.concatenate([[0], np.sort(g.integers(0, T, 3)), [T - seed]])))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    note("capture a training pass")
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(1, 5):
        fill(seed)
        eager = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b), seed


def test_other_streams():
    """On a stream given by its number, and on a current one that is not the default: the same results, many calls in a
    row with nothing waited for between, each with a workspace of its own."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    g = np.random.default_rng(3)
    x = torch_random(torch, g, 500)
    q, k, v = x.split([HQ, H, H], 1)
    cu = ints(torch, [0, 200, 500])
    want = gdn.attn_prompt(q, k, v, cu)
    grads = gdn.attn_prompt_bwd(q, k, v, *want, want[0], cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    note("other streams")
    got = []
    for i in range(6):
        o = gdn.attn_prompt(q, k, v, cu, stream=s.cuda_stream)
        got.append((*o, *gdn.attn_prompt_bwd(q, k, v, *o, o[0], cu, stream=s.cuda_stream)))
    with torch.cuda.stream(s):
        o = gdn.attn_prompt(q, k, v, cu)
        got.append((*o, *gdn.attn_prompt_bwd(q, k, v, *o, o[0], cu)))
        # the default stream, given by its number (zero), from another current one
        s.synchronize()
        o = gdn.attn_prompt(q, k, v, cu, stream=torch.cuda.default_stream().cuda_stream)
    named = gdn.attn_prompt(scale=None, cu_seqlens=cu, v=v, k=k, q=q, stream=s.cuda_stream)
    s.synchronize()
    torch.cuda.synchronize()
    got.append((*named, *grads))
    for r in got:
        for a, b in zip((*want, *grads), r):
            assert torch.equal(a, b)
    assert torch.equal(o[0], want[0])


def test_buffers_of_the_caller():
    """Outputs, statistics and workspace passed in: written in place and returned; a workspace that is too small, or
    tensors of other shapes, types and layouts are refused before anything is written."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    from test_gpu_attn_decode import make
    q, kc, vc, ks, vs, table, lens = make(torch, np.random.default_rng(4), [100, 3], 4, 2, 64, 16, "int8", extra_width=600)
    dev = [t.cuda() for t in (q, kc, vc, ks, vs)] + [ints(torch, table), ints(torch, lens)]
    want = gdn.attn_decode(*dev)
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    need = gdn.gdn_attn_decode_workspace_bytes(2, 4, 2, 64, 16, table.shape[1])
    got = gdn.attn_decode(*dev, out=out, lse=lse, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert got[0] is out and got[1] is lse and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(gdn.GdnError, match="WORKSPACE"):
        gdn.attn_decode(*dev, workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    x = torch_random(torch, np.random.default_rng(5), 20)
    q, k, v = x.split([HQ, H, H], 1)
    cu = ints(torch, [0, 20])
    for bad in (dict(q=q.float()), dict(k=k[:19]), dict(v=v.transpose(0, 1).contiguous().transpose(0, 1)), dict(q=q[:, :5]),
                dict(k=k.expand(20, H, D)[:1].expand(20, H, D)), dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu[:0]),
                dict(out=torch.zeros(20, HQ, D, device="cuda")), dict(lse=torch.zeros(20, HQ, device="cuda")),
                dict(q=x[:, ::2][:, :HQ])):
        with pytest.raises((ValueError, TypeError, gdn.GdnError)):
            gdn.attn_prompt(**{**dict(q=q, k=k, v=v, cu_seqlens=cu), **bad})
    with pytest.raises(gdn.GdnError, match="ALIGN"):
        gdn.attn_prompt(q, k, v, ints(torch, [7, 0, 20])[1:])


def test_empty_calls():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    x = torch.zeros(0, HQ + 2 * H, D, dtype=torch.bfloat16, device="cuda")
    q, k, v = x.split([HQ, H, H], 1)
    out, lse = gdn.attn_prompt(q, k, v, ints(torch, [0, 0]))
    assert out.shape == (0, HQ, D) and lse.shape == (HQ, 0)
    assert [g.shape[0] for g in gdn.attn_prompt_bwd(q, k, v, out, lse, out, ints(torch, [0]))] == [0, 0, 0]
    kc, ks = torch.zeros(3, H, BT, D, dtype=torch.int8, device="cuda"), torch.zeros(3, H, device="cuda")
    gdn.cache_append(k, v, ints(torch, []), kc, kc.clone(), ks, ks.clone())
    y = torch.zeros(2, HQ, D, dtype=torch.bfloat16, device="cuda")
    for table, lens in ((torch.zeros(2, 0), [5, 0]), (torch.zeros(2, 4), [0, 0])):  # no room for tokens, no tokens
        out, lse = gdn.attn_decode(y, kc, kc, ks, ks, table.int().cuda(), ints(torch, lens))
        assert (out == 0).all() and (lse == -float("inf")).all()
    none = kc[:0], kc[:0], ks[:0], ks[:0]
    out, lse = gdn.attn_decode(y, *none, ints(torch, [[0], [1]]), ints(torch, [4, 5]))
    assert (out == 0).all() and (lse == -float("inf")).all()
    # rows, but no sequence: zeros where the call allocates
    z = torch.full((9, HQ + 2 * H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, k, v = z.split([HQ, H, H], 1)
    for cu in ([0], [0, 0], [9, 9], [4, 4, 4]):
        out, lse = gdn.attn_prompt(q, k, v, ints(torch, cu))
        grads = gdn.attn_prompt_bwd(q, k, v, out, lse, out, ints(torch, cu))
        assert all((t == 0).all() for t in (out, lse, *grads))
