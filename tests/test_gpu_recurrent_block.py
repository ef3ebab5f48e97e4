"""A recurrent block of a hybrid as a user runs it: norm with the residual, projection, short convolution, scan (or the
delta rule), norm of the next block; prompts, then single tokens; its gradients; on other streams, captured and replayed."""
import numpy as np
import pytest

from gpu_util import down, note, torch_dev
from oracle import block as ref

pytestmark = pytest.mark.gpu

WIDTH, H, P, G, N, TAPS = 256, 4, 64, 1, 64, 4
INNER, CONV = H * P, H * P + 2 * G * N


class Block:
    """One layer's parameters and calls; the projections are torch products."""

    def __init__(self, torch, seed=0):
        import linear_attention_sequence_gated_amd as gdn
        self.torch, self.gdn = torch, gdn
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.norm_w, self.next_w = (1 + 0.1 * r(WIDTH)).bfloat16(), (1 + 0.1 * r(WIDTH)).bfloat16()
        self.w_in, self.w_out = (r(CONV + 8, WIDTH) * WIDTH ** -0.5).bfloat16(), (r(WIDTH, INNER) * INNER ** -0.5).bfloat16()
        self.conv_w, self.conv_b = (r(CONV, TAPS) * 0.5).bfloat16(), (0.1 * r(CONV)).bfloat16()
        self.a, self.D, self.bias = -1 - 3 * torch.rand(H, generator=g, device="cuda"), r(H), r(H) - 2

    def split(self, rows):
        t = rows.shape[0]
        x, B, C = rows.split([INNER, G * N, G * N], 1)
        return x.view(t, H, P), B.view(t, G, N), C.view(t, G, N)

    def prompt(self, hidden, residual, cu):
        gdn = self.gdn
        y, res = gdn.rms_norm(hidden, self.norm_w, residual)
        z = y @ self.w_in.t()
        rows, conv_state = gdn.short_conv(z[:, :CONV], self.conv_w, cu, bias=self.conv_b)
        x, B, C = self.split(rows)
        out, S = gdn.ssm_scan(x, z[:, CONV:CONV + H], self.a, B, C, cu, D=self.D, dt_bias=self.bias)
        codes, scale, res = gdn.rms_norm_quant(out.view(-1, INNER) @ self.w_out.t(), self.next_w, res)
        return codes, scale, res, conv_state, S

    def token(self, hidden, residual, conv_state, S):
        gdn = self.gdn
        y, res = gdn.rms_norm(hidden, self.norm_w, residual)
        z = y @ self.w_in.t()
        x, B, C = self.split(gdn.short_conv_step(z[:, :CONV], self.conv_w, conv_state, bias=self.conv_b))
        out = gdn.ssm_step(x, z[:, CONV:CONV + H], self.a, B, C, S, D=self.D, dt_bias=self.bias)
        return gdn.rms_norm_quant(out.view(-1, INNER) @ self.w_out.t(), self.next_w, res)


def value(codes, scale):
    return (codes.float().view(*scale.shape, -1) * scale[..., None]).view(codes.shape)


def reference(b, hidden, residual, cu):
    """The same in 64 bits, from the numbers that the parameters hold; roundings of rows between the operators as there."""
    import torch
    d = lambda t: down(t).astype(np.float64)  # noqa: E731
    bf = lambda v: d(torch.from_numpy(v.astype(np.float32)).bfloat16())  # noqa: E731
    s = bf(d(hidden) + d(residual))
    y = bf(ref.rms_norm(s, d(b.norm_w), 1e-6)[0])
    z = bf(y @ d(b.w_in).T)
    rows = bf(ref.short_conv(z[:, :CONV], d(b.conv_w), d(b.conv_b), cu)[0])
    t = len(rows)
    x, B, C = rows[:, :INNER].reshape(t, H, P), rows[:, INNER:INNER + G * N].reshape(t, G, N), rows[:, INNER + G * N:].reshape(t, G, N)
    out, S = ref.ssm_scan(x, z[:, CONV:CONV + H], d(b.a), B, C, d(b.D), d(b.bias), cu)
    h = bf(bf(out).reshape(t, INNER) @ d(b.w_out).T)
    s2 = bf(h + s)
    return ref.rms_norm(s2, d(b.next_w), 1e-6)[0], S


def test_prompt_then_tokens():
    torch = torch_dev()
    b = Block(torch)
    cu, more = [0, 70, 71, 200], 5
    g = torch.Generator(device="cuda").manual_seed(3)
    full = [n + more for n in np.diff(cu)]
    cu_full = np.concatenate([[0], np.cumsum(full)])
    hidden, residual = (torch.randn(cu_full[-1], WIDTH, generator=g, device="cuda").bfloat16() for _ in range(2))
    begin = torch.cat([torch.arange(cu_full[i], cu_full[i] + n) for i, n in enumerate(np.diff(cu))]).cuda()
    codes, scale, _, conv_state, S = b.prompt(hidden[begin], residual[begin], torch.tensor(cu, dtype=torch.int32, device="cuda"))
    got = torch.zeros(cu_full[-1], WIDTH, device="cuda")
    got[begin] = value(codes, scale)
    for i in range(more):
        at = torch.tensor([cu_full[r] + n + i for r, n in enumerate(np.diff(cu))], device="cuda")
        codes, scale, _ = b.token(hidden[at], residual[at], conv_state, S)
        got[at] = value(codes, scale)
    want, S_want = reference(b, hidden, residual, cu_full)
    # e4m3 rounds to half a step, 2^-4 of a value at most, 2^-4 / sqrt(3) in the root mean square; the bf16 rows before it 2^-8 each
    rel = np.linalg.norm(down(got) - want) / np.linalg.norm(want)
    relS = np.linalg.norm(down(S) - S_want) / np.linalg.norm(S_want)
    print(f"[parity] block: {rel:.2e}, states {relS:.2e}", flush=True)
    assert rel <= 2.0 ** -4 / 3 ** 0.5 + 2.0 ** -6 and relS <= 2.0 ** -6


def test_convolution_before_the_delta_rule():
    """q, k and v of the delta-rule layer from one projection through one convolution."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    import oracle
    from oracle.prologue import prologue_fwd
    T, heads, d = 96, 3, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    z = torch.randn(T, 3 * heads * d, generator=g, device="cuda").bfloat16()
    w = (torch.randn(3 * heads * d, 4, generator=g, device="cuda") * 0.5).bfloat16()
    rows, _ = gdn.short_conv(z, w, torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    q, k, v = (x.reshape(1, T, heads, d).contiguous() for x in rows.split(heads * d, 1))
    a, bt = (torch.randn(1, T, heads, generator=g, device="cuda") for _ in range(2))
    out, S = gdn.chunk_fwd_prologue(q, k, v, a, bt, 1.0)
    n = lambda t: down(t)  # noqa: E731
    want, S_want = prologue_fwd(n(q), n(k), n(v), n(a), n(bt), 1.0)
    assert np.linalg.norm(down(out) - want) <= 2e-2 * np.linalg.norm(want) and np.linalg.norm(down(S) - S_want) <= 2e-2 * np.linalg.norm(S_want)
    conv, _, _ = ref.short_conv(down(z).astype(np.float64), down(w).astype(np.float64), np.zeros(3 * heads * d), [0, T])
    assert np.linalg.norm(down(rows) - conv) <= 4e-3 * np.linalg.norm(conv)


def test_gradients_through_the_block():
    """conv -> scan -> norm: the gradients chained, against the references' chained."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    cu, t = [0, 50, 51, 130], 130
    g = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    z, cw, cb = r(t, CONV).bfloat16(), (0.5 * r(CONV, TAPS)).bfloat16(), (0.1 * r(CONV)).bfloat16()
    dt, a, D, bias, nw = r(t, H), -1 - r(H).abs(), r(H), r(H) - 2, 1 + 0.1 * r(INNER)
    go = r(t, INNER).bfloat16()
    offs = torch.tensor(cu, dtype=torch.int32, device="cuda")
    rows, _ = gdn.short_conv(z, cw, offs, bias=cb)
    x, B, C = rows[:, :INNER].view(t, H, P), rows[:, INNER:INNER + G * N].view(t, G, N), rows[:, INNER + G * N:].view(t, G, N)
    y, _ = gdn.ssm_scan(x, dt, a, B, C, offs, D=D, dt_bias=bias)
    gy, gnw = gdn.rms_norm_bwd(y.view(t, INNER), nw, go)
    grows = torch.empty_like(rows)
    parts = grows[:, :INNER].view(t, H, P), grows[:, INNER:INNER + G * N].view(t, G, N), grows[:, INNER + G * N:].view(t, G, N)
    gx, gdt, ga, gB, gC, gD, gbias, _ = gdn.ssm_scan_bwd(x, dt, a, B, C, gy.view(t, H, P), offs, D=D, dt_bias=bias, grad_x=parts[0],
                                                        grad_B=parts[1], grad_C=parts[2])
    gz, gcw, gcb, _ = gdn.short_conv_bwd(z, cw, grows, offs, bias=cb)
    d = lambda v: down(v).astype(np.float64)  # noqa: E731
    c_rows = d(rows)
    c_in = c_rows[:, :INNER].reshape(t, H, P), c_rows[:, INNER:INNER + G * N].reshape(t, G, N), c_rows[:, INNER + G * N:].reshape(t, G, N)
    wy, wnw, _ = ref.rms_norm_bwd(d(y).reshape(t, INNER), d(nw), 1e-6, d(go))
    w = ref.ssm_scan_bwd(c_in[0], d(dt), d(a), c_in[1], c_in[2], d(D), d(bias), cu, wy.reshape(t, H, P))
    wrows = np.concatenate([w[0].reshape(t, -1), w[3].reshape(t, -1), w[4].reshape(t, -1)], 1)
    (wz, wcw, wcb, _), _ = ref.short_conv_bwd(d(z), d(cw), d(cb), cu, wrows)
    # rows of bf16 between the operators, and inside the scan, each 2^-8 / sqrt(3) off at most in the mean square: four of them
    for name, u, v in (("norm", gnw, wnw), ("z", gz, wz), ("conv weight", gcw, wcw), ("conv bias", gcb, wcb), ("D", gD, w[5]), ("a", ga, w[2]),
                       ("bias", gbias, w[6]), ("dt", gdt, w[1])):
        rel = np.linalg.norm(down(u) - v) / np.linalg.norm(v)
        print(f"[parity] {name}: {rel:.2e}", flush=True)
        assert rel <= 4 * 2.0 ** -8, name


def test_on_another_stream_and_captured():
    """A step of the block on a stream of its own, then captured: every replay gives the eager result, with new inputs in the
    same places, the program's own work between the replays, and another graph's replay in between."""
    torch = torch_dev()
    b = Block(torch)
    R = 3
    g = torch.Generator(device="cuda").manual_seed(1)
    hidden, residual = (torch.randn(R, WIDTH, generator=g, device="cuda").bfloat16() for _ in range(2))
    conv0, S0 = torch.randn(R, TAPS - 1, CONV, generator=g, device="cuda").bfloat16(), torch.randn(R, H, N, P, generator=g, device="cuda")
    cu = torch.tensor([0, 90, 200], dtype=torch.int32, device="cuda")
    ph, pr = (torch.randn(200, WIDTH, generator=g, device="cuda").bfloat16() for _ in range(2))

    def token(h, r):
        conv, S = conv0.clone(), S0.clone()
        codes, scale, res = b.token(h, r, conv, S)
        return [codes.view(torch.int8), scale, res, conv, S]

    def prompt(h, r):
        codes, *rest = b.prompt(h, r, cu)
        return [codes.view(torch.int8), *rest]

    for call, h, r in ((token, hidden, residual), (prompt, ph, pr)):
        want = call(h, r)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = call(h, r)
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(u, v) for u, v in zip(want, other))
        graphs = []
        for _ in range(2):
            hh, rr = h.clone(), r.clone()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = call(hh, rr)
            graphs.append((graph, hh, rr, got))
        for i in range(3):
            for k, (graph, hh, rr, got) in enumerate(graphs):
                h2, r2 = (h * (1 + i + k)).bfloat16(), (r - i).bfloat16()
                hh.copy_(h2), rr.copy_(r2)
                graph.replay()
                now = [v.clone() for v in got]
                eager = call(h2, r2)
                torch.cuda.synchronize()
                assert all(torch.equal(u, v) for u, v in zip(now, eager)), (call.__name__, i, k)


def test_gradients_captured():
    """The backward calls in a graph: replays with new gradients give the eager results."""
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    t, cu = 600, torch.tensor([0, 300, 301, 600], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, B, C, dt = r(t, H, P).bfloat16(), r(t, G, N).bfloat16(), r(t, G, N).bfloat16(), r(t, H).bfloat16()
    a, D, bias = -1 - r(H).abs(), r(H), r(H) - 2
    w, nw, go = r(INNER, TAPS), 1 + 0.1 * r(INNER), r(t, H, P).bfloat16()

    def grads(go):
        flat = go.view(t, INNER)
        return [*gdn.ssm_scan_bwd(x, dt, a, B, C, go, cu, D=D, dt_bias=bias)[:7], *gdn.short_conv_bwd(x.view(t, INNER), w, flat, cu)[:2],
                *gdn.rms_norm_bwd(x.view(t, INNER), nw, flat)]

    want = grads(go)
    buf = go.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = grads(buf)
    for i in range(3):
        new = (go * (1 + i)).bfloat16()
        buf.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        eager = grads(new)
        assert all(torch.equal(u, v) for u, v in zip(got, eager)), i
        if i == 0:
            assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_stream_argument():
    torch = torch_dev()
    import linear_attention_sequence_gated_amd as gdn
    x, w = torch.randn(40, 64, device="cuda"), torch.ones(64, device="cuda")
    want, _ = gdn.rms_norm(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = gdn.rms_norm(x, w, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want)
