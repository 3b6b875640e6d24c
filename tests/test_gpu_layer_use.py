"""The layer operators as a program uses them: the layer of examples/tile_layer.py
on a plan's buffers against a 64-bit layer, experts dealt by a router, other
streams, graphs, far offsets, device arrays out of range, repeatability, gradients
against differences, and the binding's refusals."""
import importlib.util
import os

import pytest
import torch

import layer_reference as L
import overlap_tiling_trapezoidal_amd as tdp
import token_reference as R
from harness import note
from synth import WORKLOADS, Workload
from test_gpu_tokens import check

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAN = float("nan")

TWO = Workload("two_batches", 2, 64, (5, 6, 10), ((1, 0), (2, 2), (2, 2)), dtype="f32", seed=19)


def example():
    spec = importlib.util.spec_from_file_location("tile_layer", os.path.join(ROOT, "examples", "tile_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def f64(t):
    return t.detach().double().cpu()


@pytest.mark.parametrize("wl", [WORKLOADS["tiny"], TWO], ids=["tiny", "two_batches"])
def test_layer_on_a_plan(wl, cuda):
    """fp32 layer, forward and every gradient, against autograd in 64 bits on the used rows.  The chain's fp32
    errors: norms and products over C <= 64, heads * D = 256 and <= 500 rows, about 1e-6 of the largest magnitudes
    each; the bound is 2e-5 of the largest entry, 4e-5 behind all seven operators."""
    note(f"layer on {wl.name}")
    plan, bufs, layer, (y, saved, out), grads = example().run(wl, heads=4, kv_heads=2, head_dim=64, device=cuda)
    torch.cuda.synchronize()
    w = {n: f64(getattr(layer, n)).requires_grad_() for n in ("w_qkv", "w_out", "q_weight", "k_weight", "scale", "shift")}
    counts = bufs["tile_count"].repeat_interleave(wl.batch).tolist()
    ranges = tdp.tdp_plan_sequences(plan)
    used = torch.zeros(y.shape[0], dtype=torch.bool)
    for (a, _), n in zip(ranges, counts):
        used[a:a + n] = True
    x0 = f64(saved[0])
    x0[~used] = 0.0
    x = x0.requires_grad_()
    pos = bufs["tile_pos"].cpu()
    freqs = [[s * 10000.0 ** (-2.0 * i / r) for i in range(r // 2)] for r, s in
             zip(layer.rope.cfg.rot_dim, (1 / 8, 1 / 32, 1 / 32))]
    i0, i1 = R.pair_index(list(layer.rope.cfg.rot_dim), "interleaved")
    win = (layer.window.step, layer.window.back, layer.window.ahead, layer.window.sinks)
    want = torch.zeros(y.shape, dtype=torch.float64)
    for s, ((a, b), n) in enumerate(zip(ranges, counts)):
        t = x[a:a + n]
        d = t - t.mean(1, keepdim=True)
        t = d / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5) * w["scale"][s % wl.batch] + w["shift"][s % wl.batch]
        qkv = (t @ w["w_qkv"].T).view(n, 8, 64)
        p = pos[6 * a:6 * b].view(3, b - a, 2)[:, :n].double().mean(-1)
        ang = torch.cat([p[c][:, None] * torch.tensor(f, dtype=torch.float64) for c, f in enumerate(freqs)], 1)[:, None]

        def turned(t, weight):
            t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * weight
            c = t.clone()
            c[..., i0] = t[..., i0] * ang.cos() - t[..., i1] * ang.sin()
            c[..., i1] = t[..., i0] * ang.sin() + t[..., i1] * ang.cos()
            return c
        q, k, v = turned(qkv[:, :4], w["q_weight"]), turned(qkv[:, 4:6], w["k_weight"]), qkv[:, 6:]
        seen = L.visible(win, n, n)
        o = [torch.softmax((q[:, h] @ k[:, h // 2].T / 8.0).masked_fill(~seen, -float("inf")), 1) @ v[:, h // 2]
             for h in range(4)]
        want[a:a + n] = torch.cat(o, 1) @ w["w_out"].T
    (0.5 * want.square().sum()).backward()

    def close(name, g, r, tol=4e-5):
        err = (g - r).abs().max()
        assert err <= tol * r.abs().max(), f"{name}: {float(err)} of {float(r.abs().max())}"
    close("y", f64(y)[used], want[used].detach(), 2e-5)
    assert (f64(y)[~used] == 0).all() and torch.isfinite(out).all()
    for n in w:
        close(n, f64(grads[n]), w[n].grad)
    close("tile_lat", f64(grads["tile_lat"])[used], x.grad[used])


def test_experts_dealt_by_a_router(cuda):
    """Tokens sorted by expert on the GPU, two products per expert, no copy to the host; against each token's own."""
    n, C, H, E = 700, 128, 264, 9
    gen = torch.Generator(device=cuda).manual_seed(1)
    x = torch.randn(n, C, generator=gen, device=cuda)
    w1, w2 = (torch.randn(E, *s, generator=gen, device=cuda) * 0.1 for s in ((H, C), (C, H)))
    choice = (torch.rand(n, generator=gen, device=cuda).square() * (E - 1)).long()   # the last expert has none
    order = torch.argsort(choice, stable=True)
    start = torch.zeros(E + 1, dtype=torch.int64, device=cuda)
    start[1:] = torch.zeros(E, dtype=torch.int64, device=cuda).index_add_(0, choice, torch.ones_like(choice)).cumsum(0)
    seqs = tdp.Sequences(E, n, row_start=start, total_rows=n)
    xs, h, y = x[order], torch.empty(n, H, device=cuda), torch.empty(n, C, device=cuda)
    note("experts")
    tdp.tdp_grouped_product(seqs, xs, w1, h, workspace=tdp.allocate_grouped_product_workspace(seqs, E, H, C, "f32", cuda))
    tdp.tdp_grouped_product(seqs, h, w2, y, workspace=tdp.allocate_grouped_product_workspace(seqs, E, C, H, "f32", cuda))
    dw = torch.full_like(w2, NAN)
    ws = tdp.allocate_grouped_product_backward_workspace(seqs, E, C, H, "f32", cuda)
    tdp.tdp_grouped_product_backward(seqs, h, w2, y, None, dw, ws)
    torch.cuda.synchronize()
    for i in range(n):
        e, t = int(choice[order[i]]), f64(xs[i])
        hid, hb = L.product(t[None], f64(w1[e]), torch.float32)
        check("hidden", h[i:i + 1], hid, hb)
        check("y", y[i:i + 1], *L.product(f64(h[i:i + 1]), f64(w2[e]), torch.float32))
    for e in range(E):
        rows = slice(int(start[e]), int(start[e + 1]))
        g, t = f64(y[rows]), f64(h[rows])
        check("dw", dw[e], g.T @ t, (n + 24) * R.U32 * (g.abs().T @ t.abs()))


class Step:
    """All three operators, forward and backward, on fixed buffers."""

    def __init__(self, cuda, dt=torch.bfloat16, S=3, rows=260, C=256, hq=4, hk=2, D=64, seed=2):
        gen = torch.Generator(device=cuda).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen, device=cuda)  # noqa: E731
        n, N = S * rows, (hq + 2 * hk) * D
        self.lens = torch.tensor([rows, rows - 37, 5], dtype=torch.int32, device=cuda)
        self.seqs = tdp.Sequences(S, rows, seq_len=self.lens)
        self.x, self.g = r(n, C).to(dt), r(n, hq, D).to(dt)
        self.w, self.b, self.p = 1 + 0.1 * r(S, C), r(S, C), (r(S, N, C) / 16).to(dt)
        self.win = tdp.make_window(step=13, back=4, sinks=20)
        e = lambda *s, t=dt: torch.empty(*s, dtype=t, device=cuda)  # noqa: E731
        self.n, self.qkv, self.o, self.lse = e(n, C), e(n, hq + 2 * hk, D), e(n, hq, D), e(hq, n, t=torch.float32)
        self.dqkv, self.dn, self.dp = e(n, hq + 2 * hk, D), e(n, C), e(S, N, C, t=torch.float32)
        self.dx, self.dw, self.db = e(n, C), e(S, C, t=torch.float32), e(S, C, t=torch.float32)
        self.hq, self.hk, self.N, self.C = hq, hk, N, C
        q = self.seqs
        self.ws = [tdp.allocate_grouped_product_workspace(q, S, N, C, dt, cuda),
                   tdp.allocate_window_attention_workspace(q, q, self.win, hq, hk, D, cuda),
                   tdp.allocate_window_attention_backward_workspace(q, q, self.win, hq, hk, D, cuda),
                   tdp.allocate_grouped_product_backward_workspace(q, S, N, C, dt, cuda),
                   tdp.allocate_layer_norm_workspace(q, C, S, cuda)]

    def run(self, stream=None):
        s, hq, hk = self.seqs, self.hq, self.hk
        cut = lambda t: (t[:, :hq], t[:, hq:hq + hk], t[:, hq + hk:])  # noqa: E731
        tdp.tdp_layer_norm(s, self.x, self.w, self.b, self.n, stream=stream)
        tdp.tdp_grouped_product(s, self.n, self.p, self.qkv.view(-1, self.N), self.ws[0], stream=stream)
        tdp.tdp_window_attention(s, s, self.win, *cut(self.qkv), self.o, self.lse, workspace=self.ws[1], stream=stream)
        tdp.tdp_window_attention_backward(s, s, self.win, *cut(self.qkv), self.o, self.lse, self.g, *cut(self.dqkv),
                                          self.ws[2], stream=stream)
        tdp.tdp_grouped_product_backward(s, self.n, self.p, self.dqkv.view(-1, self.N), self.dn, self.dp, self.ws[3],
                                         stream=stream)
        tdp.tdp_layer_norm_backward(s, self.x, self.w, self.dn, self.dx, self.dw, self.db, self.ws[4], stream=stream)

    def results(self):
        return [t.clone() for t in (self.n, self.qkv, self.o, self.lse, self.dqkv, self.dn, self.dp, self.dx, self.dw,
                                    self.db)]

    def scramble(self):
        for t in (self.n, self.qkv, self.o, self.lse, self.dqkv, self.dn, self.dp, self.dx, self.dw, self.db, *self.ws):
            if t is not None:
                t.view(torch.uint8).fill_(0x5A)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_graph_replays_match_eager(dt, cuda):
    """One capture of the whole step, replayed with other inputs and lengths, eager work between the replays."""
    st, s = Step(cuda, dt), torch.cuda.Stream(cuda)
    note(f"graph of the step {dt}")
    st.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        st.run(torch.cuda.current_stream())
    for i in range(4):
        st.x.add_(0.25)
        st.lens.copy_(torch.tensor([260 - 7 * i, 100 + i, i], dtype=torch.int32))
        st.scramble()
        st.run()
        torch.cuda.synchronize()
        want = st.results()
        st.scramble()
        graph.replay()
        torch.cuda.synchronize()
        assert same(st.results(), want), f"replay {i}"
        assert all(torch.isfinite(t).all() for t in (st.dx, st.dp, st.dw))


def test_two_streams_and_repeats(cuda):
    """Two steps at once on streams of their own give what each gives alone, bit for bit, again and again."""
    a, b = Step(cuda, seed=3), Step(cuda, torch.float32, seed=4)
    note("two streams")
    a.run()
    b.run()
    torch.cuda.synchronize()
    want = a.results(), b.results()
    s, t = torch.cuda.Stream(cuda), torch.cuda.Stream(cuda)
    for _ in range(3):
        a.scramble()
        b.scramble()
        torch.cuda.synchronize()
        for _ in range(2):
            a.run(s)
            b.run(t)
        torch.cuda.synchronize()
        assert same(a.results(), want[0]) and same(b.results(), want[1])


def test_far_rows(cuda):
    """Sequences behind more than 2^31 elements, of rows, keys and weights."""
    C, rows, n = 2048, 1_100_000, 40
    gen = torch.Generator().manual_seed(6)
    big = torch.full((rows, C), NAN, dtype=torch.bfloat16, device=cuda)
    assert big.numel() > 2 ** 31
    x = torch.randn(n, C, generator=gen).bfloat16()
    big[-n:] = x.to(cuda)
    rr = torch.tensor([[rows - n, rows]], dtype=torch.int64, device=cuda)
    seqs = tdp.Sequences(1, n, row_range=rr, total_rows=rows)
    note("far rows: layer norm")
    y = torch.full_like(big, NAN)
    tdp.tdp_layer_norm(seqs, big, None, None, y)
    torch.cuda.synchronize()
    check("norm", y[-n:], *L.layer_norm(x, torch.ones(C), torch.zeros(C), 1e-5, torch.bfloat16))
    assert torch.isnan(y[-n - 1]).all()
    note("far rows: product")
    w = (torch.randn(64, C, generator=gen) / 45).bfloat16()
    out = torch.full((rows, 64), NAN, dtype=torch.bfloat16, device=cuda)
    ws = tdp.allocate_grouped_product_workspace(seqs, 1, 64, C, torch.bfloat16, cuda)
    tdp.tdp_grouped_product(seqs, big, w.to(cuda), out, workspace=ws)
    dx, dw = y, torch.empty(64, C, device=cuda)
    dy = torch.full_like(out, NAN)
    g = torch.randn(n, 64, generator=gen).bfloat16()
    dy[-n:] = g.to(cuda)
    ws = tdp.allocate_grouped_product_backward_workspace(seqs, 1, 64, C, torch.bfloat16, cuda)
    tdp.tdp_grouped_product_backward(seqs, big, w.to(cuda), dy, dx, dw, ws)
    torch.cuda.synchronize()
    check("product", out[-n:], *L.product(x, w, torch.bfloat16))
    check("dx", dx[-n:], *L.product(g, w.T, torch.bfloat16))
    g, x = g.double(), x.double()
    check("dw", dw, g.T @ x, (n + 24) * R.U32 * (g.abs().T @ x.abs()))
    del y, dx, out, dy
    note("far rows: window attention over a cache")
    kv = big.view(rows, 16, 128)
    kc = torch.randn(400, 16, 128, generator=gen).bfloat16()
    kv[-400:] = kc.to(cuda)
    rr = torch.tensor([[rows - 400, rows]], dtype=torch.int64, device=cuda)
    cache, new = tdp.Sequences(1, 400, row_range=rr, total_rows=rows), tdp.Sequences(1, 2)
    win = tdp.make_window(back=99, sinks=5)
    q = torch.randn(2, 8, 128, generator=gen).bfloat16()
    o = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=cuda)
    ws = tdp.allocate_window_attention_workspace(new, cache, win, 8, 8, 128, cuda)
    tdp.tdp_window_attention(new, cache, win, q.to(cuda), kv[:, :8], kv[:, 8:], o, workspace=ws)
    torch.cuda.synchronize()
    seen = L.visible((1, 99, 0, 5), 400, 2)
    for h in range(8):
        want, bound, *_ = L.window_attention(q[:, h], kc[:, h], kc[:, 8 + h], seen, 128 ** -0.5, torch.bfloat16)
        check("cache", o[:, h], want, bound)
    # many experts' weights: the last ones lie past 2^31 elements
    note("far weights")
    E, K, N = 9, 16384, 16384
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device=cuda)
    assert w[:-1].numel() >= 2 ** 31
    w[-1, -8:] = torch.randn(8, K, generator=gen).to(cuda).bfloat16()
    start = torch.tensor([0] * E + [3], dtype=torch.int64, device=cuda)
    seqs = tdp.Sequences(E, 3, row_start=start, total_rows=3)
    x = torch.randn(3, K, generator=gen).bfloat16()
    y = torch.empty(3, N, dtype=torch.bfloat16, device=cuda)
    ws = tdp.allocate_grouped_product_workspace(seqs, E, N, K, torch.bfloat16, cuda)
    tdp.tdp_grouped_product(seqs, x.to(cuda), w, y, workspace=ws)
    torch.cuda.synchronize()
    assert (y[:, :-8] == 0).all()
    check("y", y[:, -8:], *L.product(x, w[-1, -8:].cpu(), torch.bfloat16))


def test_device_arrays_out_of_range_are_clamped(cuda):
    """Ranges and lengths that leave the tensors: no access outside them, the rows inside as usual."""
    n, C = 100, 64
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(n, C, generator=gen)
    guard = torch.full((3 * n, C), 7.0, device=cuda)
    xd, y = x.to(cuda), guard[n:2 * n]
    rr = torch.tensor([[-50, 10], [10, 5], [20, 1000], [5000, 9000]], dtype=torch.int64, device=cuda)
    ln = torch.tensor([-3, 4, 1 << 30, 9], dtype=torch.int32, device=cuda)
    seqs = tdp.Sequences(4, n, row_range=rr, total_rows=n, seq_len=ln)
    one = torch.ones(C)
    note("clamped ranges")
    tdp.tdp_layer_norm(seqs, xd, None, None, y)
    torch.cuda.synchronize()
    check("norm", y[20:], *L.layer_norm(x[20:], one, 0 * one, 1e-5, torch.float32))
    assert (y[:10] == 0).all() and (y[10:20] == 7).all()
    y.fill_(7)
    w = torch.randn(2, C, C, generator=gen)
    ws = tdp.allocate_grouped_product_workspace(seqs, 2, C, C, "f32", cuda)
    tdp.tdp_grouped_product(seqs, xd, w.to(cuda), y, workspace=ws)
    dw = torch.empty(2, C, C, device=cuda)
    ws = tdp.allocate_grouped_product_backward_workspace(seqs, 2, C, C, "f32", cuda)
    tdp.tdp_grouped_product_backward(seqs, xd, w.to(cuda), xd, None, dw, ws)
    torch.cuda.synchronize()
    check("product", y[20:], *L.product(x[20:], w[0], torch.float32))
    assert (y[:10] == 0).all() and (y[10:20] == 7).all() and (dw[1] == 0).all()
    xx = x[20:].double()
    check("dw", dw[0], xx.T @ xx, 104 * R.U32 * (xx.abs().T @ xx.abs()))
    y.fill_(7)
    win, q = tdp.make_window(back=9, sinks=2), xd.view(n, 1, C)
    tdp.tdp_window_attention(seqs, seqs, win, q, q, q, y.view(n, 1, C))
    torch.cuda.synchronize()
    want, bound, *_ = L.window_attention(x[20:], x[20:], x[20:], L.visible((1, 9, 0, 2), 80, 80), C ** -0.5, torch.float32)
    check("window", y[20:], want, bound)
    assert (y[:10] == 0).all() and (y[10:20] == 7).all()
    assert (guard[:n] == 7).all() and (guard[2 * n:] == 7).all()


def test_gradients_against_differences(cuda):
    """<gradients, direction> of the product and of window attention against central differences in 64 bits."""
    gen = torch.Generator().manual_seed(10)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    # the difference's own error is h^2 = 1e-10 times third derivatives of the size of the values
    h = 1e-5
    n, K, N = 45, 72, 40
    x, w, g, vx, vw = r(n, K), r(N, K) / 8, r(n, N), r(n, K), r(N, K)
    f = lambda t: ((x.double() + t * vx) @ (w.double() + t * vw).T * g).sum()  # noqa: E731
    seqs = tdp.Sequences(1, n)
    dx, dw = torch.empty(n, K, device=cuda), torch.empty(N, K, device=cuda)
    ws = tdp.allocate_grouped_product_backward_workspace(seqs, 1, N, K, "f32", cuda)
    note("product differences")
    tdp.tdp_grouped_product_backward(seqs, x.to(cuda), w.to(cuda), g.to(cuda), dx, dw, ws)
    torch.cuda.synchronize()
    terms = f64(dx) * vx, f64(dw) * vw
    got, mag = sum(t.sum() for t in terms), sum(t.abs().sum() for t in terms)
    assert abs(got - (f(h) - f(-h)) / (2 * h)) <= 1e-6 * mag

    n, hq, hk, D, win = 90, 4, 2, 32, (9, 2, 1, 12)
    q, k, v, g = r(n, hq, D), r(n, hk, D), r(n, hk, D), r(n, hq, D)
    vq, vk, vv = r(n, hq, D), r(n, hk, D), r(n, hk, D)
    seen = L.visible(win, n, n)

    def f(t):
        qq, kk, vv_ = q.double() + t * vq, k.double() + t * vk, v.double() + t * vv
        s = 0.0
        for i in range(hq):
            p = torch.softmax((qq[:, i] @ kk[:, i // 2].T * D ** -0.5).masked_fill(~seen, -float("inf")), 1)
            s = s + (p @ vv_[:, i // 2] * g[:, i]).sum()
        return s
    seqs, wd = tdp.Sequences(1, n), tdp.make_window(*win)
    dev = [t.to(cuda) for t in (q, k, v)]
    o, lse = torch.empty(n, hq, D, device=cuda), torch.empty(hq, n, device=cuda)
    grads = [torch.empty_like(t) for t in dev]
    note("window differences")
    tdp.tdp_window_attention(seqs, seqs, wd, *dev, o, lse)
    ws = tdp.allocate_window_attention_backward_workspace(seqs, seqs, wd, hq, hk, D, cuda)
    tdp.tdp_window_attention_backward(seqs, seqs, wd, *dev, o, lse, g.to(cuda), *grads, ws)
    torch.cuda.synchronize()
    terms = [f64(a) * b for a, b in zip(grads, (vq, vk, vv))]
    got, mag = sum(t.sum() for t in terms), sum(t.abs().sum() for t in terms)
    assert abs(got - (f(h) - f(-h)) / (2 * h)) <= 1e-6 * mag


def test_binding_refuses(cuda):
    """Tensors that do not fit are refused before anything is enqueued."""
    s = tdp.Sequences(2, 10)
    x, y, w = torch.zeros(20, 64, device=cuda), torch.zeros(20, 64, device=cuda), torch.ones(64, device=cuda)
    ws = tdp.allocate_layer_norm_workspace(s, 64, 1, cuda)
    p, dw = torch.zeros(2, 64, 64, device=cuda), torch.zeros(2, 64, 64, device=cuda)
    bad = [
        lambda: tdp.tdp_layer_norm(s, x[:19], w, None, y),
        lambda: tdp.tdp_layer_norm(s, x.cpu(), w, None, y),
        lambda: tdp.tdp_layer_norm(s, x, w, None, y.bfloat16()),
        lambda: tdp.tdp_layer_norm(s, x, w[:32], None, y),
        lambda: tdp.tdp_layer_norm(s, x, w.double(), None, y),
        lambda: tdp.tdp_layer_norm(s, x, torch.ones(3, 64, device=cuda), None, y),
        lambda: tdp.tdp_layer_norm(s, x, w, torch.ones(2, 64, device=cuda), y),
        lambda: tdp.tdp_layer_norm(s, x, w, None, x[:1].expand(20, 64)),
        lambda: tdp.tdp_layer_norm(s, x.t().contiguous().t(), w, None, y),
        lambda: tdp.tdp_layer_norm(s, x, w, None, None),
        lambda: tdp.tdp_layer_norm(s, x.half(), w, None, y.half()),
        lambda: tdp.tdp_layer_norm_backward(s, x, w, x, y, w, w, ws[:64]),
        lambda: tdp.tdp_layer_norm_backward(s, x, w, x, y, w, w, None),
        lambda: tdp.allocate_layer_norm_workspace(s, 60, 1, cuda),
        lambda: tdp.tdp_grouped_product(s, x, p[0, 0], y),
        lambda: tdp.tdp_grouped_product(s, x, p[:, :, :32], y),
        lambda: tdp.tdp_grouped_product(s, x, p.bfloat16(), y),
        lambda: tdp.tdp_grouped_product(s, x, torch.zeros(3, 64, 64, device=cuda), y),
        lambda: tdp.tdp_grouped_product(s, x, p, y[:, :32]),
        lambda: tdp.tdp_grouped_product(s, x, p.transpose(1, 2), y),
        lambda: tdp.tdp_grouped_product_backward(s, x, p, x, y, dw.bfloat16()),
        lambda: tdp.tdp_grouped_product_backward(s, x, p, x, y, dw[0]),
        lambda: tdp.tdp_grouped_product_backward(s, x, p, x, y[:5], dw),
        lambda: tdp.tdp_window_attention(s, s, tdp.make_window(step=0), *[x.view(20, 2, 32)] * 3, y.view(20, 2, 32)),
        lambda: tdp.tdp_window_attention(s, s, tdp.make_window(back=-2), *[x.view(20, 2, 32)] * 3, y.view(20, 2, 32)),
        lambda: tdp.tdp_window_attention(s, tdp.Sequences(1, 20), tdp.make_window(), *[x.view(20, 2, 32)] * 3,
                                         y.view(20, 2, 32)),
        lambda: tdp.tdp_window_attention_backward(s, s, tdp.make_window(), *[x.view(20, 2, 32)] * 4, None,
                                                  *[x.view(20, 2, 32)] * 4, ws),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, tdp.TdpError)):
            call()
            raise AssertionError(f"call {i} was not refused")
    torch.cuda.synchronize()
    assert (y == 0).all()
