"""The token operators as a program uses them: the layer of
examples/tile_attention.py on a plan's buffers against a 64-bit layer, other
streams, graphs, 4-D tensors, repeatability, long offsets, device arrays out of
range, very negative scores, gradients against differences, and the binding's
refusals."""
import importlib.util
import math
import os

import pytest
import torch

import overlap_tiling_trapezoidal_amd as tdp
import test_gpu_tokens as G
import token_reference as R
from harness import note
from synth import WORKLOADS, Workload

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAN = float("nan")

SMALL_COND = Workload("small_cond", 2, 64, (4, 8, 10), ((2, 1), (2, 2), (2, 2)), num_cond=96, num_ref=24,
                      dtype="f32", seed=9)


def example():
    spec = importlib.util.spec_from_file_location("tile_attention", os.path.join(ROOT, "examples", "tile_attention.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("wl", [WORKLOADS["tiny"], SMALL_COND], ids=["tiny", "small_cond"])
def test_layer_on_a_plan(wl, cuda):
    """fp32 layer, forward and every gradient, against autograd in 64 bits on the used rows.  The chain's fp32
    errors: products over C <= 64, heads * D = 256 and <= 500 keys, about 1e-6 of the largest magnitudes each; the
    bound is 2e-5 of the largest entry."""
    note(f"layer on {wl.name}")
    plan, bufs, layer, (y, saved, out), grads = example().run(wl, heads=4, kv_heads=2, head_dim=64, device=cuda)
    torch.cuda.synchronize()
    f64 = lambda t: t.detach().double().cpu()  # noqa: E731
    w = {n: f64(getattr(layer, n)).requires_grad_() for n in ("w_qkv", "w_out", "q_weight", "k_weight")}
    x = f64(saved[0]).requires_grad_()
    pos = bufs["tile_pos"].cpu()
    freqs = [[s * 10000.0 ** (-2.0 * i / r) for i in range(r // 2)] for r, s in
             zip(layer.rope.cfg.rot_dim, (1 / 8, 1 / 32, 1 / 32))]
    i0, i1 = R.pair_index(list(layer.rope.cfg.rot_dim), "interleaved")
    counts = bufs["tile_count"].repeat_interleave(wl.batch).tolist()
    want, used = torch.zeros(y.shape, dtype=torch.float64), torch.zeros(y.shape[0], dtype=torch.bool)
    for (a, b), n in zip(tdp.tdp_plan_sequences(plan), counts):
        qkv = (x[a:a + n] @ w["w_qkv"].T).view(n, 8, 64)
        p = pos[6 * a:6 * b].view(3, b - a, 2)[:, :n].double().mean(-1)
        ang = torch.cat([p[d][:, None] * torch.tensor(f, dtype=torch.float64) for d, f in enumerate(freqs)], 1)[:, None]

        def turned(t, weight):
            t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * weight
            c = t.clone()
            c[..., i0] = t[..., i0] * ang.cos() - t[..., i1] * ang.sin()
            c[..., i1] = t[..., i0] * ang.sin() + t[..., i1] * ang.cos()
            return c
        q, k, v = turned(qkv[:, :4], w["q_weight"]), turned(qkv[:, 4:6], w["k_weight"]), qkv[:, 6:]
        o = torch.cat([torch.softmax(q[:, h] @ k[:, h // 2].T / 8.0, 1) @ v[:, h // 2] for h in range(4)], 1)
        want[a:a + n] = o @ w["w_out"].T
        used[a:a + n] = True
    (0.5 * want.square().sum()).backward()
    got = f64(y)

    def close(name, g, r):
        err = (g - r).abs().max()
        assert err <= 2e-5 * r.abs().max(), f"{name}: {float(err)} of {float(r.abs().max())}"
    close("y", got[used], want[used].detach())
    assert torch.isfinite(out).all()
    for n in w:
        close(n, f64(grads[n]), w[n].grad)
    close("tile_lat", f64(grads["tile_lat"])[used], x.grad[used])


def attn_inputs(cuda, dt=torch.bfloat16, n=300, hq=4, hk=2, D=64, seed=3):
    gen = torch.Generator().manual_seed(seed)
    seqs = tdp.Sequences(2, n, seq_len=torch.tensor([n, n - 37], dtype=torch.int32, device=cuda))
    q = torch.randn(2 * n, hq, D, generator=gen).to(dt).to(cuda)
    k, v = (torch.randn(2 * n, hk, D, generator=gen).to(dt).to(cuda) for _ in range(2))
    return seqs, q, k, v


def forward_backward(seqs, q, k, v, g, ws, wsb, stream=None):
    out, lse = torch.empty_like(q), torch.empty(q.shape[1], q.shape[0], device=q.device)
    grads = [torch.empty_like(t) for t in (q, k, v)]

    def call():
        tdp.tdp_attention(seqs, seqs, q, k, v, out, lse, workspace=ws, stream=stream)
        tdp.tdp_attention_backward(seqs, seqs, q, k, v, out, lse, g, *grads, wsb, stream=stream)
    return call, [out, lse, *grads]


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph(cuda):
    seqs, q, k, v = attn_inputs(cuda)
    g = torch.randn_like(q)
    ws = tdp.allocate_attention_workspace(seqs, seqs, 4, 2, 64, cuda)
    wsb = tdp.allocate_attention_backward_workspace(seqs, seqs, 4, 2, 64, cuda)
    rope = tdp.tdp_rope_create(tdp.make_rope_config(64, (24, 20, 20)))
    pos = torch.rand(6 * seqs.total_rows, device=cuda) * 100
    w = torch.rand(64, device=cuda)
    wsn = tdp.allocate_qk_norm_rope_workspace(rope, seqs, 4, 2, cuda)
    nq, nk = torch.empty_like(q), torch.empty_like(k)
    dn = [torch.empty_like(q), torch.empty_like(k), torch.empty(64, device=cuda), torch.empty(64, device=cuda)]
    attn, outs = forward_backward(seqs, nq, nk, v, g, ws, wsb)

    def call(stream=None):
        tdp.tdp_qk_norm_rope(rope, seqs, pos, q, k, w, w, nq, nk, stream=stream)
        if stream is None:
            attn()
        tdp.tdp_qk_norm_rope_backward(rope, seqs, pos, q, k, w, w, nq, nk, *dn, wsn, stream=stream)
    note("eager")
    call()
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs + dn + [nq, nk]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in dn + [nq, nk]:
        t.fill_(NAN)
    side.wait_stream(torch.cuda.current_stream())
    note("another stream")
    call(stream=side)
    torch.cuda.synchronize()
    for t, r in zip(dn + [nq, nk], ref[len(outs):]):
        assert torch.equal(t, r)
    note("capture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        for t in outs + dn + [nq, nk]:
            t.fill_(NAN)
        note(f"replay {i}")
        graph.replay()
        torch.cuda.synchronize()
        for t, r in zip(outs + dn + [nq, nk], ref):
            assert torch.equal(t, r)
        (q.float().sum() + 1).item()   # the program's own work between replays


def test_four_dimensional_and_broadcast_tensors(cuda):
    """(S, T, H, D) and head-major tensors give the packed form's bits; a key head broadcast over sequences and rows
    of stride 0 are read as what they stand for."""
    S, T, D = 2, 70, 64
    gen = torch.Generator().manual_seed(8)
    seqs = tdp.Sequences(S, T, seq_len=torch.tensor([T, 41], dtype=torch.int32, device=cuda))
    q, k, v, g = (torch.randn(S * T, 2, D, generator=gen).to(cuda) for _ in range(4))
    ws = tdp.allocate_attention_backward_workspace(seqs, seqs, 2, 2, D, cuda)

    def run(q, k, v, g, like):
        out, lse = like(), torch.empty(2, S * T, device=cuda)
        grads = [like() for _ in range(3)]
        note("attention")
        tdp.tdp_attention(seqs, seqs, q, k, v, out, lse)
        tdp.tdp_attention_backward(seqs, seqs, q, k, v, out, lse, g, *grads, ws)
        torch.cuda.synchronize()
        return [t.reshape(S * T, 2, D) for t in (out, *grads)]
    flat = run(q, k, v, g, lambda: torch.empty(S * T, 2, D, device=cuda))
    four = [t.view(S, T, 2, D) for t in (q, k, v, g)]
    for a, b in zip(flat, run(*four, lambda: torch.empty(S, T, 2, D, device=cuda))):
        assert torch.equal(a, b)
    major = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in four]
    for a, b in zip(flat, run(*major, lambda: torch.empty(S, 2, T, D, device=cuda).transpose(1, 2))):
        assert torch.equal(a, b)
    # one key and value row for all rows, sequences and heads: their expanded and their copied form
    one = [torch.randn(1, 1, 1, D, generator=gen).to(cuda).expand(S, T, 2, D) for _ in range(2)]
    mk = lambda: torch.empty(S, T, 2, D, device=cuda)  # noqa: E731
    for a, b in zip(run(four[0], *one, four[3], mk), run(four[0], *[t.contiguous() for t in one], four[3], mk)):
        assert torch.equal(a, b)
    # queries and their gradients of stride 0
    ones = [torch.randn(1, 1, 1, D, generator=gen).to(cuda).expand(S, T, 2, D) for _ in range(2)]
    for a, b in zip(run(ones[0], *four[1:3], ones[1], mk),
                    run(ones[0].contiguous(), *four[1:3], ones[1].contiguous(), mk)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_scores_far_below_zero(dt, cuda):
    """Every score near -400: weights are recomputed from an lse whose negative would overflow exp on the padding of
    a key block (70 keys in blocks of 32 and 64)."""
    gen = torch.Generator().manual_seed(4)
    n, D = 70, 64
    seqs = tdp.Sequences(1, n)
    base = torch.full((n, 1, D), 7.0)
    q = (base + 0.25 * torch.randn(n, 1, D, generator=gen)).to(dt)
    k = (-base + 0.25 * torch.randn(n, 1, D, generator=gen)).to(dt)
    v, g = (torch.randn(n, 1, D, generator=gen).to(dt) for _ in range(2))
    dev = [t.to(cuda) for t in (q, k, v, g)]
    out, lse = torch.empty_like(dev[0]), torch.empty(1, n, device=cuda)
    grads = [torch.empty_like(dev[0]) for _ in range(3)]
    note("far scores")
    tdp.tdp_attention(seqs, seqs, *dev[:3], out, lse)
    tdp.tdp_attention_backward(seqs, seqs, *dev[:3], out, lse, dev[3], *grads,
                               tdp.allocate_attention_backward_workspace(seqs, seqs, 1, 1, D, cuda))
    torch.cuda.synchronize()
    assert lse.max() < -300
    o, ob, _, _ = R.attention(q[:, 0], k[:, 0], v[:, 0], None, D ** -0.5, dt)
    G.check("out", out[:, 0], o, ob)
    r = R.attention(q[:, 0], k[:, 0], v[:, 0], None, D ** -0.5, dt, out.cpu()[:, 0], g[:, 0])
    for name, t in zip(("dq", "dk", "dv"), grads):
        G.check(name, t[:, 0], *r[name])


def test_device_arrays_out_of_range_are_clamped(cuda):
    """Ranges past the tensors or reversed and lengths below zero or past the range: as their clamped values."""
    D, rows = 64, 64
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(rows, 1, D, generator=gen).to(cuda) for _ in range(3))
    bad = tdp.Sequences(4, 40, row_range=torch.tensor([[-5, 20], [30, 20], [20, 50], [50, 900]], device=cuda),
                        total_rows=rows, seq_len=torch.tensor([99, 7, -3, 14], dtype=torch.int32, device=cuda))
    good = tdp.Sequences(4, 40, row_range=torch.tensor([[0, 20], [30, 30], [20, 50], [50, 64]], device=cuda),
                         total_rows=rows, seq_len=torch.tensor([20, 0, 0, 14], dtype=torch.int32, device=cuda))
    rope = tdp.tdp_rope_create(tdp.make_rope_config(D, (24, 20, 20)))
    pos = torch.rand(6 * rows, device=cuda)
    res = []
    for s in (bad, good):
        out, y = torch.full_like(q, -1.0), torch.full_like(q, -1.0)
        note("clamped")
        tdp.tdp_rope_apply(rope, s, pos, q, y)
        tdp.tdp_attention(s, s, q, k, v, out, workspace=tdp.allocate_attention_workspace(s, s, 1, 1, D, cuda))
        torch.cuda.synchronize()
        res.append((out, y))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert (res[0][0][20:50] == 0).all()


def test_offsets_past_32_bits(cuda):
    """Tensors of more than 2^31 elements: the last rows turned, attended and differentiated as they are alone."""
    n, H, D = 140_000, 128, 128                      # 2.29e9 elements of bf16
    x = torch.zeros(n, H, D, dtype=torch.bfloat16, device=cuda)
    tail = 200
    gen = torch.Generator(device=cuda).manual_seed(1)
    x[-tail:] = torch.randn(tail, H, D, generator=gen, device=cuda)
    ranges = torch.tensor([[0, 5], [n - tail, n]], device=cuda)
    long = tdp.Sequences(2, tail, row_range=ranges, total_rows=n)
    short = tdp.Sequences(1, tail)
    rope = tdp.tdp_rope_create(tdp.make_rope_config(D, (44, 42, 42)))
    pos = torch.rand(6 * n, device=cuda)
    y = torch.empty_like(x)
    note("rope past 2^31")
    tdp.tdp_rope_apply(rope, long, pos, x, y)
    ref = torch.empty_like(x[-tail:])
    tdp.tdp_rope_apply(rope, short, pos[6 * (n - tail):], x[-tail:].contiguous(), ref)
    torch.cuda.synchronize()
    assert torch.equal(y[-tail:], ref)
    lse, lse1 = torch.empty(H, n, device=cuda), torch.empty(H, tail, device=cuda)
    note("attention past 2^31")
    tdp.tdp_attention(long, long, x, x, x, y, lse)
    out = torch.empty_like(ref)
    xs = x[-tail:].contiguous()
    tdp.tdp_attention(short, short, xs, xs, xs, out, lse1)
    torch.cuda.synchronize()
    assert torch.equal(y[-tail:], out) and torch.equal(lse[:, -tail:], lse1)
    g = torch.empty_like(x)
    grads = [torch.empty_like(ref) for _ in range(3)]
    note("gradients past 2^31")
    tdp.tdp_attention_backward(short, short, xs, xs, xs, out, lse1, out, *grads,
                               tdp.allocate_attention_backward_workspace(short, short, H, H, D, cuda))
    ws = tdp.allocate_attention_backward_workspace(long, long, H, H, D, cuda)
    g2, g3 = torch.empty_like(x), torch.empty_like(x)
    tdp.tdp_attention_backward(long, long, x, x, x, y, lse, y, g, g2, g3, ws)
    torch.cuda.synchronize()
    for a, b in zip((g, g2, g3), grads):
        assert torch.equal(a[-tail:], b)


def test_gradients_against_differences(cuda):
    """Central differences of the 64-bit formula along random directions (step 1e-5: truncation and cancellation below
    1e-8) against the fp32 kernels' gradients, within their bounds."""
    gen = torch.Generator().manual_seed(6)
    n, D = 45, 40
    q, k, v, g = (torch.randn(n, 1, D, generator=gen) for _ in range(4))
    dev = [t.to(cuda) for t in (q, k, v, g)]
    seqs = tdp.Sequences(1, n)
    out, lse = torch.empty_like(dev[0]), torch.empty(1, n, device=cuda)
    grads = [torch.empty_like(dev[0]) for _ in range(3)]
    note("differences")
    tdp.tdp_attention(seqs, seqs, *dev[:3], out, lse)
    tdp.tdp_attention_backward(seqs, seqs, *dev[:3], out, lse, dev[3], *grads,
                               tdp.allocate_attention_backward_workspace(seqs, seqs, 1, 1, D, cuda))
    torch.cuda.synchronize()
    args = [t[:, 0].double() for t in (q, k, v)]
    r = R.attention(*args, None, D ** -0.5, torch.float32, out.cpu()[:, 0], g[:, 0])
    loss = lambda a: (R.attention(*a, None, D ** -0.5, torch.float32)[0] * g[:, 0].double()).sum()  # noqa: E731
    for i, name in enumerate(("dq", "dk", "dv")):
        d = torch.randn(n, D, generator=gen).double()
        hi = [t + 1e-5 * d if j == i else t for j, t in enumerate(args)]
        lo = [t - 1e-5 * d if j == i else t for j, t in enumerate(args)]
        want = (loss(hi) - loss(lo)) / 2e-5
        got = (grads[i][:, 0].double().cpu() * d).sum()
        assert abs(got - want) <= (r[name][1] * d.abs()).sum() + 1e-7, name

    rope = tdp.tdp_rope_create(tdp.make_rope_config(D, (16, 12, 12)))
    freqs = [[10000.0 ** (-2.0 * i / s) for i in range(s // 2)] for s in (16, 12, 12)]
    rot = ((16, 12, 12), freqs, "interleaved", "middle")
    pos = torch.rand(3, n, 2, generator=gen) * 50
    w = 1 + 0.3 * torch.randn(D, generator=gen)
    dq, dk = torch.empty_like(dev[0]), torch.empty_like(dev[0])
    dwq, dwk = torch.empty(2, D, device=cuda)
    wd = w.to(cuda)
    tdp.tdp_qk_norm_rope_backward(rope, seqs, pos.reshape(-1).to(cuda), dev[0], dev[1], wd, wd, dev[3], dev[2], dq, dk,
                                  dwq, dwk, tdp.allocate_qk_norm_rope_workspace(rope, seqs, 1, 1, cuda))
    torch.cuda.synchronize()
    f = lambda x, w: (R.norm_rope(x, w, pos, rot, 1e-6, torch.float32)[0] * g.double()).sum()  # noqa: E731
    _, bx, _, bw = R.norm_rope_backward(q, w, g, pos, rot, 1e-6, torch.float32)
    d = torch.randn(n, 1, D, generator=gen).double()
    want = (f(q.double() + 1e-5 * d, w.double()) - f(q.double() - 1e-5 * d, w.double())) / 2e-5
    assert abs((dq.double().cpu() * d).sum() - want) <= (bx * d.abs()).sum() + 1e-7
    d = torch.randn(D, generator=gen).double()
    want = (f(q.double(), w.double() + 1e-5 * d) - f(q.double(), w.double() - 1e-5 * d)) / 2e-5
    assert abs((dwq.double().cpu() * d).sum() - want) <= (bw * d.abs()).sum() + 1e-7


def test_binding_refusals(cuda):
    seqs, q, k, v = attn_inputs(cuda)
    out = torch.empty_like(q)
    ok = dict(q=q, k=k, v=v, out=out)

    def refused(match, **kw):
        a = {**ok, **kw}
        with pytest.raises((ValueError, tdp.TdpError), match=match):
            tdp.tdp_attention(kw.get("seqs", seqs), seqs, a["q"], a["k"], a["v"], a["out"], a.get("lse"),
                              key_bias=a.get("bias"))
    refused("on a GPU", q=q.cpu())
    refused("on cuda", k=k.cpu())
    refused("bfloat16", v=v.float())
    refused("rows", k=k[:-1])
    refused("contiguous elements", v=torch.empty(600, 2, 128, dtype=q.dtype, device=cuda)[..., ::2])
    refused("overlap itself", out=out[:1].expand(600, 4, 64))
    refused("multiple", q=torch.empty(600, 3, 64, dtype=q.dtype, device=cuda),
            out=torch.empty(600, 3, 64, dtype=q.dtype, device=cuda))
    refused("lse", lse=torch.empty(4, 599, device=cuda))
    refused("key_bias", bias=torch.empty(599, device=cuda))
    refused("is required", v=None)
    with pytest.raises(ValueError, match="float32 or torch.bfloat16"):
        tdp.tdp_attention(seqs, seqs, *(t.half() for t in (q, k, v)), out.half())
    one, long = tdp.Sequences(2, 1), tdp.Sequences(2, 9000)
    qo = torch.empty(2, 2, 64, device=cuda)
    kl = torch.empty(18000, 2, 64, device=cuda)
    with pytest.raises(ValueError, match="workspace"):
        tdp.tdp_attention(one, long, qo, kl, kl, torch.empty_like(qo))
    with pytest.raises(ValueError):
        tdp.Sequences(2, 9, total_rows=19)
    with pytest.raises(ValueError):
        tdp.Sequences(2, 9, row_start=torch.zeros(2, dtype=torch.int64, device=cuda), total_rows=18)
