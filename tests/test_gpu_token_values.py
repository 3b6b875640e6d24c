"""Values at the edge of the token operators' formulas: a norm without eps,
values that are not finite in dims that do not turn, scores of 1e9 and more
and the gradients' weights computed again from their lse."""
import math

import pytest
import torch

import overlap_tiling_trapezoidal_amd as tdp
import test_gpu_tokens as G
import token_reference as R
from harness import note

pytestmark = pytest.mark.gpu
DT, NAN, INF = G.DT, float("nan"), math.inf


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("D,hq,hk", [(128, 3, 1), (32, 4, 2), (64, 17, 5), (256, 1, 3), (40, 7, 1)])
def test_norm_without_eps(D, hq, hk, pairing, dtype, cuda):
    """eps = 0 with head counts that leave lanes without a head: forward and gradients, weights' among them."""
    dt = DT[dtype]
    rot_dims = (D // 2, D // 4, 0)
    case = (D, rot_dims, hq, hk, (9, 6), (9, 5), True, pairing, "middle", "packed", 100.0)
    gen, seqs, rows, rope, pos, planes, rot = G.rope_setup(case, dtype, cuda, 31)
    q, k, gq, gk = (G.poisoned(gen, seqs, rows, h, D, dt) for h in (hq, hk, hq, hk))
    wq, wk = (1 + 0.3 * torch.randn(D, generator=gen) for _ in range(2))
    qd, kd, gqd, gkd = (G.to_device(t, cuda, "packed") for t in (q, k, gq, gk))
    yq, yk, dq, dk = (G.to_device(torch.full_like(t, NAN), cuda, "packed") for t in (q, k, q, k))
    dwq, dwk = torch.full((2, D), NAN, device=cuda)
    note(f"norm without eps {D} {hq} {hk} {dtype}")
    tdp.tdp_qk_norm_rope(rope, seqs, pos, qd, kd, wq.to(cuda), wk.to(cuda), yq, yk, eps=0.0)
    tdp.tdp_qk_norm_rope_backward(rope, seqs, pos, qd, kd, wq.to(cuda), wk.to(cuda), gqd, gkd, dq, dk, dwq, dwk,
                                  tdp.allocate_qk_norm_rope_workspace(rope, seqs, hq, hk, cuda), eps=0.0)
    torch.cuda.synchronize()
    for x, w, g, y, dx, dw in ((q, wq, gq, yq, dq, dwq), (k, wk, gk, yk, dk, dwk)):
        want_dw, bound_dw = torch.zeros(D).double(), torch.zeros(D).double()
        for (a, c, n), p in zip(rows, planes):
            G.check("y", y[a:a + n], *R.norm_rope(x[a:a + n], w, p, rot, 0.0, dt))
            v, b, w1, b1 = R.norm_rope_backward(x[a:a + n], w, g[a:a + n], p, rot, 0.0, dt)
            G.check("dx", dx[a:a + n], v, b)
            want_dw, bound_dw = want_dw + w1, bound_dw + b1
        G.check("dw", dw, want_dw, bound_dw)


def same(a, b):
    """Equal values, signs of zeros among them, or both not a number."""
    a, b = a.detach().float().cpu(), b.detach().float().cpu()
    return bool(((a.view(torch.int32) == b.view(torch.int32)) | (a.isnan() & b.isnan())).all())


# head_dim, rot dims, heads, rows: the general form (two and four passes) and the one for few heads
PASS = [(64, (24, 0, 16), 12, 7), (128, (40, 20, 20), 16, 5), (32, (12, 0, 0), 2, 19), (256, (64, 64, 64), 1, 6),
        (40, (2, 2, 2), 1, 30), (64, (0, 0, 0), 3, 9)]


def partial(D, rot_dims, heads, n, pairing, dtype, cuda, seed):
    case = (D, rot_dims, heads, heads, (n,), (n,), False, pairing, "middle", "rows", 100.0)
    gen, seqs, rows, rope, pos, planes, rot = G.rope_setup(case, dtype, cuda, seed)
    return gen, seqs, rope, pos, planes[0], rot


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("case", PASS, ids=[f"d{c[0]}-h{c[2]}" for c in PASS])
def test_dims_that_do_not_turn_pass_unchanged(case, pairing, dtype, cuda):
    """Infinities, NaN and zeros of either sign beyond the turned dims come out as they are and touch nothing else."""
    (D, rot_dims, heads, n), dt = case, DT[dtype]
    gen, seqs, rope, pos, planes, rot = partial(*case, pairing, dtype, cuda, 41)
    first = sum(rot_dims)
    x = torch.randn(n, heads, D, generator=gen).to(dt)
    x[0, :, first] = INF
    x[1, :, first + 1] = -INF
    x[2, :, D - 1] = NAN
    x[3, :, first:] = -0.0
    x[4, 0, first::2] = torch.finfo(dt).max
    xd = x.to(cuda)
    for inverse in (False, True):
        y = torch.full_like(xd, 7.0)
        note(f"partial rotation {case} {pairing} {dtype}")
        tdp.tdp_rope_apply(rope, seqs, pos, xd, y, inverse=inverse)
        torch.cuda.synchronize()
        assert same(y[..., first:], x[..., first:])
        if first:
            want, mag = R.turn(x.double(), planes, *rot, inverse=inverse)
            bound = 12 * R.U32 * mag + R.half_step(dt) * want.abs()
            G.check("turned", y[..., :first], want[..., :first], bound[..., :first])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("case", PASS, ids=[f"d{c[0]}-h{c[2]}" for c in PASS])
def test_norm_keeps_values_that_do_not_turn_apart(case, pairing, dtype, cuda):
    """An infinite weight in a dim that does not turn reaches that dim of the output alone; an output gradient that is
    not finite there reaches that dim of the weight's gradient alone (and, through the mean, its own head's dx)."""
    (D, rot_dims, heads, n), dt = case, DT[dtype]
    gen, seqs, rope, pos, planes, rot = partial(*case, pairing, dtype, cuda, 42)
    d = sum(rot_dims) + 2
    others = [i for i in range(D) if i != d]
    x, g = (torch.randn(n, heads, D, generator=gen).to(dt) for _ in range(2))
    w = 1 + 0.3 * torch.randn(D, generator=gen)
    xd, w_inf = x.to(cuda), w.clone()
    w_inf[d] = INF
    y, y2 = torch.full_like(xd, 7.0), torch.full_like(xd, 7.0)
    note(f"norm with an infinite weight {case} {pairing} {dtype}")
    tdp.tdp_qk_norm_rope(rope, seqs, pos, xd, xd, w_inf.to(cuda), w_inf.to(cuda), y, y2, eps=1e-5)
    torch.cuda.synchronize()
    want, bound = R.norm_rope(x, w, planes, rot, 1e-5, dt)
    for t in (y, y2):
        G.check("others", t[..., others], want[..., others], bound[..., others])
        assert same(t[..., d], torch.where(x[..., d].float() > 0, INF, -INF))
    bad = g.clone()
    bad[n // 2, 0, d] = NAN
    dx, dx2 = torch.full_like(xd, 7.0), torch.full_like(xd, 7.0)
    dw, dw2 = torch.full((2, D), 7.0, device=cuda)
    ws = tdp.allocate_qk_norm_rope_workspace(rope, seqs, heads, heads, cuda)
    note(f"norm gradients with a NaN {case} {pairing} {dtype}")
    tdp.tdp_qk_norm_rope_backward(rope, seqs, pos, xd, xd, w.to(cuda), w.to(cuda), bad.to(cuda), bad.to(cuda), dx, dx2,
                                  dw, dw2, ws, eps=1e-5)
    torch.cuda.synchronize()
    want, bound, want_dw, bound_dw = R.norm_rope_backward(x, w, g, planes, rot, 1e-5, dt)
    keep = torch.ones(n, heads, dtype=torch.bool)
    keep[n // 2, 0] = False
    for t, tw in ((dx, dw), (dx2, dw2)):
        G.check("dx", t.cpu()[keep], want[keep], bound[keep])
        G.check("dw", tw[others], want_dw[others], bound_dw[others])
        assert math.isnan(tw[d].item())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("rows,keys", [(200, 130), (3, 1200)], ids=["whole", "keys-split"])
@pytest.mark.parametrize("spread", [3e4, 3e5, 1e7])
def test_attention_of_huge_scores(spread, rows, keys, D, dtype, cuda):
    """Scores of 1e9 to 1e15: every row whose largest score leads by more than the fp32 errors of two dot products and
    what makes the other weights vanish gives that key's value, exactly, and its score as lse."""
    dt, scale = DT[dtype], D ** -0.5
    gen = torch.Generator().manual_seed(52)
    q, k, v = (torch.randn(n, 1, D, generator=gen) for n in (rows, keys, keys))
    q, k, v = ((t * s).to(dt) for t, s in ((q, spread), (k, spread), (v, 1.0)))
    qs, ks = tdp.Sequences(1, rows), tdp.Sequences(1, keys)
    out, lse = torch.empty(rows, 1, D, dtype=dt, device=cuda), torch.empty(1, rows, device=cuda)
    note(f"huge scores {spread} {rows} {D} {dtype}")
    tdp.tdp_attention(qs, ks, q.to(cuda), k.to(cuda), v.to(cuda), out, lse,
                      workspace=tdp.allocate_attention_workspace(qs, ks, 1, 1, D, cuda))
    torch.cuda.synchronize()
    s = scale * q[:, 0].double() @ k[:, 0].double().T
    err = (D + 4) * R.U32 * scale * (q[:, 0].double().abs() @ k[:, 0].double().abs().T).max(1).values
    two = s.topk(2, 1)
    lead = two.values[:, 0] - two.values[:, 1] > 2 * err + 120   # exp(-120) vanishes in fp32
    assert lead.sum() > rows // 2 and s.max() > 1e9
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert torch.equal(out[:, 0].cpu()[lead], v[two.indices[:, 0], 0][lead])
    top = two.values[:, 0]
    assert ((lse[0].double().cpu() - top).abs() <= err + 4 * R.U32 * top.abs())[lead].all()


def bounded_gradients(cuda, dt, D, spread, bias, scale, most, seed):
    """Attention of 200 rows over 130 keys and its gradients.  Whatever weight in [0, most] a key is given,
    |dv_j| <= most sum_i |do_i|, |dp - delta| <= D max|do| (max|v| + max|o|) =: z, |dq_i| <= most scale n z max|k| and
    |dk_j| <= most scale m z max|q|; each may be off by roundings of 2^-7 altogether."""
    m, n = 200, 130
    gen = torch.Generator().manual_seed(seed)
    qs, ks = tdp.Sequences(1, m), tdp.Sequences(1, n)
    q, g = (torch.randn(m, 1, D, generator=gen) for _ in range(2))
    k, v = (torch.randn(n, 1, D, generator=gen) for _ in range(2))
    q, k, v, g = ((t * s).to(dt).to(cuda) for t, s in ((q, spread), (k, spread), (v, 1.0), (g, 1.0)))
    bd = None if bias is None else torch.full((n,), bias, device=cuda)
    out, lse = torch.empty_like(q), torch.empty(1, m, device=cuda)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    note(f"bounded gradients {spread} {bias} {D} {dt}")
    tdp.tdp_attention(qs, ks, q, k, v, out, lse, key_bias=bd, scale=scale)
    tdp.tdp_attention_backward(qs, ks, q, k, v, out, lse, g, dq, dk, dv,
                               tdp.allocate_attention_backward_workspace(qs, ks, 1, 1, D, cuda), key_bias=bd,
                               scale=scale)
    torch.cuda.synchronize()
    top = lambda t: t.detach().double().abs().max().item()  # noqa: E731
    z = most * D * top(g) * (top(v) + top(out))
    for name, t, limit in (("out", out, top(v)), ("dv", dv, most * g.double().abs().sum(0).max().item()),
                           ("dq", dq, scale * n * z * top(k)), ("dk", dk, scale * m * z * top(q))):
        assert torch.isfinite(t).all(), f"{name} is not finite"
        assert top(t) <= (1 + 2.0 ** -7) * limit, f"{name}: {top(t)} above {limit}"
    return q, k, v, g, lse, dq


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bias", [-1.2e9, -2.5e9, 1.7e9])
def test_gradients_with_huge_biases(bias, D, dtype, cuda):
    """Every key's bias huge: fp32 scores keep next to nothing of q . k, lse is rounded by tens, and a weight computed
    again from it must not pass one."""
    bounded_gradients(cuda, DT[dtype], D, 1.0, bias, 40.0, 1.0, 51)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("spread", [3e4, 3e5])
def test_gradients_of_huge_scores(spread, D, dtype, cuda):
    """Scores of 1e9 to 1e12 without a bias: no weight above 2^4.  Rows with a clear leader hold its value as their
    output, so dp - delta there is two fp32 dot products of the same numbers, and dq no more than that makes it."""
    scale = D ** -0.5
    q, k, v, g, lse, dq = (t[:, 0].double().cpu() for t in
                           bounded_gradients(cuda, DT[dtype], D, spread, None, scale, 16.0, 52))
    s = scale * q @ k.T
    err = (D + 4) * R.U32 * scale * (q.abs() @ k.abs().T).max(1).values
    two = s.topk(2, 1)
    first = two.indices[:, 0]
    lead = two.values[:, 0] - two.values[:, 1] > 2 * err + 2.0 ** -20 * two.values[:, 0].abs() + 120
    assert lead.sum() > 100 and s.max() > 1e9
    same_dots = 2 * (D + 4) * R.U32 * (g.abs() * v[first].abs()).sum(1, keepdim=True)
    limit = 16 * scale * same_dots * k[first].abs() * (1 + 2.0 ** -6)
    assert (dq.abs() <= limit)[lead].all()
