"""GPU parity of the layer norm and its gradients with the 64-bit reference
(tests/layer_reference.py), within its derived bounds.

Every unused row of every input holds NaN and every output starts as NaN, so a
row that leaks in or is not written shows.  Inputs are seeded.
"""
import pytest
import torch

import layer_reference as L
import overlap_tiling_trapezoidal_amd as tdp
from harness import note
from test_gpu_tokens import DT, NAN, check, check_rest, layout

pytestmark = pytest.mark.gpu

CASES = [
    # channels, caps, lens, ragged ranges, weight rows, layout, offset of the rows
    (8, (70,) * 3, (70, 1, 0), False, 1, "rows", 0.0),
    (64, (9, 33, 40), (9, 33, 17), True, 3, "wide", 3.0),
    (72, (41,) * 2, (41, 40), False, 2, "seqs", 0.0),
    (128, (75,) * 4, (75,) * 4, False, 1, "rows", -5.0),
    (200, (18, 5, 1), (17, 5, 1), True, 1, "wide", 0.0),
    (512, (13, 4), (13, 3), True, 2, "rows", 100.0),
    (520, (6,) * 5, (6, 5, 0, 1, 6), False, 2, "wide", 0.0),
    (1024, (11,), (11,), False, 1, "rows", 0.0),
    (2048, (9, 10, 1), (9, 7, 1), True, 1, "wide", 20.0),
    (2056, (5,) * 3, (5, 4, 0), False, 3, "rows", 0.0),
    (4104, (4,) * 2, (4, 3), False, 1, "wide", 1.0),
    (8192, (3, 5), (3, 5), True, 2, "rows", 0.0),
]
IDS = [f"c{c[0]}-{c[5]}-{c[4]}" for c in CASES]


def rows_like(seqs, x, cuda, kind):
    """On the GPU: contiguous, columns of a wider tensor, or (sequences, rows, channels) with gaps between sequences."""
    if kind == "wide":
        w = torch.full((x.shape[0], x.shape[1] + 24), NAN, dtype=x.dtype, device=cuda)
        w[:, 8:-16] = x.to(cuda)
        return w[:, 8:-16]
    if kind == "seqs":
        w = torch.full((seqs.num_seqs, seqs.max_rows + 2, x.shape[1]), NAN, dtype=x.dtype, device=cuda)
        w[:, :-2] = x.view(seqs.num_seqs, seqs.max_rows, -1).to(cuda)
        return w[:, :-2]
    return x.to(cuda)


def setup(case, dtype, cuda, seed):
    C, caps, lens, ragged, sets, kind, offset = case
    gen = torch.Generator().manual_seed(seed)
    seqs, rows = layout(caps, lens, cuda, ragged)
    def values(shift=0.0):
        x = (torch.randn(seqs.total_rows, C, generator=gen) + shift).to(DT[dtype])
        keep = torch.zeros(seqs.total_rows, dtype=torch.bool)
        for a, _, n in rows:
            keep[a:a + n] = True
        x[~keep] = NAN
        return x
    w, b = 1.0 + 0.3 * torch.randn(sets, C, generator=gen), 0.5 * torch.randn(sets, C, generator=gen)
    return seqs, rows, values, w, b


def flat(t):
    return t.reshape(-1, t.shape[-1])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_layer_norm(case, dtype, cuda):
    C, caps, lens, ragged, sets, kind, offset = case
    seqs, rows, values, w, b = setup(case, dtype, cuda, 11)
    x = values(offset)
    xd, y = rows_like(seqs, x, cuda, kind), rows_like(seqs, torch.full_like(x, NAN), cuda, kind)
    wd, bd = w.to(cuda), b.to(cuda)
    note(f"layer norm {case} {dtype}")
    tdp.tdp_layer_norm(seqs, xd, wd, bd, y, eps=1e-5)
    torch.cuda.synchronize()
    check_rest("y", flat(y), rows)
    for s, (a, c, n) in enumerate(rows):
        want, bound = L.layer_norm(x[a:a + n], w[s % sets], b[s % sets], 1e-5, DT[dtype])
        check("y", flat(y)[a:a + n], want, bound)
    # without weights, and in place
    tdp.tdp_layer_norm(seqs, xd, None, None, y, eps=1e-5)
    tdp.tdp_layer_norm(seqs, xd, wd, bd, xd, eps=1e-5)
    torch.cuda.synchronize()
    one, zero = torch.ones(C), torch.zeros(C)
    for s, (a, c, n) in enumerate(rows):
        check("plain", flat(y)[a:a + n], *L.layer_norm(x[a:a + n], one, zero, 1e-5, DT[dtype]))
        want, bound = L.layer_norm(x[a:a + n], w[s % sets], b[s % sets], 1e-5, DT[dtype])
        check("in place", flat(xd)[a:a + n], want, bound)
        assert (flat(xd)[a + n:a + c] == 0).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_layer_norm_backward(case, dtype, cuda):
    C, caps, lens, ragged, sets, kind, offset = case
    seqs, rows, values, w, b = setup(case, dtype, cuda, 12)
    x, dy = values(offset), values()
    xd, gd = rows_like(seqs, x, cuda, kind), rows_like(seqs, dy, cuda, kind)
    dx = rows_like(seqs, torch.full_like(x, NAN), cuda, kind)
    wd = w.to(cuda)
    dw, db = torch.full((sets, C), NAN, device=cuda), torch.full((sets, C), NAN, device=cuda)
    ws = tdp.allocate_layer_norm_workspace(seqs, C, sets, cuda)
    ws.fill_(255)
    note(f"layer norm gradients {case} {dtype}")
    tdp.tdp_layer_norm_backward(seqs, xd, wd, gd, dx, dw, db, ws, eps=1e-5)
    torch.cuda.synchronize()
    check_rest("dx", flat(dx), rows)
    sums = torch.zeros(4, sets, C, dtype=torch.float64)
    for s, (a, c, n) in enumerate(rows):
        g, gb, *parts = L.layer_norm_backward(x[a:a + n], w[s % sets], dy[a:a + n], 1e-5, DT[dtype])
        check("dx", flat(dx)[a:a + n], g, gb)
        for i, p in enumerate(parts):
            sums[i, s % sets] += p
    check("dw", dw, sums[0], sums[1])
    check("db", db, sums[2], sums[3])
    # in place of dy, without the sums, and bit for bit again
    again = torch.empty_like(dw)
    tdp.tdp_layer_norm_backward(seqs, xd, wd, gd, gd, again, None, ws, eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(again, dw)
    for a, c, n in rows:
        assert torch.equal(flat(gd)[a:a + c], flat(dx)[a:a + c])


def test_layer_norm_gradient_against_differences(cuda):
    """The directional derivative of sum(y * g) by central differences in 64 bits meets <dx, v>, <dw, vw>, <db, vb>."""
    C, gen = 136, torch.Generator().manual_seed(5)
    seqs, rows = layout((20, 7), (19, 7), cuda, True)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, g, v = rnd(seqs.total_rows, C), rnd(seqs.total_rows, C), rnd(seqs.total_rows, C)
    w, b, vw, vb = 1 + 0.2 * rnd(C), rnd(C), rnd(C), rnd(C)
    used = torch.cat([torch.arange(a, a + n) for a, _, n in rows])
    def f(t):
        xx = x[used].double() + t * v[used].double()
        d = xx - xx.mean(1, keepdim=True)
        y = d / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-3) * (w.double() + t * vw) + (b.double() + t * vb)
        return (y * g[used].double()).sum()
    h = 1e-5
    want = (f(h) - f(-h)) / (2 * h)
    dx, dw, db = torch.empty(seqs.total_rows, C, device=cuda), torch.empty(C, device=cuda), torch.empty(C, device=cuda)
    ws = tdp.allocate_layer_norm_workspace(seqs, C, 1, cuda)
    note("layer norm differences")
    tdp.tdp_layer_norm_backward(seqs, x.to(cuda), w.to(cuda), g.to(cuda), dx, dw, db, ws, eps=1e-3)
    torch.cuda.synchronize()
    terms = [(dx.cpu()[used].double() * v[used]), dw.cpu().double() * vw, db.cpu().double() * vb]
    got, mag = sum(t.sum() for t in terms), sum(t.abs().sum() for t in terms)
    # the difference's own error, h^2 times a third derivative of the size of the values, is 1e-10 of them
    assert abs(got - want) <= 1e-6 * mag, (float(got), float(want))


def test_layer_norm_values(cuda):
    """Rows of one value give the bias; a NaN or an infinity stays in its row; far offsets keep their digits."""
    C = 256
    seqs = tdp.Sequences(1, 6)
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(6, C, generator=gen)
    x[0] = 3.0
    x[2, 5] = NAN
    x[3, 7] = float("inf")
    x[4] = 1e6 + 64 * x[4].round()   # whole numbers: exact in fp32
    xd, y, b = x.to(cuda), torch.empty(6, C, device=cuda), torch.randn(C, generator=gen)
    note("layer norm values")
    tdp.tdp_layer_norm(seqs, xd, None, b.to(cuda), y, eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(y[0].cpu(), b)
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    for i in (1, 4, 5):
        check(f"row {i}", y[i:i + 1], *L.layer_norm(x[i:i + 1], torch.ones(C), b, 1e-5, torch.float32))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("offset", [100.0, 1e3, -1e4, 1e6])
@pytest.mark.parametrize("C", [8, 136, 520, 2048, 4104, 8192])
def test_layer_norm_far_rows(C, offset, dtype, cuda):
    """Rows far from zero: the error scales with their spread, not with their offset, in outputs and gradients."""
    gen, rows = torch.Generator().manual_seed(C), 5
    seqs = tdp.Sequences(1, rows)
    x = (offset + torch.randn(rows, C, generator=gen)).to(DT[dtype])
    x[1] = offset + 100 * torch.randn(C, generator=gen)
    x[2, C // 2] = -offset   # an element far from the others
    dy = torch.randn(rows, C, generator=gen).to(DT[dtype])
    w, b = 1.0 + 0.3 * torch.randn(C, generator=gen), 0.5 * torch.randn(C, generator=gen)
    xd, wd, y, dx = x.to(cuda), w.to(cuda), torch.empty_like(x, device=cuda), torch.empty_like(x, device=cuda)
    dw, db = torch.empty(C, device=cuda), torch.empty(C, device=cuda)
    note(f"layer norm far rows {C} {offset} {dtype}")
    tdp.tdp_layer_norm(seqs, xd, wd, b.to(cuda), y, eps=1e-5)
    tdp.tdp_layer_norm_backward(seqs, xd, wd, dy.to(cuda), dx, dw, db, tdp.allocate_layer_norm_workspace(seqs, C, 1, cuda),
                                eps=1e-5)
    torch.cuda.synchronize()
    check("y", y, *L.layer_norm(x, w, b, 1e-5, DT[dtype], L.far_parts))
    g, gb, w1, w1b, b1, b1b = L.layer_norm_backward(x, w, dy, 1e-5, DT[dtype], L.far_parts)
    check("dx", dx, g, gb)
    check("dw", dw, w1, w1b)
    check("db", db, b1, b1b)
