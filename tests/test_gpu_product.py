"""GPU parity of the grouped products and their gradients with the 64-bit
reference (tests/layer_reference.py), within its derived bounds.

Every unused row of every input holds NaN and every output starts as NaN, so a
row that leaks in or is not written shows.  Inputs are seeded.
"""
import pytest
import torch

import layer_reference as L
import overlap_tiling_trapezoidal_amd as tdp
from harness import note
from test_gpu_layer_norm import flat, rows_like
from test_gpu_tokens import DT, NAN, check, check_rest, layout
from token_reference import U32

pytestmark = pytest.mark.gpu

CASES = [
    # in, out features, caps, lens, ragged ranges, weights, layout
    (8, 8, (1,), (1,), False, 1, "rows"),
    (128, 384, (75,) * 4, (75,) * 4, False, 1, "rows"),
    (72, 40, (33, 20, 64), (33, 0, 63), True, 3, "wide"),
    (136, 264, (130,) * 2, (130, 1), False, 2, "seqs"),
    (64, 64, (300, 5, 200), (299, 5, 130), True, 1, "wide"),
    (1000, 72, (20, 31), (20, 30), True, 2, "rows"),                        # few rows: the contraction split
    (520, 2056, (3, 0, 40, 7, 0, 1, 2), (3, 0, 40, 7, 0, 1, 2), True, 7, "wide"),   # experts, some without rows
    (264, 1032, (70,) * 6, (70, 69, 0, 1, 70, 64), False, 2, "rows"),
    (2048, 136, (500,), (490,), False, 1, "rows"),                          # dW split over rows
    (72, 328, (90,) * 70, tuple(90 if i % 3 else i for i in range(70)), False, 1, "rows"),     # more than 64 sequences
    (72, 328, (9,) * 130, tuple(9 if i % 3 else i % 9 for i in range(130)), True, 5, "wide"),
]
IDS = [f"{c[0]}to{c[1]}-{len(c[2])}x{c[2][0]}-w{c[5]}-{c[6]}" for c in CASES]
# tiles of 256 by 256 rows and features
BIG = [
    (72, 4104, (1500, 900, 700), (1500, 899, 1), True, 3, "wide"),
    (328, 4096, (3400,), (3333,), False, 1, "rows"),
]
BIG += [   # a few tiles beyond a whole round of 256
    (72, 4096, (4300,), (4290,), False, 1, "rows"),
    (72, 4104, (2100, 1100, 1000), (2100, 1090, 1000), True, 3, "wide"),
]
BIG_IDS = [f"{c[0]}to{c[1]}-{len(c[2])}" for c in BIG]
# in, out features, sequences, rows, weights: every tile and form of the launch, split and whole, of y or of dx
TILES = [
    (136, 72, 12, 2500, 1), (136, 72, 40, 300, 40), (72, 2056, 12, 520, 3), (72, 72, 12, 5000, 1), (72, 72, 12, 2500, 2),
    (2056, 72, 3, 2500, 1), (8200, 72, 5, 33, 5), (136, 2056, 12, 33, 1), (72, 1032, 40, 33, 4), (72, 72, 40, 200, 1),
    (4104, 72, 12, 33, 2), (8200, 72, 40, 33, 1), (72, 1032, 40, 130, 1), (8200, 264, 12, 130, 1), (72, 8200, 5, 130, 1),
    (72, 72, 70, 40, 70),
]

# as those with one weight, whose tiles are of the tensors' rows, with several
TILES += [
    (136, 72, 12, 2500, 2), (72, 72, 12, 5000, 2), (2056, 72, 3, 2500, 2), (136, 2056, 12, 33, 3), (72, 72, 40, 200, 3),
    (8200, 72, 40, 33, 3), (72, 1032, 40, 130, 3), (8200, 264, 12, 130, 3), (72, 8200, 5, 130, 2),
]
# one weight for sequences that end anywhere in a tile
SHARED = [
    (136, 264, (46,) * 24, tuple(46 - 5 * (i % 3) for i in range(24)), True, 1, "wide"),
    (72, 2056, tuple(i % 5 for i in range(600)), tuple(max(0, i % 5 - i % 2) for i in range(600)), True, 1, "rows"),
    (136, 264, (1,) * 700, (1, 0) * 350, True, 1, "rows"),
    (264, 136, (46,) * 50, (0,) * 30 + tuple(range(20)), False, 1, "rows"),        # whole tiles without a used row
    (264, 136, (46,) * 50, (0,) * 30 + tuple(range(20)), False, 1, "seqs"),        # rows apart: tiles of sequences
    (2056, 72, (20,) * 7, (20, 0, 3, 20, 20, 1, 20), True, 1, "wide"),             # few rows: the contraction split
    (72, 4104, (150,) * 30, tuple(150 - i for i in range(30)), True, 1, "wide"),   # large tiles and some beyond a round
    (4104, 72, (150,) * 30, tuple(150 - i for i in range(30)), True, 1, "wide"),   # the same of dx
]


def setup(case, dtype, cuda, seed):
    K, N, caps, lens, ragged, E, kind = case
    gen = torch.Generator().manual_seed(seed)
    seqs, rows = layout(caps, lens, cuda, ragged)
    if ragged:   # experts' rows are known on the device only: any may hold all
        seqs = tdp.Sequences(len(caps), seqs.total_rows, row_range=seqs._keep[0], total_rows=seqs.total_rows,
                             seq_len=seqs._keep[1])
    def values(width):
        x = torch.randn(seqs.total_rows, width, generator=gen).to(DT[dtype])
        keep = torch.zeros(seqs.total_rows, dtype=torch.bool)
        for a, _, n in rows:
            keep[a:a + n] = True
        x[~keep] = NAN
        return x
    w = (torch.randn(E, N, K, generator=gen) * K ** -0.5).to(DT[dtype])
    return seqs, rows, values, w


def check_forward(case, dtype, cuda, seed):
    K, N, caps, lens, ragged, E, kind = case
    seqs, rows, values, w = setup(case, dtype, cuda, seed)
    x = values(K)
    xd, y = rows_like(seqs, x, cuda, kind), rows_like(seqs, torch.full((seqs.total_rows, N), NAN, dtype=x.dtype), cuda, kind)
    ws = tdp.allocate_grouped_product_workspace(seqs, E, N, K, DT[dtype], cuda)
    if ws is not None:
        ws.fill_(0xff)
    note(f"product {case[:2]} {case[5:]} {dtype} workspace {0 if ws is None else len(ws)}")
    tdp.tdp_grouped_product(seqs, xd, w.to(cuda), y, workspace=ws)
    torch.cuda.synchronize()
    check_rest("y", flat(y), rows)
    for s, (a, c, n) in enumerate(rows):
        check("y", flat(y)[a:a + n], *L.product(x[a:a + n], w[s % E], DT[dtype]))


def check_backward(case, dtype, cuda, seed):
    K, N, caps, lens, ragged, E, kind = case
    dt = DT[dtype]
    seqs, rows, values, w = setup(case, dtype, cuda, seed)
    x, dy = values(K), values(N)
    xd, gd = rows_like(seqs, x, cuda, kind), rows_like(seqs, dy, cuda, kind)
    dx, dw = rows_like(seqs, torch.full_like(x, NAN), cuda, kind), torch.full((E, N, K), NAN, device=cuda)
    ws = tdp.allocate_grouped_product_backward_workspace(seqs, E, N, K, dt, cuda)
    if ws is not None:
        ws.fill_(0xff)
    wd = w.to(cuda)
    note(f"product gradients {case[:2]} {case[5:]} {dtype} workspace {0 if ws is None else len(ws)}")
    tdp.tdp_grouped_product_backward(seqs, xd, wd, gd, dx, dw, ws)
    torch.cuda.synchronize()
    check_rest("dx", flat(dx), rows)
    want, bound = torch.zeros(E, N, K, dtype=torch.float64), torch.zeros(E, N, K, dtype=torch.float64)
    for s, (a, c, n) in enumerate(rows):
        check("dx", flat(dx)[a:a + n], *L.product(dy[a:a + n], w[s % E].T, dt))
        xs, gs = x[a:a + n].double(), dy[a:a + n].double()
        want[s % E] += gs.T @ xs
        bound[s % E] += gs.abs().T @ xs.abs()
    # a chain of all rows of a weight and a join's 16
    check("dw", dw, want, (sum(lens) + 24) * U32 * bound)
    # one at a time: the same, bit for bit
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    if kind == "rows":
        tdp.tdp_grouped_product_backward(seqs, xd, wd, gd, dx2, None, ws)
        tdp.tdp_grouped_product_backward(seqs, xd, wd, gd, None, dw2, ws)
        torch.cuda.synchronize()
        assert torch.equal(dw, dw2)
        for a, c, n in rows:
            assert torch.equal(dx[a:a + c], dx2[a:a + c])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_grouped_product(case, dtype, cuda):
    check_forward(case, dtype, cuda, 41)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_grouped_product_backward(case, dtype, cuda):
    check_backward(case, dtype, cuda, 42)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", TILES, ids=["x".join(map(str, c)) for c in TILES])
def test_grouped_product_tiles(case, dtype, cuda):
    K, N, S, n, E = case
    full = (K, N, (n,) * S, tuple(n - 3 * (i % 5) for i in range(S)), False, E, "rows")
    check_forward(full, dtype, cuda, 47)
    check_backward(full, dtype, cuda, 48)


@pytest.mark.parametrize("case", BIG, ids=BIG_IDS)
def test_grouped_product_large_tiles(case, cuda):
    check_forward(case, "bf16", cuda, 43)
    K, N, *rest = case
    check_backward((N, K, *rest), "bf16", cuda, 44)      # dx of many features


def test_grouped_product_large_tiles_of_weights(cuda):
    check_backward((1032, 1000, (70, 300, 1, 65, 130, 90, 80, 0, 3, 64, 66, 20), (70, 299, 1, 65, 130, 90, 80, 0, 3, 64, 66, 20),
                    True, 12, "wide"), "bf16", cuda, 45)


@pytest.mark.parametrize("dtype", list(DT))
def test_broadcast_rows(dtype, cuda):
    """Inputs whose rows are one row (stride 0): the end of a sequence repeats nothing."""
    K, N, n = 72, 40, 37
    gen = torch.Generator().manual_seed(46)
    seqs = tdp.Sequences(1, n, seq_len=torch.tensor([n - 2], dtype=torch.int32, device=cuda))
    x, dy = (torch.randn(1, k, generator=gen).to(DT[dtype]) for k in (K, N))
    w = torch.randn(N, K, generator=gen).to(DT[dtype])
    xd, gd = x.to(cuda).expand(n, K), dy.to(cuda).expand(n, N)
    y, dx = torch.full((n, N), NAN, dtype=x.dtype, device=cuda), torch.full((n, K), NAN, dtype=x.dtype, device=cuda)
    dw = torch.empty(N, K, device=cuda)
    note(f"broadcast rows {dtype}")
    ws = tdp.allocate_grouped_product_workspace(seqs, 1, N, K, DT[dtype], cuda)
    tdp.tdp_grouped_product(seqs, xd, w.to(cuda), y, workspace=ws)
    ws = tdp.allocate_grouped_product_backward_workspace(seqs, 1, N, K, DT[dtype], cuda)
    tdp.tdp_grouped_product_backward(seqs, xd, w.to(cuda), gd, dx, dw, ws)
    torch.cuda.synchronize()
    for got, want in ((y, L.product(x, w, DT[dtype])), (dx, L.product(dy, w.T, DT[dtype]))):
        check("rows", got[:n - 2], want[0].expand(n - 2, -1), want[1].expand(n - 2, -1))
        assert (got[n - 2:] == 0).all()
    one = dy.double().T @ x.double()
    check("dw", dw, (n - 2) * one, (n + 24) * U32 * n * one.abs())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", SHARED, ids=[f"{c[0]}to{c[1]}-{len(c[2])}x{c[2][0]}-{c[6]}" for c in SHARED])
def test_grouped_product_shared_weight(case, dtype, cuda):
    check_forward(case, dtype, cuda, 49)
    check_backward(case, dtype, cuda, 50)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("E", [1, 2])
def test_grouped_product_row_limit(E, dtype, cuda):
    """Ranges longer than max_rows: rows past it are left alone."""
    K, N, limit = 72, 136, 30
    ranges = [(3, 48), (48, 78), (80, 80), (80, 200), (200, 201), (201, 290)]
    lens = (45, 29, 0, 30, 1, 12)
    rows = [(a, min(b - a, limit), min(b - a, n, limit)) for (a, b), n in zip(ranges, lens)]
    seqs = tdp.Sequences(len(ranges), limit, row_range=torch.tensor(ranges, dtype=torch.int64, device=cuda), total_rows=300,
                         seq_len=torch.tensor(lens, dtype=torch.int32, device=cuda))
    gen = torch.Generator().manual_seed(51)
    x, dy = (torch.full((300, k), NAN).to(DT[dtype]) for k in (K, N))
    for a, _, n in rows:
        x[a:a + n], dy[a:a + n] = torch.randn(n, K, generator=gen), torch.randn(n, N, generator=gen)
    w = (torch.randn(E, N, K, generator=gen) * K ** -0.5).to(DT[dtype])
    xd, gd, wd = x.to(cuda), dy.to(cuda), w.to(cuda)
    y, dx, dw = torch.full_like(gd, NAN), torch.full_like(xd, NAN), torch.empty(E, N, K, device=cuda)
    note(f"row limit {E} {dtype}")
    ws = tdp.allocate_grouped_product_workspace(seqs, E, N, K, DT[dtype], cuda)
    tdp.tdp_grouped_product(seqs, xd, wd, y, workspace=ws)
    ws = tdp.allocate_grouped_product_backward_workspace(seqs, E, N, K, DT[dtype], cuda)
    tdp.tdp_grouped_product_backward(seqs, xd, wd, gd, dx, dw, ws)
    torch.cuda.synchronize()
    check_rest("y", y, rows)
    check_rest("dx", dx, rows)
    want, bound = torch.zeros(E, N, K, dtype=torch.float64), torch.zeros(E, N, K, dtype=torch.float64)
    for s, (a, _, n) in enumerate(rows):
        check("y", y[a:a + n], *L.product(x[a:a + n], w[s % E], DT[dtype]))
        check("dx", dx[a:a + n], *L.product(dy[a:a + n], w[s % E].T, DT[dtype]))
        want[s % E] += dy[a:a + n].double().T @ x[a:a + n].double()
        bound[s % E] += dy[a:a + n].double().abs().T @ x[a:a + n].double().abs()
    check("dw", dw, want, (sum(n for _, _, n in rows) + 24) * U32 * bound)
