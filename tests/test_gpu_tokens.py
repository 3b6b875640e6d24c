"""GPU parity of the rotation, the norms, attention and their gradients with
the 64-bit reference (tests/token_reference.py), within its derived bounds.

Every unused row of every input holds NaN and every output starts as NaN, so a
row that leaks in or is not written shows.  Inputs are seeded.
"""
import math

import pytest
import torch

import overlap_tiling_trapezoidal_amd as tdp
import token_reference as R
from harness import note

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


def layout(caps, lens, cuda, ragged, group=1):
    """Sequences and the (start, cap, len) of each, with two unowned rows before every range when ragged."""
    rows, ranges = [], []
    at = 0
    for c, n in zip(caps, lens):
        at += 2 if ragged else 0
        rows.append((at, c, n))
        ranges.append((at, at + c))
        at += c
    sl = torch.tensor(lens[::group], dtype=torch.int32, device=cuda)
    if not ragged:
        return tdp.Sequences(len(caps), caps[0], seq_len=sl, len_group=group), rows
    rr = torch.tensor(ranges, dtype=torch.int64, device=cuda)
    return tdp.Sequences(len(caps), max(caps), row_range=rr, total_rows=at + 1, seq_len=sl, len_group=group), rows


def poisoned(gen, seqs, rows, heads, dim, dt, layout_kind="rows"):
    """CPU values (rows, heads, dim) with NaN outside the used rows."""
    x = torch.randn(seqs.total_rows, heads, dim, generator=gen).to(dt)
    keep = torch.zeros(seqs.total_rows, dtype=torch.bool)
    for a, _, n in rows:
        keep[a:a + n] = True
    x[~keep] = NAN
    return x


def to_device(x, cuda, strided):
    """On the GPU: contiguous, or as a slice of a wider packed tensor, or head-major."""
    if strided == "packed":
        wide = torch.full((x.shape[0], x.shape[1] + 3, x.shape[2]), NAN, dtype=x.dtype, device=cuda)
        wide[:, 2:-1] = x.to(cuda)
        return wide[:, 2:-1]
    if strided == "heads":
        return x.transpose(0, 1).contiguous().to(cuda).transpose(0, 1)
    return x.to(cuda)


def check(name, got, want, bound):
    got = got.detach().double().cpu()
    assert torch.isfinite(got).all(), f"{name}: {(~torch.isfinite(got)).sum()} values are not finite"
    bad = (got - want).abs() > bound
    worst = ((got - want).abs() / bound.clamp_min(1e-300)).max() if bad.any() else 0
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} out of bound, worst {float(worst):.2f} of it"


def check_rest(name, out, rows, filled=0.0):
    """Unused rows of the sequences are `filled`, rows outside them untouched (NaN)."""
    out = out.detach().float().cpu()
    owned = torch.zeros(out.shape[0], dtype=torch.bool)
    for a, c, n in rows:
        owned[a:a + c] = True
        assert (out[a + n:a + c] == filled).all(), f"{name}: unused rows are not {filled}"
    assert torch.isnan(out[~owned]).all(), f"{name}: rows outside the sequences were written"


# ---- rotation and norms ----------------------------------------------------

ROPE = [
    # head dim, rot dims, heads q, k, caps, lens, ragged, pairing, point, strided, spread of positions
    (32, (12, 10, 10), 4, 4, (75,) * 4, (75,) * 4, False, "interleaved", "middle", "rows", 100.0),
    (128, (44, 42, 42), 5, 2, (33, 40, 1), (33, 17, 0), True, "halves", "middle", "packed", 4000.0),
    (64, (24, 20, 20), 16, 4, (9, 9), (9, 1), False, "halves", "start", "heads", 1e5),
    (8, (2, 2, 2), 1, 1, (130,), (129,), False, "interleaved", "start", "rows", 10.0),
    (16, (8, 0, 8), 3, 1, (5, 6), (5, 6), True, "halves", "middle", "packed", 1e6),
    (40, (16, 12, 12), 7, 7, (64,), (64,), False, "interleaved", "middle", "packed", 1000.0),
    (72, (0, 72, 0), 2, 2, (7, 3), (7, 2), True, "halves", "start", "heads", 1000.0),
    (96, (32, 32, 32), 6, 3, (21,), (20,), False, "halves", "middle", "rows", 1000.0),
    (256, (100, 78, 78), 2, 1, (10,), (10,), False, "interleaved", "middle", "rows", 1000.0),
    (128, (0, 0, 0), 2, 2, (12,), (11,), False, "interleaved", "middle", "rows", 1.0),
]
ROPE_IDS = [f"d{c[0]}-{c[7]}-{c[9]}-{i}" for i, c in enumerate(ROPE)]


def rope_setup(case, dtype, cuda, seed):
    D, rot_dims, hq, hk, caps, lens, ragged, pairing, point, strided, spread = case
    gen = torch.Generator().manual_seed(seed)
    seqs, rows = layout(caps, lens, cuda, ragged)
    freqs = [[1000.0 ** (-2.0 * i / max(r, 1)) for i in range(r // 2)] for r in rot_dims]
    rope = tdp.tdp_rope_create(tdp.make_rope_config(D, rot_dims, freqs=freqs, pairing=pairing, point=point))
    pos = torch.full((6 * seqs.total_rows,), NAN)
    planes = []
    for a, c, n in rows:
        p = torch.full((3, c, 2), NAN)
        s = (torch.rand(3, n, generator=gen) - 0.25) * spread
        p[:, :n, 0], p[:, :n, 1] = s, s + torch.rand(3, n, generator=gen) * 32
        pos[6 * a:6 * (a + c)] = p.reshape(-1)
        planes.append(p[:, :n])
    return gen, seqs, rows, rope, pos.to(cuda), planes, (rot_dims, freqs, pairing, point)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", ROPE, ids=ROPE_IDS)
def test_rope_apply(case, dtype, cuda):
    dt, D, hq, strided = DT[dtype], case[0], case[2], case[9]
    gen, seqs, rows, rope, pos, planes, rot = rope_setup(case, dtype, cuda, 1)
    x = poisoned(gen, seqs, rows, hq, D, dt)
    xd = to_device(x, cuda, strided)
    for inverse in (False, True):
        y = to_device(torch.full_like(x, NAN), cuda, strided)
        note(f"rope {case} {dtype} inverse={inverse}")
        tdp.tdp_rope_apply(rope, seqs, pos, xd, y, inverse=inverse)
        torch.cuda.synchronize()
        check_rest("y", y, rows)
        for (a, c, n), p in zip(rows, planes):
            want, mag = R.turn(x[a:a + n].double(), p, *rot, inverse=inverse)
            # cos and sin: angle within 3 * 2^-26 turns (4.8 u), the functions 2 u, two products and a sum 3 u
            check("y", y[a:a + n], want, 12 * R.U32 * mag + R.half_step(dt) * want.abs())
    # in place, and its own inverse up to two roundings
    z = xd.clone(memory_format=torch.preserve_format) if strided == "rows" else to_device(x, cuda, strided)
    tdp.tdp_rope_apply(rope, seqs, pos, z, z, inverse=True)
    torch.cuda.synchronize()
    for a, c, n in rows:
        assert torch.equal(z[a:a + n], y[a:a + n])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", ROPE, ids=ROPE_IDS)
def test_qk_norm_rope(case, dtype, cuda):
    dt, D, hq, hk, strided = DT[dtype], case[0], case[2], case[3], case[9]
    gen, seqs, rows, rope, pos, planes, rot = rope_setup(case, dtype, cuda, 2)
    q, k = (poisoned(gen, seqs, rows, h, D, dt) for h in (hq, hk))
    for t in (q, k):
        a, c, n = rows[0]
        if n:
            t[a, 0] = 0.0       # a head of zeros: eps alone
    wq, wk = (1 + 0.3 * torch.randn(D, generator=gen) for _ in range(2))
    qd, kd = to_device(q, cuda, strided), to_device(k, cuda, strided)
    yq, yk = (to_device(torch.full_like(t, NAN), cuda, strided) for t in (q, k))
    note(f"norm rope {case} {dtype}")
    tdp.tdp_qk_norm_rope(rope, seqs, pos, qd, kd, wq.to(cuda), wk.to(cuda), yq, yk, eps=1e-5)
    torch.cuda.synchronize()
    for name, x, w, y in (("q", q, wq, yq), ("k", k, wk, yk)):
        check_rest(name, y, rows)
        for (a, c, n), p in zip(rows, planes):
            check(name, y[a:a + n], *R.norm_rope(x[a:a + n], w, p, rot, 1e-5, dt))
    # without weights, in place
    tdp.tdp_qk_norm_rope(rope, seqs, pos, qd, kd, None, None, qd, kd, eps=1e-5)
    torch.cuda.synchronize()
    for name, x, y in (("q", q, qd), ("k", k, kd)):
        for (a, c, n), p in zip(rows, planes):
            check(name, y[a:a + n], *R.norm_rope(x[a:a + n], torch.ones(D), p, rot, 1e-5, dt))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", ROPE, ids=ROPE_IDS)
def test_qk_norm_rope_backward(case, dtype, cuda):
    dt, D, hq, hk, strided = DT[dtype], case[0], case[2], case[3], case[9]
    gen, seqs, rows, rope, pos, planes, rot = rope_setup(case, dtype, cuda, 3)
    q, k, gq, gk = (poisoned(gen, seqs, rows, h, D, dt) for h in (hq, hk, hq, hk))
    wq, wk = (1 + 0.3 * torch.randn(D, generator=gen) for _ in range(2))
    qd, kd, gqd, gkd = (to_device(t, cuda, strided) for t in (q, k, gq, gk))
    dq, dk = (to_device(torch.full_like(t, NAN), cuda, strided) for t in (q, k))
    dwq, dwk = torch.full((2, D), NAN, device=cuda)
    ws = tdp.allocate_qk_norm_rope_workspace(rope, seqs, hq, hk, cuda)
    note(f"norm rope backward {case} {dtype}")
    tdp.tdp_qk_norm_rope_backward(rope, seqs, pos, qd, kd, wq.to(cuda), wk.to(cuda), gqd, gkd, dq, dk, dwq, dwk, ws,
                                  eps=1e-5)
    torch.cuda.synchronize()
    for name, x, w, g, dx, dw in (("q", q, wq, gq, dq, dwq), ("k", k, wk, gk, dk, dwk)):
        check_rest(name, dx, rows)
        want_dw, bound_dw = torch.zeros(D).double(), torch.zeros(D).double()
        for (a, c, n), p in zip(rows, planes):
            v, b, w1, b1 = R.norm_rope_backward(x[a:a + n], w, g[a:a + n], p, rot, 1e-5, dt)
            check("d" + name, dx[a:a + n], v, b)
            want_dw, bound_dw = want_dw + w1, bound_dw + b1
        check("dw" + name, dw, want_dw, bound_dw)
    # in place over the outputs' gradients, weights' gradients not wanted: the same dx
    tdp.tdp_qk_norm_rope_backward(rope, seqs, pos, qd, kd, wq.to(cuda), wk.to(cuda), gqd, gkd, gqd, gkd, None, None, ws,
                                  eps=1e-5)
    torch.cuda.synchronize()
    for dx, g in ((dq, gqd), (dk, gkd)):
        for a, c, n in rows:
            assert torch.equal(dx[a:a + c], g[a:a + c])


# ---- attention --------------------------------------------------------------

ATTN = [
    # q caps, q lens, k caps, k lens (None: the queries'), q heads, k heads, D, bias, ragged, strided
    ((1,), (1,), None, None, 1, 1, 8, None, False, "rows"),
    ((75,) * 4, (75,) * 4, None, None, 2, 2, 32, None, False, "rows"),
    ((128, 33, 65), (128, 31, 64), None, None, 2, 1, 64, None, True, "packed"),
    ((200, 129), (199, 0), None, None, 4, 2, 128, None, True, "heads"),
    ((130,), (130,), (1,), (1,), 3, 1, 40, None, False, "rows"),
    ((60,) * 2, (60, 7), (257,) * 2, (256, 0), 4, 1, 72, None, False, "packed"),
    ((70,) * 3, (70, 70, 1), (77,) * 3, (77, 60, 77), 4, 2, 64, "pad", False, "rows"),
    ((40,) * 2, (40, 40), (64,) * 2, (64, 64), 2, 2, 128, "all", False, "rows"),
    ((40,) * 2, (40, 40), (64,) * 2, (64, 64), 2, 2, 96, "lowest", False, "rows"),
    ((50,), (50,), (90,), (90,), 2, 1, 64, "random", False, "heads"),
    ((1,) * 2, (1, 1), (1500,) * 2, (1500, 1111), 8, 2, 128, None, False, "rows"),       # keys split
    ((3,), (3,), (2049,), (2000,), 2, 1, 64, "pad", False, "rows"),                      # keys split
]
ATTN_IDS = [f"{'x'.join(map(str, c[0]))}-h{c[4]}.{c[5]}-d{c[6]}-{c[7]}-{c[9]}" for c in ATTN]


def attn_setup(case, dt, cuda, seed):
    qc, ql, kc, kl, hq, hk, D, bias_kind, ragged, strided = case
    gen = torch.Generator().manual_seed(seed)
    qseqs, qrows = layout(qc, ql, cuda, ragged)
    kseqs, krows = (qseqs, qrows) if kc is None else layout(kc, kl, cuda, ragged)
    q = poisoned(gen, qseqs, qrows, hq, D, dt)
    k, v = (poisoned(gen, kseqs, krows, hk, D, dt) for _ in range(2))
    bias = None
    if bias_kind:
        bias = torch.full((kseqs.total_rows,), NAN)
        for i, (a, c, n) in enumerate(krows):
            b = torch.zeros(n)
            if bias_kind == "pad":
                b[n // 3:n // 3 + n // 2] = -math.inf
            elif bias_kind == "random":
                b = 3 * torch.randn(n, generator=gen)
            elif bias_kind == "all":
                b[:] = -math.inf
            elif i == 0:
                b[1::2] = torch.finfo(torch.float32).min
            else:
                b[:] = torch.finfo(torch.bfloat16).min
            bias[a:a + n] = b
            out = b <= -1e30      # a key that takes no part may hold anything
            k[a:a + n][out] = NAN
            v[a:a + n][out] = math.inf
    return gen, qseqs, qrows, kseqs, krows, q, k, v, bias


def run_forward(case, dt, cuda, seed, scale=None):
    gen, qseqs, qrows, kseqs, krows, q, k, v, bias = attn_setup(case, dt, cuda, seed)
    hq, hk, D, strided = case[4], case[5], case[6], case[9]
    dev = [to_device(t, cuda, strided) for t in (q, k, v)]
    out = to_device(torch.full_like(q, NAN), cuda, strided)
    lse = torch.full((hq, qseqs.total_rows), NAN, device=cuda)
    ws = tdp.allocate_attention_workspace(qseqs, kseqs, hq, hk, D, cuda)
    bd = None if bias is None else bias.to(cuda)
    note(f"attention {case} {dt}")
    tdp.tdp_attention(qseqs, kseqs, *dev, out, lse, key_bias=bd, scale=scale, workspace=ws)
    torch.cuda.synchronize()
    return gen, qseqs, qrows, kseqs, krows, q, k, v, bias, dev, out, lse, bd


def heads_of(case, qrows, krows):
    hq, hk = case[4], case[5]
    for (qa, qc, qn), (ka, kc, kn) in zip(qrows, krows):
        for h in range(hq):
            yield slice(qa, qa + qn), slice(ka, ka + kn), h, h // (hq // hk)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", ATTN, ids=ATTN_IDS)
def test_attention(case, dtype, cuda):
    dt, D = DT[dtype], case[6]
    _, _, qrows, _, krows, q, k, v, bias, _, out, lse, _ = run_forward(case, dt, cuda, 5)
    check_rest("out", out, qrows)
    check_rest("lse", lse.t(), qrows, -math.inf)
    for qr, kr, h, g in heads_of(case, qrows, krows):
        o, ob, l, lb = R.attention(q[qr, h], k[kr, g], v[kr, g], None if bias is None else bias[kr], D ** -0.5, dt)
        check("out", out[qr, h], o, ob)
        live = torch.isfinite(l)
        got = lse[h, qr].double().cpu()
        assert (got[~live] == -math.inf).all()
        check("lse", got[live], l[live], lb[live])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", ATTN, ids=ATTN_IDS)
def test_attention_backward(case, dtype, cuda):
    dt, D, strided, hk = DT[dtype], case[6], case[9], case[5]
    gen, qseqs, qrows, kseqs, krows, q, k, v, bias, dev, out, lse, bd = run_forward(case, dt, cuda, 6)
    g = poisoned(gen, qseqs, qrows, case[4], D, dt)
    gd = to_device(g, cuda, strided)
    dq, dk, dv = (to_device(torch.full_like(t, NAN), cuda, strided) for t in (q, k, v))
    ws = tdp.allocate_attention_backward_workspace(qseqs, kseqs, case[4], hk, D, cuda)
    ws.fill_(0xff)
    for a, c, n in qrows:   # unused rows of the forward's results may hold anything too
        out[a + n:a + c] = NAN
        lse[:, a + n:a + c] = NAN
    note(f"attention backward {case} {dt}")
    tdp.tdp_attention_backward(qseqs, kseqs, *dev, out, lse, gd, dq, dk, dv, ws, key_bias=bd)
    torch.cuda.synchronize()
    check_rest("dq", dq, qrows)
    check_rest("dk", dk, krows)
    check_rest("dv", dv, krows)
    oc = out.cpu()
    sums = {}
    for qr, kr, h, gh in heads_of(case, qrows, krows):
        r = R.attention(q[qr, h], k[kr, gh], v[kr, gh], None if bias is None else bias[kr], D ** -0.5, dt,
                        oc[qr, h], g[qr, h])
        check("dq", dq[qr, h], *r["dq"])
        for name in ("dk", "dv"):
            a = sums.setdefault((name, kr.start, gh), [kr, 0.0, 0.0])
            a[1], a[2] = a[1] + r[name][0], a[2] + r[name][1]
    for (name, _, gh), (kr, val, bound) in sums.items():
        check(name, (dk if name == "dk" else dv)[kr, gh], val, bound)
