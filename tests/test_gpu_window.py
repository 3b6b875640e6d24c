"""GPU parity of attention within a sliding window with first rows in view, and
of its gradients, with the 64-bit reference (tests/layer_reference.py), within
its derived bounds.

Every unused row and every key that no query sees holds NaN or infinity, and
every output starts as NaN.  Inputs are seeded.
"""
import math

import pytest
import torch

import layer_reference as L
import overlap_tiling_trapezoidal_amd as tdp
from harness import note
import test_gpu_tokens as tokens
from test_gpu_tokens import DT, NAN, check, check_rest, layout, poisoned, to_device

pytestmark = pytest.mark.gpu
ALL = tdp.TDP_WINDOW_ALL

CASES = [
    # q caps, q lens, k caps, k lens (None: the queries'), q heads, k heads, D, window (step, back, ahead, sinks),
    # ragged ranges, layout
    ((1,), (1,), None, None, 1, 1, 8, (1, 0, 0, 0), False, "rows"),
    ((300,), (300,), None, None, 2, 1, 64, (1, 63, 0, 4), False, "packed"),
    ((260, 70), (257, 70), None, None, 1, 1, 128, (1, ALL, 0, 0), True, "rows"),          # causal
    ((130,) * 2, (130, 1), None, None, 4, 2, 32, (1, 0, 0, 3), False, "heads"),           # itself and the first
    ((250, 200), (249, 200), None, None, 2, 2, 128, (40, 1, 0, 40), True, "rows"),        # frames and the first
    ((250,), (250,), None, None, 2, 1, 40, (33, 1, 1, 0), False, "rows"),                 # both ways
    ((200, 31), (190, 31), None, None, 3, 3, 96, (7, ALL, ALL, 0), True, "packed"),       # all
    ((513,), (513,), None, None, 1, 1, 72, (64, 2, 0, 100), False, "rows"),               # sinks across blocks
    ((700,), (700,), None, None, 6, 1, 64, (1, 100, 0, 70), False, "rows"),               # sinks end inside a block
    ((1,) * 3, (1, 1, 1), (900,) * 3, (900, 333, 0), 8, 2, 128, (1, 511, 0, 4), False, "rows"),   # new tokens
    ((1,) * 2, (1, 0), (3000,) * 2, (2999, 3000), 4, 4, 64, (1, 1500, 0, 64), False, "rows"),     # keys split
    ((5,) * 2, (5, 5), (40,) * 2, (3, 40), 2, 1, 128, (1, 7, 0, 2), False, "rows"),       # queries before the first key
    ((64,), (64,), (400,), (390,), 2, 1, 64, (32, 3, 0, 32), True, "heads"),              # newest frames over a cache
    ((90,), (90,), (77,), (77,), 2, 2, 32, (8, 2, 1, 200), False, "rows"),                # sinks past the end
    ((2,), (2,), (9,), (9,), 1, 1, 64, (1 << 24, ALL, ALL, ALL), False, "rows"),          # the largest values
    ((600,) * 28, tuple(600 - 20 * i for i in range(28)), None, None, 8, 8, 32, (1, ALL, 0, 0), False, "rows"),  # chunks
    ((1300,) * 2, (1300, 1200), None, None, 16, 16, 32, (1, 100, 0, 130), False, "rows"),  # first rows' blocks split
    ((1300,) * 2, (1300, 1200), None, None, 16, 16, 32, (50, 3, 1, 50), False, "packed"),
    ((700,) * 2, (700, 611), None, None, 4, 2, 96, (1, ALL, 0, 0), False, "rows"),         # parts of many rows joined
    ((300, 211), (300, 17), (2100, 2000), (2099, 40), 8, 2, 40, (1, 1500, 0, 64), True, "packed"),
]
IDS = [f"{'x'.join(map(str, c[0]))}-h{c[4]}.{c[5]}-d{c[6]}-{'.'.join(map(str, c[7]))}" for c in CASES]


def setup(case, dt, cuda, seed):
    qc, ql, kc, kl, hq, hk, D, window, ragged, strided = case
    gen = torch.Generator().manual_seed(seed)
    qseqs, qrows = layout(qc, ql, cuda, ragged)
    kseqs, krows = (qseqs, qrows) if kc is None else layout(kc, kl, cuda, ragged)
    q = poisoned(gen, qseqs, qrows, hq, D, dt)
    k, v = (poisoned(gen, kseqs, krows, hk, D, dt) for _ in range(2))
    seen = [L.visible(window, kn, qn) for (_, _, qn), (_, _, kn) in zip(qrows, krows)]
    for m, (a, _, n) in zip(seen, krows):   # a key that no query sees may hold anything
        out = ~m.any(0)
        k[a:a + n][out] = NAN
        v[a:a + n][out] = math.inf
    return gen, qseqs, qrows, kseqs, krows, q, k, v, seen


def forward(case, dt, cuda, seed):
    gen, qseqs, qrows, kseqs, krows, q, k, v, seen = setup(case, dt, cuda, seed)
    hq, hk, D, strided = case[4], case[5], case[6], case[9]
    win = tdp.make_window(*case[7])
    dev = [to_device(t, cuda, strided) for t in (q, k, v)]
    out = to_device(torch.full_like(q, NAN), cuda, strided)
    lse = torch.full((hq, qseqs.total_rows), NAN, device=cuda)
    ws = tdp.allocate_window_attention_workspace(qseqs, kseqs, win, hq, hk, D, cuda)
    if ws is not None:
        ws.fill_(0xff)
    note(f"window attention {case} {dt}")
    tdp.tdp_window_attention(qseqs, kseqs, win, *dev, out, lse, workspace=ws)
    torch.cuda.synchronize()
    return gen, qseqs, qrows, kseqs, krows, q, k, v, seen, win, dev, out, lse


def heads_of(case, qrows, krows, seen):
    hq, hk = case[4], case[5]
    for (qa, _, qn), (ka, _, kn), m in zip(qrows, krows, seen):
        for h in range(hq):
            yield slice(qa, qa + qn), slice(ka, ka + kn), h, h // (hq // hk), m


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_window_attention(case, dtype, cuda):
    dt, D = DT[dtype], case[6]
    _, _, qrows, _, krows, q, k, v, seen, _, _, out, lse = forward(case, dt, cuda, 31)
    check_rest("out", out, qrows)
    check_rest("lse", lse.t(), qrows, -math.inf)
    for qr, kr, h, g, m in heads_of(case, qrows, krows, seen):
        o, ob, l, lb = L.window_attention(q[qr, h], k[kr, g], v[kr, g], m, D ** -0.5, dt)
        check("out", out[qr, h], o, ob)
        live = torch.isfinite(l)
        got = lse[h, qr].double().cpu()
        assert (got[~live] == -math.inf).all()
        check("lse", got[live], l[live], lb[live])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_window_attention_backward(case, dtype, cuda):
    dt, D, hk, strided = DT[dtype], case[6], case[5], case[9]
    gen, qseqs, qrows, kseqs, krows, q, k, v, seen, win, dev, out, lse = forward(case, dt, cuda, 32)
    g = poisoned(gen, qseqs, qrows, case[4], D, dt)
    gd = to_device(g, cuda, strided)
    dq, dk, dv = (to_device(torch.full_like(t, NAN), cuda, strided) for t in (q, k, v))
    ws = tdp.allocate_window_attention_backward_workspace(qseqs, kseqs, win, case[4], hk, D, cuda)
    ws.fill_(0xff)
    for a, c, n in qrows:
        out[a + n:a + c] = NAN
        lse[:, a + n:a + c] = NAN
    note(f"window attention backward {case} {dt}")
    tdp.tdp_window_attention_backward(qseqs, kseqs, win, *dev, out, lse, gd, dq, dk, dv, ws)
    torch.cuda.synchronize()
    check_rest("dq", dq, qrows)
    check_rest("dk", dk, krows)
    check_rest("dv", dv, krows)
    oc, sums = out.cpu(), {}
    for qr, kr, h, gh, m in heads_of(case, qrows, krows, seen):
        r = L.window_attention(q[qr, h], k[kr, gh], v[kr, gh], m, D ** -0.5, dt, oc[qr, h], g[qr, h])
        check("dq", dq[qr, h], *r["dq"])
        for name in ("dk", "dv"):
            a = sums.setdefault((name, kr.start, gh), [kr, 0.0, 0.0])
            a[1], a[2] = a[1] + r[name][0], a[2] + r[name][1]
    for (name, _, gh), (kr, val, bound) in sums.items():
        check(name, (dk if name == "dk" else dv)[kr, gh], val, bound)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("heads,dim", [(4, 64), (2, 128)])
def test_window_that_holds_everything_is_plain_attention(heads, dim, dtype, cuda):
    """The same results, bit for bit, as tdp_attention where nothing is masked."""
    dt, gen = DT[dtype], torch.Generator(device=cuda).manual_seed(3)
    seqs = tdp.Sequences(2, 333, seq_len=torch.tensor([333, 200], dtype=torch.int32, device=cuda))
    q, k, v, g = (torch.randn(666, heads, dim, generator=gen, device=cuda).to(dt) for _ in range(4))
    win, res = tdp.make_window(back=None, ahead=None), []
    note(f"window of everything {heads} {dim} {dtype}")
    for w in (None, win):
        o, dq, dk, dv = (torch.empty_like(q) for _ in range(4))
        lse = torch.empty(heads, 666, device=cuda)
        if w is None:
            tdp.tdp_attention(seqs, seqs, q, k, v, o, lse)
            ws = tdp.allocate_attention_backward_workspace(seqs, seqs, heads, heads, dim, cuda)
            tdp.tdp_attention_backward(seqs, seqs, q, k, v, o, lse, g, dq, dk, dv, ws)
        else:
            tdp.tdp_window_attention(seqs, seqs, w, q, k, v, o, lse)
            ws = tdp.allocate_window_attention_backward_workspace(seqs, seqs, w, heads, heads, dim, cuda)
            tdp.tdp_window_attention_backward(seqs, seqs, w, q, k, v, o, lse, g, dq, dk, dv, ws)
        res.append((o, lse, dq, dk, dv))
    torch.cuda.synchronize()
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_window_prompt_and_token_by_token_agree(cuda):
    """A prompt at once and its tokens one by one over the growing cache: within two roundings of the type."""
    n, hq, hk, D = 150, 4, 2, 64
    gen = torch.Generator(device=cuda).manual_seed(9)
    q, k, v = (torch.randn(n, h, D, generator=gen, device=cuda).bfloat16() for h in (hq, hk, hk))
    win = tdp.make_window(back=40, sinks=3)
    whole, one = torch.empty_like(q), torch.empty_like(q)
    s = tdp.Sequences(1, n)
    note("prompt and token by token")
    tdp.tdp_window_attention(s, s, win, q, k, v, whole)
    used = torch.zeros(1, dtype=torch.int32, device=cuda)
    cache, new = tdp.Sequences(1, n, seq_len=used), tdp.Sequences(1, 1)
    ws = tdp.allocate_window_attention_workspace(new, cache, win, hq, hk, D, cuda)
    for i in range(n):
        used += 1
        tdp.tdp_window_attention(new, cache, win, q[i:i + 1], k, v, one[i:i + 1], workspace=ws)
    torch.cuda.synchronize()
    mag = v.abs().max().float()
    # weights of one row rounded at different maxima: 2^-8 of them each, and the outputs' roundings
    assert ((whole.float() - one.float()).abs() <= 4 * 2.0 ** -8 * mag).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("bias", [None, "pad", "lowest"])
def test_attention_parts_of_many_rows(bias, dtype, cuda):
    tokens.test_attention(((330,) * 2, (330, 301), (1100,) * 2, (1099, 530), 4, 1, 72, bias, False, "rows"), dtype, cuda)
