"""Launches of the token operators that tests/test_gpu_tokens.py does not make,
against the same 64-bit reference: rows split over workgroups in the gradients
of keys and values, every ending of their three-buffer walk, biases over many
key blocks, rows handed from block to block in the rotation and the norms, four
passes of heads at once, attention on a stream of its own and in a graph."""
import math

import pytest
import torch

import overlap_tiling_trapezoidal_amd as tdp
import test_gpu_tokens as G
import token_reference as R
from harness import note

pytestmark = pytest.mark.gpu
DT, NAN = G.DT, float("nan")

# q caps, q lens, k caps, k lens, q heads, k heads, head_dim, bias, ragged, strided, as in G.ATTN
ATTN = {
    # query rows times heads of a key head >= 1024 against few keys: rows split, parts that start inside a head
    "split-3": ((400,) * 2, (390, 130), (77,) * 2, (77, 60), 4, 1, 64, None, False, "rows"),
    "split-4-d40-random": ((700,), (690,), (90,), (90,), 6, 2, 40, "random", False, "rows"),
    "split-2-d128-pad": ((300,) * 3, (300, 0, 299), (130,) * 3, (130, 130, 1), 4, 1, 128, "pad", False, "packed"),
    "split-2-d128-group-1": ((1100, 700), (1100, 650), (40, 33), (40, 33), 1, 1, 128, None, True, "heads"),
    "split-3-no-keys": ((400,) * 2, (400, 400), (64,) * 2, (0, 64), 4, 1, 128, None, False, "rows"),
    # 2, 3, 5, 6 blocks of 64 rows for each key block, and 4 and 8 with two heads
    "blocks-2-3-5-6": ((128, 150, 300, 380), (128, 150, 300, 380), (90, 20, 128, 64), (90, 20, 128, 64), 1, 1, 128, None,
                       True, "rows"),
    "blocks-shared": ((150, 65), (129, 65), (129, 70), (129, 70), 4, 2, 128, None, True, "packed"),
    # six and seven key blocks with a bias, some of them all out, four row blocks
    "bias-d96-pad": ((200,) * 2, (200, 180), (400,) * 2, (400, 390), 2, 1, 96, "pad", False, "rows"),
    "bias-d128-random": ((200,) * 2, (200, 180), (420,) * 2, (420, 330), 2, 2, 128, "random", False, "packed"),
    "bias-d128-lowest": ((200,) * 2, (200, 180), (400,) * 2, (400, 390), 2, 2, 128, "lowest", False, "heads"),
    "bias-d64-pad": ((70,) * 2, (70, 33), (600,) * 2, (600, 555), 2, 1, 64, "pad", False, "rows"),
    # 20 heads of 128 and 40 of 64
    "heads-20": ((90,), (90,), (90,), (90,), 20, 20, 128, None, False, "packed"),
    "heads-40": ((90,), (80,), (90,), (80,), 40, 40, 64, None, False, "packed"),
}


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("name", list(ATTN))
def test_attention(name, dtype, cuda):
    G.test_attention(ATTN[name], dtype, cuda)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("name", list(ATTN))
def test_attention_backward(name, dtype, cuda):
    G.test_attention_backward(ATTN[name], dtype, cuda)


@pytest.mark.parametrize("q_rows,k_rows", [(400, 77), (3, 2049)], ids=["rows-split", "keys-split"])
def test_attention_on_another_stream_and_in_a_graph(q_rows, k_rows, cuda):
    """Both attention calls with split work: the eager bits on a side stream and in every replay."""
    gen = torch.Generator().manual_seed(12)
    qs, ks = tdp.Sequences(2, q_rows), tdp.Sequences(2, k_rows)
    q, g = (torch.randn(2 * q_rows, 4, 64, generator=gen).to(torch.bfloat16).to(cuda) for _ in range(2))
    k, v = (torch.randn(2 * k_rows, 1, 64, generator=gen).to(torch.bfloat16).to(cuda) for _ in range(2))
    ws = tdp.allocate_attention_workspace(qs, ks, 4, 1, 64, cuda)
    wsb = tdp.allocate_attention_backward_workspace(qs, ks, 4, 1, 64, cuda)
    outs = [torch.empty_like(q), torch.empty(4, 2 * q_rows, device=cuda), *(torch.empty_like(t) for t in (q, k, v))]

    def call(stream=None):
        tdp.tdp_attention(qs, ks, q, k, v, outs[0], outs[1], workspace=ws, stream=stream)
        tdp.tdp_attention_backward(qs, ks, q, k, v, outs[0], outs[1], g, *outs[2:], wsb, stream=stream)

    def clear():
        for t in outs:
            t.fill_(NAN)
    note("eager")
    call()
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs]
    assert all(torch.isfinite(t).all() for t in ref)
    side = torch.cuda.Stream()
    clear()
    side.wait_stream(torch.cuda.current_stream())
    note("another stream")
    call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    graph = torch.cuda.CUDAGraph()
    note("capture")
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        clear()
        note(f"replay {i}")
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
        (q.float().sum() + 1).item()   # the program's own work between replays


# ---- rotation and norms: several blocks of rows per workgroup -------------------

def short(n, longest):
    """n sequences of 1 .. longest rows of which none, one or all are used."""
    caps = tuple(1 + (7 * i) % longest for i in range(n))
    return caps, tuple((0, 1, c)[i % 3] for i, c in enumerate(caps))


# head_dim, rot dims, heads q, k, sequences, longest, pairing, point, strided (as in G.ROPE)
ROWS = {
    # 9000 blocks of four rows: two in a row per workgroup of the forward, 14 to 74 of the backward
    "d128-5.2-interleaved": (128, (44, 42, 42), 5, 2, 3000, 11, "interleaved", "middle", "rows"),
    "d128-5.2-halves": (128, (44, 42, 42), 5, 2, 3000, 11, "halves", "start", "packed"),
    # the same with the four-pass form (16 heads fill four passes of four)
    "d72-16.3-halves": (72, (24, 24, 24), 16, 3, 3000, 11, "halves", "middle", "rows"),
    "d72-16.3-interleaved": (72, (24, 20, 20), 16, 3, 3000, 11, "interleaved", "middle", "packed"),
    # few heads: eight rows per wave side by side, two blocks of 32 rows per workgroup
    "d32-2.1-halves": (32, (12, 10, 10), 2, 1, 4200, 40, "halves", "middle", "rows"),
    # four-pass form, one block per workgroup
    "d128-16.5-interleaved": (128, (44, 42, 42), 16, 5, 40, 9, "interleaved", "middle", "packed"),
    "d128-20.3-halves": (128, (44, 42, 42), 20, 3, 40, 9, "halves", "middle", "heads"),
    "d64-40.40-halves": (64, (24, 20, 20), 40, 40, 40, 9, "halves", "middle", "packed"),
}


def setup(name, dtype, cuda, seed):
    D, rot_dims, hq, hk, n, longest, pairing, point, strided = ROWS[name]
    caps, lens = short(n, longest)
    case = (D, rot_dims, hq, hk, caps, lens, True, pairing, point, strided, 1000.0)
    gen, seqs, rows, rope, pos, planes, rot = G.rope_setup(case, dtype, cuda, seed)
    used, owned = (torch.zeros(seqs.total_rows, dtype=torch.bool) for _ in range(2))
    for a, c, m in rows:
        owned[a:a + c] = True
        used[a:a + m] = True
    return gen, seqs, rows, rope, pos, torch.cat(planes, 1), rot, used, owned


def check_rows(name, got, used, owned, want, bound):
    got = got.detach().double().cpu()
    assert (got[owned & ~used] == 0).all(), f"{name}: unused rows are not 0"
    assert torch.isnan(got[~owned]).all(), f"{name}: rows outside the sequences were written"
    G.check(name, got[used], want, bound)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("name", list(ROWS))
def test_rows_forward(name, dtype, cuda):
    dt, (D, _, hq, hk, *_, strided) = DT[dtype], ROWS[name]
    gen, seqs, rows, rope, pos, planes, rot, used, owned = setup(name, dtype, cuda, 21)
    q, k = (G.poisoned(gen, seqs, rows, h, D, dt) for h in (hq, hk))
    wq, wk = (1 + 0.3 * torch.randn(D, generator=gen) for _ in range(2))
    dev = [G.to_device(t, cuda, strided) for t in (q, k)]
    for x, xd in ((q, dev[0]), (k, dev[1])):
        y = G.to_device(torch.full_like(x, NAN), cuda, strided)
        note(f"rope {name} {dtype}")
        tdp.tdp_rope_apply(rope, seqs, pos, xd, y)
        torch.cuda.synchronize()
        want, mag = R.turn(x[used].double(), planes, *rot)
        # as in G.test_rope_apply: angles 4.8 u, cos and sin 2 u, two products and a sum 3 u
        check_rows("y", y, used, owned, want, 12 * R.U32 * mag + R.half_step(dt) * want.abs())
    outs = [G.to_device(torch.full_like(t, NAN), cuda, strided) for t in (q, k)]
    note(f"norm rope {name} {dtype}")
    tdp.tdp_qk_norm_rope(rope, seqs, pos, *dev, wq.to(cuda), wk.to(cuda), *outs, eps=1e-5)
    torch.cuda.synchronize()
    for x, w, y in ((q, wq, outs[0]), (k, wk, outs[1])):
        check_rows("y", y, used, owned, *R.norm_rope(x[used], w, planes, rot, 1e-5, dt))


def sum_chain(D, heads, other, blocks):
    """Additions one weight gradient passes through: a lane's rows, its wave, the workgroup, the partial sums (768
    workgroups shared by queries and keys in proportion to their heads, 16 strided sums each, joined)."""
    lanes = 1
    while lanes * 8 < D:
        lanes *= 2
    per = 64 // lanes
    wgs = min(blocks, max(1, 768 * heads // (heads + other) - 1))
    return math.ceil(blocks / wgs) * math.ceil(heads / per) + int(math.log2(per)) + 2 + math.ceil(768 / 16) + 16


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("name", list(ROWS))
def test_rows_backward(name, dtype, cuda):
    dt, (D, _, hq, hk, n, longest, _, _, strided) = DT[dtype], ROWS[name]
    gen, seqs, rows, rope, pos, planes, rot, used, owned = setup(name, dtype, cuda, 22)
    q, k, gq, gk = (G.poisoned(gen, seqs, rows, h, D, dt) for h in (hq, hk, hq, hk))
    wq, wk = (1 + 0.3 * torch.randn(D, generator=gen) for _ in range(2))
    dev = [G.to_device(t, cuda, strided) for t in (q, k)]
    grads = [G.to_device(t, cuda, strided) for t in (gq, gk)]
    outs = [G.to_device(torch.full_like(t, NAN), cuda, strided) for t in (q, k)]
    dws = [torch.full((D,), NAN, device=cuda) for _ in range(2)]
    ws = tdp.allocate_qk_norm_rope_workspace(rope, seqs, hq, hk, cuda)
    ws.fill_(0xff)
    note(f"norm rope backward {name} {dtype}")
    tdp.tdp_qk_norm_rope_backward(rope, seqs, pos, *dev, wq.to(cuda), wk.to(cuda), *grads, *outs, *dws, ws, eps=1e-5)
    torch.cuda.synchronize()
    blocks = n * ((longest + 3) // 4)
    for x, w, g, dx, dw, heads in ((q, wq, gq, outs[0], dws[0], hq), (k, wk, gk, outs[1], dws[1], hk)):
        want, bound, want_dw, bound_dw = R.norm_rope_backward(x[used], w, g[used], planes, rot, 1e-5, dt)
        check_rows("dx", dx, used, owned, want, bound)
        # the reference's 140 u: 40 u per term and a chain of 100 additions
        chain = sum_chain(D, heads, hq + hk - heads, blocks)
        G.check("dw", dw, want_dw, bound_dw * max(1.0, (40 + chain) / 140))
