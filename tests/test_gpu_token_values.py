"""Values at the edge of the token operators' formulas: a norm without eps."""
import pytest
import torch

import overlap_tiling_trapezoidal_amd as tdp
import test_gpu_tokens as G
import token_reference as R
from harness import note

pytestmark = pytest.mark.gpu
DT, NAN = G.DT, float("nan")


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
