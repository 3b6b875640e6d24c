"""examples/tile_attention.py beyond one extract: the rows in use are those of the
last one."""
import pytest
import torch

import test_gpu_token_use as U
from harness import note

pytestmark = pytest.mark.gpu


def test_layer_follows_the_used_rows(cuda):
    """A layer made while the slots held fewer rows gives what one made afterwards does, forward and backward."""
    note("layer made before the extract")
    mod = U.example()
    plan, bufs, layer, _, _ = mod.run(U.SMALL_COND, heads=4, kv_heads=2, head_dim=64, device=cuda)
    counts = bufs["tile_count"].clone()
    bufs["tile_count"].fill_(1)
    early = mod.TileAttention(plan, bufs, 4, 2, 64)
    bufs["tile_count"].copy_(counts)
    res = []
    for one in (early, layer):
        y, saved = one.forward(bufs["tile_lat"], bufs["tile_pos"])
        grads = one.backward(y, saved)
        res.append([y, *(grads[n] for n in sorted(grads))])
    torch.cuda.synchronize()
    for a, b in zip(*res):
        assert torch.isfinite(b).all() and torch.equal(a, b)
