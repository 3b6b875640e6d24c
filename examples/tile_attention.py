"""One attention layer of a tiled denoiser, forward and backward, on the buffers
of a plan.

    extract -> q, k, v projections -> per-head norms with the three-axis rotation
            -> attention over each tile's used rows -> output projection -> blend

All tiles run in one call per operator: the plan's slots are the sequences, the
positions are tile_pos and the used rows tile_count, both as tdp_extract leaves
them on the GPU.  Run it as `python examples/tile_attention.py [workload]`.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import overlap_tiling_trapezoidal_amd as tdp  # noqa: E402


class TileAttention:
    """Weights, buffers and handles of one layer over one plan."""

    def __init__(self, plan, bufs, heads, kv_heads, head_dim, seed=0):
        dev = bufs["tile_lat"].device
        dt = bufs["tile_lat"].dtype
        gen = torch.Generator(device=dev).manual_seed(seed)
        C = plan.cfg.channels
        self.heads, self.kv_heads, self.dim, self.channels = heads, kv_heads, head_dim, C
        init = lambda o, i: (torch.randn(o, i, generator=gen, device=dev) * i ** -0.5).to(dt)  # noqa: E731
        self.w_qkv, self.w_out = init((heads + 2 * kv_heads) * head_dim, C), init(C, heads * head_dim)
        self.q_weight, self.k_weight = torch.ones(2, head_dim, device=dev)
        self.seqs = tdp.plan_sequences(plan, bufs["tile_count"], dev)
        side = head_dim // 3 // 2 * 2
        self.rope = tdp.tdp_rope_create(tdp.make_rope_config(
            head_dim, (head_dim - 2 * side, side, side), scale=(1 / 8, 1 / 32, 1 / 32)))
        # every row's slot and place in its sequence
        self.tile_count = bufs["tile_count"]
        self.slot = torch.zeros(self.seqs.total_rows, dtype=torch.int64, device=dev)
        self.place = torch.full((self.seqs.total_rows,), self.seqs.max_rows, dtype=torch.int32, device=dev)
        for s, (a, b) in enumerate(tdp.tdp_plan_sequences(plan)):
            self.slot[a:b] = s // plan.cfg.batch
            self.place[a:b] = torch.arange(b - a, dtype=torch.int32, device=dev)

    def used(self):
        """The rows that the last extract wrote, (rows, 1): a slot's others may hold anything."""
        return (self.place < self.tile_count[self.slot])[:, None]

    def forward(self, tile_lat, tile_pos):
        rows = self.seqs.total_rows
        hq, hk, D = self.heads, self.kv_heads, self.dim
        x = torch.where(self.used(), tile_lat.view(rows, self.channels), 0)
        qkv = (x @ self.w_qkv.T).view(rows, hq + 2 * hk, D)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        qn, kn = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty(
            rows, hk, D, dtype=q.dtype, device=q.device)
        tdp.tdp_qk_norm_rope(self.rope, self.seqs, tile_pos, q, k, self.q_weight, self.k_weight, qn, kn)
        out = torch.empty(rows, hq, D, dtype=q.dtype, device=q.device)
        lse = torch.empty(hq, rows, device=q.device)
        ws = tdp.allocate_attention_workspace(self.seqs, self.seqs, hq, hk, D, q.device)
        tdp.tdp_attention(self.seqs, self.seqs, qn, kn, v, out, lse, workspace=ws)
        y = out.view(rows, hq * D) @ self.w_out.T
        return y, (x, q, k, v, qn, kn, out, lse, tile_pos)

    def backward(self, dy, saved):
        """Gradients of the tile rows and of every weight."""
        x, q, k, v, qn, kn, out, lse, tile_pos = saved
        rows = self.seqs.total_rows
        hq, hk, D = self.heads, self.kv_heads, self.dim
        dy = torch.where(self.used(), dy, 0)
        d_w_out = dy.T @ out.view(rows, hq * D)
        dout = (dy @ self.w_out).view(rows, hq, D)
        dqkv = torch.empty(rows, hq + 2 * hk, D, dtype=dy.dtype, device=dy.device)
        dq, dk, dv = dqkv[:, :hq], dqkv[:, hq:hq + hk], dqkv[:, hq + hk:]
        ws = tdp.allocate_attention_backward_workspace(self.seqs, self.seqs, hq, hk, D, dy.device)
        tdp.tdp_attention_backward(self.seqs, self.seqs, qn, kn, v, out, lse, dout, dq, dk, dv, ws)
        dwq, dwk = torch.empty(2, D, device=dy.device)
        ws = tdp.allocate_qk_norm_rope_workspace(self.rope, self.seqs, hq, hk, dy.device)
        tdp.tdp_qk_norm_rope_backward(self.rope, self.seqs, tile_pos, q, k, self.q_weight, self.k_weight, dq, dk,
                                      dq, dk, dwq, dwk, ws)
        flat = dqkv.view(rows, -1)
        return {"tile_lat": flat @ self.w_qkv, "w_qkv": flat.T @ x, "w_out": d_w_out, "q_weight": dwq,
                "k_weight": dwk}


def run(workload, heads=8, kv_heads=4, head_dim=64, device="cuda"):
    """Extract, one layer, blend; returns the plan, its buffers, the layer, its results and gradients."""
    from synth import make_inputs
    wl = workload
    dev = torch.device(device)
    inp = make_inputs(wl)
    plan = tdp.tdp_plan_create(tdp.make_config(wl.batch, wl.channels, wl.shape, wl.tiling, wl.num_cond,
                                               in_dtype=wl.dtype))
    if wl.dtype == "bf16":
        lat = torch.from_numpy(inp["latent"].view("int16")).view(torch.bfloat16).to(dev)
    else:
        lat = torch.from_numpy(inp["latent"]).to(dev)
    bufs = tdp.allocate_extract_outputs(plan, dev)
    tdp.tdp_extract(plan, lat, torch.from_numpy(inp["pos"]).to(dev), **bufs)
    layer = TileAttention(plan, bufs, heads, kv_heads, head_dim)
    y, saved = layer.forward(bufs["tile_lat"], bufs["tile_pos"])
    out = tdp.allocate_output(plan, dev)
    tdp.tdp_blend(plan, y.view(-1), bufs["cond_row"], bufs["cond_k"], out)
    grads = layer.backward(y, saved)   # of half the sum of squares of the tile outputs
    return plan, bufs, layer, (y, saved, out), grads


def main():
    from synth import WORKLOADS
    name = sys.argv[1] if len(sys.argv) > 1 else "conditioned"
    plan, bufs, layer, (y, saved, out), grads = run(WORKLOADS[name])
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(10):
        y, saved = layer.forward(bufs["tile_lat"], bufs["tile_pos"])
        layer.backward(y, saved)
    torch.cuda.synchronize()
    print(f"{name}: {layer.seqs.num_seqs} tiles x batch, {layer.seqs.total_rows} rows, forward and backward "
          f"{(time.perf_counter() - t) * 100:.2f} ms")


if __name__ == "__main__":
    main()
