"""A layer of a tiled denoiser that looks at few frames, forward and backward, on
the buffers of a plan.

    extract -> layer norm, scaled and shifted per batch element -> q, k, v projection
            -> per-head norms with the three-axis rotation -> attention over the frames
               near a row's own and the first -> output projection -> blend

Every operator takes the used rows of all tiles in one call; nothing is copied to
the host and unused rows need no masking.  The plan's tiles have equal planes (a
window counts in frames) and no conditioning tokens.  Run it as
`python examples/tile_layer.py [workload]`.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import overlap_tiling_trapezoidal_amd as tdp  # noqa: E402


class TileLayer:
    """Weights, buffers and handles of one layer over one plan."""

    def __init__(self, plan, bufs, heads, kv_heads, head_dim, back=1, seed=0):
        dev, dt = bufs["tile_lat"].device, bufs["tile_lat"].dtype
        gen = torch.Generator(device=dev).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
        C, B = plan.cfg.channels, plan.cfg.batch
        planes = {tuple(tdp.tdp_plan_tile(plan, t).shape)[1:] for t in tdp.held_tiles(plan)}
        if len(planes) != 1 or plan.cfg.num_cond:
            raise ValueError("the layer's window needs tiles of equal planes and no conditioning tokens")
        (h, w), = planes
        self.heads, self.kv_heads, self.dim, self.channels = heads, kv_heads, head_dim, C
        init = lambda o, i: (randn(o, i) * i ** -0.5).to(dt)  # noqa: E731
        self.w_qkv, self.w_out = init((heads + 2 * kv_heads) * head_dim, C), init(C, heads * head_dim)
        self.scale, self.shift = 1 + 0.1 * randn(B, C), 0.1 * randn(B, C)   # of each batch element
        self.q_weight, self.k_weight = torch.ones(2, head_dim, device=dev)
        self.seqs = tdp.plan_sequences(plan, bufs["tile_count"], dev)
        self.window = tdp.make_window(step=h * w, back=back, sinks=h * w)
        side = head_dim // 3 // 2 * 2
        self.rope = tdp.tdp_rope_create(tdp.make_rope_config(
            head_dim, (head_dim - 2 * side, side, side), scale=(1 / 8, 1 / 32, 1 / 32)))

    def _product(self, x, weight):
        y = torch.empty(x.shape[0], weight.shape[0], dtype=x.dtype, device=x.device)
        ws = tdp.allocate_grouped_product_workspace(self.seqs, 1, *weight.shape, x.dtype, x.device)
        tdp.tdp_grouped_product(self.seqs, x, weight, y, workspace=ws)
        return y

    def _product_backward(self, x, weight, dy):
        dx, dw = torch.empty_like(x), torch.empty(weight.shape, device=x.device)
        ws = tdp.allocate_grouped_product_backward_workspace(self.seqs, 1, *weight.shape, x.dtype, x.device)
        tdp.tdp_grouped_product_backward(self.seqs, x, weight, dy, dx, dw, ws)
        return dx, dw

    def _split(self, qkv):
        t = qkv.view(qkv.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        return t[:, :self.heads], t[:, self.heads:self.heads + self.kv_heads], t[:, self.heads + self.kv_heads:]

    def forward(self, tile_lat, tile_pos):
        rows, hq, hk, D = self.seqs.total_rows, self.heads, self.kv_heads, self.dim
        x = tile_lat.view(rows, self.channels)
        n = torch.empty_like(x)
        tdp.tdp_layer_norm(self.seqs, x, self.scale, self.shift, n)
        q, k, v = self._split(self._product(n, self.w_qkv))
        qn, kn = (torch.empty(rows, h, D, dtype=x.dtype, device=x.device) for h in (hq, hk))
        tdp.tdp_qk_norm_rope(self.rope, self.seqs, tile_pos, q, k, self.q_weight, self.k_weight, qn, kn)
        out, lse = torch.empty_like(qn), torch.empty(hq, rows, device=x.device)
        ws = tdp.allocate_window_attention_workspace(self.seqs, self.seqs, self.window, hq, hk, D, x.device)
        tdp.tdp_window_attention(self.seqs, self.seqs, self.window, qn, kn, v, out, lse, workspace=ws)
        y = self._product(out.view(rows, hq * D), self.w_out)
        return y, (x, n, q, k, v, qn, kn, out, lse, tile_pos)

    def backward(self, dy, saved):
        """Gradients of the tile rows and of every weight."""
        x, n, q, k, v, qn, kn, out, lse, tile_pos = saved
        rows, hq, hk, D = self.seqs.total_rows, self.heads, self.kv_heads, self.dim
        dout, d_w_out = self._product_backward(out.view(rows, hq * D), self.w_out, dy)
        dqkv = torch.empty(rows, (hq + 2 * hk) * D, dtype=dy.dtype, device=dy.device)
        dq, dk, dv = self._split(dqkv)
        ws = tdp.allocate_window_attention_backward_workspace(self.seqs, self.seqs, self.window, hq, hk, D, dy.device)
        tdp.tdp_window_attention_backward(self.seqs, self.seqs, self.window, qn, kn, v, out, lse,
                                          dout.view(rows, hq, D), dq, dk, dv, ws)
        dwq, dwk = torch.empty(2, D, device=dy.device)
        ws = tdp.allocate_qk_norm_rope_workspace(self.rope, self.seqs, hq, hk, dy.device)
        tdp.tdp_qk_norm_rope_backward(self.rope, self.seqs, tile_pos, q, k, self.q_weight, self.k_weight, dq, dk,
                                      dq, dk, dwq, dwk, ws)
        dn, d_w_qkv = self._product_backward(n, self.w_qkv, dqkv)
        dscale, dshift = torch.empty_like(self.scale), torch.empty_like(self.shift)
        ws = tdp.allocate_layer_norm_workspace(self.seqs, self.channels, len(self.scale), dy.device)
        tdp.tdp_layer_norm_backward(self.seqs, x, self.scale, dn, dn, dscale, dshift, ws)
        return {"tile_lat": dn, "w_qkv": d_w_qkv, "w_out": d_w_out, "q_weight": dwq, "k_weight": dwk,
                "scale": dscale, "shift": dshift}


def run(workload, heads=8, kv_heads=4, head_dim=64, device="cuda"):
    """Extract, one layer, blend; returns the plan, its buffers, the layer, its results and gradients."""
    from synth import make_inputs
    wl, dev = workload, torch.device(device)
    inp = make_inputs(wl)
    plan = tdp.tdp_plan_create(tdp.make_config(wl.batch, wl.channels, wl.shape, wl.tiling, wl.num_cond,
                                               in_dtype=wl.dtype))
    if wl.dtype == "bf16":
        lat = torch.from_numpy(inp["latent"].view("int16")).view(torch.bfloat16).to(dev)
    else:
        lat = torch.from_numpy(inp["latent"]).to(dev)
    bufs = tdp.allocate_extract_outputs(plan, dev)
    tdp.tdp_extract(plan, lat, torch.from_numpy(inp["pos"]).to(dev), **bufs)
    layer = TileLayer(plan, bufs, heads, kv_heads, head_dim)
    y, saved = layer.forward(bufs["tile_lat"], bufs["tile_pos"])
    out = tdp.allocate_output(plan, dev)
    tdp.tdp_blend(plan, y.view(-1), bufs["cond_row"], bufs["cond_k"], out)
    grads = layer.backward(y, saved)   # of half the sum of squares of the tile outputs
    return plan, bufs, layer, (y, saved, out), grads


def main():
    from synth import WORKLOADS
    name = sys.argv[1] if len(sys.argv) > 1 else "ltx"
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
