"""64-bit reference of the layer operators, on the CPU, and error bounds.

Each function returns the value and a bound on what the operator may be off:
u = 2^-24 per fp32 operation along the longest chain, and half a step of the
tensors' type for each rounding to it.
"""
import torch

from token_reference import U32, half_step


def _norm_parts(x, eps):
    """(differences, their error, r, its relative error) of rows x (rows, C)."""
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = d.square().mean(1, keepdim=True)
    r = 1.0 / torch.sqrt(var + eps)
    # a sum over a row: at most 32 terms in a lane, 8 joins, one product: 48 u with room
    dm = 48 * U32 * x.abs().mean(1, keepdim=True)
    dd = dm + U32 * d.abs()
    dvar = 50 * U32 * var + 2 * d.abs().mean(1, keepdim=True) * dm + dm * dm
    return d, dd, r, 0.5 * dvar / (var + eps) + 3 * U32


def layer_norm(x, w, b, eps, dtype):
    x, w, b = x.double(), w.double(), b.double()
    d, dd, r, dr = _norm_parts(x, eps)
    n = d * r * w
    y = n + b
    return y, dd * r * w.abs() + n.abs() * (dr + 3 * U32) + U32 * y.abs() + half_step(dtype) * y.abs()


def layer_norm_backward(x, w, dy, eps, dtype):
    """(dx, bound, dw, bound, db, bound); the sums over these rows alone."""
    x, w, dy = x.double(), w.double(), dy.double()
    d, dd, r, dr = _norm_parts(x, eps)
    n, g = d * r, dy * w
    mg, c = g.mean(1, keepdim=True), (g * d).mean(1, keepdim=True) * r * r
    dx = r * (g - mg - d * c)
    dmg = 50 * U32 * g.abs().mean(1, keepdim=True)
    dc = r * r * (52 * U32 * (g * d).abs().mean(1, keepdim=True) + (g.abs() * dd).mean(1, keepdim=True)) + \
        c.abs() * (2 * dr + 4 * U32)
    bound = r * (dmg + d.abs() * dc + c.abs() * dd + 4 * U32 * (g.abs() + mg.abs() + (d * c).abs())) + \
        dx.abs() * (dr + 2 * U32) + half_step(dtype) * dx.abs()
    # a weight's sum: a workgroup's rows, its lanes and waves, then the workgroups: below 100 in a chain here
    dw, db = (dy * n).sum(0), dy.sum(0)
    dwb = (dy.abs() * (dd * r + n.abs() * (dr + 103 * U32))).sum(0)
    return dx, bound, dw, dwb, db, 100 * U32 * dy.abs().sum(0)
