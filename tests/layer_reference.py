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


def far_parts(x, eps):
    """The same where the mean's own error is taken out again: what is left of it scales with the row's spread,
    not with its offset."""
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = d.square().mean(1, keepdim=True)
    r = 1.0 / torch.sqrt(var + eps)
    first = 48 * U32 * x.abs().mean(1, keepdim=True)
    # differences from the first mean are no larger than |d| + first; their mean is a sum like the first
    dm = 48 * U32 * (d.abs().mean(1, keepdim=True) + first)
    dd = dm + U32 * (2 * d.abs() + first)
    ddm = dd.mean(1, keepdim=True)
    dvar = 50 * U32 * var + 2 * (d.abs() * dd).mean(1, keepdim=True) + ddm * ddm + dd.square().mean(1, keepdim=True)
    return d, dd, r, 0.5 * dvar / (var + eps) + 3 * U32


def layer_norm(x, w, b, eps, dtype, parts=_norm_parts):
    x, w, b = x.double(), w.double(), b.double()
    d, dd, r, dr = parts(x, eps)
    n = d * r * w
    y = n + b
    return y, dd * r * w.abs() + n.abs() * (dr + 3 * U32) + U32 * y.abs() + half_step(dtype) * y.abs()


def layer_norm_backward(x, w, dy, eps, dtype, parts=_norm_parts):
    """(dx, bound, dw, bound, db, bound); the sums over these rows alone."""
    x, w, dy = x.double(), w.double(), dy.double()
    d, dd, r, dr = parts(x, eps)
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


def visible(window, n, q):
    """(q, n) truth: key j takes part for query i, straight from the definition."""
    step, back, ahead, sinks = window
    t = torch.div(torch.arange(q)[:, None] + (n - q), step, rounding_mode="floor")
    j = torch.arange(n)[None, :]
    return (j < (t + 1 + ahead) * step) & ((j >= (t - back) * step) | (j < sinks))


def window_attention(q, k, v, seen, scale, dtype, o_given=None, dout=None):
    """One head: q (m, D), k and v (n, D), seen (m, n).  Forward: (o, bound, lse, bound); with dout and the
    forward's stored o the gradients: a dict of name -> (value, bound)."""
    q, k, v = q.double(), k.double().clone(), v.double().clone()
    D, (m, n) = q.shape[1], seen.shape
    k[~seen.any(0)] = 0.0
    v[~seen.any(0)] = 0.0
    live = seen.any(1)
    zero = torch.zeros(m, dtype=torch.float64)
    s = torch.where(seen, scale * q @ k.T, -float("inf"))
    top = torch.where(live, s.max(1).values if n else zero, zero)
    e = torch.exp(s - top[:, None])
    l = e.sum(1)
    p = e / torch.where(live, l, torch.ones_like(l))[:, None]
    lse = torch.where(live, top + torch.log(l), -float("inf"))
    o = p @ v
    # a weight before its normalisation: the score's dot product, its scaling and the exponent
    sm = torch.where(seen, s.abs(), zero[:, None])
    ds = (D + 4) * U32 * scale * (q.abs() @ k.abs().T) + 6 * U32 * (sm + top.abs()[:, None]) + 4 * U32
    ds = torch.where(seen, ds, zero[:, None])
    dmax = ds.max(1).values if n else zero
    rnd = half_step(dtype) if dtype == torch.bfloat16 else 0.0
    o_bound = (2 * dmax[:, None] + (n + 20) * U32 + rnd) * (p @ v.abs()) + half_step(dtype) * o.abs()
    lse_bound = torch.where(live, dmax + (n + 20) * U32 + 2 * U32 * lse.abs(), zero)
    if dout is None:
        return o, o_bound, lse, lse_bound
    g, og = dout.double(), o_given.double()
    dp, delta = g @ v.T, (g * og).sum(1, keepdim=True)
    z = p * (dp - delta)
    pe = p * (ds + lse_bound[:, None])
    ze = pe * (dp - delta).abs() + p * (D + 4) * U32 * (g.abs() @ v.abs().T + (g.abs() * og.abs()).sum(1, keepdim=True))
    ze = ze + rnd * z.abs() + 2 * U32 * z.abs()
    res = {}
    for name, zz, ee, x, chain in (("dq", z, ze, k, n + 20), ("dk", z.T, ze.T, q, m + 20)):
        val = scale * zz @ x
        res[name] = (val, scale * (ee + chain * U32 * zz.abs()) @ x.abs() + half_step(dtype) * val.abs())
    dv = p.T @ g
    res["dv"] = (dv, (pe.T + (rnd + (m + 20) * U32) * p.T) @ g.abs() + half_step(dtype) * dv.abs())
    return res


def product(x, w, dtype):
    """x (m, K) times w (N, K) transposed: (y, bound).  K products and sums in one chain, a join's at most 16."""
    x, w = x.double(), w.double()
    y = x @ w.T
    return y, (x.shape[1] + 24) * U32 * (x.abs() @ w.abs().T) + half_step(dtype) * y.abs()
