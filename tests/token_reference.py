"""64-bit reference of the token operators, on the CPU, and error bounds.

Each function returns the value and a bound on what the operator may be off:
u = 2^-24 per fp32 operation along the longest chain, and half a step of the
tensors' type for each rounding to it.
"""
import math

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    """Relative size of one rounding to a stored type (0 where it is fp32: counted in units of U32)."""
    return torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else U32


def pair_index(rot_dims, pairing):
    first, second, off = [], [], 0
    for r in rot_dims:
        for i in range(r // 2):
            first.append(off + (2 * i if pairing == "interleaved" else i))
            second.append(off + (2 * i + 1 if pairing == "interleaved" else i + r // 2))
        off += r
    return first, second


def turn(x, pos, rot_dims, freqs, pairing, point, inverse=False):
    """x (rows, heads, D) float64 turned by pos (3, rows, 2); also the pair magnitude |x0| + |x1| per element."""
    p = pos.double()
    p = (p[..., 0] + p[..., 1]) / 2 if point == "middle" else p[..., 0]
    ang = torch.cat([p[a][:, None] * torch.tensor(f, dtype=torch.float64)[None, :] for a, f in enumerate(freqs)], 1)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    if inverse:
        s = -s
    i0, i1 = pair_index(rot_dims, pairing)
    y, mag = x.clone(), x.abs()
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
    mag[..., i0] = mag[..., i1] = a.abs() + b.abs()
    return y, mag


def pair_mag(m, rot_dims, pairing):
    """Sum of a magnitude over each element's pair."""
    i0, i1 = pair_index(rot_dims, pairing)
    out = m.clone()
    out[..., i0] = out[..., i1] = m[..., i0] + m[..., i1]
    return out


def norm_rope(x, w, pos, rot, eps, dtype):
    """(y, bound) of turn(x * r * w)."""
    x = x.double()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    y, mag = turn(x * r * w.double(), pos, *rot)
    # sum of squares: 8 products and 5 joins, halved by the root; r, r * w, x * (r w): 12 u; the turn: 12 u
    return y, 24 * U32 * mag + half_step(dtype) * y.abs()


def norm_rope_backward(x, w, dy, pos, rot, eps, dtype):
    """(dx, bound, dw, bound)."""
    x, w = x.double(), w.double()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    n, mag = turn(dy.double(), pos, *rot, inverse=True)
    g, gm = n * w, mag * w.abs()
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdim=True))
    bound = 40 * U32 * r * (gm + x.abs() * r * r * (gm * x.abs()).mean(-1, keepdim=True)) + half_step(dtype) * dx.abs()
    dw = (n * x * r).sum((0, 1))
    # each term 40 u; per lane and workgroup a chain, then joins: below 100 u for the sizes tested
    return dx, bound, dw, 140 * U32 * (mag * x.abs() * r).sum((0, 1))


def attention(q, k, v, bias, scale, dtype, o_given=None, dout=None):
    """One head: q (m, D), k and v (n, D), bias (n) or None.  Forward: (o, bound, lse, bound); with dout and the
    forward's stored o also the gradients: a dict of name -> (value, bound)."""
    q, k, v = q.double(), k.double(), v.double()
    D, n = q.shape[1], k.shape[0]
    b = torch.zeros(n, dtype=torch.float64) if bias is None else bias.double().clone()
    out = b <= -1e30
    b[out] = -math.inf
    k, v = k.clone(), v.clone()
    k[out] = 0.0
    v[out] = 0.0
    s = scale * q @ k.T + b
    live = torch.isfinite(s).any(1) if n else torch.zeros(q.shape[0], dtype=torch.bool)
    m = torch.where(live, s.max(1).values if n else torch.zeros(q.shape[0], dtype=torch.float64), torch.zeros(1).double())
    e = torch.exp(s - m[:, None])
    l = e.sum(1)
    p = torch.where(live[:, None], e / torch.where(l > 0, l, torch.ones_like(l))[:, None], torch.zeros_like(e))
    lse = torch.where(live, m + torch.log(l), torch.full_like(l, -math.inf))
    o = p @ v
    # relative error of a weight before its normalisation: the score's dot product, its scaling and exponent
    sm = torch.where(torch.isfinite(s), s.abs(), torch.zeros_like(s))
    ds = (D + 4) * U32 * scale * (q.abs() @ k.abs().T) + 6 * U32 * (sm + m.abs()[:, None]) + 4 * U32
    dmax = ds.max(1).values if n else torch.zeros(q.shape[0], dtype=torch.float64)
    rnd = half_step(dtype) if dtype == torch.bfloat16 else 0.0
    pv = p @ v.abs()
    o_bound = (2 * dmax[:, None] + (n + 20) * U32 + rnd) * pv + half_step(dtype) * o.abs()
    lse_bound = torch.where(live, dmax + (n + 20) * U32 + 2 * U32 * lse.abs(), torch.zeros_like(lse))
    if dout is None:
        return o, o_bound, lse, lse_bound
    g = dout.double()
    og = o_given.double()
    dp, delta = g @ v.T, (g * og).sum(1, keepdim=True)
    z = p * (dp - delta)
    pe = p * (ds + torch.where(live, lse_bound, torch.zeros_like(lse))[:, None])            # error of a weight
    ze = pe * (dp - delta).abs() + p * (D + 4) * U32 * (g.abs() @ v.abs().T + (g.abs() * og.abs()).sum(1, keepdim=True))
    ze = ze + rnd * z.abs() + 2 * U32 * z.abs()
    M = q.shape[0]
    res = {}
    for name, zz, ee, x in (("dq", z, ze, k), ("dk", z.T, ze.T, q)):
        val = scale * zz @ x
        chain = (n if name == "dq" else M) + 20
        res[name] = (val, scale * (ee + chain * U32 * zz.abs()) @ x.abs() + half_step(dtype) * val.abs())
    dv = p.T @ g
    res["dv"] = (dv, (pe.T + (rnd + (M + 20) * U32) * p.T) @ g.abs() + half_step(dtype) * dv.abs())
    return res
