"""Cases of the tile self-attention operators and their plain forms.

A tile's rows go through per-head norms of queries and keys with the
three-axis rotation of their positions, then attention over the used rows of
the tile's slot.  Each case runs one of these operators, forward or backward,
over the slots of a plan (or of one rank's share): `run` either calls the
package's entry points (`own`) or computes the same from elementary torch
operations in 32 bits; `exact` follows the definitions in 64 bits.

Rows past a slot's used count hold NaN in every input, as a slot's unused
rows may hold anything; outputs there are zero.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_POS_SCALE = (8.0, 32.0, 32.0)   # position units per latent cell
_EPS = 1e-6
_THETA = 10000.0


def _case(name, op, grid, tiles, dtype, heads, kv_heads, dim, **kw):
    c = {"name": name, "op": op, "dtype": dtype, "batch": 1,
         "f": grid[0], "h": grid[1], "w": grid[2],
         "nf": tiles[0][0], "of": tiles[0][1], "nh": tiles[1][0], "oh": tiles[1][1],
         "nw": tiles[2][0], "ow": tiles[2][1],
         "cond": 0, "world": 1, "heads": heads, "kv_heads": kv_heads, "dim": dim,
         "pairing": "interleaved", "point": "middle", "queries": 0, "keys": 0, "bias": False}
    c.update(kw)
    return c


_TINY = ((3, 8, 8), ((1, 0), (2, 2), (2, 2)))
_LTX = ((16, 16, 24), ((1, 0), (2, 4), (2, 4)))
_FULL = ((16, 32, 48), ((1, 0), (2, 8), (2, 8)))
_4K = ((16, 68, 120), ((1, 0), (4, 8), (4, 16)))
_COND = ((16, 32, 48), ((2, 2), (3, 6), (3, 8)))


def listed():
    return [
        # the smallest plan: four tiles of 75 rows, one small fp32 tensor; launch latency
        _case("rope_tiny", "rope", *_TINY, "f32", 4, 4, 32),
        # values of positions alone rotated (no norm) for every tile of the 4K-class plan at once
        _case("rope_4k", "rope", *_4K, "bf16", 16, 16, 128),
        # queries and keys of the 6144-token latent's tiles, slices of one packed projection
        _case("norm_ltx", "norm", *_LTX, "bf16", 32, 32, 128),
        # two batch elements, conditioning rows, used counts on the device, half-split pairs, fp32
        _case("norm_conditioned", "norm", *_COND, "f32", 8, 4, 64, batch=2, cond=1024, pairing="halves"),
        # gradients of the smallest plan's norms
        _case("norm_bwd_tiny", "norm_bwd", *_TINY, "f32", 4, 2, 32),
        # a training step's norm gradients on the 24576-token latent's tiles
        _case("norm_bwd_full", "norm_bwd", *_FULL, "bf16", 16, 16, 128, pairing="halves"),
        # attention inside the smallest plan's tiles, fp32
        _case("attn_tiny", "attn", *_TINY, "f32", 4, 4, 32),
        # a rank's share (4 of 16 tiles) of the 4K-class plan: the largest work
        _case("attn_4k_rank", "attn", *_4K, "bf16", 12, 12, 128, world=4),
        # tile rows attending a prompt of 512 tokens with padding, shared key heads
        _case("attn_prompt", "attn", *_FULL, "bf16", 16, 4, 64, keys=512, bias=True),
        # one readout token per batch element attending all rows of the latent
        _case("attn_one", "attn", (16, 32, 48), ((1, 0), (1, 0), (1, 0)), "bf16", 32, 8, 128, batch=2, queries=1),
        # a training step's attention gradients on the 6144-token latent's tiles
        _case("attn_bwd_ltx", "attn_bwd", *_LTX, "bf16", 16, 16, 128),
        # gradients with conditioning rows, used counts on the device and shared key heads
        _case("attn_bwd_conditioned", "attn_bwd", *_COND, "bf16", 8, 2, 64, batch=2, cond=1024),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "norm", "norm_bwd", "attn", "attn", "attn", "attn_bwd", "attn_bwd"])
        grid, tiles = [], []
        for lo, hi in ((1, 16), (4, 68), (4, 120)):
            d = _log_int(rng, lo, hi)
            n = rng.randint(1, 4)
            n = n if n <= d else 1
            o = rng.randint(0, d // (n + 1)) if n > 1 else 0
            grid.append(d)
            tiles.append((n, o))
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        kv = _log_int(rng, 1, 16)
        group = rng.choice([1, 1, 2, 4])
        c = _case(None, op, grid, tiles, dtype, kv * group, kv, rng.choice([32, 40, 64, 64, 72, 96, 128, 128]),
                  batch=rng.choice([1, 1, 2]), pairing=rng.choice(["interleaved", "halves"]),
                  point=rng.choice(["middle", "start"]))
        c.pop("name")
        if rng.random() < 0.4:
            c["cond"] = _log_int(rng, 1, 1024)
        if rng.random() < 0.25:
            c["world"] = rng.randint(2, 4)
        if op == "attn":
            kind = rng.choice(["self", "self", "prompt", "few"])
            if kind == "prompt":
                c["keys"], c["bias"] = _log_int(rng, 1, 1024), rng.random() < 0.7
            elif kind == "few":
                c["queries"] = _log_int(rng, 1, 24)
        elif op == "attn_bwd" and rng.random() < 0.3:
            c["keys"], c["bias"] = _log_int(rng, 1, 1024), rng.random() < 0.7
        w = work(c)
        widths = {n * c["dim"] for n in (kv, 2 * kv, kv * group, kv * (group + 1), kv * (group + 2))}
        if 3072 in widths:   # row widths this repository does not use
            continue
        if op.startswith("attn"):
            if w["flops"] <= (4e12 if dtype == "bf16" else 5e11) and w["bytes"] <= 2e9:
                return c
        elif w["bytes"] <= 2e9:
            return c


# ---------------------------------------------------------------------------
# geometry of the slots
# ---------------------------------------------------------------------------

def _slots(case):
    """Per held tile: (origin, shape); uniform capacity for a rank's share."""
    ivs = []
    for d, n, o in ((case["f"], case["nf"], case["of"]), (case["h"], case["nh"], case["oh"]),
                    (case["w"], case["nw"], case["ow"])):
        a = [i * (d - o) // n for i in range(n + 1)]
        ivs.append([(a[i], a[i + 1] + o) for i in range(n)])
    tiles = [(f, h, w) for f in ivs[0] for h in ivs[1] for w in ivs[2]]
    tiles = tiles[::case["world"]]
    shapes = [tuple(e - s for s, e in t) for t in tiles]
    gens = [f * h * w for f, h, w in shapes]
    caps = [g + case["cond"] for g in gens]
    if case["world"] > 1:
        caps = [max(caps)] * len(caps)
    return shapes, gens, caps


def _kept(case, n, seed):
    """Kept conditioning rows per tile: a quarter (the reference tokens) to all."""
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    nc = case["cond"]
    return [int(torch.randint(nc // 4, nc + 1, (1,), generator=g)) if nc else 0 for _ in range(n)]


def _tile_sequences(case, seed):
    """(capacities, used lengths) per sequence, slot-major then batch."""
    _, gens, caps = _slots(case)
    kept = _kept(case, len(gens), seed)
    cap, used = [], []
    for g, c, k in zip(gens, caps, kept):
        cap += [c] * case["batch"]
        used += [g + k] * case["batch"]
    return cap, used


def _layout(case, seed):
    """The tile rows' sequences, and the queries' and keys' of an attention case."""
    tile = _tile_sequences(case, seed)
    q = k = tile
    if case["queries"]:
        q = ([case["queries"]] * len(tile[0]),) * 2
    if case["keys"]:
        n = case["keys"]
        g = torch.Generator().manual_seed(seed * 7919 + 29)
        k = ([n] * len(tile[0]), [n if case["bias"] else int(torch.randint((n + 1) // 2, n + 1, (1,), generator=g))
                                  for _ in tile[0]])
    return tile, q, k


def _starts(cap):
    out = [0]
    for c in cap:
        out.append(out[-1] + c)
    return out


def _rot_dims(dim):
    side = dim // 3 // 2 * 2
    return (dim - 2 * side, side, side)


def _freqs(dim):
    return [[_THETA ** (-2.0 * i / r) / s for i in range(r // 2)] for r, s in zip(_rot_dims(dim), _POS_SCALE)]


def work(case):
    cap, used = _tile_sequences(case, 0)
    e = 2 if case["dtype"] == "bf16" else 4
    rows, urows, D = sum(cap), sum(used), case["dim"]
    hq, hk = case["heads"], case["kv_heads"]
    if case["op"] == "rope":
        return {"bytes": (rows + urows) * hq * D * e + 24 * urows, "flops": 3 * urows * hq * D}
    if case["op"] == "norm":
        return {"bytes": (rows + urows) * (hq + hk) * D * e + 24 * urows + 8 * D, "flops": 8 * urows * (hq + hk) * D}
    if case["op"] == "norm_bwd":
        return {"bytes": (rows + 2 * urows) * (hq + hk) * D * e + 24 * urows + 16 * D,
                "flops": 16 * urows * (hq + hk) * D}
    _, (qc, qu), (kc, ku) = _layout(case, 0)
    pairs = sum(a * b for a, b in zip(qu, ku))
    bias = 4 * sum(ku) if case["bias"] else 0
    if case["op"] == "attn":
        return {"bytes": (sum(qc) + sum(qu)) * hq * D * e + 2 * sum(ku) * hk * D * e + bias,
                "flops": 4 * D * hq * pairs}
    return {"bytes": ((3 * sum(qu) + sum(qc)) * hq + 2 * (sum(ku) + sum(kc)) * hk) * D * e + 4 * sum(qu) * hq + bias,
            "flops": 10 * D * hq * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _poison(x, cap, used):
    r = 0
    for c, u in zip(cap, used):
        x[r + u:r + c] = float("nan")
        r += c


def _positions(case, seed, cap, used):
    """Tile positions as the gather lays them out: per sequence three planes of cap [start, end) pairs."""
    shapes, gens, _ = _slots(case)
    gen = torch.Generator(device="cuda").manual_seed(seed * 31 + 5)
    out, s = [], 0
    for shape, n in zip(shapes, gens):
        axes = torch.meshgrid(*[torch.arange(d, device="cuda") for d in shape], indexing="ij")
        for _ in range(case["batch"]):
            p = torch.full((3, cap[s], 2), float("nan"), device="cuda")
            m = used[s] - n
            for a in range(3):
                start = axes[a].reshape(-1).float() * _POS_SCALE[a]
                p[a, :n, 0], p[a, :n, 1] = start, start + _POS_SCALE[a]
                if m:
                    c0 = torch.randint(0, shape[a], (m,), generator=gen, device="cuda").float() * _POS_SCALE[a]
                    if a == 0:   # the leading kept rows are reference tokens at negative times
                        c0[:m // 4] = -8.0 * torch.randint(1, 5, (m // 4,), generator=gen, device="cuda").float()
                    p[a, n:n + m, 0], p[a, n:n + m, 1] = c0, c0 + _POS_SCALE[a]
            out.append(p.reshape(-1))
            s += 1
    return torch.cat(out)


def _sequences(case, cap, used, group):
    import overlap_tiling_trapezoidal_amd as tdp
    full = cap == used
    lens = None if full else torch.tensor(used[::group], dtype=torch.int32, device="cuda")
    if len(set(cap)) == 1:
        return tdp.Sequences(len(cap), cap[0], seq_len=lens, len_group=group)
    start = torch.tensor(_starts(cap), dtype=torch.int64, device="cuda")
    return tdp.Sequences(len(cap), max(cap), row_start=start, total_rows=sum(cap), seq_len=lens, len_group=group)


def _rope_handle(case):
    import overlap_tiling_trapezoidal_amd as tdp
    return tdp.tdp_rope_create(tdp.make_rope_config(case["dim"], _rot_dims(case["dim"]), freqs=_freqs(case["dim"]),
                                                    pairing=case["pairing"], point=case["point"]))


def _packed(gen, rows, hq, hk, dim, dt, cap, used):
    """Queries, keys and values as slices of one packed projection."""
    x = _randn(gen, rows, hq + 2 * hk, dim).to(dt)
    _poison(x, cap, used)
    return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]


def prepare(case, seed):
    dt, dim, hq, hk, op = _DT[case["dtype"]], case["dim"], case["heads"], case["kv_heads"], case["op"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    (cap, used), (qcap, qused), (kcap, kused) = _layout(case, seed)
    st = {"case": case, "scale": 1.0 / math.sqrt(dim)}
    if not op.startswith("attn"):
        st.update(cap=cap, used=used, pos=_positions(case, seed, cap, used))
        rows = sum(cap)
        if op == "rope":
            st["x"] = _randn(gen, rows, hq, dim).to(dt)
            _poison(st["x"], cap, used)
            if own:
                st["y"] = torch.empty(rows, hq, dim, dtype=dt, device="cuda")
        else:
            st["q"], st["k"], _ = _packed(gen, rows, hq, hk, dim, dt, cap, used)
            st["wq"] = 1.0 + 0.2 * _randn(gen, dim)
            st["wk"] = 1.0 + 0.2 * _randn(gen, dim)
            if op == "norm_bwd":
                st["gq"], st["gk"], _ = _packed(gen, rows, hq, hk, dim, dt, cap, used)
            if own:
                st["yq"] = torch.empty(rows, hq, dim, dtype=dt, device="cuda")
                st["yk"] = torch.empty(rows, hk, dim, dtype=dt, device="cuda")
        if own:
            import overlap_tiling_trapezoidal_amd as tdp
            st["rope"] = _rope_handle(case)
            st["seqs"] = _sequences(case, cap, used, case["batch"])
            if op == "norm_bwd":
                st["dwq"], st["dwk"] = torch.empty(2, dim, device="cuda")
                st["ws"] = tdp.allocate_qk_norm_rope_workspace(st["rope"], st["seqs"], hq, hk, "cuda")
        return st

    qr, kr = sum(qcap), sum(kcap)
    st.update(cap=qcap, used=qused, kcap=kcap, kused=kused, bias=None)
    if case["queries"] or case["keys"]:
        st["q"] = _randn(gen, qr, hq, dim).to(dt)
        _poison(st["q"], qcap, qused)
        kv = _randn(gen, kr, 2 * hk, dim).to(dt)
        _poison(kv, kcap, kused)
        st["k"], st["v"] = kv[:, :hk], kv[:, hk:]
    else:
        st["q"], st["k"], st["v"] = _packed(gen, qr, hq, hk, dim, dt, qcap, qused)
    if case["bias"]:   # prompt padding: the last tokens of each prompt are masked out
        b = torch.zeros(kr, device="cuda")
        r = 0
        for c in kcap:
            pad = int(torch.randint(0, c // 2 + 1, (1,), generator=gen, device="cuda"))
            b[r + c - pad:r + c] = float("-inf")
            r += c
        st["bias"] = b
    if op == "attn_bwd":
        st["do"] = _randn(gen, qr, hq, dim).to(dt)
        _poison(st["do"], qcap, qused)
        st["o"], st["lse"] = _plain_attention(st)
    if own:
        import overlap_tiling_trapezoidal_amd as tdp
        st["qseqs"] = _sequences(case, qcap, qused, case["batch"] if not case["queries"] else 1)
        st["kseqs"] = st["qseqs"] if not (case["queries"] or case["keys"]) else \
            _sequences(case, kcap, kused, 1 if case["keys"] else case["batch"])
        if op == "attn":
            st["y"] = torch.empty(qr, hq, dim, dtype=dt, device="cuda")
            st["ws"] = tdp.allocate_attention_workspace(st["qseqs"], st["kseqs"], hq, hk, dim, "cuda")
        else:
            st["dq"] = torch.empty(qr, hq, dim, dtype=dt, device="cuda")
            st["dk"] = torch.empty(kr, hk, dim, dtype=dt, device="cuda")
            st["dv"] = torch.empty(kr, hk, dim, dtype=dt, device="cuda")
            st["ws"] = tdp.allocate_attention_backward_workspace(st["qseqs"], st["kseqs"], hq, hk, dim, "cuda")
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _angles(case, pos, row, cap, used):
    """cos and sin (used, pairs) of one sequence; angles in 64 bits."""
    p = pos[6 * row:6 * (row + cap)].view(3, cap, 2)[:, :used].double()
    p = (p[..., 0] + p[..., 1]) / 2 if case["point"] == "middle" else p[..., 0]
    ang = torch.cat([p[a, :, None] * torch.tensor(f, dtype=torch.float64, device=p.device)
                     for a, f in enumerate(_freqs(case["dim"]))], dim=1)
    return torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]


def _pair_index(case, device):
    first, second, off = [], [], 0
    for r in _rot_dims(case["dim"]):
        for i in range(r // 2):
            first.append(off + (2 * i if case["pairing"] == "interleaved" else i))
            second.append(off + (2 * i + 1 if case["pairing"] == "interleaved" else i + r // 2))
        off += r
    return torch.tensor(first, device=device), torch.tensor(second, device=device)


def _rotate(case, x, cos, sin, i0, i1):
    y = x.clone()
    a, b = x[..., i0], x[..., i1]
    y[..., i0] = a * cos - b * sin
    y[..., i1] = a * sin + b * cos
    return y


def _per_sequence(st):
    i0, i1 = _pair_index(st["case"], st["pos"].device)
    r = 0
    for c, u in zip(st["cap"], st["used"]):
        cos, sin = _angles(st["case"], st["pos"], r, c, u)
        yield slice(r, r + u), cos, sin, i0, i1
        r += c


def _plain_rope(st):
    x = st["x"]
    y = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
    for rows, cos, sin, i0, i1 in _per_sequence(st):
        y[rows] = _rotate(st["case"], x[rows].float(), cos, sin, i0, i1).to(x.dtype)
    return y


def _plain_norm(st):
    outs = [torch.zeros(t.shape, dtype=t.dtype, device=t.device) for t in (st["q"], st["k"])]
    for rows, cos, sin, i0, i1 in _per_sequence(st):
        for t, w, y in zip((st["q"], st["k"]), (st["wq"], st["wk"]), outs):
            x = t[rows].float()
            n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w
            y[rows] = _rotate(st["case"], n, cos, sin, i0, i1).to(t.dtype)
    return outs


def _plain_norm_backward(st):
    dim = st["case"]["dim"]
    grads = [torch.zeros(t.shape, dtype=t.dtype, device=t.device) for t in (st["q"], st["k"])]
    dws = [torch.zeros(dim, dtype=torch.float64, device="cuda") for _ in range(2)]
    for rows, cos, sin, i0, i1 in _per_sequence(st):
        for j, (t, g, w) in enumerate(((st["q"], st["gq"], st["wq"]), (st["k"], st["gk"], st["wk"]))):
            x = t[rows].float()
            dn = _rotate(st["case"], g[rows].float(), cos, -sin, i0, i1)
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
            dws[j] += (dn * x * r).sum((0, 1), dtype=torch.float64)
            gw = dn * w
            grads[j][rows] = (r * (gw - x * (r * r) * (gw * x).mean(-1, keepdim=True))).to(t.dtype)
    return grads + [d.float() for d in dws]


def _blocks(st):
    """(query rows, key rows, kv head, query heads) of pieces whose scores stay near 1 GiB in 32 bits."""
    group = st["case"]["heads"] // st["case"]["kv_heads"]
    q0 = k0 = 0
    for qc, qu, kc, ku in zip(st["cap"], st["used"], st["kcap"], st["kused"]):
        heads = max(1, min(st["case"]["kv_heads"], (1 << 28) // max(1, qu * ku * group)))
        step = max(1, min(qu, (1 << 28) // max(1, ku * group)))
        for h in range(0, st["case"]["kv_heads"], heads):
            for a in range(0, qu, step):
                hk = slice(h, min(h + heads, st["case"]["kv_heads"]))
                yield (slice(q0 + a, q0 + min(a + step, qu)), slice(k0, k0 + ku), hk,
                       slice(hk.start * group, hk.stop * group))
        q0, k0 = q0 + qc, k0 + kc


def _head_major(x, rows, heads, group=1):
    """(kv heads, group * rows, D) in 32 bits: the group's query heads stacked over their shared key head."""
    t = x[rows, heads].float().transpose(0, 1)
    return t.reshape(t.shape[0] // group, group * t.shape[1], t.shape[2])


def _row_major(t, group):
    """(rows, query heads, D) from (kv heads, group * rows, D)."""
    return t.reshape(t.shape[0] * group, t.shape[1] // group, t.shape[2]).transpose(0, 1)


def _scores(st, q, k, krows):
    s = torch.bmm(q, k.transpose(1, 2).contiguous()) * st["scale"]
    return s if st["bias"] is None else s + st["bias"][krows]


def _plain_attention(st):
    q, group = st["q"], st["case"]["heads"] // st["case"]["kv_heads"]
    o = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.full((q.shape[1], q.shape[0]), float("-inf"), device=q.device)
    for qr, kr, hk, hq in _blocks(st):
        s = _scores(st, _head_major(q, qr, hq, group), _head_major(st["k"], kr, hk), kr)
        m = s.amax(-1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        y = torch.bmm(p, _head_major(st["v"], kr, hk)) / torch.where(l > 0, l, torch.ones_like(l))
        o[qr, hq] = _row_major(y, group).to(q.dtype)
        lse[hq, qr] = (m + torch.log(l)).reshape(hq.stop - hq.start, -1)
    return o, lse


def _plain_attention_backward(st):
    q, k, v, group = st["q"], st["k"], st["v"], st["case"]["heads"] // st["case"]["kv_heads"]
    dq = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    dk, dv = (torch.zeros(k.shape, device=q.device) for _ in range(2))
    for qr, kr, hk, hq in _blocks(st):
        qf, kf = _head_major(q, qr, hq, group), _head_major(k, kr, hk)
        vf, g = _head_major(v, kr, hk), _head_major(st["do"], qr, hq, group)
        lse = st["lse"][hq, qr].reshape(kf.shape[0], -1, 1)
        s = _scores(st, qf, kf, kr)
        p = torch.where(torch.isinf(lse), torch.zeros_like(s), torch.exp(s - lse))
        delta = (g * _head_major(st["o"], qr, hq, group)).sum(-1, keepdim=True)
        ds = p * (torch.bmm(g, vf.transpose(1, 2).contiguous()) - delta) * st["scale"]
        dq[qr, hq] = _row_major(torch.bmm(ds, kf), group).to(q.dtype)
        dk[kr, hk] += torch.bmm(ds.transpose(1, 2).contiguous(), qf).transpose(0, 1)
        dv[kr, hk] += torch.bmm(p.transpose(1, 2).contiguous(), g).transpose(0, 1)
    return [dq, dk.to(k.dtype), dv.to(v.dtype)]


def run(st):
    op = st["case"]["op"]
    if not own:
        if op == "attn":
            return _plain_attention(st)[0]
        return {"rope": _plain_rope, "norm": _plain_norm, "norm_bwd": _plain_norm_backward,
                "attn_bwd": _plain_attention_backward}[op](st)
    import overlap_tiling_trapezoidal_amd as tdp
    if op == "rope":
        tdp.tdp_rope_apply(st["rope"], st["seqs"], st["pos"], st["x"], st["y"])
        return st["y"]
    if op == "norm":
        tdp.tdp_qk_norm_rope(st["rope"], st["seqs"], st["pos"], st["q"], st["k"], st["wq"], st["wk"],
                             st["yq"], st["yk"], eps=_EPS)
        return [st["yq"], st["yk"]]
    if op == "norm_bwd":
        tdp.tdp_qk_norm_rope_backward(st["rope"], st["seqs"], st["pos"], st["q"], st["k"], st["wq"], st["wk"],
                                      st["gq"], st["gk"], st["yq"], st["yk"], st["dwq"], st["dwk"], st["ws"],
                                      eps=_EPS)
        return [st["yq"], st["yk"], st["dwq"], st["dwk"]]
    if op == "attn":
        tdp.tdp_attention(st["qseqs"], st["kseqs"], st["q"], st["k"], st["v"], st["y"], key_bias=st["bias"],
                          scale=st["scale"], workspace=st["ws"])
        return st["y"]
    tdp.tdp_attention_backward(st["qseqs"], st["kseqs"], st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"],
                               st["dq"], st["dk"], st["dv"], st["ws"], key_bias=st["bias"], scale=st["scale"])
    return [st["dq"], st["dk"], st["dv"]]


# ---------------------------------------------------------------------------
# definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_turned(case, x, pos, row, cap, sign):
    """Rows (used, heads, D) turned by their positions as complex numbers, one pair at a time."""
    p = pos[6 * row:6 * (row + cap)].view(3, cap, 2)[:, :x.shape[0]].double()
    p = p.mean(-1) if case["point"] == "middle" else p[..., 0]
    y, off = x.clone(), 0
    for a, (r, freqs) in enumerate(zip(_rot_dims(case["dim"]), _freqs(case["dim"]))):
        for i, f in enumerate(freqs):
            u, v = (off + 2 * i, off + 2 * i + 1) if case["pairing"] == "interleaved" else (off + i, off + i + r // 2)
            z = torch.complex(x[..., u], x[..., v]) * torch.exp(1j * sign * f * p[a])[:, None]
            y[..., u], y[..., v] = z.real, z.imag
        off += r
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op, D = case["op"], case["dim"]
    group = case["heads"] // case["kv_heads"]
    if op == "rope":
        out, r = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda"), 0
        for c, u in zip(st["cap"], st["used"]):
            out[r:r + u] = _exact_turned(case, st["x"][r:r + u].double(), st["pos"], r, c, 1.0)
            r += c
        return out
    if op in ("norm", "norm_bwd"):
        outs, dws = [], []
        for name, w in (("q", st["wq"]), ("k", st["wk"])):
            x = st[name]
            out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
            dw, r = torch.zeros(D, dtype=torch.float64, device="cuda"), 0
            for c, u in zip(st["cap"], st["used"]):
                xs = x[r:r + u].double()
                rms = torch.sqrt(xs.square().sum(-1, keepdim=True) / D + _EPS)
                unit = xs / rms
                if op == "norm":
                    out[r:r + u] = _exact_turned(case, unit * w.double(), st["pos"], r, c, 1.0)
                else:   # d(unit)/dx = (I - unit unit^T / D) / rms
                    dn = _exact_turned(case, st["g" + name][r:r + u].double(), st["pos"], r, c, -1.0)
                    dw += torch.einsum("rhd,rhd->d", dn, unit)
                    dn = dn * w.double()
                    out[r:r + u] = (dn - unit * (dn * unit).sum(-1, keepdim=True) / D) / rms
                r += c
            outs.append(out)
            dws.append(dw)
        return outs if op == "norm" else outs + dws
    q, k, v = st["q"], st["k"], st["v"]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros(k.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    q0 = k0 = 0
    for qc, qu, kc, ku in zip(st["cap"], st["used"], st["kcap"], st["kused"]):
        step = max(1, (1 << 27) // max(1, ku))
        for h in range(case["heads"]):
            ks, vs = k[k0:k0 + ku, h // group].double(), v[k0:k0 + ku, h // group].double()
            for a in range(q0, q0 + qu, step):
                b = min(a + step, q0 + qu)
                qs = q[a:b, h].double()
                s = qs @ ks.T / math.sqrt(D)
                if st["bias"] is not None:
                    s += st["bias"][k0:k0 + ku].double()
                p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
                if op == "attn":
                    o[a:b, h] = p @ vs
                    continue
                g = st["do"][a:b, h].double()
                ds = p * (g @ vs.T - (g * st["o"][a:b, h].double()).sum(-1, keepdim=True)) / math.sqrt(D)
                o[a:b, h] = ds @ ks
                dk[k0:k0 + ku, h // group] += ds.T @ qs
                dv[k0:k0 + ku, h // group] += p.T @ g
        q0, k0 = q0 + qc, k0 + kc
    return o if op == "attn" else [o, dk, dv]
