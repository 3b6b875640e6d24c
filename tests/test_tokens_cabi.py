"""Host side of the token operators: a plan's sequences, the rotation's
configuration and every refusal (nothing is enqueued, so no GPU is needed)."""
import ctypes

import pytest

import overlap_tiling_trapezoidal_amd as tdp
from synth import WORKLOADS

P = 1 << 20   # a 16-byte aligned address that no refused call reads
NULL = ctypes.c_void_p(None)


@pytest.mark.parametrize("name", ["tiny", "ltx", "conditioned"])
@pytest.mark.parametrize("world,rank", [(1, 0), (3, 0), (3, 2)])
def test_plan_sequences_follow_the_slots(name, world, rank):
    wl = WORKLOADS[name]
    cfg = tdp.make_config(wl.batch, wl.channels, wl.shape, wl.tiling, wl.num_cond, in_dtype=wl.dtype)
    plan = tdp.tdp_plan_create(cfg) if world == 1 else tdp.tdp_plan_create_rank(cfg, world, rank)
    want = []
    for t in tdp.held_tiles(plan):
        info = tdp.tdp_plan_tile(plan, t)
        row = info.lat_offset // wl.channels
        assert info.pos_offset == 6 * row
        want += [(row + b * info.capacity, row + (b + 1) * info.capacity) for b in range(wl.batch)]
    assert tdp.tdp_plan_sequences(plan) == want
    assert want[-1][1] <= tdp.tdp_plan_sizes(plan).tile_pos_floats // 6


def test_plan_sequences_null():
    assert tdp.load_library().tdp_plan_sequences(None, (ctypes.c_int64 * 2)()) == tdp.TDP_EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=12), tdp.TDP_ESHAPE),
    (dict(head_dim=0, rot_dims=(0, 0, 0)), tdp.TDP_ESHAPE),
    (dict(head_dim=264), tdp.TDP_ESHAPE),
    (dict(rot_dims=(3, 10, 10), freqs=[[1.0], [1.0] * 5, [1.0] * 5]), tdp.TDP_ESHAPE),
    (dict(rot_dims=(-2, 10, 10), freqs=[[], [1.0] * 5, [1.0] * 5]), tdp.TDP_ESHAPE),
    (dict(rot_dims=(12, 12, 10)), tdp.TDP_ESHAPE),
    (dict(pairing=2), tdp.TDP_EINVAL),
    (dict(point=-1), tdp.TDP_EINVAL),
    (dict(freqs=[[float("nan")] * 6, [1.0] * 5, [1.0] * 5]), tdp.TDP_EINVAL),
    (dict(freqs=[[1.0] * 6, [2e6] * 5, [1.0] * 5]), tdp.TDP_EINVAL),
])
def test_rope_config_errors(kw, status):
    args = dict(head_dim=32, rot_dims=(12, 10, 10))
    args.update(kw)
    with pytest.raises(tdp.TdpError) as ei:
        tdp.tdp_rope_create(tdp.make_rope_config(**args))
    assert ei.value.status == status


def test_rope_config_counts_frequencies():
    with pytest.raises(ValueError):
        tdp.make_rope_config(32, (12, 10, 10), freqs=[[1.0] * 5, [1.0] * 5, [1.0] * 5])
    lib = tdp.load_library()
    out = ctypes.c_void_p()
    cfg = tdp.make_rope_config(32, (12, 10, 10)).cfg
    assert lib.tdp_rope_create(ctypes.byref(cfg), None, ctypes.byref(out)) == tdp.TDP_EINVAL
    assert lib.tdp_rope_create(None, None, ctypes.byref(out)) == tdp.TDP_EINVAL
    lib.tdp_rope_destroy(None)


def seqs(**kw):
    s = tdp.tdp_seqs()
    s.num_seqs, s.max_rows, s.total_rows, s.len_group = 4, 75, 300, 1
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def heads(n=2, **kw):
    h = tdp.tdp_heads()
    h.data, h.heads, h.head_stride, h.row_stride, h.seq_stride = P, n, 32, 32 * n, 75 * 32 * n
    for k, v in kw.items():
        setattr(h, k, v)
    return h


BAD_SEQS = [
    (dict(num_seqs=0, total_rows=1), tdp.TDP_EINVAL), (dict(len_group=0), tdp.TDP_EINVAL),
    (dict(max_rows=0, total_rows=1), tdp.TDP_ESHAPE), (dict(max_rows=(1 << 24) + 1), tdp.TDP_ESHAPE),
    (dict(total_rows=299), tdp.TDP_EINVAL), (dict(total_rows=1 << 31), tdp.TDP_ESHAPE),
    (dict(row_range=P + 4), tdp.TDP_EINVAL), (dict(seq_len=P + 2), tdp.TDP_EINVAL),
]
BAD_HEADS = [
    (dict(data=None), tdp.TDP_EINVAL), (dict(data=P + 8), tdp.TDP_EINVAL), (dict(heads=0), tdp.TDP_ESHAPE),
    (dict(heads=65537), tdp.TDP_ESHAPE), (dict(row_stride=-64), tdp.TDP_EINVAL), (dict(head_stride=33), tdp.TDP_EINVAL),
    (dict(seq_stride=2), tdp.TDP_EINVAL),
]


def rope_call(s=None, x=None, y=None, rope="rope", pos=P, dtype=tdp.TDP_F32):
    lib = tdp.load_library()
    r = tdp.tdp_rope_create(tdp.make_rope_config(32, (12, 10, 10)))
    ref = lambda v, d: ctypes.byref(v if v is not None else d)  # noqa: E731
    return lib.tdp_rope_apply(r.handle if rope else None, ref(s, seqs()), pos, ref(x, heads()), ref(y, heads(data=2 * P)),
                              dtype, 0, NULL)


@pytest.mark.device_abi
def test_rope_apply_refusals():
    for kw, status in BAD_SEQS:
        assert rope_call(s=seqs(**kw)) == status, kw
    for kw, status in BAD_HEADS:
        assert rope_call(x=heads(**kw)) == status, kw
        assert rope_call(y=heads(**kw)) == status, kw
    assert rope_call(rope=None) == tdp.TDP_EINVAL
    assert rope_call(pos=None) == tdp.TDP_EINVAL
    assert rope_call(pos=P + 4) == tdp.TDP_EINVAL
    assert rope_call(dtype=2) == tdp.TDP_EINVAL
    assert rope_call(y=heads(3)) == tdp.TDP_EINVAL
    assert rope_call(x=heads(), y=heads(row_stride=128)) == tdp.TDP_EINVAL
    assert "in place" in tdp.tdp_last_error()
    # one workgroup per 4 rows of 256 threads: 2^31 - 1 rows leave 32 bits
    big = seqs(num_seqs=1000, max_rows=2_000_000, total_rows=2_000_000_000)
    assert rope_call(s=big) == tdp.TDP_ESHAPE and "work-items" in tdp.tdp_last_error()


def norm_call(backward, eps=1e-6, ws=P, dtype=tdp.TDP_F32, **kw):
    lib = tdp.load_library()
    r = tdp.tdp_rope_create(tdp.make_rope_config(32, (12, 10, 10)))
    t = {n: kw.get(n, heads(data=(i + 1) * P)) for i, n in enumerate(("q", "k", "gq", "gk", "oq", "ok"))}
    b = {n: ctypes.byref(v) for n, v in t.items()}
    s, w = ctypes.byref(kw.get("s", seqs())), kw.get("w", P)
    if backward:
        return lib.tdp_qk_norm_rope_backward(r.handle, s, P, b["q"], b["k"], w, P, b["gq"], b["gk"], b["oq"], b["ok"], P,
                                             P, eps, dtype, ws, NULL)
    return lib.tdp_qk_norm_rope(r.handle, s, P, b["q"], b["k"], w, P, b["oq"], b["ok"], eps, dtype, NULL)


@pytest.mark.device_abi
@pytest.mark.parametrize("backward", [False, True])
def test_qk_norm_rope_refusals(backward):
    for kw, status in BAD_SEQS:
        assert norm_call(backward, s=seqs(**kw)) == status, kw
    for name in ("q", "k", "oq", "ok") + (("gq", "gk") if backward else ()):
        for kw, status in BAD_HEADS:
            assert norm_call(backward, **{name: heads(**kw)}) == status, (name, kw)
    assert norm_call(backward, eps=-1.0) == tdp.TDP_EINVAL
    assert norm_call(backward, eps=float("nan")) == tdp.TDP_EINVAL
    assert norm_call(backward, eps=float("inf")) == tdp.TDP_EINVAL
    assert norm_call(backward, w=P + 2) == tdp.TDP_EINVAL
    assert norm_call(backward, dtype=7) == tdp.TDP_EINVAL
    assert norm_call(backward, oq=heads(3, data=5 * P)) == tdp.TDP_EINVAL
    if backward:
        assert norm_call(True, ws=None) == tdp.TDP_EINVAL
        assert norm_call(True, ws=P + 8) == tdp.TDP_EINVAL
        assert norm_call(True, gk=heads(1, data=4 * P), ok=heads(1, data=6 * P)) == tdp.TDP_EINVAL


NAMES = ("q", "k", "v", "o", "do", "dq", "dk", "dv")


def attn_call(backward, scale=0.1, dim=32, ws=P, lse=P, bias=None, dtype=tdp.TDP_BF16, **kw):
    lib = tdp.load_library()
    b = {n: ctypes.byref(kw.get(n, heads(data=(i + 1) * P))) for i, n in enumerate(NAMES)}
    qs, ks = ctypes.byref(kw.get("qs", seqs())), ctypes.byref(kw.get("ks", seqs()))
    if backward:
        return lib.tdp_attention_backward(qs, ks, b["q"], b["k"], b["v"], bias, b["o"], lse, b["do"], b["dq"], b["dk"],
                                          b["dv"], scale, dim, dtype, ws, NULL)
    return lib.tdp_attention(qs, ks, b["q"], b["k"], b["v"], bias, b["o"], lse, scale, dim, dtype, ws, NULL)


@pytest.mark.device_abi
@pytest.mark.parametrize("backward", [False, True])
def test_attention_refusals(backward):
    for kw, status in BAD_SEQS:
        assert attn_call(backward, qs=seqs(**kw)) == status, kw
        assert attn_call(backward, ks=seqs(**kw)) == status, kw
    for name in NAMES if backward else NAMES[:4]:
        for kw, status in BAD_HEADS:
            assert attn_call(backward, **{name: heads(**kw)}) == status, (name, kw)
        assert attn_call(backward, **{name: heads(3)}) == tdp.TDP_EINVAL, name
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert attn_call(backward, scale=scale) == tdp.TDP_EINVAL
    for dim in (0, 4, 36, 136):
        assert attn_call(backward, dim=dim) == tdp.TDP_ESHAPE
    for name in ("q", "k", "v") + (("do",) if backward else ()):
        assert attn_call(backward, **{name: heads(row_stride=1 << 25)}) == tdp.TDP_ESHAPE   # 2^26 bytes of bf16
        assert "row stride" in tdp.tdp_last_error()
    assert attn_call(backward, dtype=5) == tdp.TDP_EINVAL
    assert attn_call(backward, bias=P + 2) == tdp.TDP_EINVAL
    assert attn_call(backward, lse=P + 1) == tdp.TDP_EINVAL
    assert attn_call(backward, ks=seqs(num_seqs=3, total_rows=225)) == tdp.TDP_EINVAL
    big = seqs(num_seqs=1, max_rows=1 << 24, total_rows=1 << 24)
    many = dict(q=heads(256), o=heads(256, data=4 * P), k=heads(2, data=2 * P), v=heads(2, data=3 * P),
                do=heads(256, data=5 * P), dq=heads(256, data=6 * P))
    assert attn_call(backward, qs=big, ks=big, **many) == tdp.TDP_ESHAPE
    if backward:
        assert attn_call(True, lse=None) == tdp.TDP_EINVAL
        assert attn_call(True, ws=None) == tdp.TDP_EINVAL
        assert attn_call(True, ws=P + 4) == tdp.TDP_EINVAL
    else:
        one, long = seqs(max_rows=1, total_rows=4), seqs(max_rows=9000, total_rows=36000)
        assert attn_call(False, qs=one, ks=long, ws=None) == tdp.TDP_EINVAL
        assert "workspace" in tdp.tdp_last_error()


def test_workspace_sizes():
    lib = tdp.load_library()
    s = seqs()
    r = tdp.tdp_rope_create(tdp.make_rope_config(32, (12, 10, 10)))
    # 4 sequences of 75 rows, 4 rows per workgroup: 76 partial rows of 2 * 32 floats
    assert lib.tdp_qk_norm_rope_workspace(r.handle, ctypes.byref(s), 2, 2) == 76 * 2 * 32 * 4
    assert lib.tdp_qk_norm_rope_workspace(r.handle, ctypes.byref(s), 0, 2) == 0
    assert lib.tdp_qk_norm_rope_workspace(None, ctypes.byref(s), 2, 2) == 0
    assert lib.tdp_attention_workspace(ctypes.byref(s), ctypes.byref(s), 2, 2, 32) == 0
    one, long = seqs(max_rows=1, total_rows=4), seqs(max_rows=9000, total_rows=36000)
    assert lib.tdp_attention_workspace(ctypes.byref(one), ctypes.byref(long), 2, 2, 32) > 0
    assert lib.tdp_attention_workspace(ctypes.byref(one), ctypes.byref(long), 3, 2, 32) == 0
    assert lib.tdp_attention_backward_workspace(ctypes.byref(s), ctypes.byref(s), 2, 2, 32) >= 2 * 300 * 4
    assert lib.tdp_attention_backward_workspace(None, ctypes.byref(s), 2, 2, 32) == 0
