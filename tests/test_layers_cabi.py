"""Host side of the layer operators: every refusal (nothing is enqueued, so no
GPU is needed) and the workspace sizes."""
import ctypes

import pytest

import overlap_tiling_trapezoidal_amd as tdp
from test_tokens_cabi import BAD_SEQS, NULL, P, seqs

BIG = dict(num_seqs=1000, max_rows=2_000_000, total_rows=2_000_000_000)
BAD_ROWS = [
    (dict(data=None), tdp.TDP_EINVAL), (dict(data=P + 8), tdp.TDP_EINVAL), (dict(row_stride=-64), tdp.TDP_EINVAL),
    (dict(row_stride=130), tdp.TDP_EINVAL), (dict(seq_stride=2), tdp.TDP_EINVAL),
    (dict(row_stride=(1 << 40) + 64), tdp.TDP_EINVAL),
]


def rows(**kw):
    r = tdp.tdp_rows()
    r.data, r.row_stride, r.seq_stride = P, 128, 75 * 128
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def ref(v, default):
    return ctypes.byref(default if v is None else v) if v != "null" else None


def norm_call(s=None, x=None, y=None, w=P, b=P, n=1, eps=1e-5, channels=128, dtype=tdp.TDP_F32):
    return tdp.load_library().tdp_layer_norm(ref(s, seqs()), ref(x, rows()), w, b, n, ref(y, rows(data=2 * P)), eps,
                                             channels, dtype, NULL)


def norm_backward_call(s=None, x=None, dy=None, dx=None, w=P, n=1, dw=P, db=P, eps=1e-5, channels=128,
                       dtype=tdp.TDP_F32, ws=P):
    return tdp.load_library().tdp_layer_norm_backward(
        ref(s, seqs()), ref(x, rows()), w, n, ref(dy, rows(data=2 * P)), ref(dx, rows(data=3 * P)), dw, db, eps,
        channels, dtype, ws, NULL)


@pytest.mark.device_abi
@pytest.mark.parametrize("call", [norm_call, norm_backward_call], ids=["forward", "backward"])
def test_layer_norm_refusals(call):
    for kw, status in BAD_SEQS:
        assert call(s=seqs(**kw)) == status, kw
    assert call(s="null") == tdp.TDP_EINVAL
    for name in ("x", "y") if call is norm_call else ("x", "dy", "dx"):
        for kw, status in BAD_ROWS:
            assert call(**{name: rows(**kw)}) == status, (name, kw)
        assert call(**{name: "null"}) == tdp.TDP_EINVAL
    for kw, status in [(dict(channels=0), tdp.TDP_ESHAPE), (dict(channels=130), tdp.TDP_ESHAPE),
                       (dict(channels=tdp.TDP_MAX_CHANNELS + 8), tdp.TDP_ESHAPE), (dict(dtype=2), tdp.TDP_EINVAL),
                       (dict(n=0), tdp.TDP_EINVAL), (dict(n=5), tdp.TDP_EINVAL), (dict(w=P + 2), tdp.TDP_EINVAL),
                       (dict(eps=-1.0), tdp.TDP_EINVAL), (dict(eps=float("nan")), tdp.TDP_EINVAL),
                       (dict(eps=float("inf")), tdp.TDP_EINVAL)]:
        assert call(**kw) == status, kw
    assert call(s=seqs(**dict(BIG, max_rows=(1 << 24), num_seqs=2 ** 20, row_range=P)), channels=2048) == tdp.TDP_ESHAPE
    if call is norm_call:
        assert call(b=P + 1) == tdp.TDP_EINVAL
        assert call(y=rows(row_stride=256)) == tdp.TDP_EINVAL and "in place" in tdp.tdp_last_error()
    else:
        for kw in (dict(dw=P + 1), dict(db=P + 2), dict(ws=None), dict(ws=P + 8)):
            assert call(**kw) == tdp.TDP_EINVAL, kw
        assert call(dx=rows(data=2 * P, row_stride=256)) == tdp.TDP_EINVAL and "in place" in tdp.tdp_last_error()
        assert call(dx=rows(row_stride=256)) == tdp.TDP_EINVAL and "in place" in tdp.tdp_last_error()


def test_layer_norm_workspace():
    lib = tdp.load_library()
    size = lambda s, c, n: lib.tdp_layer_norm_workspace(ctypes.byref(s), c, n)  # noqa: E731
    assert size(seqs(), 128, 1) > 0
    assert size(seqs(), 128, 1) % 256 == 0
    assert size(seqs(), 128, 4) >= size(seqs(num_seqs=1, total_rows=75), 128, 1)
    # two partial rows at least for each set of weights
    assert size(seqs(num_seqs=4, max_rows=1, total_rows=4), 8192, 4) >= 4 * 2 * 8192 * 4
    for c, n in ((0, 1), (12, 1), (tdp.TDP_MAX_CHANNELS + 8, 1), (128, 0), (128, 5)):
        assert size(seqs(), c, n) == 0, (c, n)
    assert size(seqs(num_seqs=0), 128, 1) == 0


def window(**kw):
    return tdp.tdp_window(*{**dict(step=1, back=7, ahead=0, sinks=2), **kw}.values())


def heads32(n=2, **kw):
    h = tdp.tdp_heads()
    h.data, h.heads, h.head_stride, h.row_stride, h.seq_stride = P, n, 32, 32 * n, 75 * 32 * n
    for k, v in kw.items():
        setattr(h, k, v)
    return h


BAD_WINDOWS = [
    (dict(step=0), tdp.TDP_ESHAPE), (dict(step=(1 << 24) + 1), tdp.TDP_ESHAPE), (dict(back=-1), tdp.TDP_EINVAL),
    (dict(ahead=-1), tdp.TDP_EINVAL), (dict(sinks=-1), tdp.TDP_EINVAL),
    (dict(back=tdp.TDP_WINDOW_ALL + 1), tdp.TDP_EINVAL), (dict(ahead=tdp.TDP_WINDOW_ALL + 1), tdp.TDP_EINVAL),
    (dict(sinks=tdp.TDP_WINDOW_ALL + 1), tdp.TDP_EINVAL),
]


def window_call(qs=None, ks=None, w=None, q=None, k=None, v=None, out=None, lse=None, scale=0.1, D=32,
                dtype=tdp.TDP_F32, ws=P):
    return tdp.load_library().tdp_window_attention(
        ref(qs, seqs()), ref(ks, seqs()), ref(w, window()), ref(q, heads32()), ref(k, heads32()), ref(v, heads32()),
        ref(out, heads32(data=2 * P)), lse, scale, D, dtype, ws, NULL)


def window_backward_call(qs=None, ks=None, w=None, q=None, k=None, v=None, out=None, lse=P, dout=None, dq=None,
                         dk=None, dv=None, scale=0.1, D=32, dtype=tdp.TDP_F32, ws=P):
    return tdp.load_library().tdp_window_attention_backward(
        ref(qs, seqs()), ref(ks, seqs()), ref(w, window()), ref(q, heads32()), ref(k, heads32()), ref(v, heads32()),
        ref(out, heads32(data=2 * P)), lse, ref(dout, heads32()), ref(dq, heads32(data=3 * P)),
        ref(dk, heads32(data=4 * P)), ref(dv, heads32(data=5 * P)), scale, D, dtype, ws, NULL)


@pytest.mark.device_abi
@pytest.mark.parametrize("call", [window_call, window_backward_call], ids=["forward", "backward"])
def test_window_attention_refusals(call):
    for kw, status in BAD_WINDOWS:
        assert call(w=window(**kw)) == status, kw
    assert call(w="null") == tdp.TDP_EINVAL
    for kw, status in BAD_SEQS:
        assert call(qs=seqs(**kw)) == status, kw
        assert call(ks=seqs(**kw)) == status, kw
    for name in ("q", "k", "v", "out") if call is window_call else ("q", "k", "v", "out", "dout", "dq", "dk", "dv"):
        for kw, status in [(dict(data=None), tdp.TDP_EINVAL), (dict(data=P + 8), tdp.TDP_EINVAL),
                           (dict(heads=0), tdp.TDP_ESHAPE), (dict(head_stride=33), tdp.TDP_EINVAL),
                           (dict(heads=3), tdp.TDP_EINVAL)]:
            assert call(**{name: heads32(**kw)}) == status, (name, kw)
    assert call(qs=seqs(num_seqs=2, total_rows=150)) == tdp.TDP_EINVAL
    for kw, status in [(dict(D=0), tdp.TDP_ESHAPE), (dict(D=36), tdp.TDP_ESHAPE), (dict(D=136), tdp.TDP_ESHAPE),
                       (dict(dtype=2), tdp.TDP_EINVAL), (dict(scale=0.0), tdp.TDP_EINVAL),
                       (dict(scale=float("nan")), tdp.TDP_EINVAL), (dict(lse=P + 2), tdp.TDP_EINVAL),
                       (dict(q=heads32(row_stride=(1 << 24))), tdp.TDP_ESHAPE)]:
        assert call(**kw) == status, kw
    if call is window_backward_call:
        assert call(lse=None) == tdp.TDP_EINVAL
        assert call(ws=None) == tdp.TDP_EINVAL and call(ws=P + 8) == tdp.TDP_EINVAL
    else:   # one query per sequence over long keys: split, so a workspace is needed
        one = dict(qs=seqs(max_rows=1, total_rows=4), ks=seqs(max_rows=4000, total_rows=16000),
                   w=window(back=tdp.TDP_WINDOW_ALL))
        assert call(**one, ws=None) == tdp.TDP_EINVAL and "workspace" in tdp.tdp_last_error()
        assert call(**one, ws=P + 8) == tdp.TDP_EINVAL


def test_window_attention_workspace():
    lib, ref = tdp.load_library(), ctypes.byref
    fwd = lambda q, k, w, hq=4, hk=2, D=64: lib.tdp_window_attention_workspace(ref(q), ref(k), ref(w), hq, hk, D)  # noqa: E731
    bwd = lambda q, k, w, hq=4, hk=2, D=64: lib.tdp_window_attention_backward_workspace(  # noqa: E731
        ref(q), ref(k), ref(w), hq, hk, D)
    one, cache = seqs(max_rows=1, total_rows=4), seqs(max_rows=4000, total_rows=16000)
    # a short window of a long cache is not worth splitting, a long one is, up to all of it
    assert fwd(one, cache, window(back=100)) == 0
    assert 0 < fwd(one, cache, window(back=1500)) < fwd(one, cache, window(back=tdp.TDP_WINDOW_ALL))
    assert fwd(one, cache, window(back=tdp.TDP_WINDOW_ALL)) == lib.tdp_attention_workspace(ref(one), ref(cache), 4, 2, 64)
    # of many key blocks only those of the first rows are split: their sums alone
    long = seqs(num_seqs=2, max_rows=40000, total_rows=80000)
    stats = 4 * 80000 * 8
    assert bwd(long, long, window(back=1000, sinks=0)) == stats
    got = bwd(long, long, window(back=1000, sinks=130)) - stats
    assert got > 0 and got % (2 * 2 * 256 * 64 * 8) == 0
    for kw, _ in BAD_WINDOWS:
        assert fwd(one, cache, window(**kw)) == 0 and bwd(one, cache, window(**kw)) == 0
    assert fwd(one, cache, window(), hq=3) == 0 and bwd(one, cache, window(), hq=3) == 0


def product_call(s=None, x=None, w=P, n=1, y=None, K=128, N=128, dtype=tdp.TDP_F32, ws=P):
    return tdp.load_library().tdp_grouped_product(ref(s, seqs()), ref(x, rows()), w, n, ref(y, rows(data=2 * P)), K, N,
                                                  dtype, ws, NULL)


def product_backward_call(s=None, x=None, w=P, n=1, dy=None, dx=None, dw=P, K=128, N=128, dtype=tdp.TDP_F32, ws=P):
    return tdp.load_library().tdp_grouped_product_backward(
        ref(s, seqs()), ref(x, rows()), w, n, ref(dy, rows(data=2 * P)), ref(dx, rows(data=3 * P)), dw, K, N, dtype, ws,
        NULL)


@pytest.mark.device_abi
@pytest.mark.parametrize("call", [product_call, product_backward_call], ids=["forward", "backward"])
def test_grouped_product_refusals(call):
    for kw, status in BAD_SEQS:
        assert call(s=seqs(**kw)) == status, kw
    assert call(s="null") == tdp.TDP_EINVAL
    for name in ("x", "y") if call is product_call else ("x", "dy", "dx"):
        for kw, status in BAD_ROWS:
            assert call(**{name: rows(**kw)}) == status, (name, kw)
    for kw, status in [(dict(x="null"), tdp.TDP_EINVAL), (dict(w=None), tdp.TDP_EINVAL), (dict(w=P + 8), tdp.TDP_EINVAL),
                       (dict(K=0), tdp.TDP_ESHAPE), (dict(N=12), tdp.TDP_ESHAPE),
                       (dict(K=tdp.TDP_MAX_FEATURES + 8), tdp.TDP_ESHAPE), (dict(N=tdp.TDP_MAX_FEATURES + 8), tdp.TDP_ESHAPE),
                       (dict(n=0), tdp.TDP_EINVAL), (dict(n=5), tdp.TDP_EINVAL), (dict(dtype=2), tdp.TDP_EINVAL),
                       (dict(x=rows(row_stride=(1 << 21) + 4)), tdp.TDP_ESHAPE)]:
        assert call(**kw) == status, kw
    # few tiles of a long contraction: it is split, so a workspace is needed
    long = dict(s=seqs(num_seqs=1, max_rows=200, total_rows=200), K=4096, N=4096)
    for ws in (None, P + 8):
        assert call(**long, ws=ws) == tdp.TDP_EINVAL and "workspace" in tdp.tdp_last_error()
    # 2^24 rows of 65536 features: more tiles than a launch holds
    many = seqs(num_seqs=100, max_rows=1 << 24, total_rows=100 << 24)
    assert call(s=many, K=65536, N=65536) == tdp.TDP_ESHAPE and "work-items" in tdp.tdp_last_error()
    if call is product_backward_call:
        assert call(dw=P + 4) == tdp.TDP_EINVAL


def test_grouped_product_workspace():
    lib = tdp.load_library()
    fwd = lambda s, n, K, N, dt=tdp.TDP_BF16: lib.tdp_grouped_product_workspace(ctypes.byref(s), n, K, N, dt)  # noqa: E731
    bwd = lambda s, n, K, N, dt=tdp.TDP_BF16: lib.tdp_grouped_product_backward_workspace(  # noqa: E731
        ctypes.byref(s), n, K, N, dt)
    few, many = seqs(max_rows=2, total_rows=8), seqs(max_rows=20000, total_rows=80000)
    long = seqs(num_seqs=1, max_rows=200, total_rows=200)    # few tiles of a long contraction: split
    assert fwd(long, 1, 4096, 4096) % (200 * 4096 * 4) == 0 and fwd(long, 1, 4096, 4096) > 0
    assert fwd(many, 1, 4096, 4096) == 0 and bwd(many, 1, 4096, 4096) == 0
    assert bwd(many, 1, 128, 128) >= 2 * 128 * 128 * 4     # one tile of weights, its rows split
    assert bwd(long, 1, 4096, 4096) >= fwd(long, 1, 4096, 4096)
    for args in ((0, 128, 128), (5, 128, 128), (1, 0, 128), (1, 128, 12), (1, 128, tdp.TDP_MAX_FEATURES + 8)):
        assert fwd(few, *args) == 0 and bwd(few, *args) == 0
    assert fwd(few, 1, 4096, 4096, 7) == 0


def test_grouped_product_workspace_of_short_sequences():
    """The gradient of a weight takes a step at least per sequence, so many short ones are split like a long one."""
    lib = tdp.load_library()
    bwd = lambda s, K, N, dt: lib.tdp_grouped_product_backward_workspace(ctypes.byref(s), 1, K, N, dt)  # noqa: E731
    for dt in (tdp.TDP_BF16, tdp.TDP_F32):
        for n, rows in ((700, 1), (600, 2), (250, 3)):
            short = seqs(num_seqs=n, max_rows=rows, total_rows=n * rows, len_group=1)
            slots = bwd(short, 136, 264, dt) // (136 * 264 * 4)   # two per part; dx needs less
            assert slots >= 2 * (n // 8 if n < 512 else 64), (dt, n, rows, slots)
        few = seqs(num_seqs=7, max_rows=1, total_rows=7, len_group=1)
        assert bwd(few, 136, 264, dt) == 0


@pytest.mark.device_abi
@pytest.mark.parametrize("call", [window_call, window_backward_call], ids=["forward", "backward"])
def test_window_attention_counts_what_it_launches(call):
    """Work is dealt in whole chunks, which may take a launch past its limit where the work alone does not."""
    n = (1 << 24) - 16
    few = seqs(num_seqs=n, max_rows=1, total_rows=n)
    one = {name: heads32(1) for name in ("q", "k", "v", "out")}
    if call is window_backward_call:
        one.update({name: heads32(1) for name in ("dout", "dq", "dk", "dv")})
    assert call(qs=few, ks=few, w=window(back=tdp.TDP_WINDOW_ALL), **one) == tdp.TDP_ESHAPE
    assert "work-items" in tdp.tdp_last_error()


ENORMOUS = dict(num_seqs=1 << 30, max_rows=1 << 24, total_rows=2 ** 31 - 1, row_range=P)


@pytest.mark.parametrize("sinks", [0, 2, (1 << 24) - 200, 1 << 25])
def test_attention_workspaces_of_enormous_counts(sinks):
    """Counts whose products pass 64 bits end in a size or a refusal, not in a division by zero."""
    lib, s, r = tdp.load_library(), seqs(**ENORMOUS), ctypes.byref
    w = window(back=5, sinks=sinks)
    for heads in (1, 4, 65535, 65536):
        rows = heads * s.total_rows * 8
        assert lib.tdp_window_attention_workspace(r(s), r(s), r(w), heads, heads, 64) == 0
        assert lib.tdp_attention_workspace(r(s), r(s), heads, heads, 64) == 0
        for got in (lib.tdp_window_attention_backward_workspace(r(s), r(s), r(w), heads, heads, 64),
                    lib.tdp_attention_backward_workspace(r(s), r(s), heads, heads, 64)):
            assert rows <= got < rows + 256
    for q, k in ((65537, 65537), (1 << 18, 1 << 18), (1 << 30, 1)):
        for got in (lib.tdp_window_attention_workspace(r(s), r(s), r(w), q, k, 64),
                    lib.tdp_window_attention_backward_workspace(r(s), r(s), r(w), q, k, 64),
                    lib.tdp_attention_workspace(r(s), r(s), q, k, 64),
                    lib.tdp_attention_backward_workspace(r(s), r(s), q, k, 64)):
            assert got == 0 and "heads" in tdp.tdp_last_error()


@pytest.mark.device_abi
@pytest.mark.parametrize("heads", [1, 4, 65536])
@pytest.mark.parametrize("call", [window_call, window_backward_call], ids=["forward", "backward"])
def test_window_attention_refuses_enormous_counts(call, heads):
    s, h = seqs(**ENORMOUS), heads32(heads, head_stride=0, row_stride=64, seq_stride=64)
    ts = ("q", "k", "v", "out") + (("dout", "dq", "dk", "dv") if call is window_backward_call else ())
    for w in (window(back=5), window(back=tdp.TDP_WINDOW_ALL, sinks=(1 << 24) - 200)):
        assert call(qs=s, ks=s, w=w, **{name: h for name in ts}) == tdp.TDP_ESHAPE
        assert "work-items" in tdp.tdp_last_error()


@pytest.mark.device_abi
@pytest.mark.parametrize("call", [norm_call, norm_backward_call, product_call, product_backward_call])
def test_layers_refuse_enormous_counts(call):
    """Past 2^30 sequences sums of counts would leave 32 bits; up to there the launch's limit is met or sizes hold."""
    lib, r = tdp.load_library(), ctypes.byref
    past = seqs(num_seqs=(1 << 30) + 1, max_rows=1, total_rows=1000, row_range=P)
    for n in (1, 1 << 20, (1 << 30) + 1):
        assert call(s=past, n=n) == tdp.TDP_ESHAPE and "2^30" in tdp.tdp_last_error()
        assert lib.tdp_layer_norm_workspace(r(past), 128, n) == 0
        for size in (lib.tdp_grouped_product_workspace, lib.tdp_grouped_product_backward_workspace):
            assert size(r(past), n, 128, 128, tdp.TDP_F32) == 0
    s = seqs(**ENORMOUS)
    for n in (1, 513, 1 << 30):
        assert call(s=s, n=n) == tdp.TDP_ESHAPE
        assert lib.tdp_layer_norm_workspace(r(s), 8192, n) == -(-512 // n) * n * 2 * 8192 * 4
