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
