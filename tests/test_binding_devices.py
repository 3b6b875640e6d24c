"""The binding makes a tensor's device current for the calls of a layer: a launch goes to the current device, and the
null stream is the current device's too.  No GPU needed."""
import ast
import contextlib
import inspect

import pytest
import torch

import overlap_tiling_trapezoidal_amd as tdp

LAYER = {"tdp_rope_apply", "tdp_qk_norm_rope", "tdp_qk_norm_rope_backward", "tdp_attention", "tdp_attention_backward",
         "tdp_window_attention", "tdp_window_attention_backward", "tdp_layer_norm", "tdp_layer_norm_backward",
         "tdp_grouped_product", "tdp_grouped_product_backward"}


@pytest.mark.parametrize("name", sorted(LAYER))
def test_layer_calls_go_through_the_device_guard(name):
    assert name in tdp.DEVICE_FUNCTIONS
    tree = ast.parse(inspect.getsource(getattr(tdp, name)))
    guarded = [a.attr for n in ast.walk(tree) if isinstance(n, ast.Call) and getattr(n.func, "id", "") == "_on"
               for a in n.args if isinstance(a, ast.Attribute) and a.attr in LAYER]
    assert guarded == [name]
    assert not [n for n in ast.walk(tree) if isinstance(n, ast.Call) and getattr(n.func, "attr", "") in LAYER]


def test_device_guard(monkeypatch):
    current, calls = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d.index
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    call = lambda *args: calls.append((current[0], args)) or 0  # noqa: E731
    for index in (0, 1):
        tdp._on(torch.device("cuda", index), call, "a", index)
    assert calls == [(0, ("a", 0)), (1, ("a", 1))] and current == [0]
    with pytest.raises(tdp.TdpError):
        tdp._on(torch.device("cuda", 1), lambda: tdp.TDP_EINVAL)
