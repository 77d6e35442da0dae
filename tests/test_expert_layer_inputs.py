"""What the expert layer of examples/expert_layer.py refuses before it hands pointers to the library, on the CPU."""
import importlib.util
import os
import types

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")

E, K, H, F, T = 8, 2, 32, 16, 5


@pytest.fixture
def example(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("expert_layer_inputs", os.path.join(ROOT, "examples", "expert_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    calls = []
    fake = types.SimpleNamespace(OUT_F32=0, OUT_BF16=1, QUANT_PLAIN=0, QUANT_GATED=1, gemm_route_plan_workspace_size=lambda *a: 0)
    for name in ("gemm_route", "gemm_route_plan", "gemm_quantize_int8", "gemm_int8_grouped", "gemm_route_combine",
                 "gemm_route_combine_backward", "gemm_route_backward"):
        setattr(fake, name, lambda *a, _n=name: calls.append(_n))
    monkeypatch.setattr(mod, "g", fake)
    layer = mod.ExpertLayer(torch.zeros(E, 2 * F, H), torch.zeros(E, H, F), K, {}, T)
    calls.clear()
    return mod, layer, calls


def inputs():
    return dict(x=torch.zeros(T, H, dtype=torch.bfloat16), logits=torch.zeros(T, E), bias=torch.zeros(E))


def test_the_right_inputs_reach_the_library(example):
    _, layer, calls = example
    layer(**inputs())
    layer(torch.zeros(T, H + 8, dtype=torch.bfloat16)[:, :H], torch.zeros(T, E + 1)[:, :E])  # rows of a wider tensor
    assert calls.count("gemm_route") == 2 and calls.count("gemm_int8_grouped") == 4
    layer.router_gradient(torch.zeros(T, E), torch.zeros(T, H, dtype=torch.bfloat16))
    assert calls[-1] == "gemm_route_backward"


@pytest.mark.parametrize("change", [
    dict(x=torch.zeros(T, H)), dict(x=torch.zeros(T, H, dtype=torch.float16)), dict(x=torch.zeros(T, H - 8, dtype=torch.bfloat16)),
    dict(x=torch.zeros(H, T, dtype=torch.bfloat16).t()), dict(x=torch.zeros(T + 1, H, dtype=torch.bfloat16)),
    dict(logits=torch.zeros(T, E, dtype=torch.bfloat16)), dict(logits=torch.zeros(T - 1, E)), dict(logits=torch.zeros(T, E - 1)),
    dict(logits=torch.zeros(E, T).t()), dict(logits=torch.zeros(T, E, dtype=torch.float64)),
    dict(bias=torch.zeros(E, dtype=torch.bfloat16)), dict(bias=torch.zeros(E - 1)), dict(bias=torch.zeros(2 * E)[::2])])
def test_other_inputs_are_refused(example, change):
    _, layer, calls = example
    with pytest.raises(ValueError):
        layer(**{**inputs(), **change})
    assert not calls


@pytest.mark.parametrize("logits,d_out", [
    (torch.zeros(T, E), torch.zeros(T, H)), (torch.zeros(T, E, dtype=torch.bfloat16), torch.zeros(T, H, dtype=torch.bfloat16)),
    (torch.zeros(T - 1, E), torch.zeros(T - 1, H, dtype=torch.bfloat16)), (torch.zeros(T, E), torch.zeros(T, H - 1, dtype=torch.bfloat16))])
def test_other_gradients_are_refused(example, logits, d_out):
    _, layer, calls = example
    layer(**inputs())
    calls.clear()
    with pytest.raises(ValueError):
        layer.router_gradient(logits, d_out)
    assert not calls


def test_weights_that_do_not_fit(example):
    mod, _, _ = example
    for w1, w2 in (((E, 2 * F, H), (E, H, F + 16)), ((E, 2 * F, H), (E - 1, H, F)), ((E, 2 * F, H), (E, H + 16, F)), ((E, 2 * F - 1, H), (E, H, F))):
        with pytest.raises(ValueError):
            mod.ExpertLayer(torch.zeros(w1), torch.zeros(w2), K, {}, T)
