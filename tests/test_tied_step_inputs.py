"""What the ends of examples/tied_step.py refuse before they hand pointers to the library, on the CPU."""
import importlib.util
import os
import types

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")

V, H, E, K, T, S = 50, 16, 8, 2, 5, 3
BF16, INT = torch.bfloat16, torch.int32


@pytest.fixture
def ends(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("tied_step_inputs", os.path.join(ROOT, "examples", "tied_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    fake = types.SimpleNamespace(OUT_F32=0, OUT_BF16=1, calls=[])
    for name in ("gemm_cross_entropy", "gemm_cross_entropy_backward", "gemm_embed_backward", "gemm_route_balance"):
        setattr(fake, name + "_workspace_size", lambda *a: 256)
    for name in ("gemm_embed", "gemm_route", "gemm_route_balance", "gemm_cross_entropy", "gemm_cross_entropy_backward",
                 "gemm_route_backward", "gemm_route_balance_backward", "gemm_embed_backward"):
        setattr(fake, name, lambda *a, _n=name: fake.calls.append(_n))
    monkeypatch.setattr(mod, "g", fake)
    out = mod.TiedEnds(V, H, E, K, T, device="cpu")
    out.calls = fake.calls
    return out


def inputs(T=T, S=S):
    table, rows, ids = torch.zeros(V, H, dtype=BF16), torch.zeros(T, H, dtype=BF16), torch.zeros(T, dtype=INT)
    logits, offsets = torch.zeros(T, E), torch.zeros(S + 1, dtype=INT)
    return dict(rows=dict(table=table, words=ids), route=dict(logits=logits, offsets=offsets),
                loss=dict(table=table, hidden=rows, targets=ids),
                loss_backward=dict(table=table, hidden=rows, targets=ids, d_losses=torch.zeros(T)),
                route_backward=dict(logits=logits, offsets=offsets, d_weights=torch.zeros(T, K)),
                rows_backward=dict(d_table=table.clone(), words=ids, d_rows=rows))


@pytest.mark.parametrize("tokens", [1, T - 1, T])
def test_up_to_the_most_tokens_reach_the_library(ends, tokens):
    for name, args in inputs(tokens, min(S, tokens)).items():
        before = len(ends.calls)
        getattr(ends, name)(**args)
        assert len(ends.calls) > before


@pytest.mark.parametrize("name", sorted(inputs()))
def test_more_tokens_than_the_buffers_hold_are_refused(ends, name):
    if name == "route_backward":
        ends.route(**inputs()["route"])
        ends.calls.clear()
    with pytest.raises(ValueError):
        getattr(ends, name)(**inputs(T + 1)[name])
    assert not ends.calls


@pytest.mark.parametrize("name", ["route", "route_backward"])
def test_more_sequences_than_the_buffers_hold_are_refused(ends, name):
    if name == "route_backward":
        ends.route(**inputs()["route"])
        ends.calls.clear()
    with pytest.raises(ValueError):
        getattr(ends, name)(**inputs(T, T + 1)[name])
    assert not ends.calls


@pytest.mark.parametrize("name,change", [
    ("rows", dict(table=torch.zeros(V, H))), ("rows", dict(words=torch.zeros(T, dtype=torch.int64))),
    ("route", dict(logits=torch.zeros(T, E + 1))), ("route", dict(offsets=torch.zeros(S + 1))),
    ("loss", dict(table=torch.zeros(V - 1, H, dtype=BF16))), ("loss", dict(targets=torch.zeros(T - 1, dtype=INT))),
    ("loss_backward", dict(hidden=torch.zeros(H, T, dtype=BF16).t())), ("loss_backward", dict(d_losses=torch.zeros(T, dtype=torch.float64))),
    ("loss_backward", dict(d_losses=torch.zeros(2 * T)[::2])), ("loss_backward", dict(table=torch.zeros(V, H))),
    ("route_backward", dict(logits=torch.zeros(T, E, dtype=BF16))), ("route_backward", dict(d_weights=torch.zeros(T, K + 1))),
    ("rows_backward", dict(d_table=torch.zeros(V, H))), ("rows_backward", dict(words=torch.zeros(T + 1, dtype=INT))),
    ("rows_backward", dict(words=torch.zeros(T, dtype=torch.int64)))])
def test_inputs_of_another_shape_are_refused(ends, name, change):
    if name == "route_backward":
        ends.route(**inputs()["route"])
        ends.calls.clear()
    with pytest.raises(ValueError):
        getattr(ends, name)(**{**inputs()[name], **change})
    assert not ends.calls
