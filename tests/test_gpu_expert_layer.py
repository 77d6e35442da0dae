"""The expert layer of examples/expert_layer.py: every call together, against the
same layer in float64 on the quantised values, with padded tokens, on a side
stream and replayed from a CUDA graph.
"""
import importlib.util
import os

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def layer64(layer, x, logits):
    """The layer's definition in 64 bits on its quantised weights and rows, its ids and (differentiable) logits.

    The rows that the layer quantised are taken as it left them, after a check that they are its inputs' within
    half a step: a value next to a half may be rounded either way, and its step would be no error.
    """
    ids, slots = layer.ids[:x.shape[0]].long(), layer.slots[:x.shape[0]].long()
    live = ids >= 0
    top = torch.where(live, logits.gather(1, ids.clamp(min=0)), torch.full_like(logits[:, :1], -1e300))
    w = torch.softmax(top, -1) * live
    out = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
    for e in range(layer.E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        r = slots[t, j]
        q, s = layer.a1[r].double(), layer.sa1[r, None].double()
        assert ((q * s - x[t].double()).abs() <= 0.5001 * s).all()
        h = (q @ layer.q1[e].double().t()) * s * layer.s1[e].double()
        gate, up = h.chunk(2, -1)
        q, s = layer.a2[r].double(), layer.sa2[r, None].double()
        assert ((q * s - gate * torch.sigmoid(gate) * up).abs() <= 0.5001 * s).all()
        y = (q @ layer.q2[e].double().t()) * s * layer.s2[e].double()
        out = out.index_add(0, t, w[t, j, None] * y)
    return out


def make(example, T, E, k, H, F, seed=0):
    import smem_swizzle_layouts_gb300 as g
    gen = torch.Generator(device=DEV).manual_seed(seed)
    w1 = torch.randn(E, 2 * F, H, generator=gen, device=DEV) * H ** -0.5
    w2 = torch.randn(E, H, F, generator=gen, device=DEV) * F ** -0.5
    layer = example.ExpertLayer(w1, w2, k, dict(score=g.ROUTE_SOFTMAX, renormalize=1), tokens=T)
    x = torch.randn(T, H, generator=gen, device=DEV).to(torch.bfloat16)
    return g, layer, x, torch.randn(T, E, generator=gen, device=DEV)


@pytest.mark.parametrize("T,E,k,H,F", [(1, 8, 2, 64, 48), (37, 16, 4, 256, 128), (600, 8, 2, 512, 256), (1500, 64, 6, 128, 64)])
def test_layer(example, T, E, k, H, F):
    g, layer, x, logits = make(example, T, E, k, H, F)
    if T > 8:
        logits[-5:] = -float("inf")  # padded tokens
    y = layer(x, logits)
    logits64 = logits.double().requires_grad_()
    ref = layer64(layer, x, logits64)
    # the output is rounded to bf16: a relative 2-norm of at most 2^-9, and fp32 sums
    assert float((y.double() - ref.detach()).norm() / ref.detach().norm()) <= 2.0 ** -9 + 1e-3
    if T > 8:
        assert (y[-5:] == 0).all() and (layer.ids[T - 5:T] == -1).all()
    d_out = torch.randn(T, H, device=DEV).to(torch.bfloat16)
    got = layer.router_gradient(logits, d_out)
    (ref * d_out.double()).sum().backward()
    want = torch.nan_to_num(logits64.grad)
    assert float((got.double() - want).norm() / want.norm()) <= 2e-3
    st, word = g.gemm_last_device_status()
    assert st == g.OK, hex(word)


def test_layer_in_a_graph(example):
    """Routing, plan and products of new inputs in a replayed graph: no size was fixed at capture."""
    g, layer, x, logits = make(example, 300, 16, 4, 256, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, logits)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = layer(x, logits)
        for seed in (1, 2):
            _, _, x2, logits2 = make(example, 300, 16, 4, 256, 128, seed)
            logits2[:, 3] += 4 * seed  # most rows to one expert
            x.copy_(x2)
            logits.copy_(logits2)
            graph.replay()
            side.synchronize()
            got = y.clone()
            assert torch.equal(got, layer(x2, logits2))
            side.synchronize()


def test_example_runs(example):
    # 8-bit weights and activations: each carries a relative error of about 127^-1 / sqrt(12) of its largest
    # value, four sigma: 0.9 %; four of them and the bf16 output
    assert example.main() < 0.04
