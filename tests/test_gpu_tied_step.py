"""The ends of a training step together, as examples/tied_step.py uses them: every gradient against the same step in
float64 under automatic differentiation, with padded tokens, and the calls replayed from a CUDA graph."""
import importlib.util
import math
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
    spec = importlib.util.spec_from_file_location("tied_step", os.path.join(ROOT, "examples", "tied_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def setup(T, V=700, H=96, E=12, seed=0, padded=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    table = (rand(V, H) * H ** -0.5).to(torch.bfloat16)
    router, directions = rand(H, E) * 0.1, rand(E, H) * 0.5
    words = torch.randint(0, V, (T,), generator=gen, device=DEV, dtype=torch.int32)
    targets = torch.randint(0, V, (T,), generator=gen, device=DEV, dtype=torch.int32)
    if padded:
        words[T - padded:], targets[T - padded:] = -1, -100
    return table, router, directions, words, targets


def step64(ends, table, router, directions, words, targets, offsets, ids, hidden_of):
    """The step in float64. The hidden rows are rounded to bf16 as the step's are; ids are those that it chose."""
    V = table.shape[0]
    t, r, d = (x.double().requires_grad_() for x in (table, router, directions))
    live_w = (words >= 0) & (words < V)
    rows = torch.where(live_w[:, None], t[words.long().clamp(0, V - 1)], 0.0) * ends.scale
    logits = rows @ r
    p = torch.softmax(logits, -1)
    live = ids >= 0
    at = ids.long().clamp(min=0)
    w = torch.where(live, p.gather(1, at), 0.0)
    hidden = rows + (w[..., None] * d[at]).sum(1)
    hidden = hidden + (hidden_of.double() - hidden).detach()  # the step's own rounding, with the identity's gradient
    lg = hidden @ t.t()
    lse = torch.logsumexp(lg, -1)
    good = (targets >= 0) & (targets < V)
    ce = torch.where(good, lse - lg.gather(1, targets.long().clamp(0, V - 1)[:, None])[:, 0], 0.0)
    n = max(int(good.sum()), 1)
    total = (ce.sum() + ends.z * torch.where(good, lse * lse, 0.0).sum()) / n
    E, k = router.shape[1], ids.shape[1]
    ends_at = offsets.tolist()
    balance = []
    for a, b in zip(ends_at[:-1], ends_at[1:]):
        on = live[a:b].any(-1)
        m = max(int(on.sum()), 1)
        f = torch.bincount(ids[a:b][live[a:b]].long(), minlength=E).double() / (k * m)
        balance.append(E * (f * (p[a:b] * on[:, None]).sum(0) / m).sum())
    total = total + ends.balance * torch.stack(balance).mean()
    total.backward()
    return total.detach(), t.grad, r.grad, d.grad


@pytest.mark.parametrize("T,padded,cuts", [(40, 0, [0, 40]), (333, 0, [0, 100, 333]), (600, 45, [0, 0, 300, 555])])
def test_a_step_against_64_bits(example, T, padded, cuts):
    table, router, directions, words, targets = setup(T, padded=padded)
    offsets = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    ends = example.TiedEnds(700, 96, 12, 3, T)
    hidden = {}
    keep = ends.loss

    def loss(t, h, y):
        hidden["rows"] = h.clone()
        return keep(t, h, y)

    ends.loss = loss
    total, d_table, d_router, d_directions = example.step(ends, table, router, directions, words, targets, offsets)
    want = step64(ends, table, router, directions, words, targets, offsets, ends.ids[:T], hidden["rows"])
    assert abs(float(total - want[0])) < 1e-4 * float(want[0])
    # bf16 on the way: dl, d hidden, the rows' gradient and the table's gradient twice are rounded, half a step of 2^-8 each
    for got, ref in ((d_table, want[1]), (d_router, want[2]), (d_directions, want[3])):
        assert float((got.double() - ref).norm()) <= 5 * 2.0 ** -8 * float(ref.norm())


def test_the_example_runs(example):
    out = example.main(steps=2)
    assert all(math.isfinite(v) for v in out)


def test_inputs_of_another_shape_are_refused(example):
    ends = example.TiedEnds(700, 96, 12, 3, 64)
    table, _, _, words, targets = setup(64)
    with pytest.raises(ValueError):
        ends.rows(table.float(), words)
    with pytest.raises(ValueError):
        ends.rows(table, words.long())
    with pytest.raises(ValueError):
        ends.rows(table, setup(65)[3])
    with pytest.raises(ValueError):
        ends.loss(table, torch.zeros(96, 64, dtype=torch.bfloat16, device=DEV).t(), targets)
    with pytest.raises(ValueError):
        example.TiedEnds(700, 100, 12, 3, 64)


def test_the_calls_together_replayed(example):
    """Both ends captured in one graph with one workspace between them, replayed on other tokens."""
    T, V, H, E, k = 300, 700, 96, 12, 3
    table, router, directions, words, targets = setup(T, padded=20)
    offsets = torch.tensor([0, 120, 280], dtype=torch.int32, device=DEV)
    ends = example.TiedEnds(V, H, E, k, T)
    logits = torch.randn(T, E, device=DEV)
    d_losses = torch.full((T,), 1.0 / T, device=DEV)
    d_weights = torch.randn(T, k, device=DEV)
    out = {}

    def run():
        out["rows"] = ends.rows(table, words)
        out["weights"], out["ids"], out["balance"] = ends.route(logits, offsets)
        out["losses"] = ends.loss(table, out["rows"], targets)
        out["d_rows"], out["d_table"] = ends.loss_backward(table, out["rows"], targets, d_losses)
        out["d_logits"] = ends.route_backward(logits, offsets, d_weights)
        ends.rows_backward(out["d_table"], words, out["d_rows"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    captured = dict(out)
    other = setup(T, seed=5, padded=70)
    for t, new in zip((table, words, targets), (other[0], other[3], other[4])):
        t.copy_(new)
    logits.copy_(torch.randn(T, E, device=DEV))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    got = {name: t.clone() for name, t in captured.items()}
    run()
    torch.cuda.synchronize()
    for name in got:
        assert torch.equal(got[name], out[name]), name
