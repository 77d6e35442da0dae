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


@pytest.mark.parametrize("V,H,most,tokens", [(32768, 1024, 257, 128), (32768, 1024, 129, 100), (700, 96, 600, 128), (700, 96, 600, 129), (700, 96, 600, 1),
                                             (700, 96, 3, 2), (20000, 1024, 20000, 19455)])
def test_fewer_tokens_than_the_buffers_hold(example, V, H, most, tokens):
    """Every call has room for a batch of any size up to the most; the results are those of buffers of that size."""
    E = 12
    table, router, directions, words, targets = setup(tokens, V, H, E, seed=most)
    offsets = torch.tensor([0, tokens // 2, tokens][-min(tokens, 2) - 1:], dtype=torch.int32, device=DEV)
    outs = [example.step(example.TiedEnds(V, H, E, 3, n), table, router, directions, words, targets, offsets) for n in (most, tokens)]
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert bool(torch.isfinite(a.float()).all()) and bool(torch.isfinite(b.float()).all())
    assert torch.equal(outs[0][1], outs[1][1])


def test_each_row_of_the_tables_gradient(example):
    """Row by row, so that a wrong one does not hide in the others' norm.

    The 64-bit step takes the rows and the hidden rows as the step rounded them. What is rounded after that, u = 2^-8 of it at
    most: dl (so that dX and the head's part of a table's row are off by u times their terms' absolute sums), dX, the rows'
    gradient, the head's part and the row at the end. An error of dX comes to the rows' gradient by 1 + |router| |directions|
    / 2 at most (norms of matrices; a softmax has a derivative of norm 1/2). 1.1 and 2^-16 are for what is done in 32 bits.
    """
    T, V, u = 500, 700, 2.0 ** -8
    table, router, directions, words, targets = setup(T, seed=3, padded=20)
    offsets = torch.tensor([0, 200, 480], dtype=torch.int32, device=DEV)
    ends = example.TiedEnds(V, 96, 12, 3, T)
    seen = {}

    def spy(name, at):
        call = getattr(ends, name)

        def wrapped(*args):
            out = call(*args)
            seen[name] = (out if at is None else args[at]).clone()
            return out

        setattr(ends, name, wrapped)

    spy("rows", None)
    spy("loss", 1)
    spy("rows_backward", 2)
    got = example.step(ends, table, router, directions, words, targets, offsets)[1]
    t, r, d = table.double().requires_grad_(), router.double(), directions.double()
    on = (words >= 0).double()[:, None]
    rows = t[words.long().clamp(min=0)] * on * ends.scale
    rows = rows + (seen["rows"].double() - rows).detach()
    p = torch.softmax(rows @ r, -1)
    ids = ends.ids[:T].long()  # every token has its experts, padded ones too: those are behind the last sequence
    hidden = rows + (p.gather(1, ids)[..., None] * d[ids]).sum(1)
    hidden = hidden + (seen["loss"].double() - hidden).detach()
    logits = hidden @ t.t()
    good = ((targets >= 0) & (targets < V)).double()
    a = good / good.sum()
    lse = torch.logsumexp(logits, -1)
    y = targets.long().clamp(0, V - 1)
    total = (a * (lse - logits.gather(1, y[:, None])[:, 0] + ends.z * lse * lse)).sum()
    cuts = offsets.tolist()
    for lo, hi in zip(cuts[:-1], cuts[1:]):
        f = torch.bincount(ids[lo:hi].flatten(), minlength=12).double() / (3 * (hi - lo))
        total = total + ends.balance / 2 * 12 * (f * p[lo:hi].mean(0)).sum()
    total.backward()
    with torch.no_grad():
        dl = torch.softmax(logits, -1) * (a * (1 + 2 * ends.z * lse))[:, None]
        dl.scatter_add_(1, y[:, None], -a[:, None])
        x, w = hidden.detach(), table.double()
        d_hidden = u * ((dl.abs() @ w.abs()).norm(dim=1) + (dl @ w).norm(dim=1))
        gain = 1 + float(torch.linalg.matrix_norm(r, 2) * torch.linalg.matrix_norm(d, 2)) / 2
        d_rows = (gain * d_hidden + u * seen["rows_backward"].double().norm(dim=1)) * on[:, 0]
        off = u * ((dl.abs().t() @ x.abs()).norm(dim=1) + (dl.t() @ x).norm(dim=1) + t.grad.norm(dim=1))
        off.index_add_(0, words.long().clamp(min=0), ends.scale * d_rows)
        err = (got.double() - t.grad).norm(dim=1)
        assert bool((err <= 1.1 * off + 2.0 ** -16 * t.grad.norm(dim=1).max()).all()), float((err / off).max())
        assert float(off.median()) < float(t.grad.norm(dim=1).median()) / 2  # a row of zeros, or another's, would show
