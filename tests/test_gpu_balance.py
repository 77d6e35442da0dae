"""The balance loss of a router, its counts, and the gradient of its logits, against float64.

Tolerances count roundings. A token's p has an exponential (two units in the last place), a sum over E and a reciprocal: within
2^-20 of itself. A mean is a sum in fp32 of at most 2^-20 more; a loss a sum of E products of such. A gradient's element is
p (c - sum p c): within 2^-19 of p (|c| + sum p |c|), and half a step of its type.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": (torch.float32, 0), "bf16": (torch.bfloat16, 1), "f16": (torch.float16, 2)}


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


def make(T, E, k, type="f32", seed=0, padded=0.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ld = E + 3
    logits = torch.full((T, ld), math.nan, dtype=TYPES[type][0], device=DEV)[:, :E]
    logits.copy_(torch.randn(T, E, generator=gen, device=DEV) * 2)
    ids = logits.float().argsort(-1, descending=True)[:, :k].to(torch.int32).contiguous()
    if padded:
        off = torch.rand(T, generator=gen, device=DEV) < padded
        logits[off], ids[off] = -math.inf, -1
    return logits, ids


def forward(g, logits, ids, score=0, offsets=None):
    T, E = logits.shape
    k, S = ids.shape[1], 1 if offsets is None else offsets.numel() - 1
    code = {v[0]: v[1] for v in TYPES.values()}[logits.dtype]
    counts, tokens = (torch.full(s, -7, dtype=torch.int32, device=DEV) for s in ((S, E), (S,)))
    means, losses = (torch.full(s, math.nan, device=DEV) for s in ((S, E), (S,)))
    n = g.gemm_route_balance_workspace_size(T, E, S)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)
    g.gemm_route_balance(T, E, logits, code, logits.stride(0), k, dict(score=score), ids, S, offsets, counts, tokens, means, losses, ws, n)
    return counts, tokens, means, losses


def backward(g, logits, ids, score, offsets, counts, tokens, dlosses, old=None):
    T, E = logits.shape
    code = {v[0]: v[1] for v in TYPES.values()}[logits.dtype]
    d = torch.full((T, E + 1), 5.0, dtype=logits.dtype, device=DEV)[:, :E]
    if old is not None:
        d.copy_(old)
    g.gemm_route_balance_backward(T, E, logits, code, logits.stride(0), ids.shape[1], dict(score=score), ids, dlosses.numel(), offsets, counts,
                                  tokens, dlosses, d, d.stride(0), int(old is not None))
    return d


def plain(logits, ids, score, offsets, dlosses=None):
    """Everything in float64, sequence by sequence, and the size of each gradient's terms."""
    T, E = logits.shape
    k = ids.shape[1]
    live = ((ids >= 0) & (ids < E)).any(-1)
    x = torch.where(live[:, None], logits.double(), 0.0)
    x.requires_grad_()
    p = torch.softmax(x, -1) if score == 0 else torch.sigmoid(x) / torch.sigmoid(x).sum(-1, keepdim=True)
    ends = [0, T] if offsets is None else offsets.clamp(0, T).tolist()
    counts, tokens, means, losses = [], [], [], []
    size = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    for s, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        b = max(a, b)
        good = ids[a:b][(ids[a:b] >= 0) & (ids[a:b] < E)]
        n = int(live[a:b].sum())
        count = torch.bincount(good.long(), minlength=E)
        mean = (p[a:b] * live[a:b, None]).sum(0) / max(n, 1)
        counts.append(count)
        tokens.append(n)
        means.append(mean)
        losses.append(E * (count.double() / (k * max(n, 1)) * mean).sum())
        if dlosses is not None:
            c = float(dlosses[s]) * E * count.double() / (k * max(n, 1)) / max(n, 1)
            q = p[a:b].detach()
            size[a:b] = q * (c.abs() + (q * c.abs()).sum(-1, keepdim=True))
    out = [torch.stack(counts).int(), torch.tensor(tokens, dtype=torch.int32, device=DEV), torch.stack(means), torch.stack(losses)]
    if dlosses is None:
        return [t.detach() for t in out]
    (out[3] * dlosses.double()).sum().backward()
    inside = torch.zeros(T, dtype=torch.bool, device=DEV)
    for a, b in zip(ends[:-1], ends[1:]):
        inside[a:b] = True
    return [t.detach() for t in out], x.grad, size, inside & live, inside


def check(g, T, E, k, score=0, cuts=None, type="f32", seed=0, padded=0.0):
    logits, ids = make(T, E, k, type, seed, padded)
    offsets = None if cuts is None else torch.tensor(cuts, dtype=torch.int32, device=DEV)
    S = 1 if cuts is None else len(cuts) - 1
    dlosses = torch.randn(S, device=DEV)
    counts, tokens, means, losses = forward(g, logits, ids, score, offsets)
    want, grad, size, live, inside = plain(logits, ids, score, offsets, dlosses)
    assert torch.equal(counts, want[0]) and torch.equal(tokens, want[1])
    assert bool(((means - want[2]).abs() <= 2.0 ** -19 * want[2] + 1e-38).all())
    assert bool(((losses - want[3]).abs() <= 2.0 ** -18 * want[3] + 1e-38).all())
    eps = torch.finfo(logits.dtype).eps / 2
    tiny = 2.0 ** -25 if logits.dtype == torch.float16 else 1e-38
    d = backward(g, logits, ids, score, offsets, counts, tokens, dlosses)
    bound = 2.0 ** -18 * size + eps * grad.abs() + tiny
    assert bool(((d.double() - grad).abs() <= bound)[live].all())
    assert not d[inside & ~live].any() and bool((d[~inside] == 5.0).all())  # rows of no sequence are left as they were
    assert bool((torch.as_strided(d, (T,), (E + 1,), E) == 5.0).all())
    old = torch.randn(T, E, device=DEV).to(logits.dtype)
    d = backward(g, logits, ids, score, offsets, counts, tokens, dlosses, old)
    total = grad + old.double()
    assert bool(((d.double() - total).abs() <= 2.0 ** -18 * size + eps * total.abs() + 2.0 ** -24 * (grad.abs() + old.double().abs()) + tiny)[live].all())
    assert torch.equal(d[~live], old[~live])


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (31, 8, 8), (32, 60, 6), (33, 64, 6), (100, 65, 4), (1000, 128, 8), (4097, 160, 10), (700, 256, 8),
                                   (5000, 384, 3), (300, 512, 32), (2000, 1000, 8), (9000, 1024, 32), (20000, 5, 1)])
def test_one_sequence(g, T, E, k, score):
    check(g, T, E, k, score, seed=T, padded=0.1 if T > 4 else 0.0)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,cuts", [(10, [0, 0, 3, 3, 10, 10]), (33, [0, 33]), (64, [2, 30, 31, 60]), (5000, [0, 1, 2, 40, 1000, 1000, 4999]),
                                    (5000, [7, 2500, 5000]), (6000, list(range(0, 6001, 7))), (40, [0, 50, 60]), (300, [-5, 100, 400])])
def test_ragged_sequences(g, T, cuts, score, type):
    check(g, T, 72, 4, score, cuts, type, seed=len(cuts), padded=0.15)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,S", [(1, 9), (5, 9), (32, 40), (30, 31), (20, 700), (300, 700), (2000, 33)])
def test_many_sequences_most_of_them_empty(g, T, S, score):
    gen = torch.Generator().manual_seed(T + S)
    cuts = torch.randint(0, min(T, 25) + 1, (S + 1,), generator=gen).sort().values
    cuts[-(S // 3):] = T  # a run of empty ones at the end, others between
    check(g, T, 12, 2, score, cuts.tolist(), seed=S, padded=0.1)


@pytest.mark.parametrize("T,E,k,S", [(600, 64, 6, 200), (500, 100, 3, 310), (900, 256, 8, 170), (300, 513, 2, 160), (400, 1024, 8, 45), (400, 1000, 5, 170)])
def test_many_sequences_of_many_experts(g, T, E, k, S):
    cuts = torch.randint(0, T + 1, (S + 1,), generator=torch.Generator().manual_seed(S)).sort().values
    check(g, T, E, k, 0, cuts.tolist(), seed=E, padded=0.1)


def test_padded_tokens_may_hold_anything(g):
    logits, ids = make(600, 64, 6, padded=0.3, seed=3)
    dead = (ids < 0).all(-1)
    want = forward(g, logits, ids)
    dl = torch.ones(1, device=DEV)
    grad = backward(g, logits, ids, 0, None, want[0], want[1], dl)
    logits[dead] = math.nan
    got = forward(g, logits, ids)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(backward(g, logits, ids, 0, None, got[0], got[1], dl), grad)


def test_masked_experts(g):
    """Experts masked with -inf have no share and no gradient; a token may have fewer ids than k, and ids that are none's."""
    logits, ids = make(500, 40, 5, seed=4)
    logits[:, 7], logits[::2, 8] = -math.inf, -math.inf
    ids[ids == 7] = -1
    ids[::3, 2:] = 40
    for score in (0, 1):
        counts, tokens, means, losses = forward(g, logits, ids, score)
        dl = torch.full((1,), 3.0, device=DEV)
        want, grad, size, live, _ = plain(logits, ids, score, None, dl)
        assert torch.equal(counts, want[0]) and torch.equal(tokens, want[1]) and float(means[0, 7]) == 0.0
        assert bool(((losses - want[3]).abs() <= 2.0 ** -18 * want[3]).all())
        d = backward(g, logits, ids, score, None, counts, tokens, dl)
        assert not d[:, 7].any()
        assert bool(((d.double() - torch.nan_to_num(grad)).abs() <= 2.0 ** -17 * size + 1e-38).all())


def test_no_live_token(g):
    logits, ids = make(200, 64, 6, seed=5)
    logits.fill_(math.nan)
    ids.fill_(-1)
    counts, tokens, means, losses = forward(g, logits, ids)
    assert not counts.any() and not tokens.any() and not means.any() and not losses.any()
    assert not backward(g, logits, ids, 0, None, counts, tokens, torch.ones(1, device=DEV)).any()


def test_no_tokens(g):
    logits, ids = torch.empty(0, 16, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    counts, tokens, means, losses = forward(g, logits, ids, 0, torch.zeros(4, dtype=torch.int32, device=DEV))
    assert not counts.any() and not tokens.any() and not means.any() and not losses.any()


@pytest.mark.parametrize("S,E", [(1, 1), (9, 70), (700, 33)])
def test_no_tokens_of_many_sequences(g, S, E):
    logits, ids = torch.empty(0, E, device=DEV), torch.empty(0, 1, dtype=torch.int32, device=DEV)
    assert g.gemm_route_balance_workspace_size(0, E, S) == 0
    counts, tokens, means, losses = forward(g, logits, ids, 0, torch.zeros(S + 1, dtype=torch.int32, device=DEV))
    assert not counts.any() and not tokens.any() and not means.any() and not losses.any()


def test_a_perfect_balance_has_loss_one(g):
    logits, ids = torch.zeros(512, 16, device=DEV), (torch.arange(1024, device=DEV) % 16).int().view(512, 2)
    counts, tokens, means, losses = forward(g, logits, ids)
    assert bool((counts == 64).all()) and int(tokens) == 512 and bool((means == 1 / 16).all()) and float(losses) == 1.0


def test_gradient_against_differences(g):
    """(loss(x + h d) - loss(x - h d)) / 2h for a random direction, in the kernel's own losses.

    With |d| <= 1 and h = 2^-5 the third derivative, at most 6 E max f, leaves h^2 of the loss; fp32 leaves 2^-21 / h.
    """
    logits, ids = make(64, 12, 3, seed=6)
    logits = logits.clone()
    d = torch.randint(-1, 2, logits.shape, device=DEV).float()
    h = 2.0 ** -5
    for score in (0, 1):
        counts, tokens, _, losses = forward(g, logits, ids, score)
        grad = backward(g, logits, ids, score, None, counts, tokens, torch.ones(1, device=DEV))
        up, down = (float(forward(g, logits + s * d, ids, score)[3]) for s in (h, -h))
        assert abs((up - down) / (2 * h) - float((grad * d).sum())) <= h * h * float(losses) + 2.0 ** -21 / h * float(losses)


def test_the_same_call_twice_and_replayed(g):
    T, E, k, S = 7000, 96, 6, 5
    logits, ids = make(T, E, k, "bf16", seed=7, padded=0.1)
    logits = logits.contiguous()
    offsets = torch.tensor([0, 100, 100, 3000, 6900, 7000], dtype=torch.int32, device=DEV)
    counts, tokens = torch.empty(S, E, dtype=torch.int32, device=DEV), torch.empty(S, dtype=torch.int32, device=DEV)
    means, losses, dl = torch.empty(S, E, device=DEV), torch.empty(S, device=DEV), torch.rand(S, device=DEV)
    d = torch.empty_like(logits)
    n = g.gemm_route_balance_workspace_size(T, E, S)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def step():
        g.gemm_route_balance(T, E, logits, 1, E, k, None, ids, S, offsets, counts, tokens, means, losses, ws, n)
        g.gemm_route_balance_backward(T, E, logits, 1, E, k, None, ids, S, offsets, counts, tokens, dl, d, E, 0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    first = [t.clone() for t in (counts, tokens, means, losses, d)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    old = [t.clone() for t in (logits, ids, offsets)]
    other = make(T, E, k, "bf16", seed=8, padded=0.3)
    logits.copy_(other[0])
    ids.copy_(other[1])
    offsets.copy_(torch.tensor([0, 1, 5000, 5001, 5002, 6000], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    want = plain(logits, ids, 0, offsets)
    assert torch.equal(counts, want[0]) and torch.equal(tokens, want[1])
    assert bool(((losses - want[3]).abs() <= 2.0 ** -18 * want[3]).all())
    for t, o in zip((logits, ids, offsets), old):
        t.copy_(o)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (counts, tokens, means, losses, d)))
