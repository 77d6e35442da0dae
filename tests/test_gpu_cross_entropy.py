"""The head's cross entropy and its gradients against float64, at the sizes and masks where tiles, pieces and splits end.

Tolerances count roundings.
Forward: sums on the tensor cores are fp32. K products of random signs are off by far less than sqrt(K) * 2^-22 of the
logits' deviation; a normaliser by that beside 2^-22 of itself for its exponentials, their sum and the logarithm.
Backward: a gradient's element is a sum of terms dl * value. dl carries one rounding to the inputs' type, at most half a
step, u of it (fp16: at least half of the smallest number, 2^-25, of dl scaled to 2^14), and the exponential 2^-18 at most;
the element one more to its own type. So an element is off by (u + 2^-18) times its terms' absolute sum and by half a step of
itself; and as the terms' half steps are independent, the norm of all errors by 2 u of the root of their squares' sum, which is
over three times what half steps of random sign leave.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": (torch.bfloat16, 1), "f16": (torch.float16, 0)}
OUT = {"f32": (torch.float32, 0), "bf16": (torch.bfloat16, 1), "f16": (torch.float16, 2)}


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


def rows(n, width, dtype, pad=0):
    """Rows on 16-byte words, with `pad` further words behind each; what lies behind a row's end is NaN."""
    ld = -(-width // 8) * 8 + 8 * pad
    return torch.full((n, ld), math.nan, dtype=dtype, device=DEV)[:, :width]


def make(T, V, K, dtype, seed=0, masked=0.0, pad=0, spread=2.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    X, W = rows(T, K, dtype, pad), rows(V, K, dtype, pad)
    X.copy_(torch.randn(T, K, generator=gen, device=DEV))
    W.copy_(torch.randn(V, K, generator=gen, device=DEV) * (spread / math.sqrt(K)))
    y = torch.randint(0, V, (T,), generator=gen, device=DEV, dtype=torch.int32)
    if masked:
        off = torch.rand(T, generator=gen, device=DEV) < masked
        y[off] = torch.where(torch.arange(int(off.sum()), device=DEV) % 2 == 0, -100, V).to(torch.int32)
    return X, W, y


def forward(g, X, W, y, stream=None):
    T, K = X.shape
    V = W.shape[0]
    losses, lse = (torch.full((T,), math.nan, device=DEV) for _ in range(2))
    n = g.gemm_cross_entropy_workspace_size(T, V)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)
    g.gemm_cross_entropy(1 if X.dtype == torch.bfloat16 else 0, T, V, K, X, X.stride(0), W, W.stride(0), y, losses, lse, ws, n,
                         stream=stream)
    return losses, lse


def forward64(X, W, y):
    logits = X.double() @ W.double().t()
    live = (y >= 0) & (y < W.shape[0])
    lse = torch.logsumexp(logits, -1)
    losses = lse - logits.gather(1, y.long().clamp(0, W.shape[0] - 1)[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return torch.where(live, losses, zero), torch.where(live, lse, zero), logits, live


def status_ok(g):
    assert g.gemm_last_device_status()[0] == g.OK


FORWARD = [(1, 1, 1), (1, 1000, 64), (2, 257, 63), (8, 4096, 512), (33, 5000, 200), (77, 50001, 129), (128, 2048, 1024),
           (129, 2047, 72), (255, 513, 300), (256, 256, 128), (257, 8200, 65), (700, 3001, 1001), (1500, 12345, 96), (65, 131, 4096)]


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("T,V,K", FORWARD)
def test_losses(g, T, V, K, type):
    X, W, y = make(T, V, K, TYPES[type][0], seed=T + V, masked=0.2 if T > 4 else 0.0, pad=T % 2)
    losses, lse = forward(g, X, W, y)
    want, want_lse, logits, _ = forward64(X, W, y)
    tol = math.sqrt(K) * 2.0 ** -22 * float(logits.std(correction=0) + 1.0) + 2.0 ** -22 * (1.0 + want_lse.abs())
    assert bool(((lse - want_lse).abs() <= tol).all()), float((lse - want_lse).abs().max())
    assert bool(((losses - want).abs() <= 2 * tol).all()), float((losses - want).abs().max())
    status_ok(g)


def backward(g, X, W, y, lse, dl, dz, x_type="same", w_type="same", accumulate=None, columns=0, want="xw", stream=None):
    T, K = X.shape
    V = W.shape[0]
    own = "bf16" if X.dtype == torch.bfloat16 else "f16"
    xt, wt = (OUT[own if t == "same" else t] for t in (x_type, w_type))
    dX = rows(T, K, xt[0]) if "x" in want else None
    dW = rows(V, K, wt[0]) if "w" in want else None
    if accumulate is not None:
        dW.copy_(accumulate)
    n = g.gemm_cross_entropy_backward_workspace_size(T, V, K, columns)
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device=DEV)
    g.gemm_cross_entropy_backward(1 if own == "bf16" else 0, T, V, K, X, X.stride(0), W, W.stride(0), y, lse, dl, dz, dX, xt[1],
                                  dX.stride(0) if dX is not None else 0, dW, wt[1], dW.stride(0) if dW is not None else 0,
                                  int(accumulate is not None), ws, n, stream=stream)
    return dX, dW


def backward64(X, W, y, lse, dl, dz):
    """Gradients with, for each, its terms' absolute sums, the norm of all terms, and the sums of its values."""
    live = (y >= 0) & (y < W.shape[0])
    a = torch.where(live, dl.double(), 0.0)
    z = torch.where(live, dz.double(), 0.0) if dz is not None else torch.zeros_like(a)
    x, w = torch.where(live[:, None], X.double(), 0.0), W.double()
    p = torch.exp(x @ w.t() - lse.double()[:, None]) * (a + z)[:, None]
    p = torch.where(live[:, None], p, 0.0)
    p[torch.arange(len(y), device=DEV), y.long().clamp(0, W.shape[0] - 1)] -= a
    top = float((a.abs() + z.abs()).max())
    q = p.abs()
    return ((p @ w, q @ w.abs(), float((p.square() @ w.square()).sum().sqrt()), top * w.abs().sum(0)),
            (p.t() @ x, q.t() @ x.abs(), float((p.square().t() @ x.square()).sum().sqrt()), top * x.abs().sum(0)))


def near(got, want, dtype, old=None):
    want, size, norm, values = want
    u, v = torch.finfo(dtype).eps / 2, torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0  # half of the smallest fp16 number
    lost = 2.0 ** -39 * values if dtype == torch.float16 else 0.0 * values  # the same of a dl scaled to 2^14
    if old is not None:
        want, size = want + old.double(), size + old.double().abs()
    err = (got.double() - want).abs()
    assert bool((err <= (1.01 * u + 2.0 ** -18) * size + v * want.abs() + tiny + lost + 1e-36).all()), float(err.max())
    assert float(err.norm()) <= 2 * u * norm + 2.0 ** -18 * float(size.norm()) + v * float(want.norm()) + (tiny + float(lost.max())) * math.sqrt(err.numel()) + 1e-36


def check_backward(g, T, V, K, type, seed=0, masked=0.0, z=False, factor=1.0, x_type="same", w_type="same", columns=0, accumulate=False,
                   pad=0):
    X, W, y = make(T, V, K, TYPES[type][0], seed=seed, masked=masked, pad=pad)
    lse = forward64(X, W, y)[1].float()
    gen = torch.Generator(device=DEV).manual_seed(seed + 1)
    dl = (torch.rand(T, generator=gen, device=DEV) + 0.5) * factor
    dz = torch.randn(T, generator=gen, device=DEV) * 0.1 * factor if z else None
    old = None
    if accumulate:
        old = torch.randn(V, K, generator=gen, device=DEV) * factor
        old = old.to(TYPES[type][0] if w_type == "same" else OUT[w_type][0])
    dX, dW = backward(g, X, W, y, lse, dl, dz, x_type, w_type, old, columns)
    want_x, want_w = backward64(X, W, y, lse, dl, dz)
    near(dX, want_x, X.dtype)
    near(dW, want_w, X.dtype, old)
    status_ok(g)


BACKWARD = [(1, 1, 1), (1, 30001, 2048), (2, 5000, 4096), (1, 3000, 4097), (2, 1217, 1500), (3, 2000, 700), (1, 7, 4090), (1, 1000, 64), (2, 257, 63), (8, 4096, 512), (33, 5000, 200), (77, 20001, 129), (128, 2048, 1024), (129, 2047, 72),
            (256, 256, 128), (257, 8200, 65), (700, 3001, 1001), (1500, 12345, 96), (300, 40000, 256)]


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("T,V,K", BACKWARD)
def test_gradients(g, T, V, K, type):
    check_backward(g, T, V, K, type, seed=T + K, masked=0.3 if T > 4 else 0.0, z=T % 2 == 0, pad=T % 2)


@pytest.mark.parametrize("K", [128, 129, 192, 193, 256, 257, 320, 321, 384, 385, 449, 512, 513, 641])
@pytest.mark.parametrize("T", [20, 300])
def test_widths_of_the_last_tile(g, T, K):
    check_backward(g, T, 3500, K, "bf16", seed=K, masked=0.1, x_type="f32" if K % 2 else "same")


def test_three_products_whose_rounds_end_together(g):
    """A launch in which the second product's units are just as many as fill what the first left of its last round: every
    unit of the third is dealt out all the same."""
    check_backward(g, 3274, 84699, 424, "bf16", seed=9)


@pytest.mark.parametrize("x_type", OUT)
@pytest.mark.parametrize("w_type", OUT)
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_types(g, x_type, w_type, accumulate):
    check_backward(g, 300, 2500, 172, "bf16", seed=5, masked=0.1, x_type=x_type, w_type=w_type, accumulate=accumulate)
    check_backward(g, 60, 700, 333, "f16", seed=6, masked=0.1, x_type=x_type, w_type=w_type, accumulate=accumulate, z=True)
    check_backward(g, 2, 3001, 203, "bf16", seed=7, x_type=x_type, w_type=w_type, accumulate=accumulate, z=True)
    check_backward(g, 1, 900, 96, "f16", seed=8, x_type=x_type, w_type=w_type, accumulate=accumulate)


@pytest.mark.parametrize("columns", [256, 512, 1024, 4096])
@pytest.mark.parametrize("T", [40, 500])
def test_pieces_of_the_vocabulary(g, T, columns):
    """Pieces that end inside the vocabulary, the last one short: of one column, of less than a part of dX's sums."""
    check_backward(g, T, 4097, 520, "bf16", seed=7, masked=0.1, columns=columns)
    check_backward(g, T, 5000, 64, "f16", seed=8, columns=columns, w_type="f32", accumulate=True)


@pytest.mark.parametrize("factor", [1e-30, 1e-6, 1.0, 65536.0, 1e30])
@pytest.mark.parametrize("type", TYPES)
def test_any_scaling_of_the_loss(g, type, factor):
    """dl is divided by its largest factor before it is rounded: tiny and huge losses keep their digits."""
    check_backward(g, 50, 900, 96, type, seed=9, factor=factor, z=True, x_type="f32", w_type="f32")


@pytest.mark.parametrize("want", ["x", "w"])
@pytest.mark.parametrize("T", [1, 2, 270])
def test_one_gradient_alone(g, T, want):
    X, W, y = make(T, 3000, 136, torch.bfloat16, seed=10, masked=0.2)
    lse = forward64(X, W, y)[1].float()
    dl = torch.rand(T, device=DEV)
    both = backward(g, X, W, y, lse, dl, None)
    alone = backward(g, X, W, y, lse, dl, None, want=want)
    i = "xw".index(want)
    assert torch.equal(both[i], alone[i]) and alone[1 - i] is None


def test_rows_without_a_loss(g):
    """Padded rows may hold anything: they have no loss, no gradient and no part in the weights' gradient."""
    X, W, y = make(200, 1000, 120, torch.bfloat16, seed=11)
    y[::3] = -1
    y[1::7] = 1000
    dead = (y < 0) | (y >= 1000)
    X[dead] = math.nan
    X[5 * 3] = math.inf
    dl, dz = torch.rand(200, device=DEV), torch.rand(200, device=DEV)
    dl[dead], dz[dead] = math.nan, math.inf
    losses, lse = forward(g, X, W, y)
    assert bool((losses[dead] == 0).all()) and bool((lse[dead] == 0).all())
    dX, dW = backward(g, X, W, y, lse, dl, dz)
    assert bool((dX[dead] == 0).all())
    Xc, dl, dz = X.clone(), dl.clone(), dz.clone()
    Xc[dead], dl[dead], dz[dead] = 0.0, 0.0, 0.0
    want_x, want_w = backward64(Xc, W, y, lse, dl, dz)
    near(dX, want_x, X.dtype)
    near(dW, want_w, X.dtype)


@pytest.mark.parametrize("T", [1, 2])
def test_few_tokens_without_a_loss(g, T):
    X, W, y = make(T, 700, 264, torch.bfloat16, seed=12)
    y[0] = -1
    X[0] = math.nan
    lse = forward(g, X, W, y)[1]
    dl = torch.full((T,), 0.5, device=DEV)
    dl[0] = math.inf
    dX, dW = backward(g, X, W, y, lse, dl, None)
    assert not dX[0].any()
    X[0], dl[0] = 0.0, 0.0
    want_x, want_w = backward64(X, W, y, lse, dl, None)
    near(dX, want_x, X.dtype)
    near(dW, want_w, X.dtype)


def test_no_token_has_a_loss(g):
    X, W, y = make(130, 700, 64, torch.float16, seed=12)
    y.fill_(-100)
    X.fill_(math.nan)
    losses, lse = forward(g, X, W, y)
    assert not losses.any() and not lse.any()
    nan = torch.full((130,), math.nan, device=DEV)
    dX, dW = backward(g, X, W, y, lse, nan, nan)
    assert not dX.any() and not dW.any()
    old = torch.randn(700, 64, device=DEV).half()
    assert torch.equal(backward(g, X, W, y, lse, nan, None, accumulate=old)[1], old)


def test_no_tokens(g):
    W = torch.zeros(300, 64, dtype=torch.bfloat16, device=DEV)
    dW = torch.full((300, 72), 7.0, dtype=torch.bfloat16, device=DEV)
    g.gemm_cross_entropy(1, 0, 300, 64, None, 64, W, 64, None, None, None, None, 0)
    for accumulate, want in ((1, 7.0), (0, 0.0)):
        g.gemm_cross_entropy_backward(1, 0, 300, 64, None, 64, W, 64, None, None, None, None, None, 0, 64, dW, 1, 72, accumulate, None, 0)
        assert bool((dW[:, :64] == want).all()) and bool((dW[:, 64:] == 7.0).all())


def test_no_tokens_and_rows_of_more_than_32_bits_of_bytes(g):
    K = 2 ** 29 + 8
    dW = torch.full((1, K), 3.0, device=DEV)
    g.gemm_cross_entropy_backward(1, 0, 1, K, None, 0, None, 0, None, None, None, None, None, 0, 0, dW, 0, K, 0, None, 0)
    assert int(torch.count_nonzero(dW)) == 0


def test_columns_behind_the_rows_are_left_alone(g):
    X, W, y = make(70, 500, 100, torch.bfloat16, seed=13)
    lse = forward64(X, W, y)[1].float()
    dX, dW = backward(g, X, W, y, lse, torch.ones(70, device=DEV), None)
    assert bool(torch.as_strided(dX, (70, 4), (104, 1), 100).isnan().all())
    assert bool(torch.as_strided(dW, (500, 4), (104, 1), 100).isnan().all())


def test_large_logits_and_lone_words(g):
    """Logits of 300 and more, whose exponentials have no fp32 value, and losses near 0, which lse alone would round."""
    X = torch.zeros(6, 64, dtype=torch.bfloat16, device=DEV)
    W = torch.zeros(700, 64, dtype=torch.bfloat16, device=DEV)
    X[:, 0] = torch.tensor([300.0, -300.0, 96.0, 17.0, 1000.0, 0.0], device=DEV)
    W[5, 0] = 1.0
    y = torch.full((6,), 5, dtype=torch.int32, device=DEV)
    losses, lse = forward(g, X, W, y)
    want, want_lse, _, _ = forward64(X, W, y)
    assert bool(((lse - want_lse).abs() <= 2.0 ** -22 * want_lse.abs() + 1e-6).all())
    # the loss of a confident token keeps its digits: within 2^-22 of the sum of exponentials, which is 1 and a little
    assert bool(((losses - want).abs() <= 2.0 ** -22 * (1.0 + want)).all())


def test_infinite_and_missing_logits(g):
    X, W, y = make(4, 600, 64, torch.bfloat16, seed=14)
    X[0], X[2] = 0.0, 0.0
    X[0, 0], X[2, 0], X[3, 3] = math.inf, 1.0, math.nan
    W[:, 0] = -W[:, 0].abs() - 0.1
    W[400, 0] = 0.5  # +inf for token 0
    losses, lse = forward(g, X, W, y)
    assert float(lse[0]) == math.inf and bool(torch.isfinite(lse[1:3]).all()) and bool(lse[3].isnan()) and bool(losses[3].isnan())
    W[400, 0] = -0.5  # every logit of token 0 is -inf now
    losses, lse = forward(g, X, W, y)
    assert float(lse[0]) == -math.inf and bool(losses[0].isnan()) and bool(torch.isfinite(losses[1:3]).all())


def test_gradient_against_differences(g):
    """The backward pass is the forward pass's: (loss(x + h d) - loss(x - h d)) / 2h along a random direction.

    Inputs are fp16 numbers on a grid of 2^-6 and steps are of 2^-3 in a few places, so x + h d is exact; the losses' sum has a
    third derivative below |d|^3 sum p, and fp32 leaves 2^-20 of the losses over 2h.
    """
    T, V, K = 20, 300, 64
    gen = torch.Generator(device=DEV).manual_seed(15)
    grid = lambda *s: ((torch.randn(*s, generator=gen, device=DEV) * 16).round() / 64).half()  # noqa: E731
    X, W = grid(T, K), grid(V, K)
    y = torch.randint(0, V, (T,), generator=gen, device=DEV, dtype=torch.int32)
    lse = forward(g, X, W, y)[1]
    dX, dW = backward(g, X, W, y, lse, torch.ones(T, device=DEV), None, x_type="f32", w_type="f32")
    h = 2.0 ** -6
    for of, grad in ((X, dX), (W, dW)):
        d = torch.randint(-1, 2, of.shape, generator=gen, device=DEV).half()
        both = []
        for sign in (h, -h):
            a, b = (X + sign * d, W) if of is X else (X, W + sign * d)
            both.append(float(forward(g, a, b, y)[0].double().sum()))
        slope = float((grad.double() * d.double()).sum())
        # the change of a logit along d has a deviation of 0.25 sqrt(2 K / 3) = 1.6: its cube over six and h^2 bound the
        # difference's own error by 20 * 4^3 / 6 * h^2 = 0.05; dl's half steps add 2^-11 of the slope's terms
        assert abs((both[0] - both[1]) / (2 * h) - slope) <= 0.06 + 2.0 ** -9 * float((grad.double() * d.double()).abs().sum()) ** 0.5


def test_side_stream_and_graph(g):
    """Both calls on a stream of the caller's, captured, and replayed on other data."""
    T, V, K = 333, 5000, 128
    X, W, y = make(T, V, K, torch.bfloat16, seed=16, masked=0.1)
    losses, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    dX, dW = torch.empty(T, K, dtype=torch.bfloat16, device=DEV), torch.empty(V, K, dtype=torch.bfloat16, device=DEV)
    dl = torch.full((T,), 1.0 / T, device=DEV)
    n, m = g.gemm_cross_entropy_workspace_size(T, V), g.gemm_cross_entropy_backward_workspace_size(T, V, K, 1024)
    ws, back = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty(m, dtype=torch.uint8, device=DEV)

    def step():
        g.gemm_cross_entropy(1, T, V, K, X, K, W, K, y, losses, lse, ws, n)
        g.gemm_cross_entropy_backward(1, T, V, K, X, K, W, K, y, lse, dl, None, dX, 1, K, dW, 1, K, 0, back, m)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    eager = [t.clone() for t in (losses, lse, dX, dW)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    X2, W2, y2 = make(T, V, K, torch.bfloat16, seed=17, masked=0.3)
    for data in ((X2, W2, y2), (X.clone(), W.clone(), y.clone())):
        for t, new in zip((X, W, y), data):
            t.copy_(new)
        for t in (losses, lse, dX, dW):
            t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse, _, _ = forward64(X, W, y)
        assert bool(((lse - want_lse).abs() < 1e-4).all())
        want_x, want_w = backward64(X, W, y, lse, dl, None)
        near(dX, want_x, X.dtype)
        near(dW, want_w, X.dtype)
    assert all(torch.equal(a, b) for a, b in zip(eager, (losses, lse, dX, dW)))


def test_the_same_call_twice_gives_the_same_bits(g):
    X, W, y = make(777, 9000, 320, torch.float16, seed=18, masked=0.3)
    dl = torch.rand(777, device=DEV)
    a = forward(g, X, W, y)
    b = forward(g, X, W, y)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    p, q = (backward(g, X, W, y, a[1], dl, None) for _ in range(2))
    assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])


@pytest.mark.parametrize("role", [1, 2])
@pytest.mark.parametrize("T", [64, 300])
def test_waits_that_run_out_are_reported(g, T, role):
    """A role that waits on a barrier nothing arrives at: the call ends, says so, and the next one is right."""
    X, W, y = make(T, 3000, 128, torch.bfloat16, seed=19)
    forward(g, X, W, y)
    status_ok(g)
    g.gemm_debug_inject_timeout(20, role)
    forward(g, X, W, y)
    status, word = g.gemm_last_device_status()
    assert status == g.ERR_TIMEOUT and word & 0xFF in (1, 2, 3)
    losses, _ = forward(g, X, W, y)
    assert bool(((losses - forward64(X, W, y)[0]).abs() < 1e-4).all())
    status_ok(g)


@pytest.mark.parametrize("role", [1, 2])
@pytest.mark.parametrize("T,columns", [(64, 0), (300, 0), (300, 256)])
def test_waits_of_the_gradients_that_run_out_are_reported(g, T, columns, role):
    X, W, y = make(T, 2000, 128, torch.bfloat16, seed=20)
    lse = forward64(X, W, y)[1].float()
    dl = torch.ones(T, device=DEV)
    good = backward(g, X, W, y, lse, dl, None, columns=columns)
    status_ok(g)
    g.gemm_debug_inject_timeout(20, role)
    backward(g, X, W, y, lse, dl, None, columns=columns)
    status, word = g.gemm_last_device_status()
    assert status == g.ERR_TIMEOUT and word & 0xFF in (1, 2, 3)
    again = backward(g, X, W, y, lse, dl, None, columns=columns)
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])
    status_ok(g)


def test_two_calls_side_by_side(g):
    """Two streams, each with its own workspace: neither sees the other."""
    cases = [make(400, 6000, 192, torch.bfloat16, seed=s, masked=0.1) for s in (21, 22)]
    dl = torch.rand(400, device=DEV)
    want = []
    for X, W, y in cases:
        losses, lse = forward(g, X, W, y)
        want.append((losses, lse) + backward(g, X, W, y, lse, dl, None))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for (X, W, y), stream in zip(cases, streams):
        with torch.cuda.stream(stream):
            for _ in range(3):
                losses, lse = forward(g, X, W, y)
                out = (losses, lse) + backward(g, X, W, y, lse, dl, None)
            got.append(out)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, z) for x, z in zip(a, b))


def test_more_than_32_bits_of_weights_and_gradients(g):
    """A head of over 2^31 elements; sampled rows against float64."""
    T, V, K = 40, 262145, 8200
    X = torch.randn(T, K, device=DEV).bfloat16()
    W = torch.empty(V, K, dtype=torch.bfloat16, device=DEV)
    for a in range(0, V, 32768):
        W[a:a + 32768] = torch.randn(min(32768, V - a), K, device=DEV) * (1.5 / math.sqrt(K))
    y = torch.randint(V - 1000, V, (T,), device=DEV, dtype=torch.int32)
    losses, lse = forward(g, X, W, y)
    logits = torch.cat([X.double() @ W[a:a + 16384].double().t() for a in range(0, V, 16384)], 1)
    want_lse = torch.logsumexp(logits, -1)
    want = want_lse - logits.gather(1, y.long()[:, None])[:, 0]
    assert bool(((losses - want).abs() < 2e-5).all()) and bool(((lse - want_lse).abs() < 2e-5).all())
    dl = torch.ones(T, device=DEV)
    dX, dW = backward(g, X, W, y, lse, dl, None)
    p = torch.exp(logits - lse.double()[:, None])
    p[torch.arange(T, device=DEV), y.long()] -= 1.0
    rows = torch.cat([torch.tensor([0, 1, 131072, V - 1], device=DEV), y.long()[:8]])
    pick = p[:, rows]
    want_rows = (pick.t() @ X.double(), pick.abs().t() @ X.double().abs(), float((pick.square().t() @ X.double().square()).sum().sqrt()),
                 X.double().abs().sum(0))
    near(dW[rows], want_rows, X.dtype)
    wx = sum(p[:, a:a + 16384] @ W[a:a + 16384].double() for a in range(0, V, 16384))
    sx = sum(p[:, a:a + 16384].abs() @ W[a:a + 16384].double().abs() for a in range(0, V, 16384))
    nx = math.sqrt(sum(float((p[:, a:a + 16384].square() @ W[a:a + 16384].double().square()).sum()) for a in range(0, V, 16384)))
    near(dX, (wx, sx, nx, torch.zeros(K, dtype=torch.float64, device=DEV)), X.dtype)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("T,K", [(1, 4096), (2, 4096), (1, 5000), (2, 16384), (3, 4096), (64, 1500), (100, 8192), (300, 520), (300, 4096), (600, 16384)])
def test_confident_tokens(g, T, K, type):
    """Targets whose logits are 25 to 35 above the rest: dl is p - 1, some 1e-9, the rest of two values that nearly agree.

    Logits that are sums of products of one sign, where truncating additions move a sum the most. The gradients are compared
    with the true ones (64-bit normalisers). A target's dl may be off by what rounding leaves of lse: five half steps of fp32
    of about 35 (in the forward pass of the reference, its join with the logarithm of the sum, its return to base e and the
    constants' product, in the backward pass of lse times log2 e), and 2^-22 for the exponential. Without tiles (one or two tokens
    of K <= 4096) the logits' sums are others than the forward pass's, whose parts of 128 take eight truncations each of at
    most a step of 2^-23 of what has been summed, 4.5 parts' in all, and as much for what a step's products lose among
    themselves.
    """
    V = 2000
    dtype = TYPES[type][0]
    X, W, y = make(T, V, K, dtype, seed=T + K, spread=1.0)
    gen = torch.Generator(device=DEV).manual_seed(K)
    y.copy_(torch.randperm(V, generator=gen, device=DEV)[:T].int())
    x = X.double()
    top = 25.0 + 10.0 * torch.rand(T, 1, generator=gen, device=DEV)
    W[y.long()] = (x * (top / x.square().sum(1, keepdim=True))).to(dtype)
    losses, lse = forward(g, X, W, y)
    want, want_lse, logits, _ = forward64(X, W, y)
    dl = torch.ones(T, device=DEV)
    dX, dW = backward(g, X, W, y, lse, dl, None, x_type="f32", w_type="f32")
    status_ok(g)
    (want_x, size_x, _, values_x), (want_w, size_w, _, values_w) = backward64(X, W, y, want_lse, dl, None)
    off = 5 * 2.0 ** -24 * 36.0 + 2.0 ** -22
    if T <= 2 and K <= 4096:
        off += 2 * 4.5 * 2.0 ** -23 * 36.0
    at = y.long()
    slack_x, slack_w = off * W[at].double().abs(), torch.zeros_like(want_w)
    slack_w[at] = off * x.abs()
    u = torch.finfo(dtype).eps / 2
    lost = 2.0 ** -39 if dtype == torch.float16 else 0.0
    for got, ref, size, values, slack in ((dX, want_x, size_x, values_x, slack_x), (dW, want_w, size_w, values_w, slack_w)):
        err = (got.double() - ref).abs()
        bound = 1.01 * slack + (1.01 * u + 2.0 ** -18) * size + lost * values + 1e-36
        assert bool((err <= bound).all()), (float(err.max()), float((err / bound).max()))


@pytest.mark.parametrize("columns", [0, 512])
@pytest.mark.parametrize("T,V,K", [(20, 1217, 513), (90, 3000, 2001), (129, 2047, 640), (257, 700, 1100), (700, 4001, 1500), (40, 131, 8192)])
def test_gradients_of_long_rows(g, T, V, K, columns):
    """Rows whose sums are taken in parts, the last one short; tiles whose columns end anywhere; pieces of the vocabulary."""
    check_backward(g, T, V, K, "bf16", seed=T, masked=0.2, z=True, columns=columns, pad=1)
    check_backward(g, T, V, K, "f16", seed=T + 1, columns=columns, x_type="f32", w_type="f32", accumulate=True)


@pytest.mark.parametrize("role", [1, 2])
@pytest.mark.parametrize("T,columns", [(64, 0), (300, 0), (300, 256)])
def test_waits_of_long_rows_gradients_that_run_out_are_reported(g, T, columns, role):
    X, W, y = make(T, 2000, 1600, torch.bfloat16, seed=23)
    lse = forward64(X, W, y)[1].float()
    dl = torch.ones(T, device=DEV)
    good = backward(g, X, W, y, lse, dl, None, columns=columns)
    status_ok(g)
    g.gemm_debug_inject_timeout(20, role)
    backward(g, X, W, y, lse, dl, None, columns=columns)
    status, word = g.gemm_last_device_status()
    assert status == g.ERR_TIMEOUT and word & 0xFF in (1, 2, 3)
    again = backward(g, X, W, y, lse, dl, None, columns=columns)
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])
    status_ok(g)


def test_long_rows_on_a_side_stream_and_replayed(g):
    """Rows whose sums are taken in parts, in pieces of the vocabulary: captured, and replayed on other data."""
    T, V, K = 200, 3000, 1104
    X, W, y = make(T, V, K, torch.bfloat16, seed=24, masked=0.1)
    lse, dl = forward64(X, W, y)[1].float(), torch.full((T,), 1.0 / T, device=DEV)
    dX, dW = torch.empty(T, K, device=DEV), torch.empty(V, K, device=DEV)
    n = g.gemm_cross_entropy_backward_workspace_size(T, V, K, 1024)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def step():
        g.gemm_cross_entropy_backward(1, T, V, K, X, K, W, K, y, lse, dl, None, dX, 0, K, dW, 0, K, 0, ws, n)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    eager = [dX.clone(), dW.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = make(T, V, K, torch.bfloat16, seed=25, masked=0.3)
    for data in (other, (X.clone(), W.clone(), y.clone())):
        for t, new in zip((X, W, y), data):
            t.copy_(new)
        lse.copy_(forward64(X, W, y)[1].float())
        dX.fill_(math.nan)
        dW.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        want_x, want_w = backward64(X, W, y, lse, dl, None)
        near(dX, want_x, X.dtype)
        near(dW, want_w, X.dtype)
    assert torch.equal(dX, eager[0]) and torch.equal(dW, eager[1])
