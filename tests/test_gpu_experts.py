"""GPU parity of the expert-layer operators around the products: routing and its
gradient, the order by expert, row quantisation, weighted sums and theirs.

The references are plain float64 (or integer) loops and numpy expressions.
Tolerances, derived: fp32 expf within 2 ulp of the exact exponential of an
argument that was rounded once (relative error |x| 2^-24, |x| <= 24 here:
1.5e-6), sums of at most 1024 positive terms taken as 32 lane sums and a tree
(at most 37 roundings: 2.3e-6), two divisions and a product (2e-7): 4e-6.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {0: torch.float32, 1: torch.bfloat16, 2: torch.float16}
HALF_ULP = {0: 2.0 ** -24, 1: 2.0 ** -8, 2: 2.0 ** -11}  # relative rounding of a result (bf16 and fp16 rounded up)
REL = 4e-6


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


def np64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ routing

def scores64(x, sigmoid):
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max(-1, keepdims=True)
        e = np.exp(x - np.where(top == -np.inf, 0.0, top))
        total = e.sum(-1, keepdims=True)
        return e / np.where(total == 0, 1.0, total)


def choice64(x, bias, r):
    """(scores, what the choice goes by with -inf where a group is not kept)."""
    s = scores64(x, r["score"])
    masked = ~(x > -np.inf)
    with_bias = np.where(masked, -np.inf, s + (0.0 if bias is None else bias))
    by = np.where(masked, -np.inf, x) if bias is None else with_bias
    G = r.get("groups", 1) or 1
    if G > 1:
        T, E = x.shape
        for t in range(T):
            values = []
            for gr in range(G):
                v = sorted((v for v in with_bias[t, gr * E // G:(gr + 1) * E // G] if v > -np.inf), reverse=True)
                values.append(sum(v[:r.get("group_top", 1) or 1]) if v else -np.inf)
            order = sorted(range(G), key=lambda i: (-values[i], i))
            for gr in order[r["groups_kept"]:]:
                by[t, gr * E // G:(gr + 1) * E // G] = -np.inf
    return s, by


def route64(x, bias, k, r):
    s, by = choice64(x, bias, r)
    T, E = x.shape
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        order = sorted((e for e in range(E) if by[t, e] > -np.inf), key=lambda e: (-by[t, e], e))[:k]
        ids[t, :len(order)] = order
        if not order:
            continue
        if r.get("renormalize"):
            if r["score"]:
                p = s[t, order]
                w[t, :len(order)] = p / (p.sum() if p.sum() else 1.0)
            else:
                e = np.exp(x[t, order] - x[t, order].max())
                w[t, :len(order)] = e / e.sum()
        else:
            w[t, :len(order)] = s[t, order]
    return w * (r.get("scale") or 1.0), ids


def run_route(g, x, bias, k, r, l_type, pad=0):
    T, E = x.shape
    buf = torch.full((T, E + pad), 7.0, device=DEV, dtype=TYPES[l_type])
    buf[:, :E] = torch.from_numpy(x).to(DEV).to(TYPES[l_type])
    b = None if bias is None else torch.from_numpy(bias).float().to(DEV)
    w = torch.full((T, k), 5.0, device=DEV)
    ids = torch.full((T, k), -9, dtype=torch.int32, device=DEV)
    g.gemm_route(T, E, buf, l_type, E + pad, b, k, r, w, ids)
    torch.cuda.synchronize()
    return np64(w), ids.cpu().numpy().astype(np.int64)


def distinct_logits(rng, T, E, l_type):
    """Logits without near ties: for each token a permutation of steps that every type holds exactly."""
    step = np.arange(E) - E // 2
    x = np.stack([rng.permutation(step) for _ in range(T)]).astype(np.float64)
    return x / (16.0 if E <= 256 else 64.0) if l_type != 1 or E <= 256 else x / 4.0


ROUTES = [
    (1, 1, 1, dict(score=0), 0, False),
    (5, 8, 2, dict(score=0, renormalize=1), 0, False),
    (7, 33, 6, dict(score=0, renormalize=1, scale=2.5), 1, False),
    (64, 64, 8, dict(score=1, renormalize=1, scale=-0.5), 2, False),
    (3, 100, 32, dict(score=1), 0, True),
    (33, 256, 8, dict(score=1, groups=8, group_top=2, groups_kept=4, renormalize=1, scale=2.5), 0, True),
    (9, 160, 6, dict(score=0, groups=8, group_top=1, groups_kept=3), 0, False),
    (6, 32, 3, dict(score=0, groups=32, group_top=1, groups_kept=5), 0, False),
    (4, 1024, 32, dict(score=0, groups=32, group_top=2, groups_kept=1, renormalize=1), 0, False),
    (5, 513, 5, dict(score=1, renormalize=0), 0, True),
    (2, 300, 1, dict(score=0), 0, True),
]


@pytest.mark.parametrize("T,E,k,r,l_type,with_bias", ROUTES)
@pytest.mark.parametrize("pad", [0, 3])
def test_route(g, T, E, k, r, l_type, with_bias, pad):
    rng = np.random.default_rng(E * 7 + T)
    x = distinct_logits(rng, T, E, l_type)
    bias = (rng.integers(-40, 41, E) / 512.0) if with_bias else None
    w, ids = run_route(g, x, bias, k, r, l_type, pad)
    s, by = choice64(x, bias, r)
    w64, ids64 = route64(x, bias, k, r)
    if with_bias:  # sums of a rounded score and a bias: any order within their rounding is right
        for t in range(T):
            got = by[t, ids[t]]
            assert (np.diff(got) <= 1e-6).all() and len(set(ids[t])) == k and (ids[t] >= 0).all()
            rest = np.delete(by[t], ids[t])
            assert not rest.size or rest.max() <= got.min() + 1e-6
        p = s[np.arange(T)[:, None], ids]
        if r.get("renormalize"):
            p = p / p.sum(-1, keepdims=True)
        w64 = p * (r.get("scale") or 1.0)
    else:
        assert (ids == ids64).all()
    np.testing.assert_allclose(w, w64, rtol=REL, atol=1e-30)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [0, 1])
def test_route_masked_experts_and_padded_tokens(g, score, renorm):
    r = dict(score=score, renormalize=renorm)
    rng = np.random.default_rng(5)
    x = distinct_logits(rng, 6, 40, 0)
    x[0] = -np.inf                       # nothing is left
    x[1, 3:] = -np.inf                   # three experts for four choices
    x[2, :] = -np.inf
    x[2, 39] = -50.0                     # one, with a tiny sigmoid
    x[3, 5] = np.finfo(np.float32).min   # the lowest finite value is an ordinary logit
    x[4, :20] = -np.inf
    w, ids = run_route(g, x, None, 4, r, 0)
    w64, ids64 = route64(x, None, 4, r)
    assert (ids == ids64).all()
    assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[1, 3] == -1) and ids[2, 0] == 39
    np.testing.assert_allclose(w, w64, rtol=REL, atol=1e-30)


def test_route_all_at_the_lowest_value(g):
    x = np.full((2, 16), float(np.finfo(np.float32).min))
    w, ids = run_route(g, x, None, 3, dict(score=0, renormalize=1), 0)
    assert (ids == [[0, 1, 2]] * 2).all()
    np.testing.assert_allclose(w, 1 / 3, rtol=REL)


def test_route_nan_and_infinity(g):
    x = np.tile(np.arange(8.0), (4, 1))
    x[1, 2] = np.nan
    x[2, 2] = np.inf
    w, ids = run_route(g, x, None, 3, dict(score=0, renormalize=1), 0)
    assert (ids[0] == [7, 6, 5]).all() and (ids[1] == [7, 6, 5]).all() and (ids[2] == [2, 7, 6]).all()
    assert np.isfinite(w[0]).all() and np.isnan(w[1]).all() and np.isnan(w[2]).all() and np.isfinite(w[3]).all()
    w, ids = run_route(g, x, None, 3, dict(score=1), 0)
    assert np.isnan(w[1]).all() and (ids[2] == [2, 7, 6]).all()
    np.testing.assert_allclose(w[2], [1.0, scores64(np.float64(7), 1), scores64(np.float64(6), 1)], rtol=REL)


def test_route_ties_go_to_the_lower_index(g):
    x = np.zeros((2, 70))
    x[0, [3, 40, 69]] = 1.0
    x[1, ::2] = -0.0                     # minus zero equals zero
    w, ids = run_route(g, x, None, 5, dict(score=0), 0)
    assert (ids[0] == [3, 40, 69, 0, 1]).all() and (ids[1] == [0, 1, 2, 3, 4]).all()
    w, ids = run_route(g, x, np.full(70, 0.25), 5, dict(score=1, groups=7, group_top=2, groups_kept=2), 0)
    assert (ids[1] == [0, 1, 2, 3, 4]).all()


def test_route_saturated_scores_keep_the_order_of_the_logits(g):
    x = np.array([[30.0, 40.0, 35.0, -200.0, -190.0]])  # sigmoids 1, 1, 1, 0, 0 in fp32
    w, ids = run_route(g, x, None, 5, dict(score=1, renormalize=1), 0)
    assert (ids == [[1, 2, 0, 4, 3]]).all()
    np.testing.assert_allclose(w, [[1 / 3, 1 / 3, 1 / 3, 0, 0]], rtol=REL)


def test_route_bias_that_forbids(g):
    x = np.tile(np.arange(6.0), (1, 1))
    b = np.array([0.0, 0, 0, 0, -np.inf, np.nan])
    w, ids = run_route(g, x, b, 4, dict(score=1), 0)
    assert (ids == [[3, 2, 1, 0]]).all()


def test_route_nothing(g):
    g.gemm_route(0, 8, None, 0, 8, None, 2, None, None, None)


# ------------------------------------------------------------------ gradient

def weights64(x, ids, r):
    s = scores64(x, r["score"])
    w = np.zeros(ids.shape)
    for t in range(x.shape[0]):
        at = [e for e in ids[t] if e >= 0]
        p = s[t, at]
        if r.get("renormalize"):
            p = p / (p.sum() if p.sum() else 1.0)
        w[t, np.nonzero(ids[t] >= 0)[0]] = p
    return w * (r.get("scale") or 1.0)


def route_grad64(x, ids, dw, r):
    s = scores64(x, r["score"])
    d = np.zeros_like(x)
    for t in range(x.shape[0]):
        j = np.nonzero(ids[t] >= 0)[0]
        at = ids[t, j]
        gw = dw[t, j] * (r.get("scale") or 1.0)
        ds = np.zeros(x.shape[1])
        if r.get("renormalize"):
            P = s[t, at].sum()
            P = P if P else 1.0
            gw = (gw - (gw * s[t, at]).sum() / P) / P
        ds[at] = gw
        d[t] = ds * s[t] * (1 - s[t]) if r["score"] else s[t] * (ds - (ds * s[t]).sum())
    return d


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("T,E,k,l_type,pad", [(1, 1, 1, 0, 0), (9, 40, 5, 0, 3), (17, 256, 8, 1, 0), (3, 1000, 32, 2, 1)])
def test_route_backward(g, score, renorm, T, E, k, l_type, pad):
    r = dict(score=score, renormalize=renorm, scale=1.5)
    rng = np.random.default_rng(T + E)
    x = distinct_logits(rng, T, E, l_type) / 8
    x = torch.from_numpy(x).to(TYPES[l_type])
    buf = torch.zeros(T, E + pad, dtype=TYPES[l_type], device=DEV)
    buf[:, :E] = x
    x = np64(x)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    if k > 2:
        ids[0, 1] = -1
        ids[T - 1, 2] = E + 3
    dw = rng.standard_normal((T, k)).astype(np.float32).astype(np.float64)
    out = torch.full((T, E + 2), 9.0, dtype=TYPES[l_type], device=DEV)
    g.gemm_route_backward(T, E, buf, l_type, E + pad, k, r, torch.from_numpy(ids.astype(np.int32)).to(DEV),
                          torch.from_numpy(dw).float().to(DEV), out, E + 2)
    got = np64(out)
    assert (got[:, E:] == 9.0).all()
    valid = np.where((ids >= 0) & (ids < E), ids, -1)
    ref = route_grad64(x, valid, dw, r)
    # the parts of each difference carry REL of the largest part
    size = 1.5 * np.abs(dw).max() * max(scores64(x, score).max(), 1.0 if renorm else 0.0)
    np.testing.assert_allclose(got[:, :E], ref, rtol=REL + HALF_ULP[l_type], atol=4 * REL * size + 2.0 ** -25)
    # against differences of the weights in 64 bits (step 1e-4: their error is below 1e-7 of the weights' scale)
    if T <= 9:
        h = 1e-4
        for t, e in {(0, int(valid[0, 0])), (T - 1, E - 1), (T // 2, int(max(valid[T // 2, 0], 0)))}:
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            diff = ((weights64(up, valid, r) - weights64(down, valid, r)) * dw)[t].sum() / (2 * h)
            assert abs(got[t, e] - diff) <= 1e-6 * size * k + 4 * REL * size + HALF_ULP[l_type] * abs(diff)


def test_route_backward_of_masked_rows(g):
    x = torch.full((3, 20), -math.inf, device=DEV)
    x[1, :3] = torch.tensor([0.5, 1.0, -1.0])
    x[2] = torch.linspace(-200, 200, 20)
    for score in (0, 1):
        for renorm in (0, 1):
            ids = torch.tensor([[-1, -1], [1, 0], [19, 0]], dtype=torch.int32, device=DEV)
            dw = torch.tensor([[3.0, 1.0], [1.0, -2.0], [1.0, 1.0]], device=DEV)
            out = torch.full((3, 20), 9.0, device=DEV)
            r = dict(score=score, renormalize=renorm)
            g.gemm_route_backward(3, 20, x, 0, 20, 2, r, ids, dw, out, 20)
            got = np64(out)
            assert (got[0] == 0).all() and np.isfinite(got).all() and (got[1, 3:] == 0).all()
            ref = route_grad64(np64(x[1:]), ids[1:].cpu().numpy(), np64(dw[1:]), r)
            np.testing.assert_allclose(got[1:], ref, rtol=REL, atol=8 * REL)


# ------------------------------------------------------------------ order by expert

def plan_ref(ids, E):
    flat = ids.reshape(-1)
    k = ids.shape[1]
    order = [p for e in range(E) for p in np.nonzero(flat == e)[0]]
    counts = np.array([(flat == e).sum() for e in range(E)])
    offsets = np.concatenate([[0], np.cumsum(counts)])
    slots = np.full(flat.size, -1)
    slots[order] = np.arange(len(order))
    tokens = np.full(flat.size, -1)
    tokens[:len(order)] = np.array(order, dtype=np.int64) // k if order else []
    return offsets, slots.reshape(ids.shape), tokens


def run_plan(g, ids, E):
    T, k = ids.shape
    dev = torch.from_numpy(ids.astype(np.int32)).to(DEV)
    offsets = torch.full((E + 2,), -7, dtype=torch.int32, device=DEV)
    slots = torch.full((T * k + 1,), -7, dtype=torch.int32, device=DEV)
    tokens = torch.full((T * k + 1,), -7, dtype=torch.int32, device=DEV)
    n = g.gemm_route_plan_workspace_size(T, E, k)
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device=DEV) if n else None
    g.gemm_route_plan(T, E, k, dev, offsets, slots, tokens, ws, n)
    o, s, t = (v.cpu().numpy() for v in (offsets, slots, tokens))
    assert o[-1] == s[-1] == t[-1] == -7  # nothing past the ends
    return o[:-1], s[:-1].reshape(T, k), t[:-1]


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 6), (16, 256, 8), (127, 5, 3), (128, 64, 8), (1025, 1, 1), (1000, 1024, 2),
                                   (5000, 60, 4), (20000, 256, 8)])
def test_plan(g, T, E, k):
    rng = np.random.default_rng(T + E + k)
    ids = rng.integers(0, E, (T, k))
    ids[rng.random((T, k)) < 0.1] = -1
    ids[rng.random((T, k)) < 0.02] = E
    ids[rng.random((T, k)) < 0.02] = -2147483648
    got = run_plan(g, ids, E)
    for a, b in zip(got, plan_ref(ids, E)):
        assert (a == b).all()


@pytest.mark.parametrize("T", [50, 4000])
def test_plan_extremes(g, T):
    for ids in (np.full((T, 2), -1), np.full((T, 2), 6), np.tile([0, 6], (T, 1))):
        for a, b in zip(run_plan(g, ids, 7), plan_ref(ids, 7)):
            assert (a == b).all()


def test_plan_nothing(g):
    offsets = torch.full((5,), -7, dtype=torch.int32, device=DEV)
    g.gemm_route_plan(0, 4, 2, None, offsets, None, None, None, 0)
    assert (offsets == 0).all()


# ------------------------------------------------------------------ quantisation

def quant_ref(x):
    """In the operator's own arithmetic: the scale by the fp32 reciprocal of 127, fp32 quotients, ties to even."""
    x = x.astype(np.float32)
    top = np.abs(x).max(-1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
    scale = (top * (np.float32(1) / np.float32(127))).astype(np.float32)
    by = np.where(scale == 0, np.float32(1), scale)[:, None]
    return np.clip(np.rint(x / by), -127, 127).astype(np.int8), scale


@pytest.mark.parametrize("x_type", [0, 1, 2])
@pytest.mark.parametrize("M,K,pad,ldq", [(1, 1, 0, 1), (3, 16, 0, 16), (5, 100, 4, 112), (2, 2048, 0, 2048), (4, 4096, 8, 4112),
                                         (2, 4101, 0, 4101), (2, 8192, 0, 8192), (1, 16384, 0, 16384), (2, 20000, 0, 20000),
                                         (3, 1000, 1, 1003)])
def test_quantize(g, x_type, M, K, pad, ldq):
    rng = np.random.default_rng(M + K)
    x = torch.from_numpy(rng.standard_normal((M, K + pad)) * np.exp(rng.uniform(-3, 3, (M, 1)))).to(TYPES[x_type])
    x[0, K // 2] = 0
    dev = x.to(DEV)
    q = torch.full((M, ldq), 99, dtype=torch.int8, device=DEV)
    s = torch.full((M,), -1.0, device=DEV)
    g.gemm_quantize_int8(M, K, dev, x_type, M, K + pad, None, g.QUANT_PLAIN, q, ldq, s)
    ref_q, ref_s = quant_ref(x[:, :K].float().numpy())
    assert (q[:, :K].cpu().numpy() == ref_q).all() and (s.cpu().numpy() == ref_s).all()
    assert (q[:, K:] == 99).all()


def test_quantize_index_and_odd_rows(g):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((6, 64))).float()
    x[1] = 0
    x[2, 5] = math.nan
    x[3, 7] = -math.inf
    x[4] = 1e-44                          # the scale rounds to 0
    index = np.array([5, 0, -1, 6, 1, 2, 3, 4, 5, 2147483647], np.int32)
    q = torch.full((10, 64), 99, dtype=torch.int8, device=DEV)
    s = torch.full((10,), -1.0, device=DEV)
    g.gemm_quantize_int8(10, 64, x.to(DEV), 0, 6, 64, torch.from_numpy(index).to(DEV), g.QUANT_PLAIN, q, 64, s)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    ref_q, ref_s = quant_ref(x[[5, 0]].numpy())
    assert (q[:2] == ref_q).all() and (s[:2] == ref_s).all() and (q[8] == ref_q[0]).all()
    for zero in (2, 3, 4, 7, 9):
        assert (q[zero] == 0).all() and s[zero] == 0
    assert np.isnan(s[5]) and np.isnan(s[6]) and (q[5] == 0).all() and (q[6] == 0).all()


@pytest.mark.parametrize("x_type,K", [(0, 64), (1, 2048), (0, 2048), (2, 33), (0, 10000)])
def test_quantize_gated(g, x_type, K):
    """silu(gate) * up in fp32 carries about 4e-7: a quotient that near a half may go either way."""
    rng = np.random.default_rng(K)
    M = 5
    x = torch.from_numpy(rng.standard_normal((M, 2 * K)) * 3).to(TYPES[x_type])
    x[0, 0] = -80.0
    q = torch.empty((M, K), dtype=torch.int8, device=DEV)
    s = torch.empty((M,), device=DEV)
    g.gemm_quantize_int8(M, K, x.to(DEV), x_type, M, 2 * K, None, g.QUANT_GATED, q, K, s)
    v = np64(x)
    v = v[:, :K] / (1 + np.exp(-v[:, :K])) * v[:, K:]
    scale = np.abs(v).max(-1) / 127
    np.testing.assert_allclose(np64(s), scale, rtol=1e-6)
    quotient = v / scale[:, None]
    assert np.abs(q.cpu().numpy() - quotient).max() <= 0.5 + 127 * 2e-6


@pytest.mark.parametrize("M", [1023, 1024, 1031, 2049])
@pytest.mark.parametrize("K", [8, 33, 256, 300, 512, 700, 1024, 1100])
def test_quantize_many_short_rows(g, M, K):
    """Numbers of rows that are no multiple of a block's, through an index with rows that do not exist."""
    rng = np.random.default_rng(M + K)
    x = torch.from_numpy(rng.standard_normal((M, K)) * np.exp(rng.uniform(-3, 3, (M, 1)))).float()
    index = rng.permutation(M).astype(np.int32)
    index[::7] = -1
    index[M - 1] = 5
    q = torch.full((M + 9, K), 99, dtype=torch.int8, device=DEV)
    s = torch.full((M + 9,), -1.0, device=DEV)
    g.gemm_quantize_int8(M, K, x.to(DEV), 0, M, K, torch.from_numpy(index).to(DEV), g.QUANT_PLAIN, q, K, s)
    ref_q, ref_s = quant_ref(x.numpy()[np.maximum(index, 0)])
    ref_q[index < 0], ref_s[index < 0] = 0, 0
    assert (q[:M].cpu().numpy() == ref_q).all() and (s[:M].cpu().numpy() == ref_s).all()
    assert (q[M:] == 99).all() and (s[M:] == -1).all()


@pytest.mark.parametrize("x_type", [0, 1])
@pytest.mark.parametrize("K", [1, 7, 8, 9, 23, 31, 256, 261, 4097, 9001])
@pytest.mark.parametrize("gated", [False, True])
def test_quantize_at_every_address(g, x_type, K, gated):
    """Rows at every distance from a 16-byte boundary, between NaN that belong to no row."""
    rng = np.random.default_rng(K)
    per = 16 // TYPES[x_type].itemsize
    W = 2 * K if gated else K
    mode = g.QUANT_GATED if gated else g.QUANT_PLAIN
    for first in range(per):
        ld, M = W + 1, 3
        x = torch.from_numpy(rng.standard_normal((M, W))).to(TYPES[x_type])
        store = torch.full((per + M * ld + 8,), math.nan, dtype=TYPES[x_type])
        store[first: first + M * ld].view(M, ld)[:, :W] = x
        dev = store.to(DEV)
        q = torch.full((first + M * (K + 3) + 8,), 99, dtype=torch.int8, device=DEV)
        s = torch.empty(M, device=DEV)
        g.gemm_quantize_int8(M, K, dev[first:], x_type, M, ld, None, mode, q[first:], K + 3, s)
        got = q[first: first + M * (K + 3)].view(M, K + 3).cpu().numpy()
        assert (got[:, K:] == 99).all() and (q[:first] == 99).all() and (q[first + M * (K + 3):] == 99).all()
        if gated:                # the same values at aligned addresses
            want = torch.empty(M, (K + 15) // 16 * 16, dtype=torch.int8, device=DEV)
            t = torch.empty(M, device=DEV)
            for m in range(M):
                g.gemm_quantize_int8(1, K, x[m: m + 1].to(DEV), x_type, 1, W, None, mode, want[m], want.stride(0), t[m:])
            v = np64(x)
            v = v[:, :K] / (1 + np.exp(-v[:, :K])) * v[:, K:]
            np.testing.assert_allclose(np64(s), np.abs(v).max(-1) / 127, rtol=1e-6)
            assert (got[:, :K] == want.cpu().numpy()[:, :K]).all() and (s == t).all()
        else:
            ref_q, ref_s = quant_ref(x.float().numpy())
            assert (got[:, :K] == ref_q).all() and (s.cpu().numpy() == ref_s).all()


def test_quantize_nothing(g):
    s = torch.full((3,), -1.0, device=DEV)
    g.gemm_quantize_int8(3, 0, None, 0, 3, 0, None, g.QUANT_PLAIN, None, 0, s)
    assert (s == 0).all()
    g.gemm_quantize_int8(0, 16, None, 0, 0, 16, None, g.QUANT_PLAIN, None, 16, None)


# ------------------------------------------------------------------ weighted sums

@pytest.mark.parametrize("y_type,d_type", [(0, 0), (1, 1), (2, 2), (0, 1), (1, 0)])
@pytest.mark.parametrize("T,N,k,pad", [(1, 1, 1, 0), (3, 64, 2, 0), (5, 1000, 6, 8), (4, 1025, 8, 3), (2, 4096, 32, 0)])
def test_combine_and_backward(g, y_type, d_type, T, N, k, pad):
    rng = np.random.default_rng(T + N + k)
    R = T * k
    slots = rng.permutation(R).reshape(T, k)
    if T > 1:
        slots[0, 0] = -1
        slots[T - 1, :] = [R + 5] + [-1] * (k - 1)
    used = [int(s) for s in slots.reshape(-1) if 0 <= s < R]
    y = torch.from_numpy(rng.standard_normal((R, N + pad))).to(TYPES[y_type])
    for r in set(range(R)) - set(used):  # rows that nothing names may hold anything
        y[r] = math.nan
    w = rng.standard_normal((T, k)).astype(np.float32)
    if T > 1:
        w[0, 0] = np.nan                 # and so may their weights
    yd, wd = y.to(DEV), torch.from_numpy(w).to(DEV)
    sd = torch.from_numpy(slots.astype(np.int32)).to(DEV)
    D = torch.full((T, N + 2), 9.0, dtype=TYPES[d_type], device=DEV)
    g.gemm_route_combine(T, N, k, yd, y_type, R, N + pad, sd, wd, D, d_type, N + 2)
    y64 = np64(y)[:, :N]
    ref, size = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j in range(k):
            if 0 <= slots[t, j] < R:
                ref[t] += w[t, j].astype(np.float64) * y64[slots[t, j]]
                size[t] += abs(w[t, j].astype(np.float64)) * np.abs(y64[slots[t, j]])
    got = np64(D)
    assert (got[:, N:] == 9.0).all()
    # k fused multiply-adds in fp32, then one rounding
    assert (np.abs(got[:, :N] - ref) <= k * 2.0 ** -24 * size + HALF_ULP[d_type] * np.abs(ref) + 2.0 ** -25).all()

    dD = torch.from_numpy(rng.standard_normal((T, N + 1))).to(TYPES[d_type])
    dY = torch.full((R, N + pad), 8.0, dtype=TYPES[y_type], device=DEV)
    dw = torch.full((T, k), 7.0, device=DEV)
    g.gemm_route_combine_backward(T, N, k, dD.to(DEV), d_type, N + 1, yd, y_type, R, N + pad, sd, wd, dY, N + pad, dw)
    dY, dw, d64 = np64(dY), np64(dw), np64(dD)[:, :N]
    for t in range(T):
        for j in range(k):
            r = slots[t, j]
            if not 0 <= r < R:
                assert dw[t, j] == 0
                continue
            ref = w[t, j].astype(np.float64) * d64[t]
            assert (np.abs(dY[r, :N] - ref) <= (HALF_ULP[y_type] + 2.0 ** -24) * np.abs(ref) + 2.0 ** -25).all()
            # a lane sums at most N / 32 + 8 products, a tree joins the lanes
            bound = (N / 32 + 16) * 2.0 ** -24 * (np.abs(d64[t]) * np.abs(y64[r])).sum()
            assert abs(dw[t, j] - (d64[t] * y64[r]).sum()) <= bound + 1e-30
    untouched = sorted(set(range(R)) - set(used))
    assert (dY[untouched] == 8.0).all() and (dY[:, N:] == 8.0).all()


@pytest.mark.parametrize("y_type,d_type", [(0, 0), (1, 1), (0, 1), (2, 0)])
@pytest.mark.parametrize("N", [1, 8, 23, 255, 264, 523, 1024, 1030, 2041])
def test_combine_at_every_address(g, y_type, d_type, N):
    """Rows of every operand at every distance from a 16-byte boundary, between NaN that belong to no row."""
    rng = np.random.default_rng(N)
    T, k, R = 3, 2, 6
    slots = torch.tensor([[5, 0], [2, 1], [3, 4]], dtype=torch.int32, device=DEV)
    w = torch.from_numpy(rng.standard_normal((T, k))).float()
    wd = w.to(DEV)

    def put(rows, dtype, first, ld):
        store = torch.full((first + rows * ld + 8,), math.nan, dtype=dtype, device=DEV)
        return store, store[first: first + rows * ld].view(rows, ld)

    for first in range(8):
        y_store, y = put(R, TYPES[y_type], first, N + 1)
        y[:, :N] = torch.from_numpy(rng.standard_normal((R, N))).to(DEV)
        d_store, D = put(T, TYPES[d_type], (3 * first) % 8, N + 3)
        g.gemm_route_combine(T, N, k, y, y_type, R, N + 1, slots, wd, D, d_type, N + 3)
        y64, w64, sl = np64(y)[:, :N], np64(w), slots.cpu().numpy()
        terms = w64[:, :, None] * y64[sl]
        ref, size = terms.sum(1), np.abs(terms).sum(1)
        assert (np.abs(np64(D)[:, :N] - ref) <= k * 2.0 ** -24 * size + HALF_ULP[d_type] * np.abs(ref) + 2.0 ** -25).all()
        assert int(torch.isnan(d_store).sum()) == d_store.numel() - T * N

        _, dD = put(T, TYPES[d_type], (5 * first + 1) % 8, N + 2)
        dD[:, :N] = torch.from_numpy(rng.standard_normal((T, N))).to(DEV)
        g_store, dY = put(R, TYPES[y_type], (first + 3) % 8, N + 5)
        dw = torch.full((T, k), 7.0, device=DEV)
        g.gemm_route_combine_backward(T, N, k, dD, d_type, N + 2, y, y_type, R, N + 1, slots, wd, dY, N + 5, dw)
        d64 = np64(dD)[:, :N]
        ref = w64[:, :, None] * d64[:, None]
        got = np64(dY)[:, :N][sl]
        assert (np.abs(got - ref) <= (HALF_ULP[y_type] + 2.0 ** -24) * np.abs(ref) + 2.0 ** -25).all()
        assert int(torch.isnan(g_store).sum()) == g_store.numel() - R * N
        products = d64[:, None] * y64[sl]
        assert (np.abs(np64(dw) - products.sum(-1)) <= (N / 32 + 16) * 2.0 ** -24 * np.abs(products).sum(-1) + 1e-30).all()


@pytest.mark.parametrize("y_type,d_type", [(1, 1), (0, 1), (0, 0)])
@pytest.mark.parametrize("T,k,N", [(512, 2, 300), (205, 5, 1024), (341, 3, 1024), (205, 5, 1023), (512, 8, 1030), (4097, 1, 1030),
                                   (241, 17, 2048), (7, 3, 256), (7, 3, 257), (7, 3, 520)])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_combine_backward_of_few_and_many_pairs(g, y_type, d_type, T, k, N, pad):
    """A row's columns walked by one warp and by several, at the numbers of pairs and columns where that changes."""
    rng = np.random.default_rng(T + N)
    R = T * k
    slots = rng.permutation(R).reshape(T, k)
    slots[T // 2, 0] = -1
    y = torch.from_numpy(rng.standard_normal((R, N + pad))).to(TYPES[y_type])
    dD = torch.from_numpy(rng.standard_normal((T, N + pad))).to(TYPES[d_type])
    w = rng.standard_normal((T, k)).astype(np.float32)
    dY = torch.full((R, N + pad), 8.0, dtype=TYPES[y_type], device=DEV)
    dw = torch.full((T, k), 7.0, device=DEV)
    g.gemm_route_combine_backward(T, N, k, dD.to(DEV), d_type, N + pad, y.to(DEV), y_type, R, N + pad,
                                  torch.from_numpy(slots.astype(np.int32)).to(DEV), torch.from_numpy(w).to(DEV), dY, N + pad, dw)
    dY, dw, d64, y64 = np64(dY), np64(dw), np64(dD)[:, :N], np64(y)[:, :N]
    assert (dY[:, N:] == 8.0).all() and dw[T // 2, 0] == 0
    left = (set(range(R)) - set(int(r) for r in slots.reshape(-1))).pop()
    assert (dY[left] == 8.0).all()
    for j in range(k):
        t = np.nonzero(slots[:, j] >= 0)[0]
        r = slots[t, j]
        ref = w[t, j].astype(np.float64)[:, None] * d64[t]
        assert (np.abs(dY[r, :N] - ref) <= (HALF_ULP[y_type] + 2.0 ** -24) * np.abs(ref) + 2.0 ** -25).all()
        products = d64[t] * y64[r]
        bound = (N / 32 + 16) * 2.0 ** -24 * np.abs(products).sum(-1) + 1e-30
        assert (np.abs(dw[t, j] - products.sum(-1)) <= bound).all()


def test_combine_backward_against_differences(g):
    """The sum is linear in the rows and in the weights: differences of the forward call are exact up to rounding."""
    rng = np.random.default_rng(8)
    T, N, k = 3, 24, 2
    y = torch.from_numpy(rng.standard_normal((6, N))).float().to(DEV)
    w = torch.from_numpy(rng.standard_normal((T, k))).float().to(DEV)
    slots = torch.tensor([[5, 0], [2, 1], [3, 4]], dtype=torch.int32, device=DEV)
    gD = torch.from_numpy(rng.standard_normal((T, N))).float().to(DEV)

    def loss(y, w):
        D = torch.empty(T, N, device=DEV)
        g.gemm_route_combine(T, N, k, y, 0, 6, N, slots, w, D, 0, N)
        return float((D.double() * gD.double()).sum())

    dY, dw = torch.zeros(6, N, device=DEV), torch.zeros(T, k, device=DEV)
    g.gemm_route_combine_backward(T, N, k, gD, 0, N, y, 0, 6, N, slots, w, dY, N, dw)
    h = 0.5
    tol = 200 * N * k * 2.0 ** -24 / h   # the roundings of two forward passes over the step
    for t, j in ((0, 0), (1, 1), (2, 0)):
        up, down = w.clone(), w.clone()
        up[t, j] += h
        down[t, j] -= h
        assert abs((loss(y, up) - loss(y, down)) / (2 * h) - float(dw[t, j])) <= tol
        r, c = int(slots[t, j]), 7 * j + 3
        up, down = y.clone(), y.clone()
        up[r, c] += h
        down[r, c] -= h
        assert abs((loss(up, w) - loss(down, w)) / (2 * h) - float(dY[r, c])) <= tol


def test_combine_past_two_to_the_31_elements(g):
    """Rows whose offset passes 2^31 elements."""
    N, R, k = 32768, 70000, 1
    y = torch.zeros(R, N, dtype=torch.bfloat16, device=DEV)
    y[R - 1] = torch.arange(N, device=DEV).remainder(256).to(torch.bfloat16)
    slots = torch.tensor([[R - 1], [0]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[2.0], [3.0]], device=DEV)
    D = torch.empty(2, N, device=DEV)
    g.gemm_route_combine(2, N, k, y, 1, R, N, slots, w, D, 0, N)
    assert (D[0] == 2.0 * y[R - 1].float()).all() and (D[1] == 0).all()
    q, s = torch.empty(1, N, dtype=torch.int8, device=DEV), torch.empty(1, device=DEV)
    g.gemm_quantize_int8(1, N, y, 1, R, N, slots[0], g.QUANT_PLAIN, q, N, s)
    ref_q, ref_s = quant_ref(y[R - 1:].float().cpu().numpy())
    assert (q.cpu().numpy() == ref_q).all() and float(s) == ref_s[0]


def test_routing_rows_past_two_to_the_31_elements(g):
    """Rows of logits, and of their gradient, whose offset passes 2^31 elements."""
    ld, E, k = 1 << 30, 40, 3
    buf = torch.empty(2 * ld + E, dtype=torch.bfloat16, device=DEV)
    x = np.stack([np.roll(np.arange(E), 7 * t) for t in range(3)]) / 8.0
    rows = buf.as_strided((3, E), (ld, 1))
    rows.copy_(torch.from_numpy(x))
    w, ids = torch.empty(3, k, device=DEV), torch.empty(3, k, dtype=torch.int32, device=DEV)
    r = dict(score=0, renormalize=1)
    g.gemm_route(3, E, buf, 1, ld, None, k, r, w, ids)
    w64, ids64 = route64(x, None, k, r)
    assert (ids.cpu().numpy() == ids64).all()
    np.testing.assert_allclose(np64(w), w64, rtol=REL)
    dw = torch.tensor([[1.0, -2.0, 0.5]] * 3, device=DEV)
    out = torch.empty_like(buf)
    g.gemm_route_backward(3, E, buf, 1, ld, k, r, ids, dw, out, ld)
    np.testing.assert_allclose(np64(out.as_strided((3, E), (ld, 1))), route_grad64(x, ids64, np64(dw), r), rtol=REL + HALF_ULP[1], atol=1e-6)


def test_combine_backward_past_two_to_the_31_elements(g):
    N, R = 32768, 70000
    y = torch.zeros(R, N, dtype=torch.bfloat16, device=DEV)
    dy = torch.zeros(R, N, dtype=torch.bfloat16, device=DEV)
    y[R - 1, :8] = 2.0
    dD = torch.ones(1, N, dtype=torch.bfloat16, device=DEV)
    slots = torch.tensor([[R - 1]], dtype=torch.int32, device=DEV)
    dw = torch.empty(1, 1, device=DEV)
    g.gemm_route_combine_backward(1, N, 1, dD, 1, N, y, 1, R, N, slots, torch.tensor([[0.5]], device=DEV), dy, N, dw)
    assert float(dw) == 16.0 and (dy[R - 1] == 0.5).all() and (dy[:4] == 0).all()


def test_kernels_in_a_row_see_each_other(g):
    """Each call reads what the one before it wrote; launches overlap the end of the kernel before."""
    rng = np.random.default_rng(21)
    T, E, k, N = 3000, 64, 4, 256
    x = torch.from_numpy(distinct_logits(rng, T, E, 0)).float().to(DEV)
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, device=DEV)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    slots, tokens = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T * k, dtype=torch.int32, device=DEV)
    n = g.gemm_route_plan_workspace_size(T, E, k)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    q, s = torch.empty(T * k, N, dtype=torch.int8, device=DEV), torch.empty(T * k, device=DEV)
    y, D = torch.empty(T * k, N, device=DEV), torch.empty(T, N, device=DEV)
    b = torch.from_numpy(rng.integers(-20, 21, (E, N, N)).astype(np.int8)).to(DEV)
    sb = torch.ones(E, N, device=DEV)
    X = torch.from_numpy(rng.standard_normal((T, N))).float().to(DEV)
    first = None
    for i in range(20):
        for t in (ids, w, off, slots, tokens, q, s, y, D):
            t.fill_(77)
        g.gemm_route(T, E, x, 0, E, None, k, dict(score=0, renormalize=1), w, ids)
        g.gemm_route_plan(T, E, k, ids, off, slots, tokens, ws, n)
        g.gemm_quantize_int8(T * k, N, X, 0, T, N, tokens, g.QUANT_PLAIN, q, N, s)
        g.gemm_int8_grouped(T * k, N, N, E, off, q, N, s, b, N, N * N, sb, y, N, 0)
        g.gemm_route_combine(T, N, k, y, 0, T * k, N, slots, w, D, 0, N)
        if first is None:
            first = D.clone()
            assert torch.isfinite(first).all() and (first != 77).any()
        assert torch.equal(D, first), i
    o, sl, tk = plan_ref(ids.cpu().numpy(), E)
    assert (off.cpu().numpy() == o).all() and (slots.cpu().numpy() == sl).all() and (tokens.cpu().numpy() == tk).all()
