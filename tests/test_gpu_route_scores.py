"""What gemm_route's choice goes by where scores are infinite, tiny or close, against float64.

Scores that the choice compares carry fp32 rounding: expf and one or two correctly rounded operations, 4 ulp in
all, and a sum with a bias half an ulp of its result. Choices are checked to be right within that.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ULP = 2.0 ** -23


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


def run(g, x, bias, k, r, dtype=torch.float32):
    x = torch.as_tensor(np.asarray(x, np.float64)).to(dtype)
    T, E = x.shape
    b = None if bias is None else torch.as_tensor(np.asarray(bias, np.float64)).float().to(DEV)
    w = torch.full((T, k), 5.0, device=DEV)
    ids = torch.full((T, k), -9, dtype=torch.int32, device=DEV)
    g.gemm_route(T, E, x.to(DEV), {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[dtype], E, b, k, r, w, ids)
    torch.cuda.synchronize()
    return w.double().cpu().numpy(), ids.cpu().numpy().astype(np.int64)


# ------------------------------------------------------------------ infinities


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinite_logit_with_a_bias(g, renorm, dtype):
    """Under softmax +inf makes the weights NaN; the experts chosen are still those with the largest s + bias."""
    x = np.tile(np.arange(8.0), (3, 1))
    x[1, 2] = x[2, 5] = np.inf
    x[2, 6] = -np.inf
    bias = np.array([0.0, 0.5, 0.0, 0.0, 0.25, 0.0, 0.0, 0.0])
    w, ids = run(g, x, bias, 3, dict(score=0, renormalize=renorm), dtype)
    assert np.isfinite(w[0]).all() and np.isnan(w[1]).all() and np.isnan(w[2]).all()
    assert (ids[1] == [2, 1, 4]).all() and (ids[2] == [5, 1, 4]).all()


@pytest.mark.parametrize("renorm", [0, 1])
def test_infinite_logits_in_groups(g, renorm):
    x = np.tile(np.arange(8.0), (2, 1))
    x[0, 1] = np.inf
    x[1, [0, 6]] = np.inf
    w, ids = run(g, x, None, 3, dict(score=0, renormalize=renorm, groups=4, group_top=1, groups_kept=2), torch.float32)
    assert np.isnan(w).all()
    assert (ids[0] == [1, 3, 2]).all()    # its own group, and of three whose scores are 0 the first
    assert (ids[1] == [0, 6, 7]).all()


# ------------------------------------------------------------------ tiny scores


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("bias", [None, 0.0])
def test_groups_of_tiny_scores_keep_their_order(g, score, bias):
    """Scores below 2^-126 are subnormal fp32 numbers, and still tell groups apart."""
    x = np.full((1, 12), -100.0)
    x[0, 0] = 0.0                                        # its group is kept in any case
    x[0, 3:6], x[0, 6:9], x[0, 9:12] = -95.0, -90.0, -97.0
    b = None if bias is None else np.full(12, bias)
    _, ids = run(g, x, b, 4, dict(score=score, groups=4, group_top=2, groups_kept=2), torch.float32)
    assert ids[0, 0] == 0 and set(ids[0, 1:]) == {6, 7, 8}


@pytest.mark.parametrize("score", [0, 1])
def test_tiny_scores_without_a_bias_of_their_own(g, score):
    x = np.array([[0.0, -95.0, -91.0, -97.0, -93.0]])
    _, ids = run(g, x, np.zeros(5), 4, dict(score=score), torch.float32)
    assert (ids == [[0, 2, 4, 1]]).all()


# ------------------------------------------------------------------ close scores


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups", [1, 8])
def test_choice_is_right_to_fp32_rounding(g, score, with_bias, groups):
    """Many tokens of close logits: no expert (or group) left out is better than one taken by more than the rounding."""
    if groups == 1 and not with_bias:
        pytest.skip("the choice goes by the logits")
    rng = np.random.default_rng(17)
    T, E, k, kept = 4000, 256, 8, 3
    x = (rng.standard_normal((T, 1)) + rng.standard_normal((T, E)) * 1e-3).astype(np.float32).astype(np.float64)
    bias = (rng.integers(-3, 4, E) / 1024.0) if with_bias else None
    _, ids = run(g, x, bias, k, dict(score=score, groups=groups, group_top=2 if groups > 1 else 1, groups_kept=kept if groups > 1 else 0), torch.float32)
    s = 1 / (1 + np.exp(-x)) if score else np.exp(x - x.max(-1, keepdims=True))
    if not score:
        s /= s.sum(-1, keepdims=True)
    v = s if bias is None else s + bias
    by = x.copy() if bias is None else v.copy()
    # a score to 4 ulp (the softmax's total, of 256 terms in 13 roundings, is common to a token), a sum to half of one of its own
    size = (4 + (0 if score else 13)) * ULP * s.max(-1) + (ULP / 2 * np.abs(v).max(-1) if with_bias else 0)
    if groups > 1:
        of = np.sort(v.reshape(T, groups, -1), -1)[..., -2:].sum(-1)
        live = np.zeros((T, groups), bool)
        np.put_along_axis(live, ids // (E // groups), True, 1)
        assert (live.sum(-1) <= kept).all()
        taken = np.where(live, of, np.inf).min(-1)
        # groups whose experts were taken are no worse than the kept-th best
        third = np.sort(of, -1)[:, -kept]
        assert (taken >= third - 2 * (2 * size + ULP * np.abs(of).max(-1))).all()
        full = live.sum(-1) == kept   # all kept groups show: the choice within them
        by = np.where(np.repeat(live, E // groups, 1), by, -np.inf)[full]
        ids, size = ids[full], size[full]
    got = np.take_along_axis(by, ids, 1)
    slack = 2 * size if bias is not None else 0 * size
    assert (np.diff(got, axis=1) <= slack[:, None]).all()
    rest = by.copy()
    np.put_along_axis(rest, ids, -np.inf, 1)
    assert (rest.max(-1) <= got[:, -1] + slack).all()
    assert all(len(set(row)) == k for row in ids.tolist())
