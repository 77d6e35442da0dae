"""What gemm_route's choice goes by where scores are infinite."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


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
