"""Calls in a row whose launches overlap the end of the kernel before: each must see what that one wrote.

Every buffer that passes between two calls is filled with another value before each run, and the inputs change from
run to run, so that a read of what stood there before shows in the results, which are compared with references of
their own (whole numbers and 8-bit products exactly, sums to the roundings of their terms).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
REL = 4e-6  # a softmax weight in fp32: expf, its argument, a sum of k terms and a division


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


def quantised(x):
    """Rows by their fp32 scale (the product with the fp32 reciprocal of 127), quotients to even."""
    scale = x.abs().amax(-1) * torch.tensor(float(np.float32(1) / np.float32(127)), device=DEV)
    return torch.round(x / scale[:, None]), scale


@pytest.mark.parametrize("T,E,k", [(3000, 64, 4), (300, 16, 2), (16, 256, 8)])
def test_every_call_sees_the_one_before(g, T, E, k):
    gen = torch.Generator(device=DEV).manual_seed(T)
    N, R, few = 256, T * k, 4
    b = torch.randint(-20, 21, (E, N, N), generator=gen, device=DEV).to(torch.int8)
    sb = torch.rand(E, N, generator=gen, device=DEV) + 0.5
    one = torch.ones(N, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    ids, slots, tokens, off = torch.empty(T, k, **i32), torch.empty(T, k, **i32), torch.empty(R, **i32), torch.empty(E + 1, **i32)
    w, dw, s = torch.empty(T, k, device=DEV), torch.empty(T, k, device=DEV), torch.empty(R, device=DEV)
    q, y, dy = torch.empty(R, N, dtype=torch.int8, device=DEV), torch.empty(R, N, device=DEV), torch.empty(R, N, device=DEV)
    yf, D, dl = torch.empty(few, N, device=DEV), torch.empty(T, N, device=DEV), torch.empty(T, E, device=DEV)
    n = g.gemm_route_plan_workspace_size(T, E, k)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    rule = dict(score=0, renormalize=1)
    steps = (torch.arange(E, device=DEV) - E // 2) / 16.0
    for i in range(8):
        x = steps[torch.rand(T, E, generator=gen, device=DEV).argsort(-1)].float()  # distinct logits
        X = torch.randn(T, N, generator=gen, device=DEV)
        for t in (ids, w, off, slots, tokens, q, s, y, yf, D, dy, dw, dl, ws):
            t.fill_(i % 3)  # values that each of them could hold
        g.gemm_route(T, E, x, 0, E, None, k, rule, w, ids)
        g.gemm_route_plan(T, E, k, ids, off, slots, tokens, ws if n else None, n)
        g.gemm_quantize_int8(R, N, X, 0, T, N, tokens, g.QUANT_PLAIN, q, N, s)
        g.gemm_int8(few, N, N, q, N, s, b, N, one, yf, N, 0)
        g.gemm_int8_grouped(R, N, N, E, off, q, N, s, b, N, N * N, sb, y, N, 0)
        g.gemm_route_combine(T, N, k, y, 0, R, N, slots, w, D, 0, N)
        g.gemm_route_combine_backward(T, N, k, D, 0, N, y, 0, R, N, slots, w, dy, N, dw)
        g.gemm_route_backward(T, E, x, 0, E, k, rule, ids, dw, dl, E)
        st, word = g.gemm_last_device_status()
        assert st == g.OK, hex(word)

        want = x.argsort(-1, descending=True)[:, :k]
        assert torch.equal(ids.long(), want)
        w64 = torch.softmax(x.double().gather(1, want), -1)
        assert ((w.double() - w64).abs() <= REL * w64).all()
        order = want.flatten().sort(stable=True).indices
        at = torch.empty_like(order)
        at[order] = torch.arange(R, device=DEV)
        counts = torch.bincount(want.flatten(), minlength=E)
        assert torch.equal(off.long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)]))
        assert torch.equal(slots.long(), at.view(T, k)) and torch.equal(tokens.long(), order // k)
        q64, s64 = quantised(X[order // k])
        assert torch.equal(q.float(), q64) and torch.equal(s, s64)
        assert torch.equal(yf, (q64[:few].double() @ b[0].double().t()).float() * s64[:few, None])
        ends = off.tolist()
        for e in range(E):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                assert torch.equal(y[lo:hi], (q64[lo:hi].double() @ b[e].double().t()).float() * s64[lo:hi, None] * sb[e])
        terms = w64[..., None] * y[at.view(T, k)].double()
        assert ((D.double() - terms.sum(1)).abs() <= (REL + k * 2.0 ** -24) * terms.abs().sum(1) + 1e-30).all()
        rows = w.double()[..., None] * D.double()[:, None]
        assert ((dy[at.view(T, k)].double() - rows).abs() <= 2.0 ** -24 * rows.abs() + 1e-30).all()
        products = D.double()[:, None] * y[at.view(T, k)].double()
        dw64 = products.sum(-1)
        assert ((dw.double() - dw64).abs() <= (N / 32 + 16) * 2.0 ** -24 * products.abs().sum(-1)).all()
        d64 = torch.zeros(T, E, dtype=torch.float64, device=DEV)
        d64.scatter_(1, want, w64 * (dw.double() - (w64 * dw.double()).sum(-1, keepdim=True)))
        assert ((dl.double() - d64).abs() <= 4 * REL * dw.double().abs().amax(-1, keepdim=True) + 1e-30).all()
