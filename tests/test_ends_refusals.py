"""What the calls at the ends of a training step refuse, before any CUDA call."""
import pytest


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


BAD, ALIGN, MORE = "ERR_INVALID_ARG", "ERR_ALIGNMENT", "ERR_UNSUPPORTED"
CALLS = {
    "gemm_cross_entropy": dict(in_type=1, T=40, V=1000, K=64, X=0x1000, ldx=64, W=0x2000, ldw=64, targets=0x3000, losses=0x4000,
                               lse=0x5000, workspace=0x6000, workspace_bytes=1 << 20),
    "gemm_cross_entropy_backward": dict(in_type=1, T=40, V=1000, K=64, X=0x1000, ldx=64, W=0x2000, ldw=64, targets=0x3000, lse=0x4000,
                                        dlosses=0x5000, dlse=0, dX=0x6000, dx_type=1, lddx=64, dW=0x7000, dw_type=1, lddw=64,
                                        accumulate=0, workspace=0x8000, workspace_bytes=1 << 26),
    "gemm_route_balance": dict(T=4000, E=64, logits=0x1000, l_type=0, ldl=64, k=6, route=None, ids=0x2000, S=3, offsets=0x3000,
                               counts=0x4000, tokens=0x5000, means=0x6000, losses=0x7000, workspace=0x8000, workspace_bytes=1 << 20),
    "gemm_route_balance_backward": dict(T=40, E=64, logits=0x1000, l_type=0, ldl=64, k=6, route=None, ids=0x2000, S=3, offsets=0x3000,
                                        counts=0x4000, tokens=0x5000, dlosses=0x6000, dlogits=0x7000, lddl=64, accumulate=0),
    "gemm_embed": dict(T=40, N=64, V=100, ids=0x1000, table=0x2000, t_type=1, ldt=64, scale=1.0, D=0x3000, d_type=0, ldd=64),
    "gemm_embed_backward": dict(T=40, N=64, V=100, ids=0x1000, dD=0x2000, d_type=1, lddd=64, scale=1.0, dtable=0x3000, t_type=0, lddt=64,
                                accumulate=0, workspace=0x4000, workspace_bytes=1 << 20),
}
NAN, INF = float("nan"), float("inf")
REFUSED = {
    "gemm_cross_entropy": [
        (dict(in_type=2), BAD), (dict(in_type=-1), BAD), (dict(T=-1), BAD), (dict(V=0), BAD), (dict(K=0), BAD), (dict(V=1 << 31), BAD),
        (dict(X=0), BAD), (dict(W=0), BAD), (dict(targets=0), BAD), (dict(ldx=56), BAD), (dict(ldw=63), BAD), (dict(ldx=1 << 40), BAD),
        (dict(losses=0), BAD), (dict(lse=0), BAD), (dict(workspace=0), BAD), (dict(workspace_bytes=100), BAD),
        (dict(X=0x1008), ALIGN), (dict(W=0x2002), ALIGN), (dict(ldx=66), ALIGN), (dict(ldw=68), ALIGN), (dict(targets=0x3002), ALIGN),
        (dict(losses=0x4001), ALIGN), (dict(lse=0x5002), ALIGN), (dict(workspace=0x6008), ALIGN),
        (dict(V=(1 << 31) - 1), MORE), (dict(T=(1 << 31) - 100), MORE), (dict(K=(1 << 31) - 100, ldx=1 << 31, ldw=1 << 31), MORE)],
    "gemm_cross_entropy_backward": [
        (dict(in_type=2), BAD), (dict(V=0), BAD), (dict(X=0), BAD), (dict(dX=0, dW=0), BAD), (dict(dx_type=3), BAD), (dict(dw_type=-1), BAD),
        (dict(lddx=56), BAD), (dict(lddw=56), BAD), (dict(lse=0), BAD), (dict(dlosses=0), BAD), (dict(workspace=0), BAD),
        (dict(dX=0x6008), ALIGN), (dict(dW=0x7004), ALIGN), (dict(lddx=68), ALIGN), (dict(lddw=68), ALIGN), (dict(lse=0x4001), ALIGN),
        (dict(dlosses=0x5002), ALIGN), (dict(dlse=0x5002), ALIGN), (dict(workspace=0x8080), ALIGN), (dict(lddx=66, dx_type=0), ALIGN)],
    "gemm_route_balance": [
        (dict(T=-1), BAD), (dict(E=0), BAD), (dict(E=1025, ldl=1025), BAD), (dict(k=0), BAD), (dict(k=33), BAD), (dict(E=5, k=6), BAD),
        (dict(l_type=3), BAD), (dict(logits=0), BAD), (dict(ids=0), BAD), (dict(ldl=63), BAD), (dict(route=dict(score=2)), BAD),
        (dict(S=-1), BAD), (dict(offsets=0), BAD), (dict(S=1 << 30), BAD), (dict(counts=0), BAD), (dict(tokens=0), BAD),
        (dict(means=0), BAD), (dict(losses=0), BAD), (dict(workspace=0), BAD), (dict(workspace_bytes=64), BAD),
        (dict(logits=0x1002), ALIGN), (dict(ids=0x2001), ALIGN), (dict(offsets=0x3002), ALIGN), (dict(counts=0x4001), ALIGN),
        (dict(means=0x6002), ALIGN), (dict(losses=0x7002), ALIGN), (dict(tokens=0x5001), ALIGN), (dict(workspace=0x8004), ALIGN)],
    "gemm_route_balance_backward": [
        (dict(E=0), BAD), (dict(k=0), BAD), (dict(counts=0), BAD), (dict(tokens=0), BAD), (dict(dlosses=0), BAD), (dict(dlogits=0), BAD),
        (dict(lddl=63), BAD), (dict(offsets=0), BAD), (dict(dlogits=0x7002), ALIGN), (dict(dlosses=0x6001), ALIGN),
        (dict(counts=0x4002), ALIGN)],
    "gemm_embed": [
        (dict(T=-1), BAD), (dict(N=-1), BAD), (dict(V=-1), BAD), (dict(ids=0), BAD), (dict(table=0), BAD), (dict(D=0), BAD), (dict(ldt=63), BAD),
        (dict(ldd=63), BAD), (dict(t_type=3), BAD), (dict(d_type=3), BAD), (dict(scale=NAN), BAD), (dict(scale=INF), BAD),
        (dict(ids=0x1002), ALIGN), (dict(table=0x2001), ALIGN), (dict(D=0x3002), ALIGN), (dict(V=(1 << 31) - 1), MORE),
        (dict(N=(1 << 31) - 1, ldt=1 << 31, ldd=1 << 31), MORE), (dict(T=1 << 30, N=1 << 20, ldt=1 << 20, ldd=1 << 20), MORE)],
    "gemm_embed_backward": [
        (dict(T=-1), BAD), (dict(ids=0), BAD), (dict(dD=0), BAD), (dict(dtable=0), BAD), (dict(lddd=63), BAD), (dict(lddt=63), BAD),
        (dict(t_type=9), BAD), (dict(scale=INF), BAD), (dict(workspace=0), BAD), (dict(workspace_bytes=100), BAD),
        (dict(dD=0x2001), ALIGN), (dict(dtable=0x3002), ALIGN), (dict(ids=0x1001), ALIGN), (dict(workspace=0x4010), ALIGN)],
}


@pytest.mark.parametrize("name,case,expect", [(n, c, e) for n, cases in REFUSED.items() for c, e in cases])
def test_refused(g, name, case, expect):
    with pytest.raises(g.GemmError) as err:
        getattr(g, name)(**{**CALLS[name], **case}, stream=0)
    assert err.value.status == getattr(g, expect)


@pytest.mark.parametrize("name,case", [
    ("gemm_cross_entropy", dict(T=0)), ("gemm_cross_entropy_backward", dict(T=0, dW=0)), ("gemm_cross_entropy_backward", dict(T=0, accumulate=1)),
    ("gemm_route_balance", dict(S=0)), ("gemm_route_balance_backward", dict(T=0)), ("gemm_route_balance_backward", dict(S=0)),
    ("gemm_embed", dict(T=0)), ("gemm_embed", dict(N=0)), ("gemm_embed_backward", dict(N=0)), ("gemm_embed_backward", dict(V=0)),
    ("gemm_embed_backward", dict(T=0, accumulate=1))])
def test_nothing_to_do(g, name, case):
    getattr(g, name)(**{**CALLS[name], **case}, stream=0)


def test_workspace_sizes(g):
    assert g.gemm_cross_entropy_workspace_size(0, 1000) == 0 and g.gemm_cross_entropy_workspace_size(40, -1) == 0
    assert g.gemm_cross_entropy_workspace_size(40, 1000) >= 40 * 8 * 8  # a partial softmax for each tile of 128 words, twice
    assert g.gemm_cross_entropy_backward_workspace_size(40, 0, 64) == 0
    assert g.gemm_route_balance_workspace_size(32, 64, 1) == 0  # one block's tokens need none
    assert g.gemm_route_balance_workspace_size(4000, 64, 3) >= 2 * 4 * 64 * 4
    assert g.gemm_route_balance_workspace_size(4000, 2000, 3) == 0
    assert g.gemm_embed_backward_workspace_size(40, 64, 100) >= 2 * 4 * 40
    assert g.gemm_embed_backward_workspace_size(40, 0, 100) == 0
