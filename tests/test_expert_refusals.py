"""What the expert-layer calls refuse, before any CUDA call."""
import pytest


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


BAD, ALIGN = "ERR_INVALID_ARG", "ERR_ALIGNMENT"
CALLS = {
    "gemm_route": dict(T=4, E=64, logits=0x1000, l_type=0, ldl=64, bias=0x2000, k=6, route=None, weights=0x3000, ids=0x4000),
    "gemm_route_backward": dict(T=4, E=64, logits=0x1000, l_type=0, ldl=64, k=6, route=None, ids=0x2000, dweights=0x3000,
                                dlogits=0x4000, lddl=64),
    "gemm_route_plan": dict(T=4000, E=64, k=6, ids=0x1000, offsets=0x2000, slots=0x3000, tokens=0x4000, workspace=0x5000,
                            workspace_bytes=1 << 20),
    "gemm_quantize_int8": dict(M=4, K=64, X=0x1000, x_type=1, x_rows=4, ldx=64, index=0, mode=0, Q=0x2000, ldq=64,
                               scales=0x3000),
    "gemm_int8": dict(M=4, N=64, K=64, A=0x1000, lda=64, scale_a=0x2000, B=0x3000, ldb=64, scale_b=0x4000, D=0x5000, ldd=64,
                      d_type=1),
    "gemm_int8_grouped": dict(M=4, N=64, K=64, E=2, offsets=0x6000, A=0x1000, lda=64, scale_a=0x2000, B=0x3000, ldb=64,
                              stride_b=4096, scale_b=0x4000, D=0x5000, ldd=64, d_type=1),
    "gemm_route_combine": dict(T=4, N=64, k=6, Y=0x1000, y_type=1, y_rows=24, ldy=64, slots=0x2000, weights=0x3000, D=0x4000,
                               d_type=1, ldd=64),
    "gemm_route_combine_backward": dict(T=4, N=64, k=6, dD=0x1000, d_type=1, lddd=64, Y=0x2000, y_type=1, y_rows=24, ldy=64,
                                        slots=0x3000, weights=0x4000, dY=0x5000, lddy=64, dweights=0x6000),
}
REFUSED = [
    ("gemm_route", dict(T=-1), BAD), ("gemm_route", dict(E=0), BAD), ("gemm_route", dict(E=1025, ldl=1025), BAD),
    ("gemm_route", dict(k=0), BAD), ("gemm_route", dict(k=33), BAD), ("gemm_route", dict(E=5, k=6), BAD),
    ("gemm_route", dict(ldl=63), BAD), ("gemm_route", dict(l_type=3), BAD), ("gemm_route", dict(logits=0), BAD),
    ("gemm_route", dict(weights=0), BAD), ("gemm_route", dict(ids=0), BAD), ("gemm_route", dict(logits=0x1002), ALIGN),
    ("gemm_route", dict(bias=0x2001), ALIGN), ("gemm_route", dict(ids=0x4002), ALIGN),
    ("gemm_route", dict(route=dict(score=2)), BAD), ("gemm_route", dict(route=dict(groups=7, groups_kept=1)), BAD),
    ("gemm_route", dict(route=dict(groups=64, groups_kept=64)), BAD), ("gemm_route", dict(route=dict(groups=8)), BAD),
    ("gemm_route", dict(route=dict(groups=8, groups_kept=9)), BAD), ("gemm_route", dict(route=dict(groups=-1)), BAD),
    ("gemm_route", dict(route=dict(groups=32, group_top=3, groups_kept=8)), BAD),
    ("gemm_route", dict(route=dict(groups=32, groups_kept=2)), BAD),  # 4 experts for 6 choices
    ("gemm_route", dict(route=dict(scale=float("nan"))), BAD),
    ("gemm_route_backward", dict(dlogits=0), BAD), ("gemm_route_backward", dict(lddl=63), BAD),
    ("gemm_route_backward", dict(ids=0), BAD), ("gemm_route_backward", dict(dweights=0), BAD),
    ("gemm_route_backward", dict(dlogits=0x4001), ALIGN), ("gemm_route_backward", dict(k=65), BAD),
    ("gemm_route_plan", dict(ids=0), BAD), ("gemm_route_plan", dict(offsets=0), BAD), ("gemm_route_plan", dict(slots=0), BAD),
    ("gemm_route_plan", dict(tokens=0), BAD), ("gemm_route_plan", dict(workspace=0), BAD),
    ("gemm_route_plan", dict(workspace_bytes=100), BAD), ("gemm_route_plan", dict(workspace=0x5001), ALIGN),
    ("gemm_route_plan", dict(T=1 << 30), BAD), ("gemm_route_plan", dict(E=2000), BAD), ("gemm_route_plan", dict(k=0), BAD),
    ("gemm_route_plan", dict(tokens=0x4002), ALIGN),
    ("gemm_quantize_int8", dict(M=-1), BAD), ("gemm_quantize_int8", dict(K=-1), BAD), ("gemm_quantize_int8", dict(x_rows=3), BAD),
    ("gemm_quantize_int8", dict(x_type=7), BAD), ("gemm_quantize_int8", dict(mode=2), BAD), ("gemm_quantize_int8", dict(ldx=63), BAD),
    ("gemm_quantize_int8", dict(ldq=63), BAD), ("gemm_quantize_int8", dict(mode=1), BAD),  # gated rows are 128 wide
    ("gemm_quantize_int8", dict(X=0), BAD), ("gemm_quantize_int8", dict(Q=0), BAD), ("gemm_quantize_int8", dict(scales=0), BAD),
    ("gemm_quantize_int8", dict(X=0x1001), ALIGN), ("gemm_quantize_int8", dict(scales=0x3002), ALIGN),
    ("gemm_quantize_int8", dict(index=0x7002), ALIGN),
    ("gemm_int8", dict(M=-1), BAD), ("gemm_int8", dict(N=1 << 31), BAD), ("gemm_int8", dict(lda=48), BAD),
    ("gemm_int8", dict(ldb=48), BAD), ("gemm_int8", dict(lda=72), ALIGN), ("gemm_int8", dict(ldb=72), ALIGN),
    ("gemm_int8", dict(A=0x1008), ALIGN), ("gemm_int8", dict(B=0x3001), ALIGN), ("gemm_int8", dict(D=0x5001), ALIGN),
    ("gemm_int8", dict(scale_a=0x2002), ALIGN), ("gemm_int8", dict(A=0), BAD), ("gemm_int8", dict(B=0), BAD),
    ("gemm_int8", dict(D=0), BAD), ("gemm_int8", dict(scale_a=0), BAD), ("gemm_int8", dict(scale_b=0), BAD),
    ("gemm_int8", dict(ldd=63), BAD), ("gemm_int8", dict(d_type=5), BAD),
    ("gemm_int8_grouped", dict(E=0), BAD), ("gemm_int8_grouped", dict(E=1025), BAD), ("gemm_int8_grouped", dict(offsets=0), BAD),
    ("gemm_int8_grouped", dict(offsets=0x6001), ALIGN), ("gemm_int8_grouped", dict(stride_b=4000), BAD),
    ("gemm_int8_grouped", dict(stride_b=4100), ALIGN), ("gemm_int8_grouped", dict(stride_b=-16), BAD),
    ("gemm_route_combine", dict(k=0), BAD), ("gemm_route_combine", dict(k=33), BAD), ("gemm_route_combine", dict(Y=0), BAD),
    ("gemm_route_combine", dict(slots=0), BAD), ("gemm_route_combine", dict(weights=0), BAD), ("gemm_route_combine", dict(D=0), BAD),
    ("gemm_route_combine", dict(ldy=63), BAD), ("gemm_route_combine", dict(ldd=63), BAD), ("gemm_route_combine", dict(y_type=3), BAD),
    ("gemm_route_combine", dict(Y=0x1001), ALIGN), ("gemm_route_combine", dict(slots=0x2002), ALIGN),
    ("gemm_route_combine_backward", dict(dD=0), BAD), ("gemm_route_combine_backward", dict(dY=0), BAD),
    ("gemm_route_combine_backward", dict(dweights=0), BAD), ("gemm_route_combine_backward", dict(lddd=63), BAD),
    ("gemm_route_combine_backward", dict(lddy=63), BAD), ("gemm_route_combine_backward", dict(d_type=-1), BAD),
    ("gemm_route_combine_backward", dict(dY=0x5001), ALIGN),
]


@pytest.mark.parametrize("name,change,status", REFUSED)
def test_refused(g, name, change, status):
    with pytest.raises(g.GemmError) as e:
        getattr(g, name)(**{**CALLS[name], **change}, stream=0)
    assert e.value.status == getattr(g, status)


def test_plan_workspace(g):
    assert g.gemm_route_plan_workspace_size(0, 64, 6) == 0
    assert g.gemm_route_plan_workspace_size(16, 64, 6) == 0
    n = g.gemm_route_plan_workspace_size(16384, 256, 8)
    assert 0 < n <= 128 * 256 * 4
    assert g.gemm_route_plan_workspace_size(16384, 2000, 8) == 0


def test_unknown_route_field(g):
    with pytest.raises(TypeError):
        g.gemm_route(**{**CALLS["gemm_route"], "route": dict(top=3)}, stream=0)


@pytest.mark.parametrize("change", [
    dict(N=1 << 28, ldd=1 << 28, ldb=1 << 36, stride_b=1 << 20),  # (N - 1) * ldb passes 64 bits
    dict(N=1 << 30, ldd=1 << 30, ldb=1 << 38, stride_b=1 << 38),
    dict(N=64, ldb=128, stride_b=63 * 128 + 48)])  # one unit short
def test_stride_between_experts_holds_a_matrix(g, change):
    with pytest.raises(g.GemmError) as e:
        g.gemm_int8_grouped(**{**CALLS["gemm_int8_grouped"], **change}, stream=0)
    assert e.value.status == g.ERR_INVALID_ARG


LONG = (1 << 31) - 256  # the step of a 32-bit counter past it would wrap


@pytest.mark.parametrize("name,change", [
    ("gemm_quantize_int8", dict(K=LONG, ldx=LONG, ldq=LONG)),
    ("gemm_quantize_int8", dict(K=LONG, ldx=2 * LONG, ldq=LONG, mode=1)),
    ("gemm_route_combine", dict(T=1, N=LONG, ldy=LONG, ldd=LONG)),
    ("gemm_route_combine_backward", dict(T=1, N=LONG, lddd=LONG, ldy=LONG, lddy=LONG)),
    ("gemm_int8", dict(M=LONG)), ("gemm_int8", dict(N=LONG, ldd=LONG)), ("gemm_int8", dict(K=LONG, lda=LONG, ldb=LONG)),
    ("gemm_int8", dict(N=LONG, ldd=LONG, K=0)),
    ("gemm_int8_grouped", dict(M=LONG)), ("gemm_int8_grouped", dict(E=1, N=LONG, ldd=LONG))])
def test_lengths_next_to_the_limit(g, name, change):
    with pytest.raises(g.GemmError) as e:
        getattr(g, name)(**{**CALLS[name], **change}, stream=0)
    assert e.value.status == g.ERR_UNSUPPORTED
