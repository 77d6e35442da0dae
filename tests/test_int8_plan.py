"""Planning of the 8-bit integer products, on the host (the library's own planner; no GPU)."""
import pytest

BLOCK = 128           # elements of K per stage
SLOWEST_US = 0.66     # a stage of a wide tile, the slowest measured


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


@pytest.mark.parametrize("M,N,E", [(16, 128, 1), (16, 128, 0), (64, 256, 0), (200, 20000, 0), (8192, 8192, 0), (70, 300, 1), (600, 300, 2)])
@pytest.mark.parametrize("K", [128, 4096, 1 << 20, 1 << 27, 1 << 30, (1 << 31) - 8193])
def test_a_wait_outlasts_a_tile(g, M, N, E, K):
    """The epilogue waits for a whole tile's K: with twice the slowest stage time it still ends in time."""
    p = g.gemm_debug_int8_plan(M, N, K, E)
    assert p["kind"] in (1, 2)
    blocks = -(-K // BLOCK)
    assert p["wait_ms"] * 1e3 >= 2 * SLOWEST_US * -(-blocks // p["shares"]) + 1e6
    if K <= 1 << 20:
        assert 2000 <= p["wait_ms"] <= 2100  # ordinary lengths give up as soon as before


@pytest.mark.parametrize("M,N,K,E,want", [
    (1, 4096, 4096, 0, (0, 1, 0, 0)), (8, 1024, 1024, 0, (0, 8, 0, 0)), (8, 4096, 4096, 0, (1, 16, 128, 4)),
    (1, 64, 1 << 17, 0, (1, 16, 128, 8)), (32, 300, 4096, 0, (1, 32, 128, 4)), (64, 300, 4096, 0, (1, 64, 128, 2)),
    (128, 20000, 2048, 0, (1, 128, 256, 1)), (200, 20000, 2048, 0, (2, 256, 256, 1)), (96, 4096, 2048, 64, (1, 16, 128, 1)),
    (8192, 4096, 2048, 64, (1, 128, 256, 1)), (32768, 4096, 2048, 64, (2, 256, 256, 1)), (32768, 128, 2048, 64, (1, 128, 256, 1))])
def test_tiles(g, M, N, K, E, want):
    p = g.gemm_debug_int8_plan(M, N, K, E)
    assert (p["kind"], p["tokens"], p["channels"], p["shares"]) == want


@pytest.mark.parametrize("change,status", [(dict(M=0), "ERR_INVALID_ARG"), (dict(N=-1), "ERR_INVALID_ARG"), (dict(K=0), "ERR_INVALID_ARG"),
                                           (dict(E=1025), "ERR_INVALID_ARG"), (dict(E=-1), "ERR_INVALID_ARG"), (dict(sms=0), "ERR_INVALID_ARG"),
                                           (dict(K=(1 << 31) - 1), "ERR_UNSUPPORTED")])
def test_refused(g, change, status):
    with pytest.raises(g.GemmError) as e:
        g.gemm_debug_int8_plan(**{**dict(M=16, N=128, K=128, E=0, sms=152), **change})
    assert e.value.status == getattr(g, status)
