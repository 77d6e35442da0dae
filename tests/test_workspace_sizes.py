"""Workspace sizes of the ends of a training step, on the host: a buffer made for the most tokens serves fewer."""
import random

import pytest


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


def counts_of_tokens(most, seed):
    """Every count up to 600, then each limit that a plan may have (powers of two, multiples of 128 and of 608) and its
    neighbours, and random ones."""
    rng = random.Random(seed)
    some = set(range(1, min(most, 600) + 1))
    for step in (128, 304, 608, 1024):
        some.update(t + d for t in range(step, min(most, 200 * step) + 1, step) for d in (-1, 0, 1))
    some.update((1 << i) + d for i in range(1, 32) for d in (-1, 0, 1))
    some.update(int(most ** rng.random()) for _ in range(2000))
    return sorted(t for t in some if 1 <= t <= most)


def never_falls(sizes):
    return all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("N,V", [(1024, 32768), (2048, 32768), (8, 100), (1, 5), (1025, 300000), (3001, 131072), (700000, 64), (20000000, 3),
                                 (96, 1 << 21), (640, 1)])
def test_table_gradient(g, N, V):
    sizes = [g.gemm_embed_backward_workspace_size(t, N, V) for t in counts_of_tokens(300000, N)]
    assert never_falls(sizes) and sizes[0] > 0


def test_table_gradient_takes_a_buffer_of_more_tokens(g):
    """19455 rows of 1024 are summed in chunks half as long as those of 20000."""
    room = g.gemm_embed_backward_workspace_size(20000, 1024, 32768)
    assert room >= 2 * 1216 * 1024 * 4 + 16 * 19455


HEADS = [(32768, 1024), (131072, 2048), (50001, 1001), (5000, 64), (300, 129), (256, 8200), (1, 1), (1000003, 4096), (1 << 28, 8), (131072, 5000)]


@pytest.mark.parametrize("sms", [152, 148, 1])
@pytest.mark.parametrize("columns", [0, 256, 16384])
@pytest.mark.parametrize("V,K", HEADS)
def test_heads_gradients(g, V, K, columns, sms):
    """More tokens never ask for less, and a call has room in what it asked for."""
    plans = [(t, g.gemm_debug_cross_entropy_plan(t, V, K, columns, sms)) for t in counts_of_tokens(300000, V + K)]
    assert never_falls([p["asked"] for _, p in plans])
    for t, p in plans[::7]:
        fit = g.gemm_debug_cross_entropy_plan(t, V, K, columns, sms, p["asked"])
        assert 0 < fit["used"] <= p["asked"]
        if fit["ctas"]:  # pieces at least as wide as was asked for
            wide = min(-(-V // 256) * 256, columns or V, max(256, (1 << 27) // t // 256 * 256))
            assert fit["pieces"] <= -(-V // wide)


@pytest.mark.parametrize("most", [3, 129, 257, 600, 5000])
@pytest.mark.parametrize("V,K", HEADS)
def test_heads_gradients_take_a_buffer_of_more_tokens(g, V, K, most):
    for columns in (0, 256, 4096):
        room = g.gemm_debug_cross_entropy_plan(most, V, K, columns)["asked"]
        for t in range(1, most + 1, 1 if most < 700 else 13):
            assert g.gemm_debug_cross_entropy_plan(t, V, K, columns, 152, room)["used"] <= room, t


@pytest.mark.parametrize("change", [dict(T=0), dict(V=0), dict(K=-1), dict(columns=-1), dict(sms=0), dict(V=(1 << 31) - 1)])
def test_no_plan_for_bad_arguments(g, change):
    with pytest.raises(g.GemmError) as e:
        g.gemm_debug_cross_entropy_plan(**{**dict(T=100, V=1000, K=64, columns=0, sms=152), **change})
    assert e.value.status == g.ERR_INVALID_ARG


@pytest.mark.parametrize("E", [1, 60, 256, 1024])
@pytest.mark.parametrize("S", [1, 2, 3, 16, 152, 700, 40000])
def test_balance_loss(g, E, S):
    sizes = [g.gemm_route_balance_workspace_size(t, E, S) for t in counts_of_tokens(300000, E + S)]
    assert never_falls(sizes)


@pytest.mark.parametrize("T", [1, 5, 32, 33, 600, 4864, 5017, 100000])
def test_balance_loss_of_fewer_sequences(g, T):
    assert never_falls([g.gemm_route_balance_workspace_size(T, 64, s) for s in range(1, 3000)])


@pytest.mark.parametrize("V", [1, 300, 131072])
def test_loss(g, V):
    assert never_falls([g.gemm_cross_entropy_workspace_size(t, V) for t in counts_of_tokens(300000, V)])


def test_loss_asks_for_what_tiles_may_need(g):
    """A reference and a sum for each token and tile, whatever the tiles' width on any number of SMs; no tile of more than 128
    tokens is narrower than 128 columns."""
    assert g.gemm_cross_entropy_workspace_size(8192, 131072) == 8192 * 1024 * 8
    rng = random.Random(5)
    for _ in range(400):
        T, V, K, sms = int(20000 ** rng.random()), int(200000 ** rng.random()), rng.choice([1, 64, 700]), rng.choice([1, 7, 132, 148, 152])
        if T * V > 1 << 28:
            continue
        units = g.gemm_debug_cross_entropy_units(T, V, K, 0, sms, -1, 0)
        tiles = len(set(units[4::8]))
        assert tiles * T * 8 <= g.gemm_cross_entropy_workspace_size(T, V)
