"""The units of the cross entropy's launches, listed on the host by the code that deals them out and that the kernel's roles walk.

Every unit of each of a launch's up to three products is dealt to one cluster exactly once: the units are distinct places of a
grid, and their rows, columns and K, clipped to the product's, fill all of it. Each cluster takes the products in one order.
"""
import random

import numpy as np
import pytest


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


def units(g, *args, **kw):
    out = g.gemm_debug_cross_entropy_units(*args, **kw)
    return None if out is None else np.ctypeslib.as_array(out).reshape(-1, 8).astype(np.int64)


def covered(u, M, N, K):
    """Distinct first rows, columns and K, each inside the product, whose boxes have its volume."""
    first, size = u[:, 2::2], u[:, 3::2] - u[:, 2::2]
    inside = bool((first >= 0).all() and (size > 0).all() and (u[:, 3::2] <= np.array([M, N, K])).all())
    return inside and len(np.unique(first, axis=0)) == len(u) and sum(int(a) * int(b) * int(c) for a, b, c in size) == M * N * K


def check_launch(g, T, V, K, columns, sms, piece, want):
    plan = g.gemm_debug_cross_entropy_plan(T, V, K, columns, sms)
    if want and not plan["ctas"]:
        return 0
    u = units(g, T, V, K, columns, sms, piece, want)
    if u is None:
        return 0
    order = {}
    for c, product in u[:, :2].tolist():
        seen = order.setdefault(c, [])
        if not seen or seen[-1] != product:
            seen.append(product)
    assert all(len(set(s)) == len(s) for s in order.values())
    assert max(order) < max(1, sms // (1 if T <= 128 else 2))
    if want == 0:
        assert covered(u, T, V, K)
        return len(u)
    size = widths(g, T, V, K, columns, sms)
    cols = min(size, V - piece * size) if piece >= 0 else 0
    after = min(size, V - (piece + 1) * size)
    sizes = {0: (T, K, cols) if want & 1 and piece >= 0 else None, 1: (cols, K, T) if want & 2 and piece >= 0 else None,
             2: (T, after, K) if after > 0 else None}
    for product, box in sizes.items():
        of = u[u[:, 1] == product]
        assert covered(of, *box) if box else not len(of), (product, box)
    return len(u)


def widths(g, T, V, K, columns, sms):
    """Columns of a piece where the pieces have at most `columns`, from the launch of the first piece's dl."""
    u = units(g, T, V, K, columns, sms, -1, 3)
    return int(u[:, 5].max())


def shapes(seed, n):
    rng = random.Random(seed)
    log = lambda lo, hi: int(lo * (hi / lo) ** rng.random())  # noqa: E731
    for _ in range(n):
        yield log(1, 20000), log(1, 200000), log(1, 6000), rng.choice([0, 0, 256, 1024, 16384]), rng.choice([152, 152, 148, 132, 60, 7, 2, 1]), rng


@pytest.mark.parametrize("seed", range(12))
def test_every_unit_is_dealt_once(g, seed):
    launches = dealt = 0
    for T, V, K, columns, sms, rng in shapes(seed, 40):
        if T * V // 65536 * max(1, K // 256) > 400000:  # a list of so many units takes seconds
            continue
        dealt += check_launch(g, T, V, K, columns, sms, -1, 0)
        u = units(g, T, V, K, columns, sms, -1, 3)
        if u is None:
            continue
        pieces = -(-V // int(u[:, 5].max()))
        for piece in {-1, 0, pieces // 2, pieces - 2, pieces - 1}:
            if -1 <= piece < pieces:
                dealt += check_launch(g, T, V, K, columns, sms, piece, rng.choice([1, 2, 3, 3]))
                launches += 1
    assert launches > 30 and dealt > 1000


@pytest.mark.parametrize("sms", [152, 148, 144, 132])
@pytest.mark.parametrize("T,V,K", [(3274, 84699, 424), (4096, 32768, 4096), (777, 50001, 1001), (8192, 131072, 2048)])
def test_launches_of_three_products(g, T, V, K, sms):
    """The first left two tiles of dl to nobody on 76 clusters, where the second product's units were rounded up past what the
    first had left of its last round."""
    columns = 16384
    for piece in (-1, 0, 1, -(-V // widths(g, T, V, K, columns, sms)) - 1):
        for want in (1, 2, 3):
            check_launch(g, T, V, K, columns, sms, piece, want)
            check_launch(g, T, V, K, 0, sms, min(piece, 0), want)


def test_what_is_not_listed(g):
    assert g.gemm_debug_cross_entropy_units(1, 1000, 64, 0, 152, -1, 3) is None  # one token has no tiles backward
    assert g.gemm_debug_cross_entropy_units(1, 1000, 64, 0, 152, -1, 0) is not None
    for bad in (dict(T=0), dict(V=0), dict(K=0), dict(sms=0), dict(piece=-2), dict(piece=1), dict(want=4), dict(want=-1), dict(columns=-1)):
        assert g.gemm_debug_cross_entropy_units(**{**dict(T=300, V=1000, K=64, columns=0, sms=152, piece=0, want=3), **bad}) is None, bad
