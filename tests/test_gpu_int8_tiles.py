"""GPU parity of the 8-bit integer products on every tile shape, each test naming the one that it is for.

Partial sums stay below 2^24 in magnitude, so the fp32 sums are the exact integers and the expected value has
no tolerance: fp32 product with one scale, then with the other, then the rounding to the output type.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {0: torch.float32, 1: torch.bfloat16, 2: torch.float16}


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


def ok(g):
    st, word = g.gemm_last_device_status()
    assert st == g.OK, hex(word)


def test_a_tile_that_takes_longer_than_two_seconds(g):
    """One tile of 2^23 blocks of K, about 0.35 us each: waits for it last as long as it does."""
    K = 1 << 30
    a = torch.zeros(1, K, dtype=torch.int8, device=DEV)
    b = torch.ones(1, K, dtype=torch.int8, device=DEV)
    a[0, 0], a[0, K // 2], a[0, K - 1] = 3, -100, 5
    one = torch.ones(1, device=DEV)
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    D = torch.full((1, 1), 77.0, device=DEV)
    assert g.gemm_debug_int8_plan(1, 1, K, 1)["kind"] == 1
    g.gemm_int8_grouped(1, 1, K, 1, off, a, K, one, b, K, K, one, D, 1, 0)
    ok(g)
    assert float(D) == -92.0
