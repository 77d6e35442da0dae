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


def matrix(gen, rows, cols, ld, lim=127):
    """rows x cols of int8 in rows of ld, what lies past a row's end not zero."""
    return torch.randint(-lim - 1, lim + 1, (rows, ld), generator=gen, device=DEV, dtype=torch.int32).to(torch.int8)


def up16(n):
    return (n + 15) // 16 * 16


def limit(K):
    """Largest magnitude whose sums over K stay below 2^24."""
    return 127 if K <= 1000 else 63 if K <= 4000 else 30


def scaled(a, b, sa, sb, d_type):
    y = a.double() @ b.double().t()
    assert float(y.abs().max()) < 2 ** 24
    return (y.float() * sa[:, None] * sb).to(TYPES[d_type])


def plan(g, M, N, K, E=0):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    p = g.gemm_debug_int8_plan(M, N, K, E, sms)
    return p["kind"], p["tokens"], p["shares"]


WIDE, PAIR = (2, 256, 1), (1, 128, 1)
# whole and partial last tiles in both directions, one block of K, an odd number of blocks, a ragged last one
DENSE = [(WIDE, 512, 20224, 2048), (WIDE, 300, 20000, 2048), (WIDE, 300, 19999, 1000), (WIDE, 600, 40960, 128), (WIDE, 300, 20000, 384),
         (WIDE, 512, 40001, 200), (WIDE, 385, 20030, 65),
         (PAIR, 128, 20224, 2048), (PAIR, 128, 20000, 2048), (PAIR, 100, 19999, 1000), (PAIR, 128, 20000, 128), (PAIR, 90, 20016, 384),
         (PAIR, 65, 40001, 200)]


@pytest.mark.parametrize("tile,M,N,K", DENSE)
@pytest.mark.parametrize("d_type", [0, 1, 2])
@pytest.mark.parametrize("sectors", [True, False])
def test_pairs_of_ctas(g, tile, M, N, K, d_type, sectors):
    """Rows of D on 32-byte boundaries, whose sectors wide tiles store whole, and others."""
    assert plan(g, M, N, K) == tile
    gen = torch.Generator(device=DEV).manual_seed(M + N + K)
    lda, ldb = up16(K) + 16, up16(K)
    ldd = (N + 15) // 16 * 16 + (16 if sectors else 1)
    a, b = matrix(gen, M, K, lda, limit(K)), matrix(gen, N, K, ldb, limit(K))
    sa, sb = (torch.rand(n, generator=gen, device=DEV) * 0.01 + 0.001 for n in (M, N))
    D = torch.full((M + 1, ldd), 3.0, dtype=TYPES[d_type], device=DEV)
    g.gemm_int8(M, N, K, a, lda, sa, b, ldb, sb, D, ldd, d_type)
    ok(g)
    assert torch.equal(D[:M, :N], scaled(a[:, :K], b[:, :K], sa, sb, d_type))
    assert (D[M] == 3.0).all() and (D[:, N:] == 3.0).all()  # nothing outside


EXPERTS = [(WIDE, 1500, 520, 384, [0, 700, 700, 1490]), (WIDE, 1500, 300, 128, [0, 1, 900, 1500]), (WIDE, 1500, 512, 2048, [7, 300, 1200, 1500]),
           (WIDE, 6000, 4101, 200, [0, 2000, 2129, 6000]),
           (PAIR, 300, 520, 384, [0, 100, 100, 290]), (PAIR, 260, 300, 2000, [0, 1, 130, 260]), (PAIR, 384, 256, 128, [0, 128, 256, 384]),
           (PAIR, 1500, 128, 640, [0, 500, 1000, 1500])]


@pytest.mark.parametrize("tile,M,N,K,offsets", EXPERTS)
@pytest.mark.parametrize("d_type", [0, 1, 2])
@pytest.mark.parametrize("sectors", [True, False])
def test_experts_on_pairs_of_ctas(g, tile, M, N, K, offsets, d_type, sectors):
    assert plan(g, M, N, K, 3) == tile
    gen = torch.Generator(device=DEV).manual_seed(M + N + K)
    ld = up16(K)
    ldd = (N + 15) // 16 * 16 + (0 if sectors else 1)
    a, b = matrix(gen, M, K, ld, limit(K)), matrix(gen, 3 * N, K, ld, limit(K))
    sa, sb = (torch.rand(n, generator=gen, device=DEV) * 0.01 + 0.001 for n in (M, 3 * N))
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    D = torch.full((M, ldd), 3.0, dtype=TYPES[d_type], device=DEV)
    g.gemm_int8_grouped(M, N, K, 3, off, a, ld, sa, b, ld, N * ld, sb, D, ldd, d_type)
    ok(g)
    want = torch.full((M, ldd), 3.0, dtype=TYPES[d_type], device=DEV)
    for e in range(3):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            want[lo:hi, :N] = scaled(a[lo:hi, :K], b[e * N:(e + 1) * N, :K], sa[lo:hi], sb[e * N:(e + 1) * N], d_type)
    assert torch.equal(D, want)


INJECTED, SPLIT = 6, 13  # wait codes


@pytest.mark.parametrize("role,tile,M,N,K,wait", [
    *[(role, WIDE, 200, 20000, 2048, INJECTED) for role in (1, 2, 6)], *[(role, PAIR, 128, 20000, 2048, INJECTED) for role in (1, 2, 3, 6)],
    (6, (1, 16, 1), 16, 20000, 1024, INJECTED), (3, (1, 64, 1), 64, 20000, 1024, INJECTED),
    *[(3, (1, t, ks), t, 300, 4096, SPLIT) for t, ks in ((16, 8), (32, 4), (64, 2))], (6, (1, 32, 4), 32, 300, 4096, INJECTED),
    (1, (1, 16, 8), 16, 300, 4096, INJECTED), (2, (1, 64, 2), 64, 300, 4096, INJECTED)])
def test_waits_run_out_on_every_tile(g, role, tile, M, N, K, wait):
    """A role that waits in vain ends the launch, and the next launch is sound."""
    assert plan(g, M, N, K) == tile
    gen = torch.Generator(device=DEV).manual_seed(role)
    a, b = matrix(gen, M, K, K, limit(K)), matrix(gen, N, K, K, limit(K))
    one = torch.ones(M + N, device=DEV)
    D = torch.empty(M, N, device=DEV)
    g.gemm_debug_inject_timeout(30, role)
    g.gemm_int8(M, N, K, a, K, one, b, K, one, D, N, 0)
    st, word = g.gemm_last_device_status()
    assert st == g.ERR_TIMEOUT and word != 0  # of the injected role, or of one that waits for it
    if wait == SPLIT:
        assert (word & 255, word >> 8) == (role, SPLIT)
    g.gemm_int8(M, N, K, a, K, one, b, K, one, D, N, 0)
    ok(g)
    assert torch.equal(D, scaled(a, b, one[:M], one[:N], 0))


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
