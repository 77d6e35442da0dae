"""GPU parity of the 8-bit integer products, dense and over experts.

Where |partial sums| stay below 2^24 the fp32 sums are the exact integers, so
the expected value has no tolerance: fp32 product with one scale, then with
the other, then the rounding to the output type. Longer sums are compared
within the roundings of their accumulation.
"""
import numpy as np
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


def up16(n):
    return (n + 15) // 16 * 16


def int8_matrix(rng, rows, cols, ld, lo=-128, hi=127):
    """rows x cols of int8 in rows of ld, what lies past a row's end not zero."""
    m = rng.integers(lo, hi + 1, (rows, ld), dtype=np.int64).astype(np.int8)
    return m, torch.from_numpy(m).to(DEV)


def expected(a, b, sa, sb, d_type):
    y = a.astype(np.int64) @ b.astype(np.int64).T
    assert np.abs(y).max(initial=0) < 2 ** 24
    f = torch.from_numpy(y).float() * torch.from_numpy(sa)[:, None] * torch.from_numpy(sb)[None]
    return f.to(TYPES[d_type])


def ok(g):
    st, word = g.gemm_last_device_status()
    assert st == g.OK, hex(word)


SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 1024), (2, 100, 65), (3, 129, 16), (15, 64, 127), (16, 257, 129), (17, 130, 1000),
          (32, 128, 64), (33, 300, 500), (63, 1, 200), (64, 64, 64), (65, 513, 130), (127, 128, 256), (128, 256, 384),
          (129, 127, 72), (255, 200, 520), (256, 128, 128), (257, 1000, 1000), (300, 4096, 250), (777, 1029, 1000)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("d_type", [0, 1, 2])
def test_product(g, M, N, K, d_type):
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    lda, ldb, ldd = up16(K) + 16 * (M % 2), up16(K) + 32 * (N % 2), N + M % 3
    a, ad = int8_matrix(rng, M, K, lda)
    b, bd = int8_matrix(rng, N, K, ldb)
    sa, sb = (rng.uniform(0.001, 0.01, n).astype(np.float32) for n in (M, N))
    D = torch.full((M + 1, ldd), 3.0, dtype=TYPES[d_type], device=DEV)
    g.gemm_int8(M, N, K, ad, lda, torch.from_numpy(sa).to(DEV), bd, ldb, torch.from_numpy(sb).to(DEV), D, ldd, d_type)
    ok(g)
    got = D.cpu()
    assert torch.equal(got[:M, :N], expected(a[:, :K], b[:, :K], sa, sb, d_type))
    assert (got[M] == 3.0).all() and (got[:, N:] == 3.0).all()  # nothing outside


def test_product_large_tiles(g):
    """More tiles than SMs on every tile width, against integer products in float64 (exact below 2^53)."""
    rng = np.random.default_rng(2)
    for M, N, K in ((5000, 2500, 640), (2100, 9000, 200), (130, 40000, 128), (40, 40000, 256), (9, 30000, 512)):
        _, ad = int8_matrix(rng, M, K, up16(K))
        _, bd = int8_matrix(rng, N, K, up16(K))
        sa, sb = torch.rand(M, device=DEV), torch.rand(N, device=DEV)
        D = torch.empty(M, N, device=DEV)
        g.gemm_int8(M, N, K, ad, ad.stride(0), sa, bd, bd.stride(0), sb, D, N, 0)
        ok(g)
        y = (ad[:, :K].double() @ bd[:, :K].double().t()).float() * sa[:, None] * sb
        assert torch.equal(D, y)


@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 32, 64, 65, 128, 200, 600])
@pytest.mark.parametrize("N,K", [(1000, 4096), (20000, 2048), (40960, 1152)])
def test_long_rows_many_times(g, M, N, K):
    """Many stages and tiles a CTA on every tile shape, launched over and over: every result the same, and right."""
    rng = np.random.default_rng(M + N)
    _, ad = int8_matrix(rng, M, K, K, -30, 30)
    _, bd = int8_matrix(rng, N, K, K, -30, 30)
    sa, sb = torch.rand(M, device=DEV), torch.rand(N, device=DEV)
    y = (ad.double() @ bd.double().t()).float() * sa[:, None] * sb
    outs = [torch.empty(M, N, device=DEV) for _ in range(12)]
    for D in outs:
        g.gemm_int8(M, N, K, ad, K, sa, bd, K, sb, D, N, 0)
    ok(g)
    assert all(torch.equal(D, y) for D in outs)


@pytest.mark.parametrize("M,K", [(1, 1), (2, 17), (3, 500), (8, 4097), (5, 9000)])
def test_few_tokens_tail_is_not_read_past_its_end(g, M, K):
    """The last row of each operand ends with its allocation's last byte."""
    rng = np.random.default_rng(K)
    N = 30
    ld = up16(K) + 16
    a = rng.integers(-128, 128, (M - 1) * ld + K).astype(np.int8)
    b = rng.integers(-128, 128, (N - 1) * ld + K).astype(np.int8)
    full = [np.concatenate([v, np.zeros(ld - K, np.int8)]).reshape(-1, ld)[:, :K] for v in (a, b)]
    sa, sb = np.ones(M, np.float32), np.full(N, 0.5, np.float32)
    D = torch.empty(M, N, device=DEV)
    g.gemm_int8(M, N, K, torch.from_numpy(a).to(DEV), ld, torch.from_numpy(sa).to(DEV), torch.from_numpy(b).to(DEV), ld,
                torch.from_numpy(sb).to(DEV), D, N, 0)
    ok(g)
    assert torch.equal(D.cpu(), expected(full[0], full[1], sa, sb, 0))


def test_few_tokens_sums_are_exact_past_two_to_the_24(g):
    """Eight tokens and fewer are summed in integers: one rounding, to fp32."""
    M, N, K = 5, 100, 100000
    a = torch.full((M, up16(K)), 127, dtype=torch.int8, device=DEV)
    b = torch.full((N, up16(K)), 127, dtype=torch.int8, device=DEV)
    b[1] = -128
    one = torch.ones(N, device=DEV)
    D = torch.empty(M, N, device=DEV)
    g.gemm_int8(M, N, K, a, up16(K), one, b, up16(K), one, D, N, 0)
    ref = torch.full((N,), 127.0 * 127 * K, dtype=torch.float64)
    ref[1] = -128.0 * 127 * K
    assert torch.equal(D.cpu(), ref.float().expand(M, N))


@pytest.mark.parametrize("M,E", [(96, 64), (1500, 64), (4000, 64), (9000, 33)])
def test_experts_many_times(g, M, E):
    rng = np.random.default_rng(M)
    N, K = 512, 2048
    _, ad = int8_matrix(rng, M, K, K, -30, 30)
    _, bd = int8_matrix(rng, E * N, K, K, -30, 30)
    sa, sb = torch.rand(M, device=DEV), torch.rand(E, N, device=DEV)
    cut = np.concatenate([[0], np.sort(rng.integers(0, M + 1, E - 1)), [M]])
    y = torch.empty(M, N, device=DEV)
    for e in range(E):
        lo, hi = int(cut[e]), int(cut[e + 1])
        y[lo:hi] = (ad[lo:hi].double() @ bd[e * N:(e + 1) * N].double().t()).float() * sa[lo:hi, None] * sb[e]
    off = torch.from_numpy(cut.astype(np.int32)).to(DEV)
    outs = [torch.empty(M, N, device=DEV) for _ in range(12)]
    for D in outs:
        g.gemm_int8_grouped(M, N, K, E, off, ad, K, sa, bd, K, N * K, sb, D, N, 0)
    ok(g)
    assert all(torch.equal(D, y) for D in outs)


def test_sums_past_two_to_the_24(g):
    M, N, K = 40, 160, 16384
    rng = np.random.default_rng(4)
    a, ad = int8_matrix(rng, M, K, K, 60, 127)
    b, bd = int8_matrix(rng, N, K, K, 60, 127)
    one = torch.ones(max(M, N), device=DEV)
    D = torch.empty(M, N, device=DEV)
    g.gemm_int8(M, N, K, ad, K, one, bd, K, one, D, N, 0)
    ok(g)
    ref = a.astype(np.int64) @ b.astype(np.int64).T
    # one rounding (or truncation) for each 16 elements of K
    assert np.abs(D.double().cpu().numpy() - ref).max() <= (K / 16) * 2.0 ** -23 * ref.max()


def test_extreme_values(g):
    """-128 in both operands: 16384 a product, exact for K = 1000."""
    M, N, K = 20, 140, 1000
    a = np.full((M, up16(K)), -128, np.int8)
    b = np.full((N, up16(K)), -128, np.int8)
    b[::2] = 127
    sa, sb = np.ones(M, np.float32), np.full(N, 0.5, np.float32)
    D = torch.empty(M, N, device=DEV)
    g.gemm_int8(M, N, K, torch.from_numpy(a).to(DEV), up16(K), torch.from_numpy(sa).to(DEV), torch.from_numpy(b).to(DEV),
                up16(K), torch.from_numpy(sb).to(DEV), D, N, 0)
    ok(g)
    assert torch.equal(D.cpu(), expected(a[:, :K], b[:, :K], sa, sb, 0))


def test_scales_that_are_not_finite(g):
    """A NaN scale makes its row NaN and no other."""
    rng = np.random.default_rng(5)
    a, ad = int8_matrix(rng, 5, 32, 32)
    b, bd = int8_matrix(rng, 6, 32, 32)
    sa = torch.tensor([1.0, float("nan"), 1.0, 0.0, 1.0], device=DEV)
    D = torch.empty(5, 6, device=DEV)
    g.gemm_int8(5, 6, 32, ad, 32, sa, bd, 32, torch.ones(6, device=DEV), D, 6, 0)
    assert torch.isnan(D[1]).all() and torch.isfinite(D[[0, 2, 3, 4]]).all() and (D[3] == 0).all()


def test_no_elements_of_k(g):
    one = torch.ones(64, device=DEV)
    D = torch.full((5, 10), 3.0, device=DEV)
    g.gemm_int8(4, 9, 0, None, 0, one, None, 0, one, D, 10, 0)
    assert (D[:4, :9] == 0).all() and (D[4] == 3).all() and (D[:, 9] == 3).all()
    off = torch.tensor([1, 2, 3], dtype=torch.int32, device=DEV)
    D.fill_(3.0)
    g.gemm_int8_grouped(5, 9, 0, 2, off, None, 0, one, None, 0, 0, one, D, 10, 0)
    assert (D[1:3, :9] == 0).all() and (D[[0, 3, 4]] == 3).all()
    g.gemm_int8(0, 9, 16, None, 16, None, None, 16, None, None, 9, 0)
    g.gemm_int8(9, 0, 16, None, 16, None, None, 16, None, None, 0, 0)


# ------------------------------------------------------------------ experts

def run_grouped(g, M, N, K, E, offsets, seed, d_type=0, gap=0):
    rng = np.random.default_rng(seed)
    lda = ldb = up16(K)
    a, ad = int8_matrix(rng, M, K, lda)
    stride = N * ldb + gap
    b = rng.integers(-128, 128, E * stride).astype(np.int8)
    bd = torch.from_numpy(b).to(DEV)
    sa = rng.uniform(0.001, 0.01, M).astype(np.float32)
    sb = rng.uniform(0.001, 0.01, (E, N)).astype(np.float32)
    D = torch.full((M + 1, N + 1), 3.0, dtype=TYPES[d_type], device=DEV)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    g.gemm_int8_grouped(M, N, K, E, off, ad, lda, torch.from_numpy(sa).to(DEV), bd, ldb, stride,
                        torch.from_numpy(sb).to(DEV), D, N + 1, d_type)
    ok(g)
    got = D.cpu()
    clamped = np.maximum.accumulate(np.clip(offsets, 0, M))
    ref = torch.full((M + 1, N + 1), 3.0, dtype=TYPES[d_type])
    for e in range(E):
        lo, hi = clamped[e], clamped[e + 1]
        be = b[e * stride:e * stride + N * ldb].reshape(N, ldb)
        ref[lo:hi, :N] = expected(a[lo:hi, :K], be[:, :K], sa[lo:hi], sb[e], d_type)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("d_type", [0, 1, 2])
def test_experts(g, d_type):
    run_grouped(g, 96, 300, 200, 8, [0, 5, 5, 40, 41, 41, 41, 90, 96], 1, d_type, gap=48)
    run_grouped(g, 700, 129, 130, 3, [0, 1, 400, 690], 2, d_type)
    run_grouped(g, 1, 70, 16, 1, [0, 1], 3, d_type)


def test_experts_rows_and_gaps(g):
    run_grouped(g, 300, 64, 64, 4, [0, 0, 0, 300, 300], 4)      # one has all
    run_grouped(g, 50, 64, 64, 4, [0, 0, 0, 0, 0], 5)           # none has any
    run_grouped(g, 50, 64, 64, 3, [10, 20, 20, 30], 6)          # rows before the first and past the last
    rng = np.random.default_rng(7)
    for E, M in ((1024, 60), (65, 2000), (33, 5000)):
        cut = np.sort(rng.integers(0, M + 1, E - 1))
        run_grouped(g, M, 40, 48, E, [0, *cut.tolist(), M], 8)


def test_experts_offsets_are_clamped(g):
    run_grouped(g, 100, 64, 64, 4, [-5, 30, 20, 2147483647, 50], 9)
    run_grouped(g, 100, 64, 64, 3, [90, 10, -2147483648, 100], 10)


def test_experts_past_two_to_the_31_bytes(g):
    """The last expert's matrix and the last rows lie past 2^31 elements."""
    E, N, K, M = 36, 8192, 8192, 40
    B = torch.zeros(E, N, K, dtype=torch.int8, device=DEV)
    rng = np.random.default_rng(11)
    b, bd = int8_matrix(rng, N, K, K, -10, 10)
    B[E - 1] = bd
    a, ad = int8_matrix(rng, M, K, K, -10, 10)
    off = torch.tensor([0] * E + [M], dtype=torch.int32, device=DEV)
    sb = torch.ones(E, N, device=DEV)
    D = torch.empty(M, N, device=DEV)
    g.gemm_int8_grouped(M, N, K, E, off, ad, K, torch.ones(M, device=DEV), B, K, N * K, sb, D, N, 0)
    ok(g)
    assert torch.equal(D, (ad.double() @ bd.double().t()).float())
    del B
    M, N, K = 70000, 32768, 16
    a, ad = int8_matrix(rng, M, K, K)
    b, bd = int8_matrix(rng, N, K, K)
    D = torch.empty(M, N, dtype=torch.float16, device=DEV)
    g.gemm_int8(M, N, K, ad, K, torch.full((M,), 0.01, device=DEV), bd, K, torch.ones(N, device=DEV), D, N, 2)
    ok(g)
    for rows in (slice(0, 64), slice(M - 64, M)):
        assert torch.equal(D[rows], ((ad[rows].double() @ bd.double().t()).float() * 0.01).half())


def test_rows_past_two_to_the_31_bytes(g):
    """Rows of A whose offset passes 2^31 bytes, dense and over experts."""
    M, lda, K, N = 70000, 32768, 64, 96
    A = torch.zeros(M, lda, dtype=torch.int8, device=DEV)
    rng = np.random.default_rng(31)
    a, ad = int8_matrix(rng, 40, K, K)
    A[M - 40:, :K] = ad
    b, bd = int8_matrix(rng, 2 * N, K, K)
    one = torch.ones(M, device=DEV)
    D = torch.empty(M, N, device=DEV)
    g.gemm_int8(M, N, K, A, lda, one, bd, K, one, D, N, 0)
    ok(g)
    assert torch.equal(D[M - 40:], (ad.double() @ bd[:N].double().t()).float()) and (D[:M - 40] == 0).all()
    off = torch.tensor([0, M - 30, M], dtype=torch.int32, device=DEV)
    g.gemm_int8_grouped(M, N, K, 2, off, A, lda, one, bd, K, N * K, one, D, N, 0)
    ok(g)
    assert torch.equal(D[M - 30:], (ad[10:].double() @ bd[N:].double().t()).float())
    assert torch.equal(D[M - 40:M - 30], (ad[:10].double() @ bd[:N].double().t()).float())


# ------------------------------------------------------------------ streams, graphs, waits that run out

def test_on_another_stream_and_in_a_graph(g):
    rng = np.random.default_rng(12)
    M, N, K = 70, 200, 300
    a, ad = int8_matrix(rng, M, K, up16(K))
    b, bd = int8_matrix(rng, N, K, up16(K))
    sa, sb = np.full(M, 0.5, np.float32), np.full(N, 0.25, np.float32)
    sad, sbd = torch.from_numpy(sa).to(DEV), torch.from_numpy(sb).to(DEV)
    ref = expected(a[:, :K], b[:, :K], sa, sb, 0)
    D = torch.zeros(M, N, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g.gemm_int8(M, N, K, ad, up16(K), sad, bd, up16(K), sbd, D, N, 0, stream=side)
    side.synchronize()
    assert torch.equal(D.cpu(), ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gemm_int8(M, N, K, ad, up16(K), sad, bd, up16(K), sbd, D, N, 0)
    D.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(D.cpu(), ref)


@pytest.mark.parametrize("role", [1, 2])
@pytest.mark.parametrize("M", [12, 100, 300])
def test_waits_run_out(g, role, M):
    N, K = 256, 1024
    rng = np.random.default_rng(13)
    a, ad = int8_matrix(rng, M, K, K)
    b, bd = int8_matrix(rng, N, K, K)
    one = torch.ones(M + N, device=DEV)
    D = torch.empty(M, N, device=DEV)
    g.gemm_debug_inject_timeout(30, role)
    g.gemm_int8(M, N, K, ad, K, one, bd, K, one, D, N, 0)
    st, word = g.gemm_last_device_status()
    assert st == g.ERR_TIMEOUT and word != 0
    g.gemm_int8(M, N, K, ad, K, one, bd, K, one, D, N, 0)
    ok(g)
    assert torch.equal(D.cpu(), expected(a, b, np.ones(M, np.float32), np.ones(N, np.float32), 0))
