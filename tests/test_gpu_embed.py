"""Rows of a token table and the table's gradient against float64.

Tolerances count roundings: a row's element is one product, rounded to fp32 and to its type (half a step of each); a
gradient's element is a sum of n values in fp32, off by at most n * 2^-24 of their absolute sum (in chunks far less), times
the factor, rounded to fp32, added to what was there, and rounded to its type.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
OUT = {"f32": (torch.float32, 0), "bf16": (torch.bfloat16, 1), "f16": (torch.float16, 2)}


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import smem_swizzle_layouts_gb300 as g
    return g


def half_step(want, dtype):
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[dtype]
    return want.abs() * torch.finfo(dtype).eps / 2 + tiny


def shape(n, width, dtype, pad, shift):
    """Rows `width` wide, `pad` elements between them, that start `shift` elements into their memory; NaN all over."""
    ld = width + pad
    flat = torch.full((n * ld + shift + 8,), math.nan, dtype=dtype, device=DEV)
    return torch.as_strided(flat, (n, width), (ld, 1), shift)


def ids_of(T, V, seed, kind="random"):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if kind == "one":
        return torch.full((T,), V // 2, dtype=torch.int32, device=DEV)
    if kind == "few":
        return torch.randint(0, min(V, 5), (T,), generator=gen, device=DEV, dtype=torch.int32) * max(1, (V - 1) // 5)
    ids = torch.randint(0, V, (T,), generator=gen, device=DEV, dtype=torch.int32)
    if kind == "bad":
        ids[::5], ids[1::7], ids[2::11] = -1, V, 2 ** 31 - 1
        ids[3::13] = -2 ** 31
    return ids


def embed(g, table, ids, scale, dtype, pad=0, shift=0, stream=None):
    T, (V, N) = ids.numel(), table.shape
    D = shape(T, N, dtype, pad, shift)
    code = {v[0]: v[1] for v in OUT.values()}
    g.gemm_embed(T, N, V, ids, table, code[table.dtype], table.stride(0), scale, D, code[dtype], D.stride(0), stream=stream)
    return D


def check_rows(table, ids, scale, D):
    V = table.shape[0]
    live = (ids >= 0) & (ids < V)
    want = torch.where(live[:, None], table[ids.long().clamp(0, V - 1)].double(), 0.0) * float(torch.tensor(scale))
    want = torch.where(live[:, None], want, 0.0)
    assert bool(((D.double() - want).abs() <= half_step(want, D.dtype) + 2.0 ** -24 * want.abs()).all())


@pytest.mark.parametrize("t_type", OUT)
@pytest.mark.parametrize("d_type", OUT)
@pytest.mark.parametrize("T,N,V,pad,shift", [(1, 1, 1, 0, 0), (1, 4096, 50, 0, 0), (5, 64, 1000, 8, 8), (300, 1001, 777, 3, 1), (257, 2048, 4000, 0, 1),
                                            (64, 24, 9, 0, 0)])
def test_rows(g, T, N, V, pad, shift, t_type, d_type):
    table = shape(V, N, OUT[t_type][0], pad, shift)
    table.copy_(torch.randn(V, N, device=DEV))
    ids = ids_of(T, V, T, "bad" if T > 8 else "random")
    D = embed(g, table, ids, 1.7, OUT[d_type][0], pad, shift)
    check_rows(table, ids, 1.7, D)
    assert bool(torch.as_strided(D, (T, pad), (N + pad, 1), shift + N).isnan().all())  # nothing behind the rows is written


def gradient(g, ids, dD, V, scale, dtype, old=None, pad=0, shift=0, stream=None):
    T, N = dD.shape
    d = shape(V, N, dtype, pad, shift)
    if old is not None:
        d.copy_(old)
    code = {v[0]: v[1] for v in OUT.values()}
    n = g.gemm_embed_backward_workspace_size(T, N, V)
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device=DEV)
    g.gemm_embed_backward(T, N, V, ids, dD, code[dD.dtype], dD.stride(0), scale, d, code[dtype], d.stride(0), int(old is not None), ws, n,
                          stream=stream)
    return d


def check_gradient(ids, dD, V, scale, d, old=None):
    scale = float(torch.tensor(scale))
    live = (ids >= 0) & (ids < V)
    at = ids[live].long()
    rows = dD[live].double()
    want = torch.zeros(V, dD.shape[1], dtype=torch.float64, device=DEV).index_add_(0, at, rows) * scale
    size = torch.zeros_like(want).index_add_(0, at, rows.abs()) * abs(scale)
    many = torch.bincount(at, minlength=V).double()[:, None]
    if old is not None:
        want, size = want + old.double(), size + old.double().abs()
    # a sum of n values passes at most 32 in its chunk, an eighth of the chunks in its group, and 8 groups
    steps = torch.minimum(many, 34 + many / 256 + 8)
    assert bool(((d.double() - want).abs() <= half_step(want, d.dtype) * (1 + 2.0 ** -8) + (steps + 2) * 2.0 ** -24 * size + 1e-38).all())
    if old is not None:
        still = many[:, 0] == 0
        assert torch.equal(d[still], old[still])


GRAD = [(1, 1, 1, "random"), (1, 4096, 50, "random"), (31, 64, 1000, "few"), (32, 40, 7, "one"), (33, 40, 7, "one"), (64, 1001, 20, "few"),
        (65, 72, 3000, "bad"), (2000, 1030, 513, "random"), (2048, 200, 70000, "bad"), (2049, 24, 262145, "random"), (5000, 1032, 40, "few"),
        (20000, 96, 1000, "random"), (9000, 129, 300000, "bad"), (70000, 16, 2, "random"), (40000, 8, 3, "one"), (300000, 8, 1 << 19, "random")]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,N,V,kind", GRAD)
def test_gradient(g, T, N, V, kind, accumulate):
    dD = torch.randn(T, N, device=DEV).bfloat16()
    ids = ids_of(T, V, T + 1, kind)
    old = torch.randn(V, N, device=DEV) if accumulate else None
    d = gradient(g, ids, dD, V, 0.7, torch.float32, old)
    check_gradient(ids, dD, V, 0.7, d, old)


@pytest.mark.parametrize("t_type", OUT)
@pytest.mark.parametrize("d_type", OUT)
@pytest.mark.parametrize("N,pad,shift", [(1000, 0, 0), (1000, 24, 8), (77, 1, 3), (136, 0, 1)])
def test_gradient_types_and_strides(g, N, pad, shift, t_type, d_type):
    dD = shape(700, N, OUT[d_type][0], pad, shift)
    dD.copy_(torch.randn(700, N, device=DEV))
    ids = ids_of(700, 90, 3, "bad")
    for old in (None, torch.randn(90, N, device=DEV).to(OUT[t_type][0])):
        d = gradient(g, ids, dD, 90, -1.3, OUT[t_type][0], old, pad, shift)
        check_gradient(ids, dD, 90, -1.3, d, old)
        assert bool(torch.as_strided(d, (90, pad), (N + pad, 1), shift + N).isnan().all())


def test_padded_rows_carry_nothing(g):
    """Rows whose id is no token's may hold anything; with none that is, the table's gradient is zeros, or stays."""
    dD = torch.randn(400, 64, device=DEV)
    ids = ids_of(400, 100, 4, "bad")
    dead = (ids < 0) | (ids >= 100)
    dD[dead] = math.nan
    d = gradient(g, ids, dD, 100, 2.0, torch.float32)
    clean = torch.where(dead[:, None], 0.0, dD)
    check_gradient(ids, clean, 100, 2.0, d)
    ids.fill_(-1)
    dD.fill_(math.nan)
    assert not gradient(g, ids, dD, 100, 2.0, torch.float32).any()
    old = torch.randn(100, 64, device=DEV)
    assert torch.equal(gradient(g, ids, dD, 100, 2.0, torch.float32, old), old)


def test_no_tokens_and_no_table(g):
    d = torch.full((30, 16), 3.0, device=DEV)
    g.gemm_embed(0, 16, 30, None, None, 0, 16, 1.0, None, 0, 16)
    g.gemm_embed_backward(0, 16, 30, None, None, 0, 16, 1.0, d, 0, 16, 1, None, 0)
    assert bool((d == 3.0).all())
    g.gemm_embed_backward(0, 16, 30, None, None, 0, 16, 1.0, d, 0, 16, 0, None, 0)
    assert not d.any()
    D = torch.full((3, 16), 3.0, device=DEV)
    g.gemm_embed(3, 16, 0, torch.zeros(3, dtype=torch.int32, device=DEV), None, 0, 16, 1.0, D, 0, 16)
    assert not D.any()


def test_the_sum_of_a_frequent_token_is_exact_where_fp32_is(g):
    """100000 ones of one token, and whole numbers of others: sums below 2^24 have one right answer."""
    T = 100000
    ids = torch.full((T,), 7, dtype=torch.int32, device=DEV)
    ids[::1000] = 3
    dD = torch.randint(-8, 9, (T, 40), device=DEV).float()
    d = gradient(g, ids, dD, 11, 1.0, torch.float32)
    want = torch.zeros(11, 40, dtype=torch.float64, device=DEV).index_add_(0, ids.long(), dD.double())
    assert torch.equal(d.double(), want)


def test_the_same_call_twice_gives_the_same_bits(g):
    dD = torch.randn(30000, 200, device=DEV)
    ids = ids_of(30000, 400, 5)
    assert torch.equal(gradient(g, ids, dD, 400, 1.0, torch.float32), gradient(g, ids, dD, 400, 1.0, torch.float32))


def test_side_stream_and_graph(g):
    T, N, V = 5000, 264, 900
    table, dD = torch.randn(V, N, device=DEV).bfloat16(), torch.randn(T, N, device=DEV).bfloat16()
    ids = ids_of(T, V, 6, "bad")
    D, d = torch.empty(T, N, device=DEV), torch.empty(V, N, device=DEV)
    n = g.gemm_embed_backward_workspace_size(T, N, V)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def step():
        g.gemm_embed(T, N, V, ids, table, 1, N, 0.5, D, 0, N)
        g.gemm_embed_backward(T, N, V, ids, dD, 1, N, 0.5, d, 0, N, 0, ws, n)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    check_rows(table, ids, 0.5, D)
    check_gradient(ids, dD, V, 0.5, d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (7, 8):
        ids.copy_(ids_of(T, V, seed, "few" if seed == 7 else "bad"))
        dD.copy_(torch.randn(T, N, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        check_rows(table, ids, 0.5, D)
        check_gradient(ids, dD, V, 0.5, d)


def test_rows_past_32_bit_offsets(g):
    """A table and rows of more than 2^31 elements."""
    N, V = 65536, 33000
    table = torch.empty(V, N, dtype=torch.bfloat16, device=DEV)
    table[-3:] = torch.randn(3, N, device=DEV)
    ids = torch.tensor([V - 1, V - 2, V - 1, V], dtype=torch.int32, device=DEV)
    D = embed(g, table, ids, 1.0, torch.float32)
    assert torch.equal(D[:3], table[[V - 1, V - 2, V - 1]].float()) and not D[3].any()
    table.zero_()
    d = gradient(g, ids, D, V, 1.0, torch.bfloat16)
    assert torch.equal(d[V - 1], (D[0] + D[2]).bfloat16()) and torch.equal(d[V - 2], D[1].bfloat16()) and not d[:V - 2].any()
