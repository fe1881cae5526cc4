"""The embedding lookup and its gradient against 64-bit references.

Tolerances: one rounding to bf16 (half a step, 2^-8 of the value) after a
product in fp32 (2^-24), and for the gradient a sum of n products in fp32, off
by at most n * 2^-24 of the sum of magnitudes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ROUND = 2.0 ** -8
F32 = 2.0 ** -24


def make_ids(kind, M, V, g):
    if kind == "same":
        return torch.full((M,), V - 1, device="cuda", dtype=torch.int64)
    if kind == "unknown":
        return torch.where(torch.arange(M, device="cuda") % 2 == 0, -1, V).long()
    if kind == "mixed":  # a few frequent ids, rare ones, unknown ones
        ids = ((V + 1.0) ** torch.rand(M, generator=g, device="cuda", dtype=torch.float64)).long() - 1
        ids.clamp_(0, V - 1)
        ids[torch.rand(M, generator=g, device="cuda") < 0.1] = -1
        return ids
    return torch.randint(0, V, (M,), generator=g, device="cuda")


@pytest.mark.parametrize("M,V,D", [(1, 1, 8), (3, 50, 264), (16, 1000, 4096), (257, 32000, 1000),
                                   (1021, 777, 2056), (5000, 129, 1032)])
@pytest.mark.parametrize("index", ["i64", "i32"])
@pytest.mark.parametrize("kind", ["random", "mixed", "unknown"])
def test_lookup(cuda_lib, M, V, D, index, kind):
    g = torch.Generator(device="cuda").manual_seed(M + V)
    ids = make_ids(kind, M, V, g)
    table = torch.randn(V, D, generator=g, device="cuda").bfloat16()
    typed = ids.to(torch.int32 if index == "i32" else torch.int64)
    out = torch.full((M, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    for scale in (1.0, 27.7):
        cuda_lib.embedding_lookup(typed, table, out, M, V, D, scale, index_type=index)
        known = (ids >= 0) & (ids < V)
        want = table[ids.clamp(0, V - 1)].double() * torch.tensor(scale, dtype=torch.float32).double()
        want[~known] = 0
        assert ((out.double() - want).abs() <= (ROUND + F32) * want.abs()).all()
        if scale == 1.0:
            assert torch.equal(out.double(), want)


def test_lookup_infinite_rows_do_not_reach_unknown_ids(cuda_lib):
    table = torch.full((4, 16), float("inf"), device="cuda", dtype=torch.bfloat16)
    table[3] = float("nan")
    ids = torch.tensor([-1, 0, 4, 3, -(1 << 40)], device="cuda")
    out = torch.full((5, 16), 7.0, device="cuda", dtype=torch.bfloat16)
    cuda_lib.embedding_lookup(ids, table, out, 5, 4, 16, 0.5)
    assert (out[[0, 2, 4]] == 0).all() and torch.isinf(out[1]).all() and torch.isnan(out[3]).all()


def grad_reference(ids, dout, V, scale, before):
    known = (ids >= 0) & (ids < V)
    at = ids[known]
    scale = torch.tensor(scale, dtype=torch.float32).double()
    total = torch.zeros(V, dout.shape[1], device="cuda", dtype=torch.float64)
    size = torch.zeros_like(total)
    total.index_add_(0, at, dout[known].double() * scale)
    size.index_add_(0, at, dout[known].double().abs() * scale)
    if before is not None:
        total += before.double()
        size += before.double().abs()
    terms = torch.bincount(at, minlength=V).double()[:, None] + 2
    return total, ROUND * total.abs() + (1 + ROUND) * terms * F32 * size


GRAD_SHAPES = [(1, 1, 8), (1, 300, 1032), (31, 7, 264), (33, 600, 2048), (1021, 1000, 1000),
               (2049, 263000, 8), (5000, 129, 1032), (16385, 40000, 512), (70001, 3000, 24)]


@pytest.mark.parametrize("M,V,D", GRAD_SHAPES)
@pytest.mark.parametrize("kind", ["random", "mixed", "same", "unknown"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(cuda_lib, M, V, D, kind, accumulate):
    g = torch.Generator(device="cuda").manual_seed(M + V)
    ids = make_ids(kind, M, V, g)
    dout = torch.randn(M, D, generator=g, device="cuda").bfloat16()
    dout[(ids < 0) | (ids >= V)] = float("nan")  # what padding may hold
    before = torch.randn(V, D, generator=g, device="cuda").bfloat16() if accumulate else None
    want, tol = grad_reference(ids, dout, V, 1.5, before)
    n = cuda_lib.gbf_workspace_size("embedding_grad", M, V, D, True)
    got = []
    for index in ("i64", "i32"):
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # holds anything
        dtable = before.clone() if accumulate else torch.full((V, D), float("nan"), device="cuda", dtype=torch.bfloat16)
        cuda_lib.embedding_grad(ids.to(torch.int32 if index == "i32" else torch.int64), dout, dtable, M, V, D, 1.5,
                                accumulate, index_type=index, workspace=ws, workspace_bytes=n)
        assert ((dtable.double() - want).abs() <= tol).all()
        got.append(dtable)
    assert torch.equal(got[0], got[1])  # a fixed order of sums


def test_gradient_of_no_positions(cuda_lib):
    dtable = torch.full((5, 16), 3.0, device="cuda", dtype=torch.bfloat16)
    ids = torch.zeros(8, device="cuda", dtype=torch.int64)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    cuda_lib.embedding_grad(ids, dtable, dtable, 0, 5, 16, accumulate=True, workspace=ws, workspace_bytes=4096)
    assert (dtable == 3).all()
    cuda_lib.embedding_grad(ids, dtable, dtable, 0, 5, 16, workspace=ws, workspace_bytes=4096)
    assert (dtable == 0).all()


def test_gradient_matches_differences_of_the_lookup(cuda_lib):
    """d/dE of sum(out * dout), by a difference in one row's values."""
    M, V, D, scale = 40, 9, 64, 0.5
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(-1, V, (M,), generator=g, device="cuda")
    table = torch.randint(-8, 8, (V, D), generator=g, device="cuda").bfloat16()
    dout = torch.randint(-3, 4, (M, D), generator=g, device="cuda").bfloat16()
    n = cuda_lib.gbf_workspace_size("embedding_grad", M, V, D, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dtable = torch.empty(V, D, device="cuda", dtype=torch.bfloat16)
    cuda_lib.embedding_grad(ids, dout, dtable, M, V, D, scale, workspace=ws, workspace_bytes=n)

    def value(t):
        out = torch.empty(M, D, device="cuda", dtype=torch.bfloat16)
        cuda_lib.embedding_lookup(ids, t, out, M, V, D, scale)
        return (out.double() * dout.double()).sum(dim=0)  # per column, exact: small integers

    for v in range(V):
        up, down = table.clone(), table.clone()
        up[v] += 2
        down[v] -= 2
        assert torch.equal((value(up) - value(down)) / 4, dtable[v].double())


def test_on_another_stream_and_in_a_graph(cuda_lib):
    M, V, D = 700, 500, 256
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(0, V, (M,), generator=g, device="cuda")
    table = torch.randn(V, D, generator=g, device="cuda").bfloat16()
    out = torch.empty(M, D, device="cuda", dtype=torch.bfloat16)
    dtable = torch.empty(V, D, device="cuda", dtype=torch.bfloat16)
    n = cuda_lib.gbf_workspace_size("embedding_grad", M, V, D, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def both(stream=None):
        cuda_lib.embedding_lookup(ids, table, out, M, V, D, stream=stream)
        cuda_lib.embedding_grad(ids, out, dtable, M, V, D, workspace=ws, workspace_bytes=n, stream=stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    both(side)
    side.synchronize()
    first = dtable.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    dtable.zero_()
    out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, dtable)
    table.mul_(2)  # the graph reads the buffers' present contents
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first * 2, dtable)


@pytest.mark.parametrize("M", [4097, 8191, 8192, 8193])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_where_the_way_of_sorting_changes(cuda_lib, M, accumulate):
    test_gradient(cuda_lib, M, 1500, 64, "mixed", accumulate)


@pytest.mark.parametrize("D", [264, 1288])
@pytest.mark.parametrize("share", [0.3, 0.7, 0.95])
def test_gradient_of_runs_over_many_pieces(cuda_lib, D, share):
    """A few ids that fill most of a long list, at its beginning, middle and end."""
    M, V = 20011, 900
    g = torch.Generator(device="cuda").manual_seed(D)
    ids = torch.randint(0, V, (M,), generator=g, device="cuda")
    often = torch.tensor([0, 400, 401, V - 1], device="cuda")
    pick = torch.rand(M, generator=g, device="cuda") < share
    ids = torch.where(pick, often[torch.randint(0, 4, (M,), generator=g, device="cuda")], ids)
    dout = torch.randn(M, D, generator=g, device="cuda").bfloat16()
    n = cuda_lib.gbf_workspace_size("embedding_grad", M, V, D, True)
    for accumulate in (False, True):
        before = torch.randn(V, D, generator=g, device="cuda").bfloat16() if accumulate else None
        want, tol = grad_reference(ids, dout, V, 1.5, before)
        got = []
        for _ in range(2):
            ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            dtable = before.clone() if accumulate else torch.full((V, D), float("nan"), device="cuda", dtype=torch.bfloat16)
            cuda_lib.embedding_grad(ids, dout, dtable, M, V, D, 1.5, accumulate, workspace=ws, workspace_bytes=n)
            assert ((dtable.double() - want).abs() <= tol).all()
            got.append(dtable)
        assert torch.equal(got[0], got[1])
