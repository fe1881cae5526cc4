"""Distillation from a teacher's top logits through a linear head, against a plain
fp64 form.

Tolerances.  A logit is a sum of chains of at most 1024 products on the tensor cores,
each off by at most 4e-9 a product of the sum S of its magnitudes, added in fp32: E =
(4e-9 min(D, 1024) + 2^-22) S.  lse and every l are off by that, the powers of two and
the shares by 2^-21 of themselves, the results by their fp32 rounding.  G is rounded to
bf16 (R = 2^-8 of it), and so are dx and dw; their sums over V or M products are one
chain.  Such bounds are far above what random errors come to, so root mean squares are
held as well: two independent roundings of up to R, uniform, come to 0.82 R."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

R = 2.0 ** -8


def inputs(M, V, D, K, seed=0, unscored=0.0, index=torch.int64, teacher=torch.float32, holes=0.2, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, D, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, D, generator=g, device="cuda") * (spread / math.sqrt(D))).bfloat16()
    ids = torch.randint(0, V, (M, K), generator=g, device="cuda")
    ids = torch.where(torch.rand(M, K, generator=g, device="cuda") < holes, -1 - ids, ids)
    ids[torch.rand(M, generator=g, device="cuda") < unscored] = V
    logits = (torch.randn(M, K, generator=g, device="cuda") * 2.5 + 8.0).to(teacher)
    return x, w, ids.to(index), logits


KINDS = {torch.int64: "i64", torch.int32: "i32", torch.bfloat16: "bf16", torch.float32: "f32"}


def sizes(x, w, ids, logits):
    return (x.shape[0], w.shape[0], x.shape[1], ids.shape[1]), dict(index_type=KINDS[ids.dtype], teacher_type=KINDS[logits.dtype])


def workspace(lib, size, grad):
    n = lib.linear_distill_workspace_size(*size, grad)
    return dict(workspace=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"), workspace_bytes=n)


def forward(lib, x, w, ids, logits, alpha=1.0, beta=1.0, stream=None):
    size, kinds = sizes(x, w, ids, logits)
    loss, lse, mean = (torch.full((n,), float("nan"), device="cuda") for n in (size[0], size[0], 1))
    lib.linear_distill(x, w, ids, logits, loss, lse, mean, *size, alpha, beta, **kinds, **workspace(lib, size, False), stream=stream)
    return loss, lse, mean


def backward(lib, x, w, ids, logits, lse, dloss=None, alpha=1.0, beta=1.0, scale=1.0, reduction="mean", skip=(), stream=None):
    size, kinds = sizes(x, w, ids, logits)
    out = {"dx": torch.full_like(x, float("nan")), "dw": torch.full_like(w, float("nan"))}
    lib.linear_distill_grad(x, w, ids, logits, lse, dloss, *(None if k in skip else v for k, v in out.items()), *size, alpha, beta,
                            scale, reduction, **kinds, **workspace(lib, size, True), stream=stream)
    return out["dx"], out["dw"]


def plain(x, w, ids, logits, alpha, beta):
    """fp64: scored rows, their logits, shares, lse, loss."""
    V = w.shape[0]
    ids, t = ids.long(), logits.double()
    valid = (ids >= 0) & (ids < V) & (t != -math.inf)
    scored = valid.any(dim=1)
    x = torch.where(scored[:, None], x.double(), 0.0)
    t = torch.where(valid, beta * t, -math.inf)
    t = torch.where(scored[:, None], t, 0.0)
    q = torch.where(valid, torch.softmax(t, dim=1), 0.0)
    l = alpha * (x @ w.double().T)
    lse = torch.logsumexp(l, dim=1)
    q = torch.zeros_like(l).scatter_add_(1, torch.where(valid, ids, 0), q)  # by column
    loss = torch.where(q > 0, q * (q.log() - l + lse[:, None]), 0.0).sum(dim=1)
    return scored, x, l, q, lse, loss


def near(x, w, alpha):
    D = x.shape[1]
    return (4e-9 * min(D, 1024) + 2.0 ** -22) * abs(alpha) * (x.abs() @ w.double().abs().T).amax(dim=1)


def check_forward(got, x, w, ids, logits, alpha=1.0, beta=1.0):
    loss, lse, mean = got
    scored, x, l, q, lse64, loss64 = plain(x, w, ids, logits, alpha, beta)
    e = near(x, w, alpha)
    assert bool((loss[~scored] == 0).all()) and bool((lse[~scored] == 0).all())
    err = (lse.double() - lse64).abs()[scored]
    assert bool((err <= (e + 2.0 ** -21 + 2.0 ** -23 * lse64.abs())[scored]).all()), float(err.max())
    tol = 2 * e + 2.0 ** -19 + 2.0 ** -23 * loss64.abs()  # shares and powers: 2^-21, times logarithms of some units
    err = (loss.double() - loss64).abs()[scored]
    assert bool((err <= tol[scored]).all()), float((err / tol[scored]).max())
    assert bool((loss >= 0).all())
    want = loss64[scored].sum() / max(1, int(scored.sum()))
    assert abs(float(mean[0]) - float(want)) <= float(tol[scored].mean() if bool(scored.any()) else 0.0) + 1e-12


def check_backward(got, x, w, ids, logits, lse, dloss=None, alpha=1.0, beta=1.0, scale=1.0, reduction="mean", rms=True):
    scored, x64, l, q, _, _ = plain(x, w, ids, logits, alpha, beta)
    w64 = w.double()
    p = (l - lse.double()[:, None]).exp()  # of the lse that was handed in
    dl = torch.ones_like(lse, dtype=torch.float64) if dloss is None else dloss.double()
    dl = torch.where(scored, dl, 0.0)
    G = dl[:, None] * (p - q)
    f = alpha * scale / (max(1, int(scored.sum())) if reduction == "mean" else 1)
    e = 2 * near(x64, w, alpha)[:, None] + 2.0 ** -21
    eg = dl.abs()[:, None] * (p * e + 2.0 ** -21 * (p + q))
    eg = R * (G.abs() + eg) + eg
    for name, grad, a, b, ea in (("dx", got[0], G, w64, eg), ("dw", got[1], G.T, x64, eg.T)):
        want = f * (a @ b)
        k = a.shape[1]
        bound = abs(f) * (ea @ b.abs() + (4e-9 * k + 2.0 ** -22) * ((a.abs() + ea) @ b.abs()))
        err = (grad.double() - want).abs()
        bound = R * (want.abs() + bound) + bound + 1e-37
        assert bool((err <= bound).all()), (name, float((err / bound).max()))
        if rms and want.numel() >= 4096:
            assert float(err.square().mean().sqrt()) <= R * float(want.square().mean().sqrt()), name
    assert bool((got[0][~scored] == 0).all())


def check(lib, x, w, ids, logits, alpha=1.0, beta=1.0, rms=True, **kw):
    got = forward(lib, x, w, ids, logits, alpha, beta)
    check_forward(got, x, w, ids, logits, alpha, beta)
    grads = backward(lib, x, w, ids, logits, got[1], alpha=alpha, beta=beta, **kw)
    check_backward(grads, x, w, ids, logits, got[1], alpha=alpha, beta=beta, rms=rms, **kw)
    assert lib.gbf_check_device_error() == 0
    return got, grads


@pytest.mark.parametrize("M,V,D,K", [
    (1, 1, 8, 1), (1, 300, 64, 3), (3, 1000, 200, 7), (16, 5001, 1024, 20), (17, 700, 1032, 130), (64, 3000, 2048, 50),
    (100, 1000, 4096, 64), (128, 555, 264, 1024), (129, 300, 72, 5), (200, 5001, 1024, 20), (256, 900, 2048, 33),
    (257, 5001, 264, 50), (300, 700, 4096, 9), (700, 3001, 1032, 128), (1030, 2000, 136, 1)])
def test_against_fp64(cuda_lib, M, V, D, K):
    check(cuda_lib, *inputs(M, V, D, K, seed=M + V, unscored=0.25 if M > 8 else 0.0))


@pytest.mark.parametrize("M,V,D,K", [(1, 700, 136, 2), (1, 5001, 1032, 40), (7, 300, 64, 3), (16, 33000, 264, 20)])
def test_few_rows_are_rounded_once(cuda_lib, M, V, D, K):
    """Up to 16 rows G is the sum of two bf16, off by R^2 of itself: the gradients are off
    by their own rounding and what the logits are off by."""
    args = inputs(M, V, D, K, seed=M + V)
    lse = forward(cuda_lib, *args)[1]
    got = backward(cuda_lib, *args, lse, reduction="sum")
    scored, x64, l, q, _, _ = plain(*args, 1.0, 1.0)
    w64 = args[1].double()
    p = (l - lse.double()[:, None]).exp()
    G = torch.where(scored[:, None], p - q, 0.0)
    eg = p * (2 * near(x64, args[1], 1.0)[:, None] + 2.0 ** -21) + 2.0 ** -21 * q + R * R * G.abs()
    for name, grad, a, b, ea in (("dx", got[0], G, w64, eg), ("dw", got[1], G.T, x64, eg.T)):
        want = a @ b
        bound = ea @ b.abs() + (8e-9 * a.shape[1] + 2.0 ** -22) * (a.abs() @ b.abs())
        err = (grad.double() - want).abs()
        assert bool((err <= R * (want.abs() + bound) + bound + 1e-37).all()), name


@pytest.mark.parametrize("M", [5, 100, 300])
@pytest.mark.parametrize("index", [torch.int64, torch.int32])
@pytest.mark.parametrize("teacher", [torch.float32, torch.bfloat16])
def test_types_scales_and_reductions(cuda_lib, M, index, teacher):
    args = inputs(M, 1500, 136, 12, seed=M, unscored=0.3, index=index, teacher=teacher)
    check(cuda_lib, *args, alpha=0.5, beta=0.25, scale=4.0)
    check(cuda_lib, *args, alpha=-1.5, beta=2.0, reduction="sum")
    dloss = torch.randn(M, device="cuda")
    check(cuda_lib, *args, dloss=dloss, reduction="sum")


@pytest.mark.parametrize("M,V,D,K", [(257, 10001, 72, 50), (300, 12000, 264, 1), (600, 9000, 1000, 128), (1030, 6000, 136, 20)])
def test_two_row_tiles_per_unit(cuda_lib, M, V, D, K):
    """Sizes whose units of work hold two row tiles; the last ones are ragged."""
    check(cuda_lib, *inputs(M, V, D, K, seed=M + V, unscored=0.25))


def edge_ids(V):
    marks = [0, 32, 64, 96, 128, 160, 192, 224, 256, 384, 512, 1024, 16384, 32768, V]
    return sorted({i for m in marks for i in (m - 1, m, m + 1) if 0 <= i < V})


@pytest.mark.parametrize("M,V,D", [(9, 700, 64), (70, 700, 72), (128, 1100, 64), (200, 700, 64), (300, 700, 72), (300, 700, 1032)])
def test_ids_at_the_edges_of_tiles(cuda_lib, M, V, D):
    """Every row holds columns on both sides of each tile's, chunk's and warp's edge, in
    falling and mixed orders."""
    x, w, _, _ = inputs(M, V, D, 1, seed=V)
    e = torch.tensor(edge_ids(V), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = e.flip(0).repeat(M, 1)
    ids[1::2] = e[torch.rand(len(ids[1::2]), len(e), generator=g, device="cuda").argsort(dim=1)]
    check(cuda_lib, x, w, ids, torch.randn(M, len(e), generator=g, device="cuda"))


def test_ids_at_the_edges_of_two_row_tiles(cuda_lib):
    x, w, _, _ = inputs(300, 10100, 72, 1, seed=4)
    g = torch.Generator(device="cuda").manual_seed(4)
    e = torch.tensor(edge_ids(10100), device="cuda")
    ids = e[torch.rand(300, len(e), generator=g, device="cuda").argsort(dim=1)]
    check(cuda_lib, x, w, ids, torch.randn(300, len(e), generator=g, device="cuda"))


@pytest.mark.parametrize("M", [40, 300])
def test_the_same_id_many_times(cuda_lib, M):
    """Entries of one id are one column with the sum of their shares."""
    x, w, ids, logits = inputs(M, 600, 72, 1024, seed=M, holes=0.0)
    ids[0::3] %= 5  # 1024 entries on five columns
    ids[1::3] = 599
    check(cuda_lib, x, w, ids, logits)


@pytest.mark.parametrize("M", [12, 100, 200, 300])
def test_entries_and_rows_left_out(cuda_lib, M):
    """Padding of any kind, and what a row without entries holds, reaches nothing."""
    x, w, ids, logits = inputs(M, 900, 136, 6, seed=M, unscored=0.3)
    ids[3] = torch.tensor([-1, 5, -100, 900, 2 ** 40, 899], device="cuda")
    logits[3, 0], logits[3, 2], logits[3, 3] = float("nan"), float("inf"), float("nan")
    logits[4] = -math.inf  # a row of nothing but minus infinity is not scored
    logits[5, :5] = -math.inf
    ids[5] = torch.arange(6, device="cuda")
    scored = plain(x, w, ids, logits, 1.0, 1.0)[0]
    assert not bool(scored[4]) and bool(scored[3]) and bool(scored[5])
    x[~scored] = float("nan")
    check(cuda_lib, x, w, ids, logits, rms=False)


@pytest.mark.parametrize("M", [4, 300])
def test_no_row_scored(cuda_lib, M):
    x, w, ids, logits = inputs(M, 300, 64, 4)
    ids[:] = -100
    x[:] = float("nan")
    (loss, lse, mean), (dx, dw) = forward(cuda_lib, x, w, ids, logits), backward(cuda_lib, x, w, ids, logits, torch.zeros(M, device="cuda"))
    for t in (loss, lse, mean, dx, dw):
        assert bool((t == 0).all())


def test_no_rows(cuda_lib):
    x, w, ids, logits = inputs(2, 300, 64, 4)
    loss, lse, mean = forward(cuda_lib, x[:0], w, ids[:0], logits[:0])
    assert float(mean) == 0.0
    assert bool((backward(cuda_lib, x[:0], w, ids[:0], logits[:0], lse)[1] == 0).all())


@pytest.mark.parametrize("M", [30, 200, 400])
def test_small_losses(cuda_lib, M):
    """A confident student of a confident teacher, and a student that is its teacher:
    losses of zero, in differences of large sums.  The errors of l leave the differences
    (both come from one product); what stays is 2^-21 of the powers and shares, times
    logarithms of some units."""
    V, D = 300, 512
    x, w, _, _ = inputs(M, V, D, 1, seed=M)
    ids = torch.randint(0, V, (M, 2), device="cuda")
    ids[:, 1] = -1
    sure = (w[ids[:, 0]].float() * 20).bfloat16()
    loss, _, _ = forward(cuda_lib, sure, w, ids, torch.zeros(M, 2, device="cuda"))
    want = plain(sure, w, ids, torch.zeros(M, 2, device="cuda"), 1.0, 1.0)[5]
    assert float(want.max()) < 1e-9 and float(loss.max()) <= 2.0 ** -20
    every = torch.arange(V, device="cuda").repeat(M, 1)
    logits = (x.double() @ w.double().T).float()
    got = forward(cuda_lib, x, w, every, logits)
    want = plain(x, w, every, logits, 1.0, 1.0)[5]
    assert float(want.abs().max()) < 1e-9
    assert float(got[0].max()) <= float(near(x.double(), w, 1.0).max()) + 2.0 ** -19


@pytest.mark.parametrize("M", [20, 100, 200, 600])
@pytest.mark.parametrize("D", [512, 4096])
def test_accuracy_for_random_signs(cuda_lib, M, D):
    """lse and loss off by no more than about 5e-7 of the sums they are made of."""
    x, w, ids, logits = inputs(M, 4000, D, 30, seed=M + D, holes=0.0)
    loss, lse, _ = forward(cuda_lib, x, w, ids, logits)
    _, _, l, q, lse64, loss64 = plain(x, w, ids, logits, 1.0, 1.0)
    size = lse64.abs() + (q * l.abs()).sum(dim=1) + 1.0
    for got, want in ((lse, lse64), (loss, loss64)):
        assert float(((got.double() - want) / size).square().mean().sqrt()) <= 5e-7


def test_one_entry_is_the_hard_targets_loss(cuda_lib):
    M, V, D = 300, 900, 264
    x, w, ids, logits = inputs(M, V, D, 1, seed=2, unscored=0.3)
    loss, lse, mean = forward(cuda_lib, x, w, ids, logits)
    grads = backward(cuda_lib, x, w, ids, logits, lse)
    a, b, c = torch.empty_like(loss), torch.empty_like(lse), torch.empty_like(mean)
    n = max(cuda_lib.gbf_workspace_size(op, M, V, D, True) for op in ("linear_ce", "linear_ce_grad"))
    ws = dict(workspace=torch.empty(n, dtype=torch.uint8, device="cuda"), workspace_bytes=n)
    t = ids[:, 0].contiguous()
    cuda_lib.linear_ce(x, w, t, a, b, c, M, V, D, **ws)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    cuda_lib.linear_ce_grad(x, w, t, lse, None, dx, dw, M, V, D, **ws)
    # the same products; the sums of powers may be cut into other tiles
    assert float((a - loss).abs().max()) <= 2.0 ** -20 * float(1.0 + lse.abs().max())
    assert torch.equal(grads[0], dx) and torch.equal(grads[1], dw)


@pytest.mark.parametrize("M", [24, 200, 600])
def test_left_out_captured_and_on_another_stream(cuda_lib, M):
    from tcgen05_tmem_bf16_gb300.graphs import CapturedChain
    args = inputs(M, 1200, 264, 9, seed=M, unscored=0.2)
    other = inputs(M, 1200, 264, 9, seed=M + 1, unscored=0.4)

    def step(args, stream=None):
        got = forward(cuda_lib, *args, stream=stream)
        return (*got, *backward(cuda_lib, *args, got[1], stream=stream))

    want, want2 = step(args), step(other)
    for skip, keep in (("dx", 1), ("dw", 0)):
        assert torch.equal(backward(cuda_lib, *args, want[1], skip=(skip,))[keep], want[3 + keep])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step(args)
    torch.cuda.synchronize()
    for a, b in zip(again, want):
        assert torch.equal(a, b)
    size, kinds = sizes(*args)
    out = [torch.empty_like(t) for t in want]
    ws = {g: workspace(cuda_lib, size, g) for g in (False, True)}

    def chain(stream):
        cuda_lib.linear_distill(*args, *out[:3], *size, **kinds, **ws[False], stream=stream)
        cuda_lib.linear_distill_grad(*args, out[1], None, *out[3:], *size, **kinds, **ws[True], stream=stream)

    graph = CapturedChain(chain)
    for b, w in ((None, want), (other, want2)):
        if b is not None:
            for dst, src in zip(args, b):
                dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(out, w):
            assert torch.equal(a, c)


def test_several_pieces_of_the_vocabulary(cuda_lib):
    """G in three pieces; columns on both sides of the pieces' edges."""
    M, V, D = 8192, 40001, 64
    x, w, ids, logits = inputs(M, V, D, 40, seed=1, unscored=0.1)
    e = torch.tensor(edge_ids(V), device="cuda")[-12:]
    ids[::2, :len(e)] = e
    check(cuda_lib, x, w, ids, logits)


def test_long_sums_in_segments(cuda_lib):
    for M, D in ((5, 8192), (100, 8192), (300, 8192)):
        check(cuda_lib, *inputs(M, 400, D, 10, seed=M))


def test_against_differences(cuda_lib):
    """Directional derivatives against differences of the fp64 loss; a random error of
    0.82 R of each value along a normal direction comes to that of the norm."""
    M, V, D = 90, 500, 72
    x, w, ids, logits = inputs(M, V, D, 7, seed=5)
    _, lse, _ = forward(cuda_lib, x, w, ids, logits)
    grads = backward(cuda_lib, x, w, ids, logits, lse, reduction="sum")
    g = torch.Generator(device="cuda").manual_seed(2)
    for k in (0, 1):
        v = torch.randn(grads[k].shape, generator=g, device="cuda", dtype=torch.float64)
        at = lambda s: float(plain(x.double() + (s * v if k == 0 else 0.0), w.double() + (s * v if k == 1 else 0.0),  # noqa: E731
                                   ids, logits, 1.0, 1.0)[5].sum())
        diff = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(float((grads[k].double() * v).sum()) - diff) <= 6 * 0.82 * R * float(grads[k].double().norm())


@pytest.mark.parametrize("M", [30, 200, 400])
def test_nothing_outside_is_written(cuda_lib, M):
    V, D, K = 700, 72, 9
    args = inputs(M, V, D, K, seed=M)
    size, kinds = sizes(*args)
    flat = {n: torch.full((c + 128,), 7.0, device="cuda", dtype=t) for n, c, t in (
        ("loss", M, torch.float32), ("lse", M, torch.float32), ("dx", M * D, torch.bfloat16), ("dw", V * D, torch.bfloat16))}
    v = {n: t[64:-64] for n, t in flat.items()}
    for grad in (False, True):
        n = cuda_lib.linear_distill_workspace_size(*size, grad)
        ws = torch.full((n + 256,), 0x55, dtype=torch.uint8, device="cuda")
        if grad:
            cuda_lib.linear_distill_grad(*args, v["lse"], None, v["dx"], v["dw"], *size, **kinds, workspace=ws, workspace_bytes=n)
        else:
            cuda_lib.linear_distill(*args, v["loss"], v["lse"], None, *size, **kinds, workspace=ws, workspace_bytes=n)
        assert bool((ws[n:] == 0x55).all())
    for t in flat.values():
        assert bool((t[:64] == 7.0).all()) and bool((t[-64:] == 7.0).all())
    check_backward((v["dx"].view(M, D), v["dw"].view(V, D)), *args, v["lse"].clone())


@pytest.mark.parametrize("M,D", [(100, 4096), (200, 64), (200, 4096), (300, 64), (300, 4096)])
def test_a_wait_that_runs_out_is_reported(cuda_lib, M, D):
    args = inputs(M, 300, D, 5, seed=M)
    want = forward(cuda_lib, *args)
    try:
        cuda_lib.gbf_set_wait_timeout_ns(20_000_000)
        cuda_lib.gbf_debug_inject_timeout(True)
        forward(cuda_lib, *args)
        assert cuda_lib.gbf_check_device_error() == 6
    finally:
        cuda_lib.gbf_debug_inject_timeout(False)
        cuda_lib.gbf_set_wait_timeout_ns(2_000_000_000)
    assert all(torch.equal(a, b) for a, b in zip(forward(cuda_lib, *args), want))


def test_a_wait_of_two_row_tiles_that_runs_out_is_reported(cuda_lib):
    args = inputs(300, 10100, 72, 5, seed=300)
    want = forward(cuda_lib, *args)
    try:
        cuda_lib.gbf_set_wait_timeout_ns(20_000_000)
        cuda_lib.gbf_debug_inject_timeout(True)
        forward(cuda_lib, *args)
        assert cuda_lib.gbf_check_device_error() == 6
    finally:
        cuda_lib.gbf_debug_inject_timeout(False)
        cuda_lib.gbf_set_wait_timeout_ns(2_000_000_000)
    assert all(torch.equal(a, b) for a, b in zip(forward(cuda_lib, *args), want))
