"""The linear cross entropy and its gradients against 64-bit references.

Tolerances, element by element from the reference's own magnitudes:
  logits  a sum of D products in fp32, off by at most D * 2^-23 * sum |x w|
          (tensor cores may cut instead of rounding: a whole step each);
  lse     the largest logit error of the row, the rounding of the scaled
          logits (2^-22 of the largest) and of the sum of exponentials (each
          2^-21, and fewer than 128 + V / 128 additions deep);
  G       the relative error of exp(l - lse), and half a step of bf16 (2^-8);
  dx, dw  the errors of G times the magnitudes of the other factor, a sum in
          fp32 of V (M) products, and half a step of bf16 on the result.
Values below 2^-126, the smallest normal value of bf16 and fp32, may be zero."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8
F32 = 2.0 ** -24
SMALLEST = 2.0 ** -126


def inputs(M, V, D, ignored, seed, spread=2.0, index="i64"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, D, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, D, generator=g, device="cuda") * spread / D ** 0.5).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    if ignored:
        off = torch.rand(M, generator=g, device="cuda") < ignored
        t[off] = torch.where(torch.rand(int(off.sum()), generator=g, device="cuda") < 0.5, -100, V)
    return x, w, t.to(torch.int32 if index == "i32" else torch.int64)


def forward(lib, x, w, t, alpha=1.0, stream=None, with_mean=True):
    M, D = x.shape
    V = w.shape[0]
    n = lib.gbf_workspace_size("linear_ce", M, V, D, True)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
    loss = torch.full((M,), float("nan"), device="cuda")
    lse = torch.full((M,), float("nan"), device="cuda")
    mean = torch.full((1,), float("nan"), device="cuda")
    index = "i32" if t.dtype == torch.int32 else "i64"
    lib.linear_ce(x, w, t, loss, lse, mean if with_mean else None, M, V, D, alpha, index_type=index, workspace=ws,
                  workspace_bytes=n, stream=stream)
    assert lib.gbf_check_device_error(stream) == 0
    return loss, lse, mean


def backward(lib, x, w, t, lse, alpha=1.0, scale=1.0, reduction="mean", dloss=None, want=("dx", "dw")):
    M, D = x.shape
    V = w.shape[0]
    n = lib.gbf_workspace_size("linear_ce_grad", M, V, D, True)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    dx = torch.full((M, D), float("nan"), device="cuda", dtype=torch.bfloat16) if "dx" in want else None
    dw = torch.full((V, D), float("nan"), device="cuda", dtype=torch.bfloat16) if "dw" in want else None
    index = "i32" if t.dtype == torch.int32 else "i64"
    lib.linear_ce_grad(x, w, t, lse, dloss, dx, dw, M, V, D, alpha, scale, reduction, index_type=index, workspace=ws,
                       workspace_bytes=n)
    assert lib.gbf_check_device_error() == 0
    return dx, dw


class Reference:
    def __init__(self, x, w, t, alpha):
        V, D = w.shape
        t = t.long()
        self.scored = (t >= 0) & (t < V)
        self.rows = torch.nonzero(self.scored)[:, 0]
        self.x, self.w, self.alpha = x[self.rows].double(), w.double(), alpha
        self.t = t[self.rows]
        self.l = alpha * self.x @ self.w.T
        self.l_err = abs(alpha) * D * 2 * F32 * (self.x.abs() @ self.w.abs().T)
        self.lse = torch.logsumexp(self.l, dim=1)
        at = torch.arange(len(self.rows), device="cuda")
        self.at = at
        lt = self.l[at, self.t]
        self.loss = self.lse - lt
        big = self.l.abs().amax(dim=1) if len(self.rows) else self.lse
        self.lse_tol = self.l_err.amax(dim=1) + 4 * F32 * big + (8 + 128 + V / 128) * F32 + F32 * self.lse.abs()
        self.loss_tol = self.lse_tol + self.l_err[at, self.t] + F32 * (lt.abs() + self.loss.abs())

    def check_forward(self, loss, lse, mean):
        assert (loss[~self.scored] == 0).all() and (lse[~self.scored] == 0).all()
        assert ((lse[self.rows].double() - self.lse).abs() <= self.lse_tol).all()
        assert ((loss[self.rows].double() - self.loss).abs() <= self.loss_tol).all()
        want = float(self.loss.mean()) if len(self.rows) else 0.0
        tol = float(self.loss_tol.mean()) + F32 * abs(want) if len(self.rows) else 0.0
        assert abs(float(mean) - want) <= tol

    def check_backward(self, dx, dw, scale=1.0, reduction="mean", dloss=None):
        f = self.alpha * scale / (max(1, len(self.rows)) if reduction == "mean" else 1)
        p = (self.l - self.lse[:, None]).exp()
        weight = torch.ones_like(self.lse) if dloss is None else dloss[self.rows].double()
        big = self.l.abs().amax(dim=1)
        rel = self.l_err + (self.lse_tol + 4 * F32 * big)[:, None] + 8 * F32
        g_err = rel * p
        g = p.clone()
        g[self.at, self.t] -= 1
        g, g_err = g * weight[:, None], g_err * weight.abs()[:, None]
        g_err = g_err * (1 + BF) + (BF + 4 * F32) * g.abs() + weight.abs()[:, None] * SMALLEST
        size = g.abs() + g_err
        if dx is not None:
            want = f * g @ self.w
            err = abs(f) * (g_err @ self.w.abs() + len(self.w) * 2 * F32 * (size @ self.w.abs()))
            self.close(dx[self.rows], want, err)
            assert (dx[~self.scored] == 0).all()
        if dw is not None:
            want = f * g.T @ self.x
            err = abs(f) * (g_err.T @ self.x.abs() + (len(self.rows) + 64) * 2 * F32 * (size.T @ self.x.abs()))
            self.close(dw, want, err)

    @staticmethod
    def close(got, want, err):
        bad = ~((got.double() - want).abs() <= err * (1 + BF) + (BF + 4 * F32) * want.abs() + SMALLEST)
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first at {torch.nonzero(bad)[0].tolist()}"


SHAPES = [(1, 1, 8), (1, 300, 64), (2, 257, 72), (33, 1000, 200), (64, 129, 1032), (129, 513, 256), (256, 256, 512),
          (257, 1111, 136), (300, 2049, 520), (513, 777, 1024), (1030, 3001, 328)]


@pytest.mark.parametrize("M,V,D", SHAPES)
@pytest.mark.parametrize("ignored", [0.0, 0.4, 1.0])
def test_loss_and_gradients(cuda_lib, M, V, D, ignored):
    for index, alpha in (("i64", 1.0), ("i32", -0.7)):
        x, w, t = inputs(M, V, D, ignored, seed=M + V, index=index)
        ref = Reference(x, w, t, torch.tensor(alpha, dtype=torch.float32).double().item())
        loss, lse, mean = forward(cuda_lib, x, w, t, alpha)
        ref.check_forward(loss, lse, mean)
        dx, dw = backward(cuda_lib, x, w, t, lse, alpha)
        ref.check_backward(dx, dw)


@pytest.mark.parametrize("M,V,D", [(5, 40000, 64), (700, 20000, 128), (2500, 70001, 64), (2500, 53256, 64), (40, 33000, 2048)])
def test_large_vocabularies(cuda_lib, M, V, D):
    """Many column tiles, several pieces of the backward pass (the last one
    shorter than the split sums of dx), split sums of dx."""
    x, w, t = inputs(M, V, D, 0.2, seed=V)
    ref = Reference(x, w, t, 1.0)
    loss, lse, mean = forward(cuda_lib, x, w, t)
    ref.check_forward(loss, lse, mean)
    dx, dw = backward(cuda_lib, x, w, t, lse)
    ref.check_backward(dx, dw)
    again = backward(cuda_lib, x, w, t, lse)  # the same bits on every run
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_weights_of_the_losses_and_their_sum(cuda_lib):
    x, w, t = inputs(200, 1500, 264, 0.3, seed=11)
    ref = Reference(x, w, t, 1.0)
    loss, lse, _ = forward(cuda_lib, x, w, t, with_mean=False)
    dloss = torch.randn(200, device="cuda")
    dloss[3:40] = 0
    dx, dw = backward(cuda_lib, x, w, t, lse, scale=0.5, reduction="sum", dloss=dloss)
    ref.check_backward(dx, dw, scale=0.5, reduction="sum", dloss=dloss)


def test_either_gradient_alone(cuda_lib):
    x, w, t = inputs(300, 900, 136, 0.3, seed=12)
    _, lse, _ = forward(cuda_lib, x, w, t)
    dx, dw = backward(cuda_lib, x, w, t, lse)
    only_x, none = backward(cuda_lib, x, w, t, lse, want=("dx",))
    assert none is None and torch.equal(dx, only_x)
    none, only_w = backward(cuda_lib, x, w, t, lse, want=("dw",))
    assert none is None and torch.equal(dw, only_w)


def test_rows_that_are_not_scored_may_hold_anything(cuda_lib):
    x, w, t = inputs(333, 700, 136, 0.5, seed=13)
    skipped = (t < 0) | (t >= 700)
    loss, lse, mean = forward(cuda_lib, x, w, t)
    dx, dw = backward(cuda_lib, x, w, t, lse)
    x[skipped] = float("nan")
    x[skipped.nonzero()[0, 0]] = float("inf")
    loss2, lse2, mean2 = forward(cuda_lib, x, w, t)
    dloss = torch.where(skipped, float("nan"), 1.0)
    dx2, dw2 = backward(cuda_lib, x, w, t, lse2, dloss=dloss)
    for a, b in ((loss, loss2), (lse, lse2), (mean, mean2), (dx, dx2), (dw, dw2)):
        assert torch.equal(a, b)


def test_a_nan_in_a_scored_row_stays_in_it(cuda_lib):
    x, w, t = inputs(300, 700, 136, 0.0, seed=14)
    loss, lse, _ = forward(cuda_lib, x, w, t)
    x[77, 5] = float("nan")
    loss2, lse2, mean2 = forward(cuda_lib, x, w, t)
    others = torch.arange(300, device="cuda") != 77
    assert torch.isnan(loss2[77]) and torch.isnan(lse2[77]) and torch.isnan(mean2)
    assert torch.equal(loss[others], loss2[others]) and torch.equal(lse[others], lse2[others])


def test_large_logits_do_not_overflow(cuda_lib):
    """Logits in the thousands: confident rows with losses of 0 and of thousands."""
    x, w, t = inputs(130, 600, 64, 0.0, seed=15, spread=400.0)
    ref = Reference(x, w, t, 1.0)
    loss, lse, mean = forward(cuda_lib, x, w, t)
    ref.check_forward(loss, lse, mean)
    dx, dw = backward(cuda_lib, x, w, t, lse)
    ref.check_backward(dx, dw)


def test_gradients_match_differences_of_the_loss(cuda_lib):
    """Central differences of the summed loss in single values.  The loss is
    smooth: the quotient's own error is at most h^2 / 6 times the third
    derivative, under 0.1 |s|^3 for a slope s of the logits; the losses of a few
    rows are each off by at most their tolerance."""
    M, V, D, h = 6, 40, 16, 2.0 ** -4
    x, w, t = inputs(M, V, D, 0.0, seed=16, spread=1.0)
    x = (x * 16).round().clamp(-32, 32).div(16).bfloat16()
    w = (w * 16).round().clamp(-32, 32).div(16).bfloat16()  # values whose neighbours at h are bf16 too
    ref = Reference(x, w, t, 1.0)
    _, lse, _ = forward(cuda_lib, x, w, t)
    dx, dw = backward(cuda_lib, x, w, t, lse, reduction="sum")
    noise = 2 * float(ref.loss_tol.sum()) * 2 / (2 * h)
    for which, grad, slope in ((x, dx, float(w.abs().max())), (w, dw, float(x.abs().max()))):
        for at in [(0, 0), (3, 7), (5, 15), (2, 9)]:
            keep = which[at].clone()
            which[at] = keep + h
            up = forward(cuda_lib, x, w, t)[0].double().sum()
            which[at] = keep - h
            down = forward(cuda_lib, x, w, t)[0].double().sum()
            which[at] = keep
            quotient = float((up - down) / (2 * h))
            tol = noise + M * h * h / 6 * 0.1 * slope ** 3 + 3 * BF * (abs(quotient) + slope)
            assert abs(float(grad[at]) - quotient) <= tol


def test_on_another_stream_and_in_a_graph(cuda_lib):
    M, V, D = 300, 5000, 128
    x, w, t = inputs(M, V, D, 0.3, seed=17)
    loss, lse, mean = forward(cuda_lib, x, w, t)
    dx, dw = backward(cuda_lib, x, w, t, lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        loss2, lse2, mean2 = forward(cuda_lib, x, w, t, stream=side)
    side.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(mean, mean2)
    n = max(cuda_lib.gbf_workspace_size(op, M, V, D, True) for op in ("linear_ce", "linear_ce_grad"))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    loss3, lse3, mean3 = torch.empty_like(loss), torch.empty_like(lse), torch.empty_like(mean)
    dx3, dw3 = torch.empty_like(dx), torch.empty_like(dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.linear_ce(x, w, t, loss3, lse3, mean3, M, V, D, workspace=ws, workspace_bytes=n)
        cuda_lib.linear_ce_grad(x, w, t, lse3, None, dx3, dw3, M, V, D, workspace=ws, workspace_bytes=n)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in ((loss, loss3), (lse, lse3), (mean, mean3), (dx, dx3), (dw, dw3)):
        assert torch.equal(a, b)
    t.fill_(-100)  # the graph sees the new targets: nothing is scored
    graph.replay()
    torch.cuda.synchronize()
    assert (loss3 == 0).all() and float(mean3) == 0 and (dx3 == 0).all() and (dw3 == 0).all()


def test_no_rows(cuda_lib):
    x, w, t = inputs(8, 64, 16, 0.0, seed=18)
    mean = torch.full((1,), 5.0, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    cuda_lib.linear_ce(x, w, t, mean, mean, mean, 0, 64, 16, workspace=ws, workspace_bytes=1 << 20)
    assert float(mean) == 0
    dw = torch.full((64, 16), 3.0, device="cuda", dtype=torch.bfloat16)
    cuda_lib.linear_ce_grad(x, w, t, mean, None, None, dw, 0, 64, 16, workspace=ws, workspace_bytes=1 << 20)
    assert (dw == 0).all()


def test_a_wait_that_runs_out_is_reported(cuda_lib):
    """The commit of the first tile is left out: the ending's bounded wait gives up."""
    x, w, t = inputs(64, 300, 64, 0.0, seed=19)
    loss, lse, _ = forward(cuda_lib, x, w, t)
    n = cuda_lib.gbf_workspace_size("linear_ce", 64, 300, 64, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(loss)
    try:
        cuda_lib.gbf_set_wait_timeout_ns(20_000_000)
        cuda_lib.gbf_debug_inject_timeout(True)
        cuda_lib.linear_ce(x, w, t, out, out, None, 64, 300, 64, workspace=ws, workspace_bytes=n)
        assert cuda_lib.gbf_check_device_error() == 6
    finally:
        cuda_lib.gbf_debug_inject_timeout(False)
        cuda_lib.gbf_set_wait_timeout_ns(2_000_000_000)
    again, _, _ = forward(cuda_lib, x, w, t)
    assert torch.equal(loss, again)


@pytest.mark.parametrize("M", [15, 16, 17, 63, 65, 127, 128, 130])
@pytest.mark.parametrize("V,D", [(900, 64), (5003, 72), (1280, 2056)])
def test_few_rows(cuda_lib, M, V, D):
    for ignored in (0.0, 0.5):
        x, w, t = inputs(M, V, D, ignored, seed=M * V)
        ref = Reference(x, w, t, 1.0)
        loss, lse, mean = forward(cuda_lib, x, w, t)
        ref.check_forward(loss, lse, mean)
        dx, dw = backward(cuda_lib, x, w, t, lse)
        ref.check_backward(dx, dw)


@pytest.mark.parametrize("M,V,D", [(200, 30000, 640), (256, 20011, 968), (40, 6000, 1032), (100, 9001, 64)])
def test_lone_row_tiles_of_short_products_again_and_again(cuda_lib, M, V, D):
    """Up to 256 rows, whose column tiles two issuers take in turn or share by K
    blocks, over many tiles per CTA pair, call after call without a wait between."""
    x, w, t = inputs(M, V, D, 0.1, seed=M + D)
    ref = Reference(x, w, t, 1.0)
    loss, lse, mean = forward(cuda_lib, x, w, t)
    ref.check_forward(loss, lse, mean)
    dx, dw = backward(cuda_lib, x, w, t, lse)
    ref.check_backward(dx, dw)
    n = max(cuda_lib.gbf_workspace_size(op, M, V, D, True) for op in ("linear_ce", "linear_ce_grad"))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = [[torch.empty_like(a) for a in (loss, lse, mean, dx, dw)] for _ in range(12)]
    for o in outs:
        cuda_lib.linear_ce(x, w, t, o[0], o[1], o[2], M, V, D, workspace=ws, workspace_bytes=n)
        cuda_lib.linear_ce_grad(x, w, t, o[1], None, o[3], o[4], M, V, D, workspace=ws, workspace_bytes=n)
    assert cuda_lib.gbf_check_device_error() == 0
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, (loss, lse, mean, dx, dw)))


@pytest.mark.parametrize("M", [3, 40, 100, 200, 300])
def test_wide_hidden_states(cuda_lib, M):
    """K over 4096: more sums per tile."""
    x, w, t = inputs(M, 700, 4104, 0.2, seed=M)
    ref = Reference(x, w, t, 1.0)
    loss, lse, mean = forward(cuda_lib, x, w, t)
    ref.check_forward(loss, lse, mean)
    dx, dw = backward(cuda_lib, x, w, t, lse)
    ref.check_backward(dx, dw)
