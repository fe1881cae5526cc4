"""Results of the linear cross entropy that a bound on any sum of D products
(test_linear_ce_gpu.py) is too wide to see."""
import pytest
import torch

from test_linear_ce_gpu import BF, F32, SMALLEST, backward, forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 16, 60, 120, 200, 300, 600])
@pytest.mark.parametrize("alpha", [1.0, 0.7, -0.3])
def test_confident_rows(cuda_lib, M, alpha):
    """All of the probability on the target: losses under 1e-9, whatever the
    logit.  The loss is a difference of one product with itself, so the errors
    of the products and of their factor are not in it; what is left is the
    rounding of the powers of two (2^-22 for the function, 2^-24 for its value and
    for its logarithm), and it is never below zero."""
    V, D = 700, 4096
    g = torch.Generator(device="cuda").manual_seed(M)
    w = (torch.randn(V, D, generator=g, device="cuda") / D ** 0.5).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    logit = torch.linspace(35.0, 1000.0 if M > 1 else 50.0, M, device="cuda")
    x = (w[t].float() * (logit / alpha)[:, None]).bfloat16()
    exact = alpha * x.double() @ w.double().T
    want = torch.logsumexp(exact, dim=1) - exact[torch.arange(M, device="cuda"), t]
    assert float(want.max()) < 1e-9
    loss, lse, mean = forward(cuda_lib, x, w, t, alpha)
    assert (loss >= 0).all() and float(mean) >= 0
    assert float(loss.max()) <= 2.0 ** -22 + 2 * 2.0 ** -24


# K blocks of 64 products that the tensor cores add up in one chain, 16 products
# per addition; an addition cuts less than a unit in the last place, 2^-23 of the
# running sum.
CHAIN = 1024
ROWS = [1, 16, 64, 100, 200, 300, 600]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("D", [1024, 4096, 65536])
def test_a_sparse_row(cuda_lib, M, D):
    """One value of x other than zero: every logit is one product, an exact one, and
    nothing is cut.  Left are the rounding of the factor 1 / ln 2 (half of 2^-23
    of the largest logit), the powers (2^-22) and their sum (fewer than 128 + V / 128
    additions deep, 2^-24 each)."""
    V = 300
    g = torch.Generator(device="cuda").manual_seed(M + D)
    w = (torch.randn(V, D, generator=g, device="cuda") * 8).bfloat16()
    x = torch.zeros(M, D, device="cuda", dtype=torch.bfloat16)
    each = torch.arange(M, device="cuda")
    at = torch.randint(0, D, (M,), generator=g, device="cuda")
    x[each, at] = torch.where(each % 2 == 0, 1.5, -2.0).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    logits = x[each, at].double()[:, None] * w[:, at].T.double()
    want = torch.logsumexp(logits, dim=1)
    loss, lse, _ = forward(cuda_lib, x, w, t)
    tol = F32 * logits.abs().amax(dim=1) + 2.0 ** -22 + (128 + V / 128) * F32 + F32 * want.abs()
    assert ((lse.double() - want).abs() <= tol).all()
    target = logits[each, t]
    tol = F32 * (want - target) + 2.0 ** -22 + (128 + V / 128) * F32 + F32 * (want - target).abs()
    assert ((loss.double() - (want - target)).abs() <= tol).all()


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("V,D", [(1000, 2048), (1000, 4096), (8000, 4096), (1000, 8192), (700, 65536)])
def test_products_of_random_signs(cuda_lib, M, V, D):
    """The additions of a chain cut 2^-25 of the running sum on average, which is
    half of its end on average: CHAIN / 16 of them take CHAIN 2^-30 of a chain's
    sum, and so of a logit, however many chains it has.  The logits' part in lse and
    in the loss is under one of their size (standard deviation 2, a mean of 4 under
    the softmax, lse of 8.5 and more): both are off by less than CHAIN 2^-30 of
    themselves, taken over the rows; fp32 adds a few 2^-24."""
    g = torch.Generator(device="cuda").manual_seed(V + D + M)
    x = torch.randn(M, D, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, D, generator=g, device="cuda") * 2 / D ** 0.5).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    logits = x.double() @ w.double().T
    want = torch.logsumexp(logits, dim=1)
    want_loss = want - logits[torch.arange(M, device="cuda"), t]
    loss, lse, mean = forward(cuda_lib, x, w, t)
    bound = CHAIN * 2.0 ** -30 + 4 * F32
    assert float((lse.double() - want).norm()) <= bound * float(want.norm())
    assert float((loss.double() - want_loss).norm()) <= bound * float(want_loss.norm())


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("D", [1024, 8192, 65536])
def test_products_of_one_sign(cuda_lib, M, D):
    """Every running sum is under its chain's end, so a chain of CHAIN / 16 additions
    cuts under CHAIN / 16 units of its end, and a logit loses under that share of
    itself; the sum of up to D / CHAIN chains is rounded to fp32 at each step."""
    V = 500
    g = torch.Generator(device="cuda").manual_seed(D + M)
    x = torch.rand(M, D, generator=g, device="cuda").bfloat16()
    w = (torch.rand(V, D, generator=g, device="cuda") * 64 / D).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    logits = x.double() @ w.double().T
    want = torch.logsumexp(logits, dim=1)
    loss, lse, _ = forward(cuda_lib, x, w, t)
    share = CHAIN / 16 * 2 * F32 + (D / CHAIN + 8) * F32
    tol = share * logits.amax(dim=1) + 2.0 ** -22 + (128 + V / 128) * F32 + F32 * want
    assert ((lse.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("M", [16, 64, 100, 200, 300, 600])
@pytest.mark.parametrize("D", [1024, 4096, 8192])
def test_gradients_of_confident_rows(cuda_lib, M, D):
    """All of the probability on the target: dx is (p - 1) w[target] with p = 1, and
    the gradient's own logits have to agree with the lse that the loss left.  p is
    off by what fp32 makes of them: lse is rounded (half of 2^-23 of it), so is its
    product with 1 / ln 2, that factor is for both, and the power (2^-22)."""
    V = 700
    g = torch.Generator(device="cuda").manual_seed(M + D)
    w = (torch.randn(V, D, generator=g, device="cuda") / D ** 0.5).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    size = torch.linspace(40.0, 400.0, M, device="cuda")
    x = (w[t].float() * size[:, None]).bfloat16()
    logits = x.double() @ w.double().T
    want = torch.logsumexp(logits, dim=1) - logits[torch.arange(M, device="cuda"), t]
    assert float(want.max()) < 1e-9
    _, lse, _ = forward(cuda_lib, x, w, t)
    dx, _ = backward(cuda_lib, x, w, t, lse, reduction="sum", want=("dx",))
    off = 4 * F32 * lse.double() + 2.0 ** -22 + 2 * F32  # of p
    others = V * 1e-9 * w.double().abs().amax()
    tol = off[:, None] * w[t].double().abs() * (1 + 2 * BF) + others + SMALLEST
    assert (dx.double().abs() <= tol).all()
