"""Results of the linear cross entropy that a bound on any sum of D products
(test_linear_ce_gpu.py) is too wide to see."""
import pytest
import torch

from test_linear_ce_gpu import forward

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
