"""The loss of a student that has nearly reached its teacher: a small sum of differences
log q + lse - l.  It is off by what lse and l are off by, up to 5e-7 of their magnitudes and
of log q's, and by the relative 2^-21 of the powers and shares: not by a share of itself."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [16, 100, 300])
@pytest.mark.parametrize("V,D,K", [(64, 64, 64), (1000, 64, 1000), (1000, 4096, 1000), (5000, 520, 20)])
@pytest.mark.parametrize("away", [0.0, 1e-3, 1e-2])
def test_small_losses(cuda_lib, M, V, D, K, away):
    gen = torch.Generator(device="cuda").manual_seed(M + V)
    x = torch.randn(M, D, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(V, D, generator=gen, device="cuda") * (2.0 / math.sqrt(D))).bfloat16()
    l = x.double() @ w.double().T
    top, ids = l.topk(K, dim=1)
    logits = (top + away * torch.randn(M, K, generator=gen, device="cuda", dtype=torch.float64)).float()
    n = cuda_lib.linear_distill_workspace_size(M, V, D, K, False)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse, mean = (torch.full((k,), float("nan"), device="cuda") for k in (M, M, 1))
    cuda_lib.linear_distill(x, w, ids.contiguous(), logits, loss, lse, mean, M, V, D, K, workspace=ws, workspace_bytes=n)
    log_q, z = torch.log_softmax(logits.double(), 1), torch.logsumexp(l, 1)
    want = (log_q.exp() * (log_q + z[:, None] - top)).sum(1)
    size = z.abs() + top.abs().amax(1) + log_q.abs().amax(1)
    assert bool((loss >= 0).all())
    err = (loss.double() - want).abs()
    assert bool((err <= 5e-7 * size + 2.0 ** -20 + 2.0 ** -23 * want).all()), float((err / size).max())
    assert abs(float(mean) - float(want.mean())) <= 5e-7 * float(size.max()) + 2.0 ** -20 + 2.0 ** -23 * float(want.max())
