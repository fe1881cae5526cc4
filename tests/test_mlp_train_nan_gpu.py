"""NaN and infinity in the gate of the block that is trained: they stay where the formula
has them, and nothing else changes (the same bits as without them)."""
import pytest
import torch

from test_mlp_train_gpu import ACTS, backward, forward, inputs

pytestmark = pytest.mark.gpu

# the swapped kernel, the one-SM kernel, CTA pairs with one and with two row tiles per unit
FORWARD = [(16, 264, 520), (1300, 72, 4104), (513, 136, 1032), (1800, 1032, 4104)]
BACKWARD = [(1, 64, 136), (40, 136, 264), (700, 520, 2056), (2500, 136, 2056)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,D,F", FORWARD)
def test_a_nan_in_the_gates_weight(cuda_lib, M, D, F, act):
    t, residual, _ = inputs(M, D, F, seed=1)
    _, g, u, h = forward(cuda_lib, t, residual, act, M, D, F)
    f = F // 2 + 1
    t["w_gate"][f, D // 3] = float("nan")
    out2, g2, u2, h2 = forward(cuda_lib, t, residual, act, M, D, F)
    keep = torch.arange(F, device="cuda") != f
    assert torch.equal(u, u2)
    assert torch.equal(g[:, keep], g2[:, keep]) and torch.equal(h[:, keep], h2[:, keep])
    assert bool(torch.isnan(g2[:, f]).all()) and bool(torch.isnan(h2[:, f]).all()) and bool(torch.isnan(out2).all())


@pytest.mark.parametrize("M,D,F", FORWARD)
def test_infinite_gates_through_relu(cuda_lib, M, D, F):
    t, residual, _ = inputs(M, D, F, seed=2)
    f, k = F - 3, D // 3
    t["w_gate"][f, k] = float("inf")
    t["x"][:, k] = torch.where(torch.arange(M, device="cuda") % 2 == 0, 1.0, -1.0)
    _, g, u, h = forward(cuda_lib, t, residual, "relu", M, D, F)
    even = torch.arange(M, device="cuda") % 2 == 0
    inf = torch.full((M,), float("inf"), device="cuda", dtype=torch.bfloat16)
    assert torch.equal(g[:, f], torch.where(even, inf, -inf))
    assert torch.equal(h[:, f], torch.where(even, inf * u[:, f].sign(), torch.zeros_like(inf)))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,D,F", BACKWARD)
def test_a_nan_in_the_kept_gate(cuda_lib, M, D, F, act):
    t, residual, dout = inputs(M, D, F, seed=3)
    _, g, u, h = forward(cuda_lib, t, residual, act, M, D, F)
    m, f = M * 2 // 3, F // 3
    g[m, f] = -1.0
    want = backward(cuda_lib, t, (g, u, h), dout, act, M, D, F)
    g[m, f] = float("nan")
    got = backward(cuda_lib, t, (g, u, h), dout, act, M, D, F)
    rows, cols = torch.arange(M, device="cuda") != m, torch.arange(F, device="cuda") != f
    assert bool(torch.isnan(got["dx"][m]).all())
    assert torch.equal(got["dx"][rows], want["dx"][rows]) and torch.equal(got["dw_down"], want["dw_down"])
    for name in ("dw_gate", "dw_up"):
        assert torch.equal(got[name][cols], want[name][cols])
    assert bool(torch.isnan(got["dw_up"][f]).all())
    if act in ("relu", "identity"):  # act' of a NaN: 0, as that of -1; 1
        assert torch.equal(got["dw_gate"][f], want["dw_gate"][f])
    else:
        assert bool(torch.isnan(got["dw_gate"][f]).all())
