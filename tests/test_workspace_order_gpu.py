"""Calls of fewer rows in a workspace that was made for the most, and of fewer gradients
in a smaller one: the results of workspaces of their own, nothing written behind."""
import pytest
import torch

from test_mlp_train_gpu import backward, forward, inputs

pytestmark = pytest.mark.gpu


def guarded(n):
    return torch.full((n + 256,), 0x55, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("D,F,most", [(64, 2048, 1000), (1024, 4096, 1000), (520, 1032, 700), (256, 8192, 2000)])
def test_mlp_grad_of_fewer_rows(cuda_lib, D, F, most):
    n = cuda_lib.gbf_workspace_size("mlp_grad", most, D, F, True)
    for M in sorted({1, 16, 129, 256, 257, 513, most // 2, most}):
        t, residual, dout = inputs(M, D, F, seed=M)
        kept = forward(cuda_lib, t, residual, "silu", M, D, F)[1:]
        want = backward(cuda_lib, t, kept, dout, "silu", M, D, F)
        got = {k: torch.full_like(v, float("nan")) for k, v in want.items()}
        ws = guarded(n)
        cuda_lib.mlp_grad(dout, t["x"], *kept, t["w_gate"], t["w_up"], t["w_down"], **got, M=M, D=D, F=F, workspace=ws,
                          workspace_bytes=n)
        assert all(torch.equal(got[k], want[k]) for k in want), M
        assert bool((ws[n:] == 0x55).all())
    assert cuda_lib.gbf_check_device_error() == 0


@pytest.mark.parametrize("M", [16, 200, 300, 1000])
def test_mlp_grad_without_dx(cuda_lib, M):
    D, F = 264, 1032
    t, residual, dout = inputs(M, D, F, seed=M)
    kept = forward(cuda_lib, t, residual, "silu", M, D, F)[1:]
    want = backward(cuda_lib, t, kept, dout, "silu", M, D, F)
    n = 2 * ((2 * M * F + 255) // 256 * 256)
    ws = guarded(n)
    got = {k: torch.full_like(v, float("nan")) for k, v in want.items()}
    args = (dout, t["x"], *kept, t["w_gate"], t["w_up"], t["w_down"], None)
    cuda_lib.mlp_grad(*args, got["dw_gate"], got["dw_up"], got["dw_down"], M, D, F, workspace=ws, workspace_bytes=n)
    assert all(torch.equal(got[k], want[k]) for k in ("dw_gate", "dw_up", "dw_down"))
    assert bool((ws[n:] == 0x55).all())
    assert cuda_lib.mlp_grad(*args, got["dw_gate"], None, None, M, D, F, workspace=ws, workspace_bytes=n - 1,
                             raise_on_error=False) == 4
    only = torch.full_like(want["dw_down"], float("nan"))
    cuda_lib.mlp_grad(*args, None, None, only, M, D, F)
    assert torch.equal(only, want["dw_down"])
