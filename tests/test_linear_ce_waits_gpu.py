"""A bounded wait that runs out in each form of the product kernel under the loss
is reported, and the next call is right again."""
import pytest
import torch

from test_linear_ce_gpu import forward, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,D", [(100, 4096), (200, 64), (200, 4096), (300, 64), (300, 4096)])
def test_a_wait_that_runs_out_is_reported(cuda_lib, M, D):
    """The commit of the first tile's last sums is left out: the ending's wait for
    them gives up after 20 ms."""
    V = 300
    x, w, t = inputs(M, V, D, 0.0, seed=M + D)
    loss, lse, _ = forward(cuda_lib, x, w, t)
    n = cuda_lib.gbf_workspace_size("linear_ce", M, V, D, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(loss)
    try:
        cuda_lib.gbf_set_wait_timeout_ns(20_000_000)
        cuda_lib.gbf_debug_inject_timeout(True)
        cuda_lib.linear_ce(x, w, t, out, out, None, M, V, D, workspace=ws, workspace_bytes=n)
        assert cuda_lib.gbf_check_device_error() == 6
    finally:
        cuda_lib.gbf_debug_inject_timeout(False)
        cuda_lib.gbf_set_wait_timeout_ns(2_000_000_000)
    again, _, _ = forward(cuda_lib, x, w, t)
    assert torch.equal(loss, again)
