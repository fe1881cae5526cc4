"""The gated block that is trained, and its gradients, over several rounds of units per CTA
pair: accumulators and ring go on from one unit to the next, row tiles end inside one."""
import pytest
import torch

from test_mlp_paths import GRAD_ROUNDS, ROUNDS
from test_mlp_train_gpu import backward, check_backward, check_forward, forward, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,D,F,path", ROUNDS)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_forward(cuda_lib, M, D, F, path, act):
    assert cuda_lib.gbf_debug_mlp_path(M, D, F)[0] == path
    t, residual, _ = inputs(M, D, F, seed=M + D + F)
    got = forward(cuda_lib, t, residual, act, M, D, F)
    check_forward(t, residual, got, act, D, F)
    again = forward(cuda_lib, t, residual, act, M, D, F)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert cuda_lib.gbf_check_device_error() == 0


@pytest.mark.parametrize("M,D,F,path", [ROUNDS[1], ROUNDS[4]])
@pytest.mark.parametrize("act", ["relu", "identity"])
def test_other_gates(cuda_lib, M, D, F, path, act):
    t, _, _ = inputs(M, D, F, seed=2)
    check_forward(t, None, forward(cuda_lib, t, None, act, M, D, F), act, D, F)


@pytest.mark.parametrize("M,D,F,path", GRAD_ROUNDS + [ROUNDS[1], ROUNDS[5]])
def test_gradients(cuda_lib, M, D, F, path):
    t, residual, dout = inputs(M, D, F, seed=M + D + F)
    got = forward(cuda_lib, t, residual, "silu", M, D, F)
    check_backward(t, got[1:], dout, backward(cuda_lib, t, got[1:], dout, "silu", M, D, F), "silu", M, D, F)
    assert cuda_lib.gbf_check_device_error() == 0


@pytest.mark.parametrize("M,D,F,path", [ROUNDS[0], ROUNDS[2], ROUNDS[3], ROUNDS[5]])
def test_nothing_outside_is_written(cuda_lib, M, D, F, path):
    t, residual, _ = inputs(M, D, F, seed=3)
    want = forward(cuda_lib, t, residual, "silu", M, D, F)
    shapes = dict(out=(M, D), g=(M, F), u=(M, F), h=(M, F))
    flat = {k: torch.full((a * b + 512,), 7.0, device="cuda", dtype=torch.bfloat16) for k, (a, b) in shapes.items()}
    v = {k: f[256:-256].view(shapes[k]) for k, f in flat.items()}
    cuda_lib.mlp_train(**t, residual=residual, **v, M=M, D=D, F=F)
    assert all(bool((f[:256] == 7.0).all()) and bool((f[-256:] == 7.0).all()) for f in flat.values())
    assert all(torch.equal(v[k], w) for k, w in zip(shapes, want))


@pytest.mark.parametrize("M,D,F,path", [ROUNDS[1], ROUNDS[3]])
def test_a_wait_that_runs_out_is_reported(cuda_lib, M, D, F, path):
    t, residual, _ = inputs(M, D, F, seed=4)
    want = forward(cuda_lib, t, residual, "silu", M, D, F)
    try:
        cuda_lib.gbf_set_wait_timeout_ns(20_000_000)
        cuda_lib.gbf_debug_inject_timeout(True)
        forward(cuda_lib, t, residual, "silu", M, D, F)
        assert cuda_lib.gbf_check_device_error() == 6
    finally:
        cuda_lib.gbf_debug_inject_timeout(False)
        cuda_lib.gbf_set_wait_timeout_ns(2_000_000_000)
    assert all(torch.equal(a, b) for a, b in zip(forward(cuda_lib, t, residual, "silu", M, D, F), want))
    assert cuda_lib.gbf_check_device_error() == 0
