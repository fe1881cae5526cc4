"""Calls of fewer rows in a workspace that was made for the most, and of fewer gradients
in a smaller one: the results of workspaces of their own, nothing written behind."""
import pytest
import torch

import test_linear_distill_gpu as distill
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


@pytest.mark.parametrize("V,D,K,most", [(600, 4104, 20, 1000), (3000, 64, 5, 300), (40001, 264, 20, 700), (1000, 2056, 8, 130)])
def test_distillation_of_fewer_rows(cuda_lib, V, D, K, most):
    """Also of hard targets: the two losses share their passes and their workspace."""
    ws = {g: guarded(cuda_lib.linear_distill_workspace_size(most, V, D, K, g)) for g in (False, True)}
    hard = {g: guarded(cuda_lib.gbf_workspace_size(op, most, V, D, True)) for g, op in ((False, "linear_ce"), (True, "linear_ce_grad"))}
    for M in sorted({1, 16, 17, 64, 65, 128, min(129, most), min(257, most), most}):
        args = distill.inputs(M, V, D, K, seed=M, unscored=0.2)
        loss, lse, mean = distill.forward(cuda_lib, *args)
        want = (loss, lse, mean, *distill.backward(cuda_lib, *args, lse))
        out = [torch.full_like(t, float("nan")) for t in want]
        size, kinds = distill.sizes(*args)
        cuda_lib.linear_distill(*args, *out[:3], *size, **kinds, workspace=ws[False], workspace_bytes=ws[False].numel() - 256)
        cuda_lib.linear_distill_grad(*args, out[1], None, *out[3:], *size, **kinds, workspace=ws[True],
                                     workspace_bytes=ws[True].numel() - 256)
        assert all(torch.equal(a, b) for a, b in zip(out, want)), M
        x, w, ids, _ = args
        t = ids[:, 0].contiguous()
        ends = [torch.full_like(v, float("nan")) for v in want]
        for k, o in enumerate((out, ends)):  # once in a workspace of its own
            n = [h.numel() - 256 if k else cuda_lib.gbf_workspace_size(op, M, V, D, True)
                 for h, op in zip(hard.values(), ("linear_ce", "linear_ce_grad"))]
            b = list(hard.values()) if k else [guarded(s) for s in n]
            cuda_lib.linear_ce(x, w, t, *o[:3], M, V, D, workspace=b[0], workspace_bytes=n[0])
            cuda_lib.linear_ce_grad(x, w, t, o[1], None, *o[3:], M, V, D, workspace=b[1], workspace_bytes=n[1])
        assert all(torch.equal(a, b) for a, b in zip(out, ends)), M
    assert all(bool((b[-256:] == 0x55).all()) for b in (*ws.values(), *hard.values()))
    assert cuda_lib.gbf_check_device_error() == 0


@pytest.mark.parametrize("V,D,most", [(3000, 4096, 5000), (3000, 1024, 20000)])
def test_embedding_grad_of_fewer_positions(cuda_lib, V, D, most):
    n = cuda_lib.gbf_workspace_size("embedding_grad", most, V, D, True)
    for M in (1, 1024, 1025, most // 2 - 60, most // 2, most):
        gen = torch.Generator(device="cuda").manual_seed(M)
        ids = torch.randint(0, V, (M,), generator=gen, device="cuda")
        dout = torch.randn(M, D, generator=gen, device="cuda").bfloat16()
        out = [torch.full((V, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        for o, b in zip(out, (n, cuda_lib.gbf_workspace_size("embedding_grad", M, V, D, True))):
            ws = guarded(b)
            cuda_lib.embedding_grad(ids, dout, o, M, V, D, workspace=ws, workspace_bytes=b)
            assert bool((ws[b:] == 0x55).all())
        assert torch.equal(*out)
