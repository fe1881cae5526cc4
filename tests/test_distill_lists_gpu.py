"""Distillation's lists and scored rows where calls follow one another through one workspace."""
import pytest
import torch

from test_linear_distill_gpu import backward, forward, inputs, sizes, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,V,D,K", [(1, 4000, 256, 40), (33, 3000, 136, 100), (100, 2000, 64, 300)])
def test_other_lists_at_the_same_addresses(cuda_lib, M, V, D, K):
    """The pass over few rows is resident while its lists are written.  Calls with other
    lists and no wait between them, each through the workspace that holds the lists of the
    call before, give the bits of calls with workspaces of their own."""
    many = [inputs(M, V, D, K, seed=s, holes=0.1 * s) for s in range(4)]
    want = []
    for args in many:
        loss, lse, mean = forward(cuda_lib, *args)
        want.append((loss, lse, mean, *backward(cuda_lib, *args, lse)))
    size, kinds = sizes(*many[0])
    ws = {g: workspace(cuda_lib, size, g) for g in (False, True)}
    got = [[torch.empty_like(t) for t in w] for w in want for _ in range(8)]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        args = many[i * 3 % 4]
        cuda_lib.linear_distill(*args, *out[:3], *size, **kinds, **ws[False])
        cuda_lib.linear_distill_grad(*args, out[1], None, *out[3:], *size, **kinds, **ws[True])
    for i, out in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(out, want[i * 3 % 4])), i
    assert cuda_lib.gbf_check_device_error() == 0


@pytest.mark.parametrize("M,V,D,K", [(20, 3000, 64, 5), (128, 1000, 64, 20), (700, 2000, 136, 20)])
def test_other_scored_rows_at_the_same_addresses(cuda_lib, M, V, D, K):
    """The same where each call scores other rows, which the kernel that lists the rows
    finds in what the one before it has just written."""
    many = [inputs(M, V, D, K, seed=s, unscored=0.3 * s) for s in range(4)]
    want = []
    for args in many:
        loss, lse, mean = forward(cuda_lib, *args)
        want.append((loss, lse, mean, *backward(cuda_lib, *args, lse)))
    size, kinds = sizes(*many[0])
    ws = {g: workspace(cuda_lib, size, g) for g in (False, True)}
    got = [[torch.empty_like(t) for t in w] for w in want for _ in range(8)]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        args = many[i * 3 % 4]
        cuda_lib.linear_distill(*args, *out[:3], *size, **kinds, **ws[False])
        cuda_lib.linear_distill_grad(*args, out[1], None, *out[3:], *size, **kinds, **ws[True])
    for i, out in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(out, want[i * 3 % 4])), i
    assert cuda_lib.gbf_check_device_error() == 0
