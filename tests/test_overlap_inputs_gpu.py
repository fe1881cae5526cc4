"""Kernels that begin while the one before still writes what they read: a chain of calls
whose inputs are the results of the calls before, at the same addresses again and again,
gives the bits of calls with a wait between them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,V", [(100, 1024, 300), (1000, 512, 2000), (3000, 1032, 2000)])
def test_norms_gradient_then_tables(cuda_lib, M, N, V):
    gen = torch.Generator(device="cuda").manual_seed(M)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").bfloat16()

    ids = torch.randint(-1, V, (M,), generator=gen, device="cuda")
    r, w = normal(M, N), normal(N)
    many = [normal(M, N) for _ in range(4)]
    n = [cuda_lib.gbf_workspace_size("add_rmsnorm_grad", M, N, 0, True), cuda_lib.gbf_workspace_size("embedding_grad", M, V, N, True)]
    ws = [torch.full((b,), 0xFF, dtype=torch.uint8, device="cuda") for b in n]
    dr, dw = torch.empty_like(r), torch.empty_like(w)

    def run(dn, table, wait):
        cuda_lib.add_rmsnorm_grad(dn, None, r, w, dr, dw, M, N, 1e-5, ws[0], n[0])
        if wait:
            torch.cuda.synchronize()
        cuda_lib.embedding_grad(ids, dr, table, M, V, N, workspace=ws[1], workspace_bytes=n[1])

    tables = [torch.empty(V, N, device="cuda", dtype=torch.bfloat16) for _ in range(36)]
    for dn, t in zip(many, tables):
        run(dn, t, True)
    torch.cuda.synchronize()
    for i in range(32):
        run(many[i * 3 % 4], tables[4 + i], False)
    assert all(torch.equal(tables[4 + i], tables[i * 3 % 4]) for i in range(32))
    assert cuda_lib.gbf_check_device_error() == 0


@pytest.mark.parametrize("M,D,F,V", [(64, 264, 520, 1000), (300, 264, 520, 1000)])
def test_block_then_loss(cuda_lib, M, D, F, V):
    gen = torch.Generator(device="cuda").manual_seed(M)

    def normal(*shape):
        return (torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5).bfloat16()

    t = dict(w_gate=normal(F, D), w_up=normal(F, D), w_down=normal(D, F))
    table, many = normal(V, D), [normal(M, D) for _ in range(4)]
    targets = torch.randint(0, V, (M,), generator=gen, device="cuda")
    targets[::3] = -1  # the others' rows are gathered
    out, g, u, h = (torch.empty(M, k, device="cuda", dtype=torch.bfloat16) for k in (D, F, F, F))
    n = [cuda_lib.gbf_workspace_size(op, M, V, D, True) for op in ("linear_ce", "linear_ce_grad")]
    ws = [torch.full((b,), 0xFF, dtype=torch.uint8, device="cuda") for b in n]

    def run(x, res, wait):
        cuda_lib.mlp_train(x, **t, residual=x, out=out, g=g, u=u, h=h, M=M, D=D, F=F)
        if wait:
            torch.cuda.synchronize()
        cuda_lib.linear_ce(out, table, targets, *res[:3], M, V, D, workspace=ws[0], workspace_bytes=n[0])
        cuda_lib.linear_ce_grad(out, table, targets, res[1], None, *res[3:], M, V, D, workspace=ws[1], workspace_bytes=n[1])

    f32 = dict(device="cuda", dtype=torch.float32)
    sets = [[torch.empty(M, **f32), torch.empty(M, **f32), torch.empty(1, **f32), torch.empty_like(out), torch.empty_like(table)]
            for _ in range(36)]
    for x, s in zip(many, sets):
        run(x, s, True)
    torch.cuda.synchronize()
    for i in range(32):
        run(many[i * 3 % 4], sets[4 + i], False)
    for i in range(32):
        assert all(torch.equal(a, b) for a, b in zip(sets[4 + i], sets[i * 3 % 4])), i
    assert cuda_lib.gbf_check_device_error() == 0
