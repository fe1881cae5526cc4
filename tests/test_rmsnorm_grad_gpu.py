"""The gradient of the fused residual add + RMSNorm against a plain fp64 form.

Tolerances.  bf16 rounds by at most R = 2^-8 of a value.  A row's sums are fp32 sums
of chains of at most 32 products and 21 joins: 2^-18 of the sum of their magnitudes;
the operations after them add some 2^-22 of each term: 2^-17 of the terms' magnitudes
is held.  dweight's sum goes over M rows: at most M 2^-24 of the magnitudes beside."""
import pytest
import torch

pytestmark = pytest.mark.gpu

R = 2.0 ** -8


def inputs(M, N, seed=0, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).bfloat16()

    return normal(M, N, std=1e-2), normal(M, N, std=1e-2) if residual else None, normal(M, N, std=3.0), normal(N, std=0.1, mean=1.0)


def call(lib, dn, dres, r, w, M, N, eps=1e-5, dr=None, dweight=True, stream=None):
    dr = torch.full((M, N), float("nan"), device="cuda", dtype=torch.bfloat16) if dr is None else dr
    dw = torch.full((N,), float("nan"), device="cuda", dtype=torch.bfloat16) if dweight else None
    n = lib.gbf_workspace_size("add_rmsnorm_grad", M, N, 0, True)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if dweight else None
    lib.add_rmsnorm_grad(dn, dres, r, w, dr, dw, M, N, eps, ws, n if dweight else 0, stream=stream)
    return dr, dw


def check(got, dn, dres, r, w, eps=1e-5):
    dr, dw = got
    dn, r, w = dn.double(), r.double(), w.double()
    M, N = r.shape
    s = 1.0 / (r.square().mean(dim=1, keepdim=True) + eps).sqrt()
    lead, back = s * dn * w, r * s ** 3 * (dn * w * r).mean(dim=1, keepdim=True)
    want = lead - back
    size = lead.abs() + r.abs() * s ** 3 * (dn * w * r).abs().mean(dim=1, keepdim=True)
    if dres is not None:
        want = want + dres.double()
        size = size + dres.double().abs()
    bound = R * want.abs() + 2.0 ** -17 * size
    err = (dr.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    if dw is None:
        return
    terms = dn * r * s
    want, size = terms.sum(dim=0), terms.abs().sum(dim=0)
    err, bound = (dw.double() - want).abs(), R * want.abs() + (2.0 ** -17 + M * 2.0 ** -24) * size
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("M,N", [(1, 8), (3, 72), (1, 1000), (77, 1000), (700, 1024), (5, 1032), (2000, 2048), (333, 2056),
                                 (1500, 4096), (2, 4104), (900, 8192), (3, 8200), (700, 16384), (1, 16384)])
@pytest.mark.parametrize("residual", [True, False])
def test_against_fp64(cuda_lib, M, N, residual):
    dn, dres, r, w = inputs(M, N, seed=M + N, residual=residual)
    check(call(cuda_lib, dn, dres, r, w, M, N), dn, dres, r, w)


@pytest.mark.parametrize("M,N", [(1, 512), (9, 280), (2500, 512), (6007, 136), (3, 520), (1301, 1000), (2, 1032), (701, 2048),
                                 (400, 12008)])
def test_several_rows_at_a_time_and_staged_rows(cuda_lib, M, N):
    """Short rows, of which a CTA takes 8, 4 or 2 at a time, more than once; long ones."""
    dn, dres, r, w = inputs(M, N, seed=M + N)
    got = call(cuda_lib, dn, dres, r, w, M, N)
    check(got, dn, dres, r, w)
    for k in (0, 1):  # dr in the place of dnorm, of dresid
        args = [dn.clone(), dres.clone()]
        again = call(cuda_lib, *args, r, w, M, N, dr=args[k])
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


def test_of_what_the_forward_stored(cuda_lib):
    """add_rmsnorm, then its gradient of the r it stored, against autograd through the
    unrounded sum: r's rounding moves the result by some R of its terms."""
    M, N = 130, 520
    dn, dres, a, w = inputs(M, N, seed=1)
    x = inputs(M, N, seed=2)[2]
    norm, resid = torch.empty_like(a), torch.empty_like(a)
    cuda_lib.add_rmsnorm(a, x, w, norm, resid, M, N, 1e-5)
    dr, dw = call(cuda_lib, dn, dres, resid, w, M, N)
    check((dr, dw), dn, dres, resid, w)
    s = (a.double() + x.double()).requires_grad_()
    w64 = w.double().requires_grad_()
    torch.autograd.backward(torch.nn.functional.rms_norm(s, (N,), w64, 1e-5), dn.double())
    want = s.grad + dres.double()
    assert float((dr.double() - want).norm() / want.norm()) <= 2 * R
    assert float((dw.double() - w64.grad).norm() / w64.grad.norm()) <= 2 * R


def test_against_differences(cuda_lib):
    """Directions in r and in the weight; the result's roundings along a normal
    direction come to R / sqrt(3) of the gradient's norm: six times that is held."""
    M, N = 20, 136
    dn, _, r, w = inputs(M, N, seed=3)
    dr, dw = call(cuda_lib, dn, None, r, w, M, N)

    def value(r, w):
        return float((r / (r.square().mean(dim=1, keepdim=True) + 1e-5).sqrt() * w * dn.double()).sum())

    g = torch.Generator(device="cuda").manual_seed(1)
    r, w = r.double(), w.double()
    for grad, at in ((dr.double(), 0), (dw.double(), 1)):
        v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        move = lambda e: value(r + e * v, w) if at == 0 else value(r, w + e * v)  # noqa: E731
        diff = (move(1e-5) - move(-1e-5)) / 2e-5
        assert abs(float((grad * v).sum()) - diff) <= 6 * R / 3 ** 0.5 * float(grad.norm())


def test_rows_of_zeros_and_special_values(cuda_lib):
    M, N = 6, 264
    dn, dres, r, w = inputs(M, N, seed=4)
    r[1] = 0.0  # s = 1 / sqrt(eps)
    dn[2] = 0.0  # only the residual's gradient is left
    r[3, 5] = float("nan")
    dr, dw = call(cuda_lib, dn, dres, r, w, M, N)
    assert torch.equal(dr[2], dres[2])
    assert bool(torch.isnan(dr[3]).all()) and bool(torch.isnan(dw).any())
    keep = [0, 1, 2, 4, 5]
    check((dr[keep], None), dn[keep], dres[keep], r[keep], w)
    zero = r[1:2]
    assert bool(torch.isfinite(dr[1]).all())
    check((dr[1:2], None), dn[1:2], dres[1:2], zero, w)


@pytest.mark.parametrize("M,N", [(40, 1000), (1300, 4096)])
def test_in_place_without_dweight_captured_and_on_a_side_stream(cuda_lib, M, N):
    from tcgen05_tmem_bf16_gb300.graphs import CapturedChain
    dn, dres, r, w = inputs(M, N, seed=5)
    dr, dw = call(cuda_lib, dn, dres, r, w, M, N)
    for k in (0, 1):  # dr in the place of dnorm, of dresid
        args = [dn.clone(), dres.clone()]
        got, _ = call(cuda_lib, *args, r, w, M, N, dr=args[k], dweight=False)
        assert torch.equal(got, dr)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(cuda_lib, dn, dres, r, w, M, N)
    torch.cuda.synchronize()
    assert torch.equal(other[0], dr) and torch.equal(other[1], dw)
    out, dw2 = torch.empty_like(dr), torch.empty_like(dw)
    n = cuda_lib.gbf_workspace_size("add_rmsnorm_grad", M, N, 0, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graph = CapturedChain(lambda s: cuda_lib.add_rmsnorm_grad(dn, dres, r, w, out, dw2, M, N, 1e-5, ws, n, stream=s))
    dn2, dres2, r2, w2 = inputs(M, N, seed=6)
    want = call(cuda_lib, dn2, dres2, r2, w2, M, N)
    for a, b in ((dn, dn2), (dres, dres2), (r, r2), (w, w2)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(dw2, want[1])


def test_no_rows_and_no_columns(cuda_lib):
    N = 64
    dw = torch.full((N,), float("nan"), device="cuda", dtype=torch.bfloat16)
    cuda_lib.add_rmsnorm_grad(None, None, None, dw, None, dw, 0, N)
    assert bool((dw == 0).all())
    cuda_lib.add_rmsnorm_grad(None, None, None, None, None, None, 5, 0)


def test_nothing_outside_is_written(cuda_lib):
    M, N = 9, 1000
    dn, dres, r, w = inputs(M, N, seed=7)
    flat = torch.full((M * N + 64,), 7.0, device="cuda", dtype=torch.bfloat16)
    n = cuda_lib.gbf_workspace_size("add_rmsnorm_grad", M, N, 0, True)
    ws = torch.full((n + 64,), 0x55, dtype=torch.uint8, device="cuda")
    dw = torch.full((N + 64,), 7.0, device="cuda", dtype=torch.bfloat16)
    cuda_lib.add_rmsnorm_grad(dn, dres, r, w, flat[32:-32], dw[32:-32], M, N, 1e-5, ws, n)
    assert bool((flat[:32] == 7.0).all()) and bool((flat[-32:] == 7.0).all())
    assert bool((dw[:32] == 7.0).all()) and bool((dw[-32:] == 7.0).all()) and bool((ws[n:] == 0x55).all())
    check((flat[32:-32].view(M, N), dw[32:-32]), dn, dres, r, w)
