"""The gradient of add + RMSNorm of rows whose values are tiny: s = 1 / rms(r) is held by
fp32, its square is not.

Tolerance, beside those of the other tests (R = 2^-8 of a value, 2^-17 of the terms'
magnitudes): the mean of r^2 is a subnormal, rounded by at most 2^-150 of 1e-40 or more,
2^-17.1 of itself, s by half of that and its third power by 1.5 times: 2^-16 of the terms
together holds both."""
import pytest
import torch

from test_rmsnorm_grad_gpu import R, call, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [264, 1000, 2048, 4096, 8192, 16384])
@pytest.mark.parametrize("rms", [1e-15, 4e-20, 1e-20])
def test_tiny_rows(cuda_lib, N, rms):
    M = 40
    dn, dres, r, w = inputs(M, N, seed=N)
    r = (r.float() * (rms / 3.0)).bfloat16()
    dr, dw = call(cuda_lib, dn, dres, r, w, M, N, eps=0.0)
    dn, r, w = dn.double(), r.double(), w.double()
    s = 1.0 / r.square().mean(dim=1, keepdim=True).sqrt()
    lead, back = s * dn * w, r * s ** 3 * (dn * w * r).mean(dim=1, keepdim=True)
    want = lead - back + dres.double()
    size = lead.abs() + dres.double().abs() + r.abs() * s ** 3 * (dn * w * r).abs().mean(dim=1, keepdim=True)
    err = (dr.double() - want).abs()
    assert bool((err <= R * want.abs() + 2.0 ** -16 * size).all())
    terms = dn * r * s
    err, want = (dw.double() - terms.sum(dim=0)).abs(), terms.sum(dim=0).abs()
    assert bool((err <= R * want + (2.0 ** -16 + M * 2.0 ** -24) * terms.abs().sum(dim=0)).all())
