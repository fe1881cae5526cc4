"""Refusals of the gated block's and the norm's training entry points: argument
errors are found on the host, before any launch and without a GPU."""
import math

import pytest

import tcgen05_tmem_bf16_gb300 as gbf

INVALID, MISALIGNED, SHAPE, WORKSPACE = 1, 2, 3, 4
P = 0x10000  # an address that is never followed
ACTS = (-1, 4)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tcgen05_tmem_bf16_gb300 import build
    build.build()
    return gbf.load()


SIZES = [
    (dict(M=-1), INVALID), (dict(D=-8), INVALID), (dict(F=-8), INVALID), (dict(act=-1), INVALID), (dict(act=4), INVALID),
    (dict(D=12), SHAPE), (dict(F=20), SHAPE), (dict(D=0), SHAPE), (dict(F=0), SHAPE), (dict(M=2 ** 24 + 1), SHAPE),
    (dict(D=2 ** 20 + 8), SHAPE), (dict(F=2 ** 20 + 8), SHAPE), (dict(M=2 ** 24, F=2 ** 20), SHAPE)]
TRAIN = ("x", "w_gate", "w_up", "w_down", "out", "g", "u", "h")
GRAD = ("dout", "x", "g", "u", "h", "w_gate", "w_up", "w_down")
GRADS = ("dx", "dw_gate", "dw_up", "dw_down")


@pytest.mark.parametrize("change,want", SIZES + [({n: None}, INVALID) for n in TRAIN]
                         + [({n: P + 8}, MISALIGNED) for n in TRAIN + ("residual",)])
def test_mlp_train_refuses(change, want):
    args = dict({n: P for n in TRAIN}, residual=None, M=4, D=16, F=24)
    assert gbf.mlp_train(**{**args, **change}, stream=0, raise_on_error=False) == want


@pytest.mark.parametrize("change,want", SIZES + [({n: None}, INVALID) for n in GRAD]
                         + [({n: P + 8}, MISALIGNED) for n in GRAD + GRADS + ("workspace",)]
                         + [({n: None for n in GRADS}, INVALID), (dict(workspace=None), WORKSPACE),
                            (dict(workspace_bytes=64), WORKSPACE)])
def test_mlp_grad_refuses(change, want):
    need = gbf.gbf_workspace_size("mlp_grad", 4, 16, 24, True)
    args = dict({n: P for n in GRAD + GRADS}, M=4, D=16, F=24, workspace=P, workspace_bytes=need)
    assert gbf.mlp_grad(**{**args, **change}, stream=0, raise_on_error=False) == want


@pytest.mark.parametrize("change,want", [
    (dict(dnorm=None), INVALID), (dict(resid=None), INVALID), (dict(weight=None), INVALID), (dict(dr=None), INVALID),
    (dict(M=-1), INVALID), (dict(N=-8), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(dnorm=P + 8), MISALIGNED), (dict(dresid=P + 8), MISALIGNED), (dict(resid=P + 8), MISALIGNED),
    (dict(weight=P + 8), MISALIGNED), (dict(dr=P + 8), MISALIGNED), (dict(dweight=P + 8), MISALIGNED),
    (dict(workspace=P + 8), MISALIGNED), (dict(N=12), SHAPE), (dict(N=16392), SHAPE), (dict(M=2 ** 31), SHAPE),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=64), WORKSPACE)])
def test_add_rmsnorm_grad_refuses(change, want):
    need = gbf.gbf_workspace_size("add_rmsnorm_grad", 4, 64, 0, True)
    args = dict(dnorm=P, dresid=P, resid=P, weight=P, dr=P, dweight=P, M=4, N=64, workspace=P, workspace_bytes=need)
    assert gbf.add_rmsnorm_grad(**{**args, **change}, stream=0, raise_on_error=False) == want


def test_workspace_sizes():
    small, large = (gbf.gbf_workspace_size("mlp_grad", m, 4096, 14336, True) for m in (1, 4096))
    assert 2 * 2 * 14336 <= small < large and large >= 2 * 2 * 4096 * 14336
    assert gbf.gbf_workspace_size("mlp_grad", 4, 12, 24, True) == 0  # refused
    assert gbf.gbf_workspace_size("add_rmsnorm_grad", 4, 64, 0, True) == 4 * 64 * 4
    assert gbf.gbf_workspace_size("add_rmsnorm_grad", 0, 64, 0, True) == 0
    assert gbf.gbf_workspace_size("add_rmsnorm_grad", 4, 16392, 0, True) == 0
