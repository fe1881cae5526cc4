"""Refusals of the distillation entry points: found on the host, before any launch
and without a GPU."""
import math

import pytest

import tcgen05_tmem_bf16_gb300 as gbf

INVALID, MISALIGNED, SHAPE, WORKSPACE = 1, 2, 3, 4
P = 0x10000  # an address that is never followed


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tcgen05_tmem_bf16_gb300 import build
    build.build()
    return gbf.load()


BAD = [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(ids=None), INVALID), (dict(logits=None), INVALID),
    (dict(M=-1), INVALID), (dict(K=-1), INVALID), (dict(alpha=math.inf), INVALID), (dict(alpha=math.nan), INVALID),
    (dict(beta=0.0), INVALID), (dict(beta=-1.0), INVALID), (dict(beta=math.inf), INVALID), (dict(beta=math.nan), INVALID),
    (dict(index_type=2), INVALID), (dict(teacher_type=2), INVALID), (dict(lse=None), INVALID),
    (dict(x=P + 8), MISALIGNED), (dict(w=P + 8), MISALIGNED), (dict(ids=P + 4), MISALIGNED), (dict(logits=P + 2), MISALIGNED),
    (dict(logits=P + 1, teacher_type="bf16"), MISALIGNED), (dict(lse=P + 2), MISALIGNED), (dict(workspace=P + 8), MISALIGNED),
    (dict(K=0), SHAPE), (dict(K=1025), SHAPE), (dict(D=12), SHAPE), (dict(D=0), SHAPE), (dict(V=0), SHAPE),
    (dict(M=2 ** 24 + 1), SHAPE), (dict(V=2 ** 26 + 1), SHAPE), (dict(D=2 ** 20 + 8), SHAPE), (dict(M=2 ** 24, V=2 ** 26), SHAPE),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=-1), WORKSPACE)]


def call(fn, change, grad, **more):
    need = gbf.linear_distill_workspace_size(4, 10, 16, 3, grad)
    args = {**dict(x=P, w=P, ids=P, logits=P, lse=P, M=4, V=10, D=16, K=3, workspace=P, workspace_bytes=need), **more, **change}
    if args["workspace_bytes"] == -1:
        args["workspace_bytes"] = need - 1
    return fn(**args, stream=0, raise_on_error=False)


@pytest.mark.parametrize("change,want", BAD + [(dict(loss=None), INVALID), (dict(loss=P + 1), MISALIGNED), (dict(mean=P + 2), MISALIGNED)])
def test_linear_distill_refuses(change, want):
    assert call(gbf.linear_distill, change, False, loss=P, mean=None) == want


@pytest.mark.parametrize("change,want", BAD + [
    (dict(dx=None, dw=None), INVALID), (dict(reduction=2), INVALID), (dict(dx=P + 8), MISALIGNED), (dict(dw=P + 8), MISALIGNED),
    (dict(dloss=P + 2), MISALIGNED)])
def test_linear_distill_grad_refuses(change, want):
    assert call(gbf.linear_distill_grad, change, True, dloss=None, dx=P, dw=P) == want


def test_workspace_sizes():
    size = gbf.linear_distill_workspace_size
    assert size(4, 10, 16, 0, False) == 0 and size(4, 10, 16, 1025, False) == 0 and size(4, 10, 12, 3, True) == 0  # refused
    assert size(-1, 10, 16, 3, False) == 0
    for grad, op in ((False, "linear_ce"), (True, "linear_ce_grad")):
        assert size(300, 1000, 64, 20, grad) >= gbf.gbf_workspace_size(op, 300, 1000, 64, True) + 300 * 21 * 8
