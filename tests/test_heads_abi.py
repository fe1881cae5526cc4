"""Refusals of the embedding and clipping entry points: argument errors are
found on the host, before any launch and without a GPU."""
import ctypes
import math

import pytest
import torch

import tcgen05_tmem_bf16_gb300 as gbf

INVALID, MISALIGNED, SHAPE, WORKSPACE = 1, 2, 3, 4
P = 0x10000  # an address that is never followed
MAX = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tcgen05_tmem_bf16_gb300 import build
    build.build()
    return gbf.load()


@pytest.mark.parametrize("change,want", [
    (dict(ids=None), INVALID), (dict(table=None), INVALID), (dict(out=None), INVALID), (dict(M=-1), INVALID),
    (dict(V=-1), INVALID), (dict(D=-8), INVALID), (dict(index_type=2), INVALID), (dict(ids=P + 4), MISALIGNED),
    (dict(ids=P + 2, index_type="i32"), MISALIGNED), (dict(table=P + 8), MISALIGNED), (dict(out=P + 2), MISALIGNED),
    (dict(D=12), SHAPE), (dict(M=MAX + 1), SHAPE), (dict(V=MAX), SHAPE), (dict(M=MAX, D=2048), SHAPE)])
def test_lookup_refuses(change, want):
    args = dict(ids=P, table=P, out=P, M=4, V=10, D=16)
    assert gbf.embedding_lookup(**{**args, **change}, stream=0, raise_on_error=False) == want


@pytest.mark.parametrize("change,want", [
    (dict(ids=None), INVALID), (dict(dout=None), INVALID), (dict(dtable=None), INVALID), (dict(M=-1), INVALID),
    (dict(accumulate=2), INVALID), (dict(index_type=-1), INVALID), (dict(dout=P + 8), MISALIGNED),
    (dict(dtable=P + 8), MISALIGNED), (dict(workspace=P + 8), MISALIGNED), (dict(D=20), SHAPE),
    (dict(M=2 ** 30 + 1), SHAPE), (dict(V=MAX), SHAPE), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=-1), WORKSPACE)])
def test_embedding_grad_refuses(change, want):
    need = gbf.gbf_workspace_size("embedding_grad", 4, 10, 16, True)
    if change.get("workspace_bytes") == -1:
        change = dict(workspace_bytes=need - 1)
    args = dict(ids=P, dout=P, dtable=P, M=4, V=10, D=16, workspace=P, workspace_bytes=need)
    assert gbf.embedding_grad(**{**args, **change}, stream=0, raise_on_error=False) == want


def clip_call(lib, tensors=2, grads=(P, P), out=None, counts=(4, 4), types=(0, 1), max_norm=1.0, eps=1e-6, norm=P,
              workspace=P, workspace_bytes=1 << 20):
    arr = lambda kind, v: None if v is None else (kind * len(v))(*v)  # noqa: E731
    return lib.gbf_clip_grad_norm(arr(ctypes.c_void_p, grads), arr(ctypes.c_void_p, out), arr(ctypes.c_int64, counts),
                              arr(ctypes.c_int, types), tensors, max_norm, eps, norm, workspace, workspace_bytes, 0)


@pytest.mark.parametrize("change,want", [
    (dict(tensors=-1), INVALID), (dict(grads=None), INVALID), (dict(counts=None), INVALID), (dict(types=None), INVALID),
    (dict(norm=None), INVALID), (dict(counts=(4, -1)), INVALID), (dict(types=(0, 2)), INVALID),
    (dict(grads=(P, None)), INVALID), (dict(out=(P, None)), INVALID), (dict(max_norm=-1.0), INVALID),
    (dict(max_norm=math.nan), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.inf), INVALID),
    (dict(grads=(P + 1, P)), MISALIGNED), (dict(grads=(P, P + 2)), MISALIGNED), (dict(out=(P, P + 2)), MISALIGNED),
    (dict(norm=P + 2), MISALIGNED), (dict(workspace=P + 4), MISALIGNED), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=100), WORKSPACE)])
def test_clip_refuses(lib, change, want):
    assert clip_call(lib, **change) == want


def test_tensor_list_refuses():
    with pytest.raises(TypeError):
        gbf.TensorList([torch.zeros(3, dtype=torch.float16)])
    with pytest.raises(ValueError):
        gbf.TensorList([torch.zeros(4, 4).t()])
    with pytest.raises(ValueError):
        gbf.clip_grad_norm([torch.zeros(3)], [torch.zeros(4)], 1.0, P, stream=0)


def test_workspace_sizes():
    assert gbf.gbf_workspace_size("embedding_grad", 0, 0, 0, True) == 0
    small = gbf.gbf_workspace_size("embedding_grad", 1024, 32000, 1024, True)
    assert 0 < small < gbf.gbf_workspace_size("embedding_grad", 65536, 32000, 1024, True)
    assert gbf.gbf_workspace_size("clip_grad_norm", 1, 0, 0, True) == 152 * 8 * 24
    assert gbf.gbf_workspace_size("clip_grad_norm", 513, 0, 0, True) == 2 * 152 * 8 * 24


def ce_args(**change):
    need = gbf.gbf_workspace_size("linear_ce", 4, 10, 16, True)
    return {**dict(x=P, w=P, targets=P, loss=P, lse=P, mean=None, M=4, V=10, D=16, workspace=P, workspace_bytes=need),
            **change}


BAD_HEADS = [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(targets=None), INVALID), (dict(M=-1), INVALID),
    (dict(alpha=math.inf), INVALID), (dict(alpha=math.nan), INVALID), (dict(index_type=2), INVALID),
    (dict(x=P + 8), MISALIGNED), (dict(w=P + 8), MISALIGNED), (dict(targets=P + 4), MISALIGNED),
    (dict(lse=P + 2), MISALIGNED), (dict(workspace=P + 8), MISALIGNED), (dict(D=12), SHAPE), (dict(D=0), SHAPE),
    (dict(V=0), SHAPE), (dict(M=2 ** 24 + 1), SHAPE), (dict(V=2 ** 26 + 1), SHAPE), (dict(D=2 ** 20 + 8), SHAPE),
    (dict(M=2 ** 24, V=2 ** 26), SHAPE), (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=64), WORKSPACE)]


@pytest.mark.parametrize("change,want", BAD_HEADS + [
    (dict(loss=None), INVALID), (dict(lse=None), INVALID), (dict(loss=P + 1), MISALIGNED), (dict(mean=P + 1), MISALIGNED)])
def test_linear_ce_refuses(change, want):
    assert gbf.linear_ce(**ce_args(**change), stream=0, raise_on_error=False) == want


@pytest.mark.parametrize("change,want", BAD_HEADS + [
    (dict(lse=None), INVALID), (dict(dx=None, dw=None), INVALID), (dict(reduction=2), INVALID),
    (dict(dx=P + 8), MISALIGNED), (dict(dw=P + 8), MISALIGNED), (dict(dloss=P + 2), MISALIGNED)])
def test_linear_ce_grad_refuses(change, want):
    need = gbf.gbf_workspace_size("linear_ce_grad", 4, 10, 16, True)
    args = dict(x=P, w=P, targets=P, lse=P, dloss=None, dx=P, dw=P, M=4, V=10, D=16, workspace=P, workspace_bytes=need)
    assert gbf.linear_ce_grad(**{**args, **change}, stream=0, raise_on_error=False) == want
