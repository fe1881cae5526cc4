"""Calls on no positions, no rows of a table and no columns with empty tensors,
whose addresses are null.  The calls without a GPU get as far as asking for one."""
import pytest
import torch

import tcgen05_tmem_bf16_gb300 as gbf

INVALID, NO_DEVICE = 1, 7
P = 0x10000  # an address that is never followed: none of these calls launches anything


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tcgen05_tmem_bf16_gb300 import build
    build.build()
    return gbf.load()


def taken(status):
    return status == (0 if torch.cuda.is_available() else NO_DEVICE)


ENDS = dict(stream=0, raise_on_error=False)


def test_lookup_of_nothing():
    e = torch.empty(0)
    assert e.data_ptr() == 0
    assert taken(gbf.embedding_lookup(e, P, e, 0, 10, 16, **ENDS))
    assert taken(gbf.embedding_lookup(e, e, e, 0, 0, 16, **ENDS))
    assert taken(gbf.embedding_lookup(P, e, e, 4, 10, 0, **ENDS))
    assert gbf.embedding_lookup(P, e, P, 4, 10, 16, **ENDS) == INVALID
    assert gbf.embedding_lookup(e, P, P, 4, 10, 16, **ENDS) == INVALID
    assert gbf.embedding_lookup(e, P, e, -1, 10, 16, **ENDS) == INVALID


def test_gradient_of_nothing():
    e = torch.empty(0)
    ends = dict(ENDS, workspace=P, workspace_bytes=1 << 20)
    assert taken(gbf.embedding_grad(e, e, P, 0, 10, 16, accumulate=True, **ends))
    assert taken(gbf.embedding_grad(P, P, e, 4, 0, 16, **ends))
    assert taken(gbf.embedding_grad(P, e, e, 4, 10, 0, **ends))
    assert gbf.embedding_grad(e, e, e, 0, 10, 16, **ends) == INVALID
    assert gbf.embedding_grad(P, e, P, 4, 10, 16, **ends) == INVALID


def test_loss_of_nothing():
    e = torch.empty(0)
    ends = dict(ENDS, workspace=P, workspace_bytes=1 << 20)
    assert taken(gbf.linear_ce(e, P, e, e, e, None, 0, 10, 16, **ends))
    assert taken(gbf.linear_ce_grad(e, P, e, e, None, e, None, 0, 10, 16, **ends))
    assert gbf.linear_ce(e, e, e, e, e, None, 0, 10, 16, **ends) == INVALID
    assert gbf.linear_ce(P, P, P, e, e, None, 4, 10, 16, **ends) == INVALID
    assert gbf.linear_ce_grad(P, P, P, P, None, e, None, 4, 10, 16, **ends) == INVALID


@pytest.mark.gpu
def test_results_of_no_positions(cuda_lib):
    V, D = 40, 64
    ids = torch.empty(0, device="cuda", dtype=torch.int64)
    x = torch.empty(0, D, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(V, D, device="cuda").bfloat16()
    f = torch.empty(0, device="cuda")
    ws = torch.empty(1 << 20, device="cuda", dtype=torch.uint8)
    ends = dict(workspace=ws, workspace_bytes=1 << 20)
    cuda_lib.embedding_lookup(ids, w, x, 0, V, D)
    for accumulate, want in ((True, 3.0), (False, 0.0)):
        dtable = torch.full((V, D), 3.0, device="cuda", dtype=torch.bfloat16)
        cuda_lib.embedding_grad(ids, x, dtable, 0, V, D, accumulate=accumulate, **ends)
        assert (dtable == want).all()
    mean = torch.full((1,), 5.0, device="cuda")
    cuda_lib.linear_ce(x, w, ids, f, f, mean, 0, V, D, **ends)
    dw = torch.full((V, D), 3.0, device="cuda", dtype=torch.bfloat16)
    cuda_lib.linear_ce_grad(x, w, ids, f, None, x.clone(), dw, 0, V, D, **ends)
    assert float(mean) == 0 and (dw == 0).all()
    # an empty table: every id is unknown
    out = torch.full((3, D), 7.0, device="cuda", dtype=torch.bfloat16)
    none = torch.empty(0, D, device="cuda", dtype=torch.bfloat16)
    cuda_lib.embedding_lookup(torch.arange(3, device="cuda"), none, out, 3, 0, D)
    assert (out == 0).all()
