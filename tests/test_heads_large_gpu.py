"""Tables of more than 2^31 values: offsets past 32 bits in every operator at a
model's two ends.  The tolerances are those of the operators' own tests."""
import pytest
import torch

from test_linear_ce_gpu import BF, F32, backward, forward

pytestmark = pytest.mark.gpu

V, D = 270_001, 8192  # 2.2e9 values


@pytest.fixture(scope="module")
def table(cuda_lib):
    g = torch.Generator(device="cuda").manual_seed(1)
    t = torch.empty(V, D, device="cuda", dtype=torch.bfloat16)
    for v0 in range(0, V, 30000):
        n = min(30000, V - v0)
        t[v0:v0 + n] = (torch.randn(n, D, generator=g, device="cuda") / 45).bfloat16()
    return t


def test_lookup_and_its_gradient(cuda_lib, table):
    ids = torch.tensor([0, V - 1, V - 2, 262_143, 262_144, 262_145, 131_072, V, -1, V - 1], device="cuda")
    M = len(ids)
    out = torch.empty(M, D, device="cuda", dtype=torch.bfloat16)
    cuda_lib.embedding_lookup(ids, table, out, M, V, D)
    known = (ids >= 0) & (ids < V)
    assert torch.equal(out[known], table[ids[known]]) and (out[~known] == 0).all()
    # a short list, and a long one that is sorted
    for copies in (1, 200):
        many = ids.repeat(copies)
        dout = torch.ones(len(many), D, device="cuda", dtype=torch.bfloat16)
        n = cuda_lib.gbf_workspace_size("embedding_grad", len(many), V, D, True)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        dtable = torch.full((V, D), float("nan"), device="cuda", dtype=torch.bfloat16)
        cuda_lib.embedding_grad(many, dout, dtable, len(many), V, D, workspace=ws, workspace_bytes=n)
        counts = torch.bincount(ids[known], minlength=V)
        rows = counts.nonzero()[:, 0]
        assert (dtable[rows].float() == (counts[rows] * copies)[:, None]).all()
        for v0 in range(0, V, 30000):  # whole numbers: every other row is zero
            part = dtable[v0:v0 + 30000]
            assert int(torch.count_nonzero(part)) == D * int((counts[v0:v0 + 30000] > 0).sum())


@pytest.mark.parametrize("M", [40, 300])
def test_linear_cross_entropy(cuda_lib, table, M):
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, D, generator=g, device="cuda").bfloat16()
    t = torch.randint(V - 5000, V, (M,), generator=g, device="cuda")
    t[1], t[2] = 5, -100
    loss, lse, mean = forward(cuda_lib, x, table, t)
    logits = torch.empty(M, V, device="cuda", dtype=torch.float64)
    size = torch.zeros(M, device="cuda", dtype=torch.float64)
    for v0 in range(0, V, 30000):
        w = table[v0:v0 + 30000].double()
        logits[:, v0:v0 + 30000] = x.double() @ w.T
        size = torch.maximum(size, (x.double().abs() @ w.abs().T).amax(dim=1))
    want = torch.logsumexp(logits, dim=1)
    tol = D * 2 * F32 * size + 8 * F32 * logits.abs().amax(dim=1) + (200 + V / 128) * F32
    scored = t >= 0
    assert ((lse.double() - want).abs()[scored] <= tol[scored]).all()
    each = torch.arange(M, device="cuda")
    at = logits[each, t.clamp(min=0)]
    assert ((loss.double() - (want - at)).abs()[scored] <= 2 * tol[scored]).all()
    dx, dw = backward(cuda_lib, x, table, t, lse, reduction="sum")
    p = (logits - want[:, None]).exp()
    p[each, t.clamp(min=0)] -= 1
    p[~scored] = 0
    # every term of a sum is off by half a step of bf16 and the logit's error
    rel = BF + 2 * float(tol.max())
    for v0 in (0, 131_072, V - 5000):
        rows = slice(v0, v0 + 5000)
        want_dw = p[:, rows].T @ x.double()
        err = rel * (p[:, rows].abs().T @ x.double().abs()) + 2.0 ** -126
        assert ((dw[rows].double() - want_dw).abs() <= err * (1 + BF) + (BF + 4 * F32) * want_dw.abs()).all()
    assert not torch.isnan(dw[::997]).any()
    want_dx, err_dx = torch.zeros(M, D, device="cuda", dtype=torch.float64), torch.zeros(M, D, device="cuda", dtype=torch.float64)
    for v0 in range(0, V, 30000):
        w = table[v0:v0 + 30000].double()
        want_dx += p[:, v0:v0 + 30000] @ w
        err_dx += rel * (p[:, v0:v0 + 30000].abs() @ w.abs())
    err_dx += V * 2 * F32 * err_dx / rel
    assert ((dx.double() - want_dx).abs() <= err_dx * (1 + BF) + (BF + 4 * F32) * want_dx.abs()).all()


def test_clipping(cuda_lib, table):
    n = cuda_lib.gbf_workspace_size("clip_grad_norm", 1, 0, 0, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    norm = torch.empty(1, device="cuda")
    out = torch.empty_like(table)
    cuda_lib.clip_grad_norm([table], [out], 1.0, norm, workspace=ws, workspace_bytes=n)
    want = sum(float(table[v0:v0 + 30000].double().square().sum()) for v0 in range(0, V, 30000)) ** 0.5
    assert abs(float(norm) - want) <= 22 * F32 * want
    for v0 in (0, 262_000, V - 1000):
        a, b = out[v0:v0 + 1000].double(), table[v0:v0 + 1000].double() / (want + 1e-6)
        assert ((a - b).abs() <= (BF + 30 * F32) * b.abs() + 2.0 ** -134).all()
