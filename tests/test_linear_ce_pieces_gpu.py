"""Vocabularies of several pieces of the backward pass, and of more than 2^31
values, with all of the probability on a few columns at the pieces' and the
offsets' edges: every one of them shows in dx, and each is a row of dw.

Tolerances: a logit of about 30 whose products are summed in chains of 64
additions that each cut less than 2^-23 of a running sum under 40 (LOGIT); p and
G from two such logits; G's and the result's rounding to bf16."""
import pytest
import torch

from test_heads_large_gpu import table  # noqa: F401  (a fixture)
from test_linear_ce_gpu import BF, F32, SMALLEST, backward, forward

pytestmark = pytest.mark.gpu

LOGIT = 64 * 2 * F32 * 40
REL = BF + 2 * LOGIT + 8 * F32 * 40  # of p and of a value of G


def check(lib, x, w, t, at, others, dx_noise, dw_noise):
    """at: the columns that hold the probability; others(lse): the sum of the other
    columns' powers; the noise: what those may add to dx and dw at most."""
    M, V = x.shape[0], w.shape[0]
    ws = w[at].double()
    logits = x.double() @ ws.T
    total = logits.exp().sum(dim=1) + others
    want_lse = total.log()
    scored = (t >= 0) & (t < V)
    n = int(scored.sum())
    hit = (t[:, None] == at[None, :]).double()
    loss, lse, mean = forward(lib, x, w, t)
    tol = LOGIT + 8 * F32 * 40 + 256 * F32
    assert ((lse.double() - want_lse).abs() <= tol)[scored].all()
    want_loss = want_lse - (logits * hit).sum(dim=1)
    assert ((loss.double() - want_loss).abs() <= 2 * tol)[scored].all()
    assert (loss[~scored] == 0).all() and (lse[~scored] == 0).all()
    dx, dw = backward(lib, x, w, t, lse)
    g = ((logits - want_lse[:, None]).exp() - hit) * scored[:, None] / n
    # p - 1 of a target is off by p's error
    g_err = REL * ((logits - want_lse[:, None]).exp() * scored[:, None] / n + g.abs())
    want = g @ ws
    err = (g_err @ ws.abs()) * (1 + BF) + (BF + 32 * F32) * want.abs() + dx_noise / n + SMALLEST
    assert ((dx.double() - want).abs() <= err).all()
    for k in range(len(at)):  # each column's part would be missed
        part = g[:, k:k + 1] * ws[k:k + 1]
        assert (part.abs() > 2 * err).any()
    want = g.T @ x.double()
    err = (g_err.T @ x.double().abs()) * (1 + BF) + (BF + (M + 64) * 2 * F32) * want.abs()
    assert ((dw[at].double() - want).abs() <= err + SMALLEST).all()
    assert (want.abs() > 2 * err).any(dim=1).all()
    for v0 in range(0, V, 1 << 18):
        rest = dw[v0:v0 + (1 << 18)].float().abs().amax(dim=1)
        inside = at[(at >= v0) & (at < v0 + (1 << 18))] - v0
        rest[inside] = 0
        assert float(rest.max()) <= dw_noise / n
    again = backward(lib, x, w, t, lse)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("M", [17, 100, 128, 200, 300])
@pytest.mark.parametrize("V", [(1 << 20) + 1000, (1 << 21) + 77])
def test_pieces_of_the_vocabulary(cuda_lib, M, V):
    """Rows of w that are zero but for those at the edges of pieces of any length
    that M gives (2^27 / M in whole tiles of 512; 2^20 for 128 rows)."""
    D = 16
    g = torch.Generator(device="cuda").manual_seed(M + V)
    cols = (1 << 27) // M // 512 * 512
    edges = {0, V - 1, (1 << 20) - 1, 1 << 20}
    for k in (1, 2, 4):
        edges |= {k * cols - 1, k * cols}
    at = torch.tensor(sorted(v for v in edges if 0 <= v < V), device="cuda")
    n = len(at)
    assert n <= D
    w = torch.zeros(V, D, device="cuda", dtype=torch.bfloat16)
    w[at] = torch.randn(n, D, generator=g, device="cuda").bfloat16()
    # three of the columns at a logit of 30, the other edges at 0
    want = torch.zeros(M, n, device="cuda", dtype=torch.float64)
    each = torch.arange(M, device="cuda")
    for k in range(3):
        want[each, (each * 3 + k) % n] = 30.0
    x = (want @ torch.linalg.pinv(w[at].double()).T).bfloat16()
    t = at[(each * 3) % n].clone()
    t[5::11] = -100
    assert float((x.double() @ w[at].double().T).max()) < 40
    # the power of a zero column, and of an edge that is off 0 by x's rounding
    check(cuda_lib, x, w, t, at, float(V - n), 0.0,
          2 * M * float(x.double().abs().max()) * 3e-12)


@pytest.mark.parametrize("M", [40, 100, 300])
def test_past_32_bits(cuda_lib, table, M):  # noqa: F811
    """A dense table of 2.2e9 values: x is made of three of its rows, one of them the
    target, on both sides of the offset 2^31 (row 262144)."""
    V, D = table.shape
    at = torch.tensor([0, 131_072, 262_143, 262_144, 262_145, V - 2, V - 1], device="cuda")
    n = len(at)
    each = torch.arange(M, device="cuda")
    rows = table[at].double()
    size = (rows * rows).sum(dim=1)
    x = torch.zeros(M, D, device="cuda", dtype=torch.float64)
    for k in range(3):
        which = (each * 3 + k) % n
        x += rows[which] * (30.0 / size[which])[:, None]
    x = x.bfloat16()
    t = at[(each * 3) % n].clone()
    t[7::13] = V
    # the other columns' powers: under 2e-6 of a row's, all together
    others = torch.zeros(M, device="cuda", dtype=torch.float64)
    largest = 0.0
    for v0 in range(0, V, 30000):
        l = x.double() @ table[v0:v0 + 30000].double().T
        inside = at[(at >= v0) & (at < v0 + 30000)] - v0
        l[:, inside] = float("-inf")
        others += l.exp().sum(dim=1)
        largest = max(largest, float(l.max()))
    p = others / (x.double() @ rows.T).exp().sum(dim=1)
    assert float(p.max()) < 2e-6 and largest < 12
    noise = 2 * float(p.max()) * float(table[:1000].abs().max()) * 2
    check(cuda_lib, x, table, t, at, others, noise, 2 * M * float(x.double().abs().max()) * 2.718 ** (largest - 26))
