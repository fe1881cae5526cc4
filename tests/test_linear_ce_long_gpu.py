"""The losses' gradients by the weight over very many rows, and by x over a very large
vocabulary, where the products of a sum have one sign: the tensor cores' additions cut, so
a long sum is taken in parts.

Tolerances.  A chain of n products is low by up to 7.5e-9 n of itself (an addition of 16
products cuts at most 2^-23): CUT for 131072.  G is rounded by up to R = 2^-8 of itself,
uniform and with either sign: over a sum of terms t seven times R / sqrt(3) sqrt(sum t^2) /
sum t; lse, the powers and the fp32 additions are off by less than 2^-18.  The last
rounding is monotone, so a result lies between the roundings of what these leave."""
import pytest
import torch

pytestmark = pytest.mark.gpu
R = 2.0 ** -8
CUT = 7.5e-9 * 131072


def between(got, want, noise, cut=CUT):
    low, high = (want * (1.0 - cut - noise)).bfloat16(), (want * (1.0 + noise)).bfloat16()
    ok = (got >= low) & (got <= high)
    assert bool(ok.all()), (int((~ok).sum()), float((got.double() / want - 1.0).mean()))


def case(M, V, D, unscored, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (1.0 + torch.rand(M, D, generator=gen, device="cuda")).bfloat16()
    w = (torch.randn(V, D, generator=gen, device="cuda") * 0.05).bfloat16()
    t = torch.randint(0, 3, (M,), generator=gen, device="cuda")  # few columns, so that the others' G has one sign
    t[torch.rand(M, generator=gen, device="cuda") < unscored] = -1
    return x, w, t


def gradients(lib, x, w, t, soft):
    (M, D), V = x.shape, w.shape[0]
    loss, lse, mean = (torch.full((n,), float("nan"), device="cuda", dtype=torch.float32) for n in (M, M, 1))
    flat = {k: torch.full((v.numel() + 512,), 7.0, device="cuda", dtype=torch.bfloat16) for k, v in (("dx", x), ("dw", w))}
    dx, dw = flat["dx"][256:-256].view(M, D), flat["dw"][256:-256].view(V, D)
    if soft:
        args = (x, w, torch.stack([t, torch.where(t < 0, -1, (t + 1) % 3)], 1).contiguous(), torch.zeros(M, 2, device="cuda"))
        n = [lib.linear_distill_workspace_size(M, V, D, 2, g) for g in (False, True)]
    else:
        n = [lib.gbf_workspace_size(op, M, V, D, True) for op in ("linear_ce", "linear_ce_grad")]
    ws = [torch.full((b + 256,), 0xFF, device="cuda", dtype=torch.uint8) for b in n]
    if soft:
        lib.linear_distill(*args, loss, lse, mean, M, V, D, 2, workspace=ws[0], workspace_bytes=n[0])
        lib.linear_distill_grad(*args, lse, None, dx, dw, M, V, D, 2, reduction="sum", workspace=ws[1], workspace_bytes=n[1])
    else:
        lib.linear_ce(x, w, t, loss, lse, mean, M, V, D, workspace=ws[0], workspace_bytes=n[0])
        lib.linear_ce_grad(x, w, t, lse, None, dx, dw, M, V, D, reduction="sum", workspace=ws[1], workspace_bytes=n[1])
    assert all(bool((f[:256] == 7.0).all()) and bool((f[-256:] == 7.0).all()) for f in flat.values())
    assert all(bool((b[k:] == 0xFF).all()) for b, k in zip(ws, n)) and lib.gbf_check_device_error() == 0
    return loss, lse, dx, dw


# 131072 rows: one chain; a piece of the vocabulary has 512 columns from there on
@pytest.mark.parametrize("M,V,D,unscored", [(131072, 600, 64, 0.0), (131073, 600, 64, 0.2), (300000, 257, 136, 0.0),
                                            (2 ** 20 + 72, 600, 64, 0.0), (2 ** 20, 300, 64, 0.3), (400000, 100, 64, 0.9995),
                                            (270000, 40, 64, 1.0)])
@pytest.mark.parametrize("soft", [False, True])
def test_weight_over_many_rows(cuda_lib, M, V, D, unscored, soft):
    x, w, t = case(M, V, D, unscored)
    loss, lse, dx, dw = gradients(cuda_lib, x, w, t, soft)
    rows = (t >= 0).nonzero()[:, 0]
    assert bool((dx[t < 0] == 0).all()) and bool((loss[t < 0] == 0).all())
    if len(rows) == 0:
        assert bool((dw == 0).all())
        return
    p = torch.softmax(x[rows].double() @ w.double().T, 1)[:, 3:]
    xs = x[rows].double()
    want = p.T @ xs
    noise = 7 * R * ((p.square().T @ xs.square()) / 3).sqrt() / want + 2.0 ** -18
    between(dw[3:], want, noise)
    # the columns with a target: p - q of either sign, within the magnitudes' share
    p = torch.softmax(x[rows].double() @ w.double().T, 1)[:, :3]
    q = torch.nn.functional.one_hot(t[rows], 3).double()
    if soft:
        q = 0.5 * (q + q.roll(1, 1))
    want, size = (p - q).T @ xs, (p - q).abs().T @ xs
    assert bool(((dw[:3].double() - want).abs() <= R * want.abs() + (CUT + R) * size).all())


@pytest.mark.parametrize("soft", [False, True])
def test_x_over_a_large_vocabulary(cuda_lib, soft):
    """So wide that one part of K would fill the pairs, and more columns than a chain."""
    M, V, D = 5, 140000, 77 * 256
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(V, D, device="cuda", dtype=torch.bfloat16).uniform_(1.0, 2.0, generator=gen)
    x = (torch.randn(M, D, generator=gen, device="cuda") * 1e-3).bfloat16()
    t = torch.randint(0, 3, (M,), generator=gen, device="cuda")
    loss, lse, dx, dw = gradients(cuda_lib, x, w, t, soft)
    l = torch.cat([x.double() @ part.double().T for part in w.split(20000)], 1)
    grad = torch.softmax(l, 1)
    if soft:
        grad[torch.arange(M), t] -= 0.5
        grad[torch.arange(M), (t + 1) % 3] -= 0.5
    else:
        grad[torch.arange(M), t] -= 1.0
    cols = torch.tensor([0, 1, 255, 256, 9999, D - 257, D - 1], device="cuda")
    some = w[:, cols].double()
    want, size = grad @ some, grad.abs() @ some
    assert bool(((dx[:, cols].double() - want).abs() <= R * want.abs() + (CUT + R) * size).all())
