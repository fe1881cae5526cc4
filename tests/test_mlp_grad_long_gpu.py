"""The gated block's gradients over many rows or hidden columns, where all products of a sum
have one sign: the tensor cores' additions cut, so a long sum is taken in parts.

Tolerances.  A chain of n products is low by up to 7.5e-9 n of itself (an addition of 16
products cuts at most 2^-23): CUT, 1e-3, for 131072.  dg and du are rounded by up to R =
2^-8 of themselves, uniform and with either sign: n of them in a sum of terms within a
factor of 8 are held to seven times R / sqrt(3 n) (their root mean square is 1.06 times
their mean).  The last rounding is monotone, so a result lies between the roundings of
want (1 - CUT - that) and want (1 + that).  (No bound on the mean of the errors: sums of
many values in [1, 2) lie so close together that all of a result may round to one number,
675400 +- 700 to 675840 where bf16's step is 4096, and the last rounding does not average
out.)"""
import pytest
import torch

from test_mlp_train_gpu import R

pytestmark = pytest.mark.gpu
CUT = 7.5e-9 * 131072


def positive(gen, *shape):
    return (1.0 + torch.rand(*shape, generator=gen, device="cuda")).bfloat16()


def case(lib, M, D, F, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, dout = positive(gen, M, D), positive(gen, M, D)
    g, u, h = (positive(gen, M, F) for _ in range(3))
    wg, wu, wd = positive(gen, F, D), positive(gen, F, D), positive(gen, D, F)
    shapes = dict(dx=(M, D), dw_gate=(F, D), dw_up=(F, D), dw_down=(D, F))
    flat = {k: torch.full((a * b + 512,), 7.0, device="cuda", dtype=torch.bfloat16) for k, (a, b) in shapes.items()}
    got = {k: f[256:-256].view(shapes[k]) for k, f in flat.items()}
    n = lib.gbf_workspace_size("mlp_grad", M, D, F, True)
    ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    lib.mlp_grad(dout, x, g, u, h, wg, wu, wd, **got, M=M, D=D, F=F, act="identity", workspace=ws, workspace_bytes=n)
    assert all(bool((f[:256] == 7.0).all()) and bool((f[-256:] == 7.0).all()) for f in flat.values())
    assert bool((ws[n:] == 0xFF).all()) and lib.gbf_check_device_error() == 0
    dh = dout.double() @ wd.double()
    dg, du = dh * u.double(), dh * g.double()
    want = dict(dx=dg @ wg.double() + du @ wu.double(), dw_gate=dg.T @ x.double(), dw_up=du.T @ x.double(),
                dw_down=dout.double().T @ h.double())
    return got, want


def check(got, want):
    M, F = want["dx"].shape[0], want["dw_gate"].shape[0]
    for k, w in want.items():
        noise = 0.0 if k == "dw_down" else 7 * R / (3 * (2 * F if k == "dx" else M)) ** 0.5
        noise += 2.0 ** -22  # the parts added in fp32
        low, high = (w * (1.0 - CUT - noise)).bfloat16(), (w * (1.0 + noise)).bfloat16()
        assert bool((got[k] >= low).all()) and bool((got[k] <= high).all()), (k, float((got[k].double() / w - 1.0).mean()))


@pytest.mark.parametrize("M,D,F", [(131072, 64, 72), (131073, 64, 72), (300000, 136, 64), (2 ** 20 + 72, 64, 72), (140000, 520, 264)])
def test_many_rows(cuda_lib, M, D, F):
    check(*case(cuda_lib, M, D, F))


@pytest.mark.parametrize("M", [40, 300])
def test_many_hidden_columns(cuda_lib, M):
    check(*case(cuda_lib, M, 64, 140000))


def test_gradients_left_out(cuda_lib):
    M, D, F = 262200, 64, 72
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, dout = positive(gen, M, D), positive(gen, M, D)
    kept = [positive(gen, M, F) for _ in range(3)]
    w = [positive(gen, F, D), positive(gen, F, D), positive(gen, D, F)]
    n = cuda_lib.gbf_workspace_size("mlp_grad", M, D, F, True)
    names = ("dx", "dw_gate", "dw_up", "dw_down")

    def run(some):
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        out = dict(zip(names, (torch.full_like(t, 7.0) for t in (x, *w))))
        cuda_lib.mlp_grad(dout, x, *kept, *w, **{k: v if k in some else None for k, v in out.items()}, M=M, D=D, F=F,
                          workspace=ws, workspace_bytes=n)
        return out

    full = run(names)
    for some in (("dw_down",), ("dw_up",), ("dx", "dw_gate"), ("dw_gate", "dw_down")):
        got = run(some)
        for k in names:
            assert torch.equal(got[k], full[k]) if k in some else bool((got[k] == 7.0).all()), (some, k)
