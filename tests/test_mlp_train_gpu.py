"""The gated block that is trained, and its gradients, against a plain fp64 form.

Tolerances.  bf16 rounds by at most R = 2^-8 of a value.  A sum of K products on
the tensor cores is off by at most chain(K) = 4e-9 K + 2^-23 of the sum of their
magnitudes (the additions cut; fp32 operations around them).  The activations take
an approximate exponential and reciprocal: 2^-20 of the values they make.  The
gradients' operands dg and du are rounded themselves, so each bound below adds up
what its operands can be off by, times the magnitudes they meet.  Such a bound is
far above what random roundings come to; so the root mean square of the errors is
held too: two independent roundings of at most R of each value, uniform, have
R / sqrt(3) each, 0.82 R together, held to R of the result's root mean square."""
import pytest
import torch

pytestmark = pytest.mark.gpu

R = 2.0 ** -8
ACTS = ("silu", "gelu_tanh", "relu", "identity")


def chain(k):
    return 4e-9 * k + 2.0 ** -23


def act64(v, act):
    f = torch.nn.functional
    return {"silu": f.silu, "relu": f.relu, "identity": lambda t: t,
            "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[act](v)


def inputs(M, D, F, seed=0, dout_std=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    return dict(x=normal(M, D), w_gate=normal(F, D, std=D ** -0.5), w_up=normal(F, D, std=D ** -0.5),
                w_down=normal(D, F, std=F ** -0.5)), normal(M, D), normal(M, D, std=dout_std)


def nan(*shape):
    return torch.full(shape, float("nan"), device="cuda", dtype=torch.bfloat16)


def forward(lib, t, residual, act, M, D, F, stream=None):
    out, g, u, h = nan(M, D), nan(M, F), nan(M, F), nan(M, F)
    lib.mlp_train(**t, residual=residual, out=out, g=g, u=u, h=h, M=M, D=D, F=F, act=act, stream=stream)
    return out, g, u, h


def backward(lib, t, kept, dout, act, M, D, F, skip=(), stream=None):
    n = lib.gbf_workspace_size("mlp_grad", M, D, F, True)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in bf16 and fp32
    grads = dict(dx=nan(M, D), dw_gate=nan(F, D), dw_up=nan(F, D), dw_down=nan(D, F))
    lib.mlp_grad(dout, t["x"], *kept, t["w_gate"], t["w_up"], t["w_down"],
                 **{k: None if k in skip else v for k, v in grads.items()}, M=M, D=D, F=F, act=act, workspace=ws,
                 workspace_bytes=n, stream=stream)
    return grads


def close(got, want, bound, what):
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), (what, float((err / (bound + 1e-300)).max()))


def check_rms(got, want, what):
    err, ref = (got.double() - want).square().mean().sqrt(), want.square().mean().sqrt()
    assert float(err) <= R * float(ref), (what, float(err / ref))


def check_forward(t, residual, got, act, D, F):
    x, wg, wu, wd = (t[n].double() for n in ("x", "w_gate", "w_up", "w_down"))
    out, g, u, h = got
    g64, u64 = x @ wg.T, x @ wu.T
    dg, du = (chain(D) * (x.abs() @ w.abs().T) for w in (wg, wu))
    close(g, g64, R * (g64.abs() + dg) + dg, "g")
    close(u, u64, R * (u64.abs() + du) + du, "u")
    a = act64(g64, act)
    h64 = a * u64
    # |act'| <= 1.13 for all of them
    dh = 1.13 * dg * (u64.abs() + du) + a.abs() * du + 2.0 ** -20 * (g64.abs() + dg) * (u64.abs() + du)
    close(h, h64, R * (h64.abs() + dh) + dh, "h")
    hs = h.double()  # the down product takes h as stored
    out64 = hs @ wd.T
    do = chain(F) * (hs.abs() @ wd.abs().T)
    if residual is not None:
        out64 = out64 + residual.double()
        do = do + 2.0 ** -23 * residual.double().abs()
    close(out, out64, R * (out64.abs() + do) + do, "out")


def gradients64(t, kept, dout, act):
    x, wg, wu, wd = (t[n].double() for n in ("x", "w_gate", "w_up", "w_down"))
    g, u, h = (v.double() for v in kept)
    g = g.requires_grad_()
    dh = dout.double() @ wd
    a = act64(g, act)
    (da,) = torch.autograd.grad(a.sum(), g)
    g, a = g.detach(), a.detach()
    return x, wg, wu, wd, g, u, h, dh, a, da


def check_backward(t, kept, dout, got, act, M, D, F, rms=True):
    x, wg, wu, wd, g, u, h, dh, a, da = gradients64(t, kept, dout, act)
    d64 = dout.double()
    ddh = chain(D) * (d64.abs() @ wd.abs())
    dg, du = dh * u * da, dh * a
    near = 2.0 ** -20 * (1.0 + g.abs())  # of the approximate activation and its derivative
    eg = (ddh * da.abs() + dh.abs() * near) * u.abs()
    eg = R * (dg.abs() + eg) + eg
    eu = ddh * a.abs() + dh.abs() * near
    eu = R * (du.abs() + eu) + eu
    want = dict(dx=dg @ wg + du @ wu, dw_gate=dg.T @ x, dw_up=du.T @ x, dw_down=d64.T @ h)
    size = dict(dx=dg.abs() @ wg.abs() + du.abs() @ wu.abs(), dw_gate=dg.abs().T @ x.abs(), dw_up=du.abs().T @ x.abs(),
                dw_down=d64.abs().T @ h.abs())
    terms = dict(dx=2 * F, dw_gate=M, dw_up=M, dw_down=M)
    operands = dict(dx=eg @ wg.abs() + eu @ wu.abs(), dw_gate=eg.T @ x.abs(), dw_up=eu.T @ x.abs(), dw_down=0.0)
    for name, w in want.items():
        e = operands[name] + chain(terms[name]) * (size[name] + operands[name])
        close(got[name], w, R * (w.abs() + e) + e, name)
        if rms and w.numel() >= 4096:
            check_rms(got[name], w, name)


SIZES = [(1, 8, 8), (1, 64, 136), (7, 72, 200), (16, 264, 520), (65, 520, 264), (128, 256, 512), (255, 136, 1032),
         (256, 512, 256), (257, 264, 520), (300, 1000, 264), (513, 136, 1032), (700, 520, 2056), (1100, 2056, 264)]


@pytest.mark.parametrize("M,D,F", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_block_and_its_gradients(cuda_lib, M, D, F, act):
    t, residual, dout = inputs(M, D, F, seed=M + D + F)
    got = forward(cuda_lib, t, residual, act, M, D, F)
    check_forward(t, residual, got, act, D, F)
    grads = backward(cuda_lib, t, got[1:], dout, act, M, D, F)
    check_backward(t, got[1:], dout, grads, act, M, D, F)
    assert cuda_lib.gbf_check_device_error() == 0


# Many tiles, which the kernels of CTA pairs and of one SM take, with one and two row tiles
# per unit.
WIDE = [(129, 72, 5000), (100, 136, 10000), (300, 264, 6000), (1300, 72, 4104), (600, 72, 12000), (2500, 136, 2056)]


@pytest.mark.parametrize("M,D,F", WIDE)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_many_tiles(cuda_lib, M, D, F, act):
    t, residual, dout = inputs(M, D, F, seed=M + D + F)
    got = forward(cuda_lib, t, residual, act, M, D, F)
    check_forward(t, residual, got, act, D, F)
    check_backward(t, got[1:], dout, backward(cuda_lib, t, got[1:], dout, act, M, D, F), act, M, D, F)
    assert cuda_lib.gbf_check_device_error() == 0


@pytest.mark.parametrize("M,D,F", [(129, 72, 5000), (1300, 72, 4104)])
def test_many_tiles_write_nothing_outside(cuda_lib, M, D, F):
    t, residual, dout = inputs(M, D, F, seed=3)
    want = forward(cuda_lib, t, residual, "silu", M, D, F)
    grads = backward(cuda_lib, t, want[1:], dout, "silu", M, D, F)
    shapes = dict(out=(M, D), g=(M, F), u=(M, F), h=(M, F), dx=(M, D), dw_gate=(F, D), dw_up=(F, D), dw_down=(D, F))
    flat = {k: torch.full((a * b + 512,), 7.0, device="cuda", dtype=torch.bfloat16) for k, (a, b) in shapes.items()}
    v = {k: f[256:-256].view(shapes[k]) for k, f in flat.items()}
    n = cuda_lib.gbf_workspace_size("mlp_grad", M, D, F, True)
    ws = torch.full((n + 256,), 0x55, dtype=torch.uint8, device="cuda")
    cuda_lib.mlp_train(**t, residual=residual, out=v["out"], g=v["g"], u=v["u"], h=v["h"], M=M, D=D, F=F)
    cuda_lib.mlp_grad(dout, t["x"], v["g"], v["u"], v["h"], t["w_gate"], t["w_up"], t["w_down"], v["dx"], v["dw_gate"],
                      v["dw_up"], v["dw_down"], M, D, F, workspace=ws, workspace_bytes=n)
    assert all(bool((f[:256] == 7.0).all()) and bool((f[-256:] == 7.0).all()) for f in flat.values())
    assert bool((ws[n:] == 0x55).all())
    assert all(torch.equal(v[k], w) for k, w in zip(("out", "g", "u", "h"), want))
    assert all(torch.equal(v[k], grads[k]) for k in grads)


@pytest.mark.parametrize("M,D,F", [(129, 72, 5000), (100, 136, 10000), (300, 264, 6000), (1300, 72, 4104)])
def test_a_wait_of_many_tiles_that_runs_out_is_reported(cuda_lib, M, D, F):
    t, residual, dout = inputs(M, D, F, seed=M)
    want = forward(cuda_lib, t, residual, "silu", M, D, F)
    grads = backward(cuda_lib, t, want[1:], dout, "silu", M, D, F)
    for call in (lambda: forward(cuda_lib, t, residual, "silu", M, D, F),
                 lambda: backward(cuda_lib, t, want[1:], dout, "silu", M, D, F)):
        try:
            cuda_lib.gbf_set_wait_timeout_ns(20_000_000)
            cuda_lib.gbf_debug_inject_timeout(True)
            call()
            assert cuda_lib.gbf_check_device_error() == 6
        finally:
            cuda_lib.gbf_debug_inject_timeout(False)
            cuda_lib.gbf_set_wait_timeout_ns(2_000_000_000)
    assert all(torch.equal(a, b) for a, b in zip(forward(cuda_lib, t, residual, "silu", M, D, F), want))
    again = backward(cuda_lib, t, want[1:], dout, "silu", M, D, F)
    assert all(torch.equal(again[k], grads[k]) for k in grads)
    assert cuda_lib.gbf_check_device_error() == 0


@pytest.mark.parametrize("act", ["relu", "identity"])
@pytest.mark.parametrize("M,D,F", [(40, 136, 264), (600, 264, 136)])
def test_other_gates(cuda_lib, act, M, D, F):
    t, _, dout = inputs(M, D, F, seed=3)
    got = forward(cuda_lib, t, None, act, M, D, F)
    check_forward(t, None, got, act, D, F)
    check_backward(t, got[1:], dout, backward(cuda_lib, t, got[1:], dout, act, M, D, F), act, M, D, F)


def test_full_width_few_rows(cuda_lib):
    """A few tokens through a block of full size: parts of K for dx."""
    M, D, F = 16, 4096, 14336
    t, residual, dout = inputs(M, D, F, seed=5)
    got = forward(cuda_lib, t, residual, "silu", M, D, F)
    check_forward(t, residual, got, "silu", D, F)
    check_backward(t, got[1:], dout, backward(cuda_lib, t, got[1:], dout, "silu", M, D, F), "silu", M, D, F)


@pytest.mark.parametrize("act", ACTS)
def test_values_far_out(cuda_lib, act):
    """Gates far from zero, up to bf16's largest: no NaN where the formula has none."""
    M, D, F = 8, 64, 64
    t, _, dout = inputs(M, D, F, seed=9)
    far = torch.tensor([0.0, -0.0, 1e-30, 5.0, -5.0, 20.0, -20.0, 88.0, -88.0, 105.0, -105.0, 300.0, -300.0, 1e19, -1e19,
                        3e38, -3e38], device="cuda").bfloat16()
    g = far.repeat(M * F // len(far) + 1)[:M * F].view(M, F).contiguous()
    u = (torch.rand(M, F, device="cuda") * 1e-3).bfloat16()
    h = torch.zeros(M, F, device="cuda", dtype=torch.bfloat16)
    only = backward(cuda_lib, t, (g, u, h), dout, act, M, D, F, skip=("dx",))
    _, _, _, _, g64, u64, _, dh, a, da = gradients64(t, (g, u, h), dout, act)
    x = t["x"].double()
    for name, d in (("dw_gate", dh * u64 * da), ("dw_up", dh * a)):
        want = d.T @ x
        assert bool(torch.isfinite(only[name]).all()), name
        # d is off by its rounding, by dh's products and by the approximate activation
        size = (d.abs().T @ x.abs())
        scale = (dh.abs() * (u64 if name == "dw_gate" else 1.0 + g64.abs())).T @ x.abs()
        ddh = chain(D) * (dout.double().abs() @ t["w_down"].double().abs())
        wide = (ddh * (1.13 * u64 if name == "dw_gate" else g64.abs() + 1.0)).T @ x.abs()
        close(only[name], want, 3 * R * size + 2.0 ** -19 * scale + 2 * wide + 1e-37, name)


@pytest.mark.parametrize("skip", [("dx",), ("dw_gate",), ("dw_up", "dw_down"), ("dx", "dw_gate", "dw_up"),
                                  ("dw_gate", "dw_up", "dw_down"), ("dx", "dw_up")])
@pytest.mark.parametrize("M", [20, 600])
def test_gradients_left_out(cuda_lib, skip, M):
    D, F = 264, 520
    t, residual, dout = inputs(M, D, F, seed=1)
    kept = forward(cuda_lib, t, residual, "silu", M, D, F)[1:]
    full = backward(cuda_lib, t, kept, dout, "silu", M, D, F)
    some = backward(cuda_lib, t, kept, dout, "silu", M, D, F, skip=skip)
    for name in full:
        if name in skip:
            assert bool(torch.isnan(some[name]).all())  # not written
        else:
            assert torch.equal(full[name], some[name])


@pytest.mark.parametrize("M", [30, 600])
def test_no_element_outside_is_written(cuda_lib, M):
    """Results in the middle of larger buffers: what surrounds them stays."""
    D, F = 136, 264
    t, residual, dout = inputs(M, D, F, seed=2)

    def middle(*shape):
        n = shape[0] * shape[1]
        flat = torch.full((n + 512,), 7.0, device="cuda", dtype=torch.bfloat16)
        return flat, flat[256:256 + n].view(shape)

    bufs = {k: middle(*s) for k, s in dict(out=(M, D), g=(M, F), u=(M, F), h=(M, F), dx=(M, D), dw_gate=(F, D), dw_up=(F, D),
                                           dw_down=(D, F)).items()}
    v = {k: b[1] for k, b in bufs.items()}
    cuda_lib.mlp_train(**t, residual=residual, out=v["out"], g=v["g"], u=v["u"], h=v["h"], M=M, D=D, F=F)
    n = cuda_lib.gbf_workspace_size("mlp_grad", M, D, F, True)
    ws = torch.full((n + 256,), 0x55, dtype=torch.uint8, device="cuda")
    cuda_lib.mlp_grad(dout, t["x"], v["g"], v["u"], v["h"], t["w_gate"], t["w_up"], t["w_down"], v["dx"], v["dw_gate"],
                      v["dw_up"], v["dw_down"], M, D, F, workspace=ws, workspace_bytes=n)
    for k, (flat, _) in bufs.items():
        assert bool((flat[:256] == 7.0).all()) and bool((flat[-256:] == 7.0).all()), k
    assert bool((ws[n:] == 0x55).all())
    check_forward(t, residual, (v["out"], v["g"], v["u"], v["h"]), "silu", D, F)


def test_no_rows(cuda_lib):
    D, F = 64, 72
    t, _, _ = inputs(4, D, F)
    t["x"] = t["x"][:0]
    e = torch.empty(0, D, device="cuda", dtype=torch.bfloat16)
    cuda_lib.mlp_train(**t, residual=None, out=e, g=None, u=None, h=None, M=0, D=D, F=F)
    dw = [nan(F, D), nan(F, D), nan(D, F)]
    cuda_lib.mlp_grad(None, None, None, None, None, t["w_gate"], t["w_up"], t["w_down"], None, *dw, M=0, D=D, F=F)
    assert all(bool((w == 0).all()) for w in dw)


def test_in_place_residual_and_agreement_with_the_inference_block(cuda_lib):
    M, D, F = 300, 264, 520
    t, residual, _ = inputs(M, D, F, seed=4)
    out = forward(cuda_lib, t, residual, "silu", M, D, F)[0]
    again = residual.clone()
    g, u, h = nan(M, F), nan(M, F), nan(M, F)
    cuda_lib.mlp_train(**t, residual=again, out=again, g=g, u=u, h=h, M=M, D=D, F=F)
    assert torch.equal(out, again)
    plain = nan(M, D)
    n = cuda_lib.gbf_workspace_size("mlp", M, D, F, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    cuda_lib.mlp_swiglu_down(t["x"], t["w_gate"], t["w_up"], t["w_down"], residual, plain, M, D, F, ws, n)
    # h of both is rounded from fp32 sums in other orders: a step of h here and there
    check_rms(out, plain.double(), "inference")


@pytest.mark.parametrize("M", [24, 600])
def test_captured_and_on_another_stream(cuda_lib, M):
    """The same bits eagerly, on a side stream, and replayed with other inputs in
    the captured buffers."""
    from tcgen05_tmem_bf16_gb300.graphs import CapturedChain
    D, F = 264, 520
    t, residual, dout = inputs(M, D, F, seed=6)
    t2, residual2, dout2 = inputs(M, D, F, seed=7)

    def step(t, residual, dout, stream=None):
        got = forward(cuda_lib, t, residual, "silu", M, D, F, stream)
        return got, backward(cuda_lib, t, got[1:], dout, "silu", M, D, F, stream=stream)

    want, want2 = step(t, residual, dout), step(t2, residual2, dout2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step(t, residual, dout)
    torch.cuda.synchronize()
    buf = dict(out=nan(M, D), g=nan(M, F), u=nan(M, F), h=nan(M, F))
    grads = dict(dx=nan(M, D), dw_gate=nan(F, D), dw_up=nan(F, D), dw_down=nan(D, F))
    n = cuda_lib.gbf_workspace_size("mlp_grad", M, D, F, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def chain_(stream):
        cuda_lib.mlp_train(**t, residual=residual, **buf, M=M, D=D, F=F, stream=stream)
        cuda_lib.mlp_grad(dout, t["x"], buf["g"], buf["u"], buf["h"], t["w_gate"], t["w_up"], t["w_down"], **grads, M=M, D=D,
                          F=F, workspace=ws, workspace_bytes=n, stream=stream)

    graph = CapturedChain(chain_)
    for a, b in ((t, want), (t2, want2)):
        for k in t:
            t[k].copy_(a[k])
        residual.copy_(residual if a is t else residual2)
        dout.copy_(dout if a is t else dout2)
        graph.replay()
        torch.cuda.synchronize()
        for k, v in zip(("out", "g", "u", "h"), b[0]):
            assert torch.equal(buf[k], v), k
        for k, v in b[1].items():
            assert torch.equal(grads[k], v), k
    for v, w in zip(other[0], want[0]):
        assert torch.equal(v, w)
    for k in want[1]:
        assert torch.equal(other[1][k], want[1][k])


def test_against_differences(cuda_lib):
    """The gradients along random directions, against differences of the fp64 block.
    An error of 0.82 R of each value, random, along a normal direction has 0.82 R of
    the gradient's norm; six times that is held, and the gradient's own part along the
    direction is as large as its norm."""
    M, D, F = 90, 136, 264
    t, _, dout = inputs(M, D, F, seed=8)
    kept = forward(cuda_lib, t, None, "silu", M, D, F)[1:]
    got = backward(cuda_lib, t, kept, dout, "silu", M, D, F)
    p = {k: v.double() for k, v in t.items()}

    def value(q):
        h = act64(q["x"] @ q["w_gate"].T, "silu") * (q["x"] @ q["w_up"].T)
        return float(((h @ q["w_down"].T) * dout.double()).sum())

    names = dict(x="dx", w_gate="dw_gate", w_up="dw_up", w_down="dw_down")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for k, name in names.items():
        for _ in range(3):
            v = torch.randn(p[k].shape, generator=gen, device="cuda", dtype=torch.float64)
            step = 1e-5
            diff = (value({**p, k: p[k] + step * v}) - value({**p, k: p[k] - step * v})) / (2 * step)
            grad = got[name].double()
            assert abs(float((grad * v).sum()) - diff) <= 6 * 0.82 * 3 * R * float(grad.norm()), name
            # (3: g, u and h kept in bf16 are roundings of their own)


def test_a_wait_that_runs_out_is_reported(cuda_lib):
    for M in (40, 600):
        D, F = 136, 264
        t, residual, dout = inputs(M, D, F, seed=M)
        want = forward(cuda_lib, t, residual, "silu", M, D, F)
        grads = backward(cuda_lib, t, want[1:], dout, "silu", M, D, F)
        try:
            cuda_lib.gbf_set_wait_timeout_ns(20_000_000)
            cuda_lib.gbf_debug_inject_timeout(True)
            backward(cuda_lib, t, want[1:], dout, "silu", M, D, F)
            assert cuda_lib.gbf_check_device_error() == 6
        finally:
            cuda_lib.gbf_debug_inject_timeout(False)
            cuda_lib.gbf_set_wait_timeout_ns(2_000_000_000)
        again = backward(cuda_lib, t, want[1:], dout, "silu", M, D, F)
        assert all(torch.equal(again[k], grads[k]) for k in grads)
        assert cuda_lib.gbf_check_device_error() == 0


def test_more_than_2_31_values(cuda_lib):
    """g, u and h of 2.3e9 values: sampled rows and columns."""
    M, D, F = 140000, 64, 16384
    t, residual, dout = inputs(M, D, F, seed=11)
    got = forward(cuda_lib, t, residual, "silu", M, D, F)
    rows = torch.tensor([0, 1, 70000, 131071, 131072, 139998, 139999], device="cuda")
    part = dict(t, x=t["x"][rows])
    check_forward(part, residual[rows], [v[rows] for v in got], "silu", D, F)
    grads = backward(cuda_lib, t, got[1:], dout, "silu", M, D, F)
    x, wg, wu, wd, g, u, h, dh, a, da = gradients64(part, [v[rows] for v in got[1:]], dout[rows], "silu")
    check_rms(grads["dx"][rows], (dh * u * da) @ wg + (dh * a) @ wu, "dx")
    cols = torch.tensor([0, 255, 256, 8191, 16383], device="cuda")
    g, u, h = (v[:, cols].double() for v in got[1:])
    dh = dout.double() @ t["w_down"][:, cols].double()
    g.requires_grad_()
    a = act64(g, "silu")
    (da,) = torch.autograd.grad(a.sum(), g)
    x = t["x"].double()
    check_rms(grads["dw_gate"][cols], (dh * u * da).T @ x, "dw_gate")
    check_rms(grads["dw_up"][cols], (dh * a.detach()).T @ x, "dw_up")
    check_rms(grads["dw_down"][:, cols], dout.double().T @ h, "dw_down")
