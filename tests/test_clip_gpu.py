"""clip_grad_norm against a 64-bit reference.

Tolerances.  The norm: a thread adds up at most 16 sums of eight squares (bf16)
or 32 sums of four (fp32) per chunk in fp32, the rest in 64 bits: off by at
most 40 * 2^-24 of the sum of squares, half of that after the root, and one
rounding to fp32.  The outputs: the factor (the norm's error and one rounding),
the product's rounding to fp32 and, for bf16, half a step (2^-8)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24
NORM_TOL = 20 * F32 + 2 * F32
OUT_TOL = {torch.float32: NORM_TOL + 3 * F32, torch.bfloat16: NORM_TOL + 3 * F32 + 2.0 ** -8}


def clip(lib, grads, out, max_norm, eps=1e-6):
    n = lib.gbf_workspace_size("clip_grad_norm", len(grads), 0, 0, True)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    norm = torch.full((1,), -1.0, device="cuda")
    lib.clip_grad_norm(grads, out, max_norm, norm, eps, workspace=ws, workspace_bytes=n)
    return norm


def reference(grads, max_norm, eps=1e-6):
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    f32 = lambda x: float(torch.tensor(x, dtype=torch.float32))  # noqa: E731
    return norm, min(1.0, f32(max_norm) / (norm + f32(eps))) if norm else 1.0


def close(got, want, tol):
    # below the normal range a result is off by up to half the smallest step of bf16
    return ((got.double() - want).abs() <= tol * want.abs() + 2.0 ** -134).all()


def check(lib, grads, max_norm, in_place):
    norm, factor = reference(grads, max_norm)
    raw = [t.clone() for t in grads]
    out = None if in_place else [torch.full_like(t, 99.0) for t in grads]
    got = clip(lib, grads, out, max_norm)
    assert abs(float(got) - norm) <= NORM_TOL * norm
    for t, r, o in zip(grads, raw, out or grads):
        assert close(o, r.double() * factor, OUT_TOL[t.dtype])
        if factor == 1.0:
            assert torch.equal(o, r)
        if not in_place:
            assert torch.equal(t, r)


SIZES = [[1], [7], [8, 9, 15], [4096, 1, 100000], [32768, 32769, 65535, 3], [1 << 20, 5, 333333], [0, 17, 0]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("kind", ["bf16", "f32", "mixed"])
@pytest.mark.parametrize("clipped", [True, False])
@pytest.mark.parametrize("in_place", [True, False])
def test_norm_and_clipping(cuda_lib, sizes, kind, clipped, in_place):
    g = torch.Generator(device="cuda").manual_seed(sum(sizes))
    types = {"bf16": [torch.bfloat16], "f32": [torch.float32], "mixed": [torch.float32, torch.bfloat16]}[kind]
    grads = [torch.randn(n, generator=g, device="cuda").to(types[i % len(types)]) for i, n in enumerate(sizes)]
    check(cuda_lib, grads, (0.25 if clipped else 4.0) * math.sqrt(sum(sizes)), in_place)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_views_at_every_offset(cuda_lib, dtype):
    """Inputs and outputs that begin at any element of a 16-byte block."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    g = torch.Generator(device="cuda").manual_seed(9)
    n = 5003
    flat = torch.randn(per * per * (n + 2 * per), generator=g, device="cuda").to(dtype)
    into = torch.full_like(flat, 55.0)
    touched = torch.zeros_like(flat, dtype=torch.bool)
    grads, out = [], []
    for i in range(per):
        for j in range(per):
            at = (i * per + j) * (n + 2 * per)
            at = -(-at // per) * per
            grads.append(flat[at + i:at + i + n])
            out.append(into[at + j:at + j + n])
            touched[at + j:at + j + n] = True
    norm, factor = reference(grads, 10.0)
    got = clip(cuda_lib, grads, out, 10.0)
    assert abs(float(got) - norm) <= NORM_TOL * norm
    for t, o in zip(grads, out):
        assert close(o, t.double() * factor, OUT_TOL[dtype])
    assert (into[~touched] == 55.0).all()


@pytest.mark.parametrize("count", [64, 65, 513, 1100])
def test_many_tensors(cuda_lib, count):
    g = torch.Generator(device="cuda").manual_seed(count)
    grads = [torch.randn(1 + 37 * i % 501, generator=g, device="cuda").to([torch.float32, torch.bfloat16][i % 2])
             for i in range(count)]
    check(cuda_lib, grads, 1.0, False)
    check(cuda_lib, grads, 1.0, True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1e-30, 1e-20, 1.0, 1e15, 1e20, 1e30])
def test_squares_beyond_the_range_of_fp32(cuda_lib, dtype, size):
    g = torch.Generator(device="cuda").manual_seed(1)
    grads = [(torch.randn(50000, generator=g, device="cuda") * size).to(dtype), torch.zeros(1000, device="cuda")]
    check(cuda_lib, grads, 30.0 * size, False)


def test_sizes_far_apart(cuda_lib):
    x = torch.zeros(40000, device="cuda")
    x[123] = 3e25
    x[30000:] = 1e-25
    check(cuda_lib, [x], 1.0, False)


def test_infinite_and_nan_values(cuda_lib):
    x = torch.ones(1000, device="cuda", dtype=torch.bfloat16)
    x[10] = float("inf")
    out = [torch.empty_like(x)]
    assert float(clip(cuda_lib, [x], out, 1.0)) == float("inf")
    assert torch.isnan(out[0][10]) and (out[0][:10] == 0).all() and (out[0][11:] == 0).all()
    x[10] = float("nan")
    assert math.isnan(float(clip(cuda_lib, [x], out, 1.0)))
    assert torch.isnan(out[0]).all()


def test_zeros_no_tensors_and_the_norm_alone(cuda_lib):
    z = torch.zeros(100, device="cuda")
    assert float(clip(cuda_lib, [z], None, 0.0, 0.0)) == 0.0 and (z == 0).all()
    assert float(clip(cuda_lib, [], None, 1.0)) == 0.0
    x = torch.full((100,), 3.0, device="cuda")
    assert float(clip(cuda_lib, [x], None, float("inf"))) == 30.0 and (x == 3).all()
    x[0] = float("inf")
    assert float(clip(cuda_lib, [x], None, float("inf"))) == float("inf") and (x[1:] == 3).all()


def test_same_bits_on_every_run_and_in_a_graph(cuda_lib):
    g = torch.Generator(device="cuda").manual_seed(2)
    grads = [torch.randn(n, generator=g, device="cuda") for n in (3000000, 777, 1234567)]
    first = clip(cuda_lib, grads, None, float("inf"))
    for _ in range(5):
        assert torch.equal(first, clip(cuda_lib, grads, None, float("inf")))
    n = cuda_lib.gbf_workspace_size("clip_grad_norm", 3, 0, 0, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    norm = torch.zeros(1, device="cuda")
    out = [torch.empty_like(t) for t in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.clip_grad_norm(grads, out, 1.0, norm, workspace=ws, workspace_bytes=n)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, norm)
    _, factor = reference(grads, 1.0)
    assert all(close(o, t.double() * factor, OUT_TOL[torch.float32]) for o, t in zip(out, grads))
