"""The operators at a model's two ends, run together as a training step."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def steps(heads, graph, n, V=1024, D=128, M=600, clusters=16):
    model = heads.TiedTable(V, D, M, alpha=4.0, graph=graph)
    g = torch.Generator(device="cuda").manual_seed(7)
    out = []
    for _ in range(n):
        prev, target = heads.clustered_text(M, V, clusters, g)
        prev[::17] = -1
        target[::13] = -100
        mean, norm = model.step(prev, target, rate=10.0)
        out.append((mean.clone(), norm.clone(), model.master.clone()))
    return model, out


def test_a_captured_step_equals_a_direct_one(cuda_lib):
    from tcgen05_tmem_bf16_gb300 import heads
    for a, b in zip(steps(heads, True, 4)[1], steps(heads, False, 4)[1]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_the_loss_falls(cuda_lib):
    from tcgen05_tmem_bf16_gb300 import heads
    _, out = steps(heads, True, 80)
    first, last = float(out[0][0]), float(out[-1][0])
    assert first > 6.0 and last < first - 1.0
    assert cuda_lib.gbf_check_device_error() == 0


def test_one_step_against_autograd(cuda_lib):
    """The clipped gradient of the tied table against 64-bit autograd of the
    same model on the bf16 table (x is rounded to bf16 on the way, as here).
    Tolerance: the logits' gradient in bf16 (2^-8 of every term, the terms'
    magnitudes bounded by their 2-norm over all values), dx and the table's two
    gradients rounded to bf16 once each."""
    from tcgen05_tmem_bf16_gb300 import heads
    V, D, M = 300, 64, 200
    model = heads.TiedTable(V, D, M, alpha=2.0, max_norm=1e-2, graph=False)
    g = torch.Generator(device="cuda").manual_seed(9)
    prev, target = heads.clustered_text(M, V, 10, g)
    prev[3], target[5] = -1, V
    table = model.table.double().requires_grad_()
    x = table[prev.clamp(min=0)] * (prev >= 0)[:, None]
    scored = target < V
    logits = 2.0 * x @ table.T
    loss = torch.nn.functional.cross_entropy(logits[scored], target[scored])
    loss.backward()
    norm = table.grad.norm()
    mean, got_norm = model.step(prev, target, rate=0.0)
    assert abs(float(mean) - float(loss)) < 1e-5 * float(loss)
    assert abs(float(got_norm) - float(norm)) < 4 * 2.0 ** -8 * float(norm)
    want = table.grad * min(1.0, 1e-2 / float(norm))
    assert float((model.dtable.double() - want).norm()) < 4 * 2.0 ** -8 * float(want.norm())
