"""A step of the student model -- every operator of a gated block's and a distilled
head's training, one after another -- against fp64 autograd of the same model."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

R = 2.0 ** -8


def batch(V, M, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, V, (M,), generator=g, device="cuda")
    ids[::7] = -1
    entries = torch.randint(0, V, (M, K), generator=g, device="cuda")
    entries[::5, K // 2:] = -1
    entries[::11] = -100
    return ids, entries, torch.randn(M, K, generator=g, device="cuda") * 2.0


def plain(model, ids, entries, logits):
    """The mean loss and the gradients before clipping, in fp64."""
    p = {k: v.double().requires_grad_() for k, v in model.parameters.items()}
    f = torch.nn.functional
    table = torch.cat([p["table"], torch.zeros(1, model.D, device="cuda", dtype=torch.float64)])
    r = table[torch.where(ids < 0, model.V, ids)]
    for l in range(model.L):
        n = f.rms_norm(r, (model.D,), p[f"norm.{l}"], model.eps)
        h = f.silu(n @ p[f"gate.{l}"].T) * (n @ p[f"up.{l}"].T)
        r = r + h @ p[f"down.{l}"].T
    n = f.rms_norm(r, (model.D,), p[f"norm.{model.L}"], model.eps)
    valid = (entries >= 0) & (entries < model.V)
    rows = valid.any(dim=1)
    t = torch.where(valid, model.beta * logits.double(), -math.inf)[rows]
    q = torch.softmax(t, dim=1)
    log_p = torch.log_softmax(model.alpha * (n @ p["table"].T), dim=1)[rows]
    q = torch.zeros_like(log_p).scatter_add_(1, entries.clamp(0, model.V - 1)[rows], q)
    loss = torch.where(q > 0, q * (q.clamp(min=1e-300).log() - log_p), 0.0).sum(dim=1).mean()
    (model.scale * loss).backward()
    return loss.detach(), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("M,D,F", [(24, 136, 264), (140, 64, 200), (600, 136, 264)])
def test_a_step_against_fp64(cuda_lib, M, D, F):
    """Each of some 9 tensors per block and 6 beside them that are stored in bf16 along
    the way is off by up to R of itself, at random; the loss, whose logits come from a
    last norm of such a stream, by as much of its terms."""
    from tcgen05_tmem_bf16_gb300.student import Student
    V, K, L = 500, 12, 2
    b = batch(V, M, K, seed=M)
    model = Student(V, D, F, L, M, K, alpha=3.0, temperature=2.0, graph=False, max_norm=math.inf)
    want, grads = plain(model, *b)
    model.ids.copy_(b[0]), model.entries.copy_(b[1]), model.logits.copy_(b[2])
    model.launch()
    n = 9 * L + 6
    assert abs(float(model.mean) - float(want)) <= math.sqrt(n) * R * float(1.0 + want)
    for k, w in grads.items():
        err = float((model.grads[k].double() - w).norm() / w.norm())
        assert err <= math.sqrt(n) * R, (k, err)
    norm = math.sqrt(sum(float(w.square().sum()) for w in grads.values()))
    assert abs(float(model.norm) - norm) <= math.sqrt(n) * R * norm
    assert cuda_lib.gbf_check_device_error() == 0


def test_captured_steps_are_the_direct_ones(cuda_lib):
    """Three steps with clipping, replayed and issued directly: the same bits."""
    from tcgen05_tmem_bf16_gb300.student import Student
    V, D, F, M, K = 700, 136, 264, 200, 9
    models = [Student(V, D, F, 2, M, K, alpha=3.0, max_norm=0.05, graph=g) for g in (True, False)]
    for i in range(3):
        b = batch(V, M, K, seed=i)
        (a, na), (c, nc) = (m.step(*b, rate=0.5) for m in models)
        torch.cuda.synchronize()
        assert torch.equal(a, c) and torch.equal(na, nc)
        for k in models[0].grads:
            assert torch.equal(models[0].grads[k], models[1].grads[k]), k
            assert torch.equal(models[0].parameters[k], models[1].parameters[k]), k


def test_two_chains_share_a_workspace(cuda_lib):
    """Two captured students on one stream, one workspace: each call of one writes what it
    reads, so replays in turn give the bits of replays alone."""
    from tcgen05_tmem_bf16_gb300.student import Student
    V, D, F, M, K = 500, 64, 136, 150, 5
    b = batch(V, M, K, seed=9)
    alone = [Student(V, D, F, 1, M, K, seed=s) for s in (1, 2)]
    want = [(float(m.step(*b)[0]), {k: v.clone() for k, v in m.grads.items()}) for m in alone]
    pair = [Student(V, D, F, 1, M, K, seed=s, graph=False) for s in (1, 2)]
    pair[1].workspace = pair[0].workspace
    from tcgen05_tmem_bf16_gb300.graphs import CapturedChain
    for m in pair:
        m.graph = CapturedChain(m.launch)
    got = [m.step(*b)[0] for m in pair]
    for m, g, (loss, grads) in zip(pair, got, want):
        assert float(g) == loss
        for k in grads:
            assert torch.equal(m.grads[k], grads[k]), k


def test_the_example_runs(cuda_lib, capsys):
    from tcgen05_tmem_bf16_gb300 import student
    student.main()
    out = capsys.readouterr().out
    assert out.count("KL from the teacher") == 6 and "nan" not in out
    assert cuda_lib.gbf_check_device_error() == 0
