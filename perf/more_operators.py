"""Measured cases of the operators that train a student model of gated blocks:
the gated MLP block that keeps what its gradient needs, with its gradient, the
gradient of the fused residual add + RMSNorm, and distillation from a teacher's
top logits through a linear head, with its gradients.

``run`` computes them in elementary torch operations in 32 bits (``own`` is
false) or through the library's entry points (``own`` is true), from the same
state.  Sizes: the widths 4096, 8192 and 14336 and the row counts 16, 64, 2048,
4096 and 8192 are the library's own workloads; the others are generic round and
odd numbers.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
GELU_C = math.sqrt(2.0 / math.pi)


def listed():
    return [
        # a few tokens through a full-size block, its gradient to follow: bound by reading the weights
        dict(name="block_16", op="block", M=16, D=4096, F=14336, act="silu", residual=True),
        # an ordinary batch
        dict(name="block_2048", op="block", M=2048, D=4096, F=14336, act="silu", residual=True),
        # a few tokens' gradient: the weights are read, and gradients as large written
        dict(name="block_grad_16", op="block_grad", M=16, D=4096, F=14336, act="silu"),
        # a small model's block with odd sizes and the other common activation
        dict(name="block_grad_1021_odd", op="block_grad", M=1021, D=1000, F=2728, act="gelu_tanh"),
        # a large batch
        dict(name="block_grad_4096", op="block_grad", M=4096, D=4096, F=14336, act="silu"),
        # a small model's last norm: nothing comes in through the residual
        dict(name="norm_grad_77", op="norm_grad", M=77, N=1000, residual=False),
        # a norm inside the residual stream of a large batch
        dict(name="norm_grad_8192", op="norm_grad", M=8192, N=4096, residual=True),
        # wide rows, an odd number of them
        dict(name="norm_grad_4099_wide", op="norm_grad", M=4099, N=8192, residual=True),
        # scoring one token of a student against a short list
        dict(name="distill_1", op="distill", M=1, V=32000, D=4096, K=8, alpha=1.0, beta=1.0, index="i64", teacher="f32", ignored=0.0),
        # scoring answers against a stored teacher: the prompts' half of the rows holds no list
        dict(name="distill_2047", op="distill", M=2047, V=128000, D=4096, K=64, alpha=1.0, beta=1.0, index="i32", teacher="bf16", ignored=0.5),
        # a small training batch: bound by reading and writing the weight
        dict(name="distill_train_64", op="distill_train", M=64, V=32000, D=4096, K=20, alpha=1.0, beta=1.0, index="i64", teacher="f32", ignored=0.0),
        # an ordinary batch with an odd vocabulary at temperature 2, lists of 50 entries and fewer
        dict(name="distill_train_4096_odd", op="distill_train", M=4096, V=50001, D=2048, K=50, alpha=0.5, beta=0.5, index="i64", teacher="bf16", ignored=0.3),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["block", "block_grad", "norm_grad", "distill", "distill_train"])
    M = spread(1, 8192)
    if op == "norm_grad":
        return dict(op=op, M=M, N=8 * spread(16, 2048), residual=rng.random() < 0.7)
    D = 8 * spread(32, 1024)
    if op in ("block", "block_grad"):
        F = 8 * spread(64, 1792)
        M = max(1, min(M, 4096 * 4096 * 14336 // (D * F)))
        act = rng.choice(["silu", "silu", "gelu_tanh", "relu"])
        return dict(op=op, M=M, D=D, F=F, act=act, residual=rng.random() < 0.7)
    V = spread(1000, 131072)
    M = max(1, min(M, 4096 * 50001 * 2048 // (V * D)))
    return dict(op=op, M=M, V=V, D=D, K=spread(1, 128), alpha=rng.choice([1.0, 0.5]), beta=rng.choice([1.0, 0.5]),
                index=rng.choice(["i64", "i32"]), teacher=rng.choice(["f32", "bf16"]), ignored=rng.choice([0.0, 0.3, 0.6]))


def scored_rows(case):
    return case["M"] - int(case["M"] * case["ignored"])


def teacher_lists(g, M, V, K):
    """Distinct ids and falling logits of a teacher's K likeliest tokens: the ids
    spread over the vocabulary like words' frequencies, in no order."""
    u = (torch.arange(K, device="cuda") + torch.rand(M, K, generator=g, device="cuda", dtype=torch.float64)) / K
    ids = ((V + 1.0) ** u).long() - 1
    k = torch.arange(K, device="cuda")
    ids = ((ids - k).cummax(dim=1).values + k).clamp_(0, V - 1)
    order = torch.rand(M, K, generator=g, device="cuda").argsort(dim=1)
    logits = torch.empty(M, K, device="cuda").normal_(8.0, 2.5, generator=g).sort(dim=1, descending=True).values
    return ids.gather(1, order), logits


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=BF16):
        return torch.empty(*shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)

    def empty(*shape, dtype=BF16):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = dict(case)
    op, M = case["op"], case["M"]
    nbytes = 0
    if op == "norm_grad":
        N = case["N"]
        s["r"], s["dnorm"], s["weight"] = normal(M, N, std=3.0), normal(M, N, std=1e-3), normal(N, std=0.1).add_(1.0)
        s["dresid"] = normal(M, N, std=1e-3) if case["residual"] else None
        s["eps"] = 1e-5
        s["dr"], s["dweight"] = empty(M, N), empty(N)
        if own:
            import tcgen05_tmem_bf16_gb300 as gbf
            nbytes = gbf.gbf_workspace_size("add_rmsnorm_grad", M, N, 0, True)
    elif op in ("block", "block_grad"):
        D, F = case["D"], case["F"]
        s["x"] = normal(M, D)
        s["wg"], s["wu"], s["wd"] = normal(F, D, std=D ** -0.5), normal(F, D, std=D ** -0.5), normal(D, F, std=F ** -0.5)
        if op == "block":
            s["res"] = normal(M, D) if case["residual"] else None
            s["out"], s["g"], s["u"], s["h"] = empty(M, D), empty(M, F), empty(M, F), empty(M, F)
        else:
            s["g"], s["u"] = normal(M, F), normal(M, F)
            s["h"] = (activation(s["g"].float(), case["act"])[0] * s["u"].float()).to(BF16)
            s["dout"] = normal(M, D, std=1e-3)
            s["dx"], s["dwg"], s["dwu"], s["dwd"] = empty(M, D), empty(F, D), empty(F, D), empty(D, F)
            if own:
                import tcgen05_tmem_bf16_gb300 as gbf
                nbytes = gbf.gbf_workspace_size("mlp_grad", M, D, F, True)
    else:
        V, D, K = case["V"], case["D"], case["K"]
        ids, logits = teacher_lists(g, M, V, K)
        # a third of the rows hold fewer entries (-1 behind the last), the ignored ones none
        length = torch.randint(1, K + 1, (M, 1), generator=g, device="cuda")
        length = torch.where(torch.rand(M, 1, generator=g, device="cuda") < 0.33, length, K)
        length[torch.randperm(M, generator=g, device="cuda")[:int(M * case["ignored"])]] = 0
        ids = torch.where(torch.arange(K, device="cuda") < length, ids, -1)
        s["ids"] = ids.to(torch.int32 if case["index"] == "i32" else torch.int64)
        s["logits"] = logits.to(BF16 if case["teacher"] == "bf16" else torch.float32)
        s["x"], s["w"] = normal(M, D), normal(V, D, std=2.0 / math.sqrt(D))
        s["loss"], s["lse"], s["mean"] = (empty(n, dtype=torch.float32) for n in (M, M, 1))
        if op == "distill_train":
            s["dx"], s["dw"] = empty(M, D), empty(V, D)
        if own:
            import tcgen05_tmem_bf16_gb300 as gbf
            nbytes = max(gbf.linear_distill_workspace_size(M, V, D, K, grad) for grad in (False, op == "distill_train"))
    if nbytes:
        s["ws"] = empty(nbytes, dtype=torch.uint8)
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import tcgen05_tmem_bf16_gb300 as gbf
    op, M = s["op"], s["M"]
    ws = dict(workspace=s["ws"], workspace_bytes=s["ws"].numel()) if "ws" in s else {}
    if op == "norm_grad":
        gbf.add_rmsnorm_grad(s["dnorm"], s["dresid"], s["r"], s["weight"], s["dr"], s["dweight"], M, s["N"], s["eps"], **ws)
        return s["dr"], s["dweight"]
    if op == "block":
        gbf.mlp_train(s["x"], s["wg"], s["wu"], s["wd"], s["res"], s["out"], s["g"], s["u"], s["h"], M, s["D"], s["F"], s["act"])
        return s["out"], s["g"], s["u"], s["h"]
    if op == "block_grad":
        gbf.mlp_grad(s["dout"], s["x"], s["g"], s["u"], s["h"], s["wg"], s["wu"], s["wd"], s["dx"], s["dwg"], s["dwu"], s["dwd"],
                     M, s["D"], s["F"], s["act"], **ws)
        return s["dx"], s["dwg"], s["dwu"], s["dwd"]
    sizes = (M, s["V"], s["D"], s["K"], s["alpha"], s["beta"])
    kinds = dict(index_type=s["index"], teacher_type=s["teacher"])
    gbf.linear_distill(s["x"], s["w"], s["ids"], s["logits"], s["loss"], s["lse"], s["mean"], *sizes, **kinds, **ws)
    if op == "distill":
        return s["loss"], s["lse"], s["mean"]
    gbf.linear_distill_grad(s["x"], s["w"], s["ids"], s["logits"], s["lse"], None, s["dx"], s["dw"], *sizes, 1.0, "mean", **kinds, **ws)
    return s["loss"], s["lse"], s["mean"], s["dx"], s["dw"]


def activation(v, act):
    """The activation and its derivative."""
    if act == "relu":
        return v.clamp(min=0.0), (v > 0).to(v.dtype)
    if act == "silu":
        t = 1.0 / (1.0 + (-v).exp())
        return v * t, t * (1.0 + v * (1.0 - t))
    z2 = 2.0 * GELU_C * (v + 0.044715 * v * v * v)  # 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z))
    t = 1.0 / (1.0 + (-z2).exp())
    return v * t, t + v * t * (1.0 - t) * 2.0 * GELU_C * (1.0 + 3.0 * 0.044715 * v * v)


def run_plain(s):
    op, M = s["op"], s["M"]
    if op == "norm_grad":
        r, dn, w = s["r"].float(), s["dnorm"].float(), s["weight"].float()
        inv = 1.0 / ((r * r).mean(dim=1, keepdim=True) + s["eps"]).sqrt()
        unit, dw = r * inv, dn * w
        dr = inv * (dw - unit * (dw * unit).mean(dim=1, keepdim=True))
        if s["dresid"] is not None:
            dr = dr + s["dresid"].float()
        return dr.to(BF16), (dn * unit).sum(dim=0).to(BF16)
    if op in ("block", "block_grad"):
        wg, wu, wd = s["wg"].float(), s["wu"].float(), s["wd"].float()
        x = s["x"].float()
        if op == "block":
            g, u = x @ wg.T, x @ wu.T
            h = (activation(g, s["act"])[0] * u).to(BF16)  # a result of its own: the down product takes it as stored
            out = h.float() @ wd.T
            if s["res"] is not None:
                out = out + s["res"].float()
            return out.to(BF16), g.to(BF16), u.to(BF16), h
        g, u, h, dout = s["g"].float(), s["u"].float(), s["h"].float(), s["dout"].float()
        dh = dout @ wd
        a, da = activation(g, s["act"])
        dg, du = dh * u * da, dh * a
        return (dg @ wg + du @ wu).to(BF16), (dg.T @ x).to(BF16), (du.T @ x).to(BF16), (dout.T @ h).to(BF16)
    x, w = s["x"].float(), s["w"].float()
    ids = s["ids"].long()
    valid = ids >= 0
    at = ids.clamp(min=0)
    scored = valid.any(dim=1)
    t = torch.where(valid, s["beta"] * s["logits"].float(), -math.inf)
    t = torch.where(scored[:, None], t - t.amax(dim=1, keepdim=True), 0.0)
    e = torch.where(valid, t.exp(), 0.0)
    total_q = e.sum(dim=1, keepdim=True).clamp(min=1e-30)
    q = e / total_q
    log_q = torch.where(valid, t - total_q.log(), 0.0)
    l = s["alpha"] * (x @ w.T)
    top = l.amax(dim=1, keepdim=True)
    p = (l - top).exp()
    total = p.sum(dim=1, keepdim=True)
    log_total = total.log()
    each = torch.where(valid, q * (log_q - ((l.gather(1, at) - top) - log_total)), 0.0)
    loss = torch.where(scored, each.sum(dim=1), 0.0)
    lse = torch.where(scored, (top + log_total)[:, 0], 0.0)
    count = scored.sum().clamp(min=1)
    mean = (loss.sum(dtype=torch.float64) / count).float().reshape(1)
    if op == "distill":
        return loss, lse, mean
    grad = (p / total).scatter_add_(1, at, -q)
    grad *= torch.where(scored, s["alpha"] / count, 0.0)[:, None]
    return loss, lse, mean, (grad @ w).to(BF16), (grad.T @ x).to(BF16)


def work(case):
    op, M = case["op"], case["M"]
    if op == "norm_grad":
        N = case["N"]
        return {"bytes": 2 * M * N * (4 if case["residual"] else 3) + 4 * N, "flops": 12 * M * N}
    if op in ("block", "block_grad"):
        D, F = case["D"], case["F"]
        weights = 2 * 3 * D * F
        if op == "block":
            return {"bytes": weights + 2 * M * D * (3 if case["residual"] else 2) + 2 * 3 * M * F, "flops": 6 * M * D * F}
        return {"bytes": 2 * weights + 2 * M * D * 3 + 2 * 3 * M * F, "flops": 12 * M * D * F}
    V, D, K = case["V"], case["D"], case["K"]
    rows = scored_rows(case)
    lists = M * K * ((4 if case["index"] == "i32" else 8) + (2 if case["teacher"] == "bf16" else 4))
    once = lists + 2 * rows * D + 2 * V * D + 8 * M + 4
    if op == "distill":
        return {"bytes": once, "flops": 2 * rows * V * D}
    return {"bytes": once + 2 * M * D + 2 * V * D, "flops": 6 * rows * V * D}


def exact(case, seed):
    s = prepare(case, seed)
    op, M = case["op"], case["M"]
    if op == "norm_grad":
        r = s["r"].double().requires_grad_()
        weight = s["weight"].double().requires_grad_()
        norm = torch.nn.functional.rms_norm(r, (case["N"],), weight, s["eps"])
        torch.autograd.backward(norm, s["dnorm"].double())
        dr = r.grad if s["dresid"] is None else r.grad.add_(s["dresid"].double())
        return dr, weight.grad
    fn = torch.nn.functional
    if op in ("block", "block_grad"):
        def gated(g, u):
            a = fn.gelu(g, approximate="tanh") if case["act"] == "gelu_tanh" else getattr(fn, case["act"])(g)
            return a * u

        x, wg, wu, wd = (s[n].double() for n in ("x", "wg", "wu", "wd"))
        if op == "block":
            g, u = fn.linear(x, wg), fn.linear(x, wu)
            h = gated(g, u)
            out = fn.linear(h.to(BF16).double(), wd)
            return (out if s["res"] is None else out.add_(s["res"])), g, u, h
        dout = s["dout"].double()
        g, u = (s[n].double().requires_grad_() for n in ("g", "u"))
        torch.autograd.backward(gated(g, u), torch.matmul(dout, wd))
        dx = torch.addmm(torch.mm(g.grad, wg), u.grad, wu)
        return dx, torch.mm(g.grad.t(), x), torch.mm(u.grad.t(), x), torch.mm(dout.t(), s["h"].double())
    ids = s["ids"].long()
    rows = torch.nonzero((ids >= 0).any(dim=1))[:, 0]
    ids, x, w = ids[rows], s["x"][rows].double(), s["w"].double()
    log_q = torch.log_softmax((s["logits"][rows].double() * case["beta"]).masked_fill_(ids < 0, -math.inf), dim=1)
    logits = torch.mm(x, w.t()).mul_(case["alpha"])
    lse_rows = torch.logsumexp(logits, dim=1)
    q = log_q.exp()
    log_p = logits.gather(1, ids.clamp(min=0)) - lse_rows[:, None]
    loss = torch.zeros(M, device="cuda", dtype=torch.float64)
    lse = torch.zeros(M, device="cuda", dtype=torch.float64)
    loss[rows] = torch.where(ids < 0, 0.0, q * (log_q - log_p)).sum(dim=1)
    lse[rows] = lse_rows
    count = max(1, rows.numel())
    mean = loss.sum().reshape(1) / count
    if op == "distill":
        return loss, lse, mean
    grad = logits.sub_(lse_rows[:, None]).exp_()
    grad.scatter_add_(1, ids.clamp(min=0), -q)
    grad *= case["alpha"] / count
    dx = torch.zeros(M, case["D"], device="cuda", dtype=torch.float64)
    dx[rows] = torch.mm(grad, w)
    return loss, lse, mean, dx, torch.mm(grad.t(), x)
