"""Measured cases of the operators at the two ends of a language model: the
embedding lookup with its gradient, the linear cross entropy over a
vocabulary with its gradients, and the global gradient norm with clipping.

``run`` computes them in elementary torch operations in 32 bits (``own`` is
false) or through the library's entry points (``own`` is true), from the same
state.  Sizes: hidden widths 4096 and 8192, the MLP width 14336 and row counts
1, 16, 64, 4096 and 8192 are the library's own workloads; the vocabularies are
generic round and odd numbers.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
IGNORE = -100  # a target that is not scored


def listed():
    return [
        # a decode step of 16 sequences looks up its next inputs
        dict(name="lookup_decode_16", op="lookup", M=16, V=32000, D=4096, scale=1.0, index="i64", pad=0.0),
        # a long prompt batch, sqrt(D) scaling, some padded positions (-1), 32-bit ids
        dict(name="lookup_prompts_16383", op="lookup", M=16383, V=128000, D=8192, scale=math.sqrt(8192.0), index="i32", pad=0.1),
        # an untied table's dense gradient from a short batch: most rows are zeros
        dict(name="embed_grad_1021", op="embed_grad", M=1021, V=32000, D=1024, scale=1.0, accumulate=False, index="i64", pad=0.05),
        # a tied table: added to the gradient that the loss left there
        dict(name="embed_grad_tied_16384", op="embed_grad", M=16384, V=128000, D=4096, scale=64.0, accumulate=True, index="i64", pad=0.0),
        # scoring one token after a decode step
        dict(name="ce_score_1", op="ce", M=1, V=32000, D=4096, alpha=1.0, index="i64", ignored=0.0),
        # scoring answers: the prompts' half of the rows is not scored
        dict(name="ce_score_2047", op="ce", M=2047, V=128000, D=4096, alpha=1.0, index="i32", ignored=0.5),
        # a small training batch: bound by reading and writing the weight
        dict(name="ce_train_64", op="ce_train", M=64, V=32000, D=4096, alpha=1.0, index="i64", ignored=0.0),
        # an ordinary batch of instruction tuning with an odd vocabulary and a logit scale
        dict(name="ce_train_4096_odd", op="ce_train", M=4096, V=50001, D=2048, alpha=0.5, index="i64", ignored=0.3),
        # a large batch of plain text
        dict(name="ce_train_8192", op="ce_train", M=8192, V=65536, D=4096, alpha=1.0, index="i64", ignored=0.0),
        # small adapters' gradients of mixed types, odd views into flat buffers, below the limit, in place
        dict(name="clip_small_in_place", op="clip", layers=10, D=512, F=64, V=0, clipped=False, in_place=True),
        # the gradients of four gated MLP blocks and a table, above the limit, into new buffers
        dict(name="clip_blocks", op="clip", layers=4, D=4096, F=14336, V=32000, clipped=True, in_place=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["lookup", "embed_grad", "ce", "ce_train", "clip"])
    D = 8 * spread(32, 1024)
    V = spread(1000, 131072)
    M = spread(1, 16384)
    index = rng.choice(["i64", "i32"])
    if op == "lookup":
        return dict(op=op, M=M, V=V, D=D, scale=rng.choice([1.0, math.sqrt(D)]), index=index, pad=rng.choice([0.0, 0.1]))
    if op == "embed_grad":
        V = min(V, 128000 * 4096 // D)
        return dict(op=op, M=M, V=V, D=D, scale=rng.choice([1.0, math.sqrt(D)]), accumulate=rng.random() < 0.5, index=index, pad=rng.choice([0.0, 0.1]))
    if op == "clip":
        D = 8 * spread(16, 512)
        return dict(op=op, layers=spread(1, 10), D=D, F=8 * spread(8, 700), V=rng.choice([0, spread(1000, 16000)]),
                    clipped=rng.random() < 0.5, in_place=False)
    M = max(1, min(M, 8192, 8192 * 65536 * 4096 // (V * D)))
    return dict(op=op, M=M, V=V, D=D, alpha=rng.choice([1.0, 0.5]), index=index, ignored=rng.choice([0.0, 0.3, 0.6]))


def valid_rows(case):
    return case["M"] - int(case["M"] * case["ignored"])


def tensor_sizes(case):
    """(elements, in 32 bits) of each gradient: per block two width-D norms (32 bits) and three matrices, a head bias of odd length, a table."""
    D, F = case["D"], case["F"]
    block = [(D, True), (F * D, False), (F * D, False), (D, True), (D * F, False)]
    return block * case["layers"] + [(2 * D + 1, True)] + ([(case["V"] * D, False)] if case["V"] else [])


def ids_like_text(g, n, V):
    """Ids whose frequency falls like 1 / rank, as words' do."""
    return ((V + 1.0) ** torch.rand(n, generator=g, device="cuda", dtype=torch.float64)).long().sub_(1).clamp_(0, V - 1)


def expected_rows(n, V):
    """How many different ids n draws of ids_like_text hold on average."""
    k = torch.arange(V, dtype=torch.float64)
    p = torch.log((k + 2) / (k + 1)) / math.log(V + 1.0)
    return float((1 - (1 - p) ** n).sum())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=BF16):
        return torch.empty(*shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)

    s = dict(case)
    op = case["op"]
    if op == "clip":
        sizes = tensor_sizes(case)
        flat = {True: normal(1 + sum(n for n, wide in sizes if wide), std=2e-3, dtype=torch.float32),
                False: normal(1 + sum(n for n, wide in sizes if not wide), std=2e-3)}
        at = {True: 1, False: 1}  # the buckets' views begin at odd elements
        s["grads"] = []
        for n, wide in sizes:
            s["grads"].append(flat[wide][at[wide]:at[wide] + n])
            at[wide] += n
        total = sum(n for n, _ in sizes)
        s["max_norm"] = 2e-3 * math.sqrt(total) * (0.3 if case["clipped"] else 3.0)
        s["out"] = s["grads"] if case["in_place"] else [torch.empty_like(t) for t in s["grads"]]
        s["norm"] = torch.empty(1, device="cuda", dtype=torch.float32)
        if own:
            import tcgen05_tmem_bf16_gb300 as gbf
            s["grad_list"] = gbf.TensorList(s["grads"])
            s["out_list"] = None if case["in_place"] else gbf.TensorList(s["out"])
            s["ws"] = torch.empty(gbf.gbf_workspace_size("clip_grad_norm", len(sizes), 0, 0, True), dtype=torch.uint8, device="cuda")
        return s

    M, V, D = case["M"], case["V"], case["D"]
    kind = torch.int32 if case["index"] == "i32" else torch.int64
    ids = ids_like_text(g, M, V)
    if op in ("lookup", "embed_grad"):
        pads = torch.randperm(M, generator=g, device="cuda")[:int(M * case["pad"])]
        ids[pads] = -1
        s["ids"] = ids.to(kind)
        if op == "lookup":
            s["table"] = normal(V, D, std=0.02)
            s["out"] = torch.empty(M, D, device="cuda", dtype=BF16)
        else:
            s["dout"] = normal(M, D, std=1e-3)
            # what a loss has left in a tied table's gradient; each pass adds to it
            s["dtable"] = normal(V, D, std=1e-2) if case["accumulate"] else torch.empty(V, D, device="cuda", dtype=BF16)
    else:
        if op == "ce" or case["ignored"] > 0:
            ids[torch.randperm(M, generator=g, device="cuda")[:int(M * case["ignored"])]] = IGNORE
        s["targets"] = ids.to(kind)
        s["x"] = normal(M, D)
        s["w"] = normal(V, D, std=2.0 / math.sqrt(D))
        s["loss"] = torch.empty(M, device="cuda", dtype=torch.float32)
        s["lse"] = torch.empty(M, device="cuda", dtype=torch.float32)
        s["mean"] = torch.empty(1, device="cuda", dtype=torch.float32)
        if op == "ce_train":
            s["dx"] = torch.empty(M, D, device="cuda", dtype=BF16)
            s["dw"] = torch.empty(V, D, device="cuda", dtype=BF16)
    if own and op != "lookup":
        import tcgen05_tmem_bf16_gb300 as gbf
        names = {"embed_grad": ["embedding_grad"], "ce": ["linear_ce"], "ce_train": ["linear_ce", "linear_ce_grad"]}[op]
        nbytes = max(gbf.gbf_workspace_size(n, M, V, D, True) for n in names)
        s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import tcgen05_tmem_bf16_gb300 as gbf
    op = s["op"]
    ws = s.get("ws")
    if op == "clip":
        gbf.clip_grad_norm(s["grad_list"], s["out_list"], s["max_norm"], s["norm"], workspace=ws, workspace_bytes=ws.numel())
        return s["norm"], s["out"]
    M, V, D = s["M"], s["V"], s["D"]
    if op == "lookup":
        gbf.embedding_lookup(s["ids"], s["table"], s["out"], M, V, D, s["scale"], index_type=s["index"])
        return s["out"]
    if op == "embed_grad":
        gbf.embedding_grad(s["ids"], s["dout"], s["dtable"], M, V, D, s["scale"], s["accumulate"], index_type=s["index"],
                           workspace=ws, workspace_bytes=ws.numel())
        return s["dtable"]
    gbf.linear_ce(s["x"], s["w"], s["targets"], s["loss"], s["lse"], s["mean"], M, V, D, s["alpha"], index_type=s["index"],
                  workspace=ws, workspace_bytes=ws.numel())
    if op == "ce":
        return s["loss"], s["lse"], s["mean"]
    gbf.linear_ce_grad(s["x"], s["w"], s["targets"], s["lse"], None, s["dx"], s["dw"], M, V, D, s["alpha"], 1.0, "mean",
                       index_type=s["index"], workspace=ws, workspace_bytes=ws.numel())
    return s["loss"], s["lse"], s["mean"], s["dx"], s["dw"]


def run_plain(s):
    op = s["op"]
    if op == "clip":
        squares = [t.float().square().sum(dtype=torch.float64) for t in s["grads"]]
        norm = torch.stack(squares).sum().sqrt()
        factor = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
        out = [(t.float() * factor).to(t.dtype) for t in s["grads"]]
        return norm.float().reshape(1), out
    M, V, D = s["M"], s["V"], s["D"]
    if op == "lookup":
        ids = s["ids"].long()
        rows = s["table"][ids.clamp(min=0)].float() * s["scale"]
        return torch.where((ids >= 0)[:, None], rows, 0.0).to(BF16)
    if op == "embed_grad":
        ids = s["ids"].long()
        rows = torch.where((ids >= 0)[:, None], s["dout"].float() * s["scale"], 0.0)
        total = s["dtable"].float() if s["accumulate"] else torch.zeros(V, D, device="cuda")
        return s["dtable"].copy_(total.index_add_(0, ids.clamp(min=0), rows))
    x, w = s["x"].float(), s["w"].float()
    targets = s["targets"].long()
    scored = targets >= 0
    at = targets.clamp(min=0)[:, None]
    logits = s["alpha"] * (x @ w.T)
    top = logits.amax(dim=1, keepdim=True)
    p = (logits - top).exp()
    total = p.sum(dim=1, keepdim=True)
    lse = top + total.log()
    loss = torch.where(scored, (lse - logits.gather(1, at))[:, 0], 0.0)
    lse = torch.where(scored, lse[:, 0], 0.0)
    count = scored.sum().clamp(min=1)
    mean = (loss.sum(dtype=torch.float64) / count).float().reshape(1)
    if op == "ce":
        return loss, lse, mean
    g = p / total
    g.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=torch.float32))
    g *= torch.where(scored, s["alpha"] / count, 0.0)[:, None]
    return loss, lse, mean, (g @ w).to(BF16), (g.T @ x).to(BF16)


def work(case):
    op = case["op"]
    if op == "clip":
        sizes = tensor_sizes(case)
        held = sum(n * (4 if wide else 2) for n, wide in sizes)
        return {"bytes": held * (1 if case["in_place"] else 2) + 4, "flops": 3 * sum(n for n, _ in sizes)}
    M, V, D = case["M"], case["V"], case["D"]
    ids = M * (4 if case["index"] == "i32" else 8)
    if op == "lookup":
        some = M - int(M * case["pad"])
        return {"bytes": ids + 2 * D * (some + M), "flops": some * D}
    if op == "embed_grad":
        some = M - int(M * case["pad"])
        # added to a gradient: the rows of the ids that occur are read and written; alone: the whole table is written
        table = 4 * D * expected_rows(some, V) if case["accumulate"] else 2 * V * D
        return {"bytes": ids + 2 * some * D + table, "flops": 2 * some * D}
    rows = valid_rows(case)
    once = ids + 2 * rows * D + 2 * V * D + 8 * M + 4
    if op == "ce":
        return {"bytes": once, "flops": 2 * rows * V * D}
    return {"bytes": once + 2 * M * D + 2 * V * D, "flops": 6 * rows * V * D}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grads"]))
        factor = min(1.0, s["max_norm"] / (norm + 1e-6))
        return torch.tensor([norm], dtype=torch.float64), [t.double() * factor for t in s["grads"]]
    M, V, D = case["M"], case["V"], case["D"]
    if op == "lookup":
        table = torch.cat([s["table"].double(), torch.zeros(1, D, device="cuda", dtype=torch.float64)])
        ids = s["ids"].long()
        return torch.nn.functional.embedding(torch.where(ids < 0, V, ids), table) * s["scale"]
    if op == "embed_grad":
        ids = s["ids"].long()
        kept = ids >= 0
        order = torch.argsort(ids[kept], stable=True)
        rows, counts = torch.unique_consecutive(ids[kept][order], return_counts=True)
        sums = torch.segment_reduce(s["dout"][kept][order].double() * s["scale"], "sum", lengths=counts)
        total = s["dtable"].double() if case["accumulate"] else torch.zeros(V, D, device="cuda", dtype=torch.float64)
        total[rows] += sums
        return total
    targets = s["targets"].long()
    rows = torch.nonzero(targets >= 0)[:, 0]
    x, w = s["x"][rows].double(), s["w"].double()
    logits = torch.matmul(x, w.t()).mul_(case["alpha"])
    lse_rows = torch.logsumexp(logits, dim=1)
    loss = torch.zeros(M, device="cuda", dtype=torch.float64)
    lse = torch.zeros(M, device="cuda", dtype=torch.float64)
    each = torch.arange(rows.numel(), device="cuda")
    loss[rows] = lse_rows - logits[each, targets[rows]]
    lse[rows] = lse_rows
    count = max(1, rows.numel())
    mean = loss.sum().reshape(1) / count
    if op == "ce":
        return loss, lse, mean
    g = logits.sub_(lse_rows[:, None]).exp_()
    g[each, targets[rows]] -= 1.0
    g *= case["alpha"] / count
    dx = torch.zeros(M, D, device="cuda", dtype=torch.float64)
    dx[rows] = torch.matmul(g, w)
    return loss, lse, mean, dx, torch.matmul(g.t(), x)
