"""A student of residual gated blocks, distilled from a teacher's top logits with the
library's operators in one captured chain: lookup, the blocks with their norms, the
distillation loss through the tied table, all gradients, and the clipped norm.

    r[0] = table[ids];  n[l] = rmsnorm(r[l]) w[l];  m[l] = mlp(n[l]);  r[l+1] = r[l] + m[l]
    loss = KL(teacher's top entries || softmax(alpha n[L] table^T))

Every residual add is the fused add + RMSNorm of the next block, and every gradient
that comes back through one is the ``dresid`` of ``add_rmsnorm_grad``.  A model with
attention puts it between the blocks.  ``python -m tcgen05_tmem_bf16_gb300.student``
distils a made-up teacher.
"""
from __future__ import annotations

import torch

from . import (TensorList, add_rmsnorm, add_rmsnorm_grad, clip_grad_norm, embedding_grad,
               embedding_lookup, gbf_workspace_size, linear_distill, linear_distill_grad,
               linear_distill_workspace_size, mlp_grad, mlp_train)
from .graphs import CapturedChain


class Student:
    """Vocabulary V, width D, hidden width F, ``blocks`` gated blocks; buffers for steps
    of ``tokens`` positions with K teacher entries each.

    ``parameters`` and ``grads`` name the bf16 tensors: "table", and per block l
    "norm.l", "gate.l", "up.l", "down.l", and the last norm "norm.L".  ``step(ids,
    entries, logits)`` copies a batch in (int64 ids [tokens], -1 a zero input; entries
    [tokens][K], outside [0, V) left out; fp32 logits [tokens][K]), replays the captured
    chain and takes one step down the clipped gradient; it returns the mean loss and
    the gradient's norm as device tensors that the next step overwrites.
    ``graph=False`` issues the launches directly."""

    def __init__(self, V: int, D: int, F: int, blocks: int, tokens: int, K: int,
                 alpha: float = 1.0, temperature: float = 1.0, act: str = "silu",
                 max_norm: float = 1.0, seed: int = 0, graph: bool = True, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.V, self.D, self.F, self.L, self.M, self.K = V, D, F, blocks, tokens, K
        # both sides' logits are divided by the temperature, the gradient multiplied by
        # its square
        self.alpha, self.beta = alpha / temperature, 1.0 / temperature
        self.scale, self.act, self.max_norm, self.eps = temperature ** 2, act, max_norm, 1e-5
        bf16 = dict(device=device, dtype=torch.bfloat16)
        f32 = dict(device=device, dtype=torch.float32)

        def random(*shape):
            return torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5

        self.master = {"table": random(V, D)}
        for l in range(blocks):
            self.master[f"norm.{l}"] = torch.ones(D, **f32)
            self.master[f"gate.{l}"], self.master[f"up.{l}"] = random(F, D), random(F, D)
            self.master[f"down.{l}"] = random(D, F)
        self.master[f"norm.{blocks}"] = torch.ones(D, **f32)
        self.parameters = {k: v.to(torch.bfloat16) for k, v in self.master.items()}
        self.grads = {k: torch.empty_like(v) for k, v in self.parameters.items()}
        self.grad_list = TensorList(self.grads.values())
        M = tokens
        self.ids = torch.zeros(M, device=device, dtype=torch.int64)
        self.entries = torch.zeros(M, K, device=device, dtype=torch.int64)
        self.logits = torch.zeros(M, K, **f32)
        self.zero, self.x = torch.zeros(M, D, **bf16), torch.empty(M, D, **bf16)
        self.r, self.n, self.m = ([torch.empty(M, D, **bf16) for _ in range(blocks + 1)]
                                  for _ in range(3))
        self.kept = [[torch.empty(M, F, **bf16) for _ in range(3)] for _ in range(blocks)]
        self.dn, self.dr = torch.empty(M, D, **bf16), torch.empty(M, D, **bf16)
        self.loss, self.lse = torch.empty(M, **f32), torch.empty(M, **f32)
        self.mean, self.norm = torch.empty(1, **f32), torch.empty(1, **f32)
        # one workspace: the calls of a step run one after another
        self.ws_bytes = max(
            linear_distill_workspace_size(M, V, D, K, False),
            linear_distill_workspace_size(M, V, D, K, True),
            gbf_workspace_size("mlp_grad", M, D, F, True),
            gbf_workspace_size("add_rmsnorm_grad", M, D, 0, True),
            gbf_workspace_size("embedding_grad", M, V, D, True),
            gbf_workspace_size("clip_grad_norm", len(self.grad_list), 0, 0, True))
        self.workspace = torch.empty(self.ws_bytes, device=device, dtype=torch.uint8)
        self.graph = CapturedChain(self.launch) if graph else None

    def launch(self, stream=None):
        """Loss, gradients and clipping of the present batch (no update)."""
        M, V, D, F, L, K = self.M, self.V, self.D, self.F, self.L, self.K
        p, d = self.parameters, self.grads
        ws = dict(workspace=self.workspace, workspace_bytes=self.ws_bytes, stream=stream)
        embedding_lookup(self.ids, p["table"], self.x, M, V, D, stream=stream)
        before, add = self.x, self.zero
        for l in range(L + 1):
            add_rmsnorm(before, add, p[f"norm.{l}"], self.n[l], self.r[l], M, D, self.eps,
                        stream=stream)
            if l < L:
                mlp_train(self.n[l], p[f"gate.{l}"], p[f"up.{l}"], p[f"down.{l}"], None,
                          self.m[l], *self.kept[l], M, D, F, self.act, stream=stream)
                before, add = self.r[l], self.m[l]
        head = (self.n[L], p["table"], self.entries, self.logits)
        linear_distill(*head, self.loss, self.lse, self.mean, M, V, D, K, self.alpha, self.beta,
                       **ws)
        linear_distill_grad(*head, self.lse, None, self.dn, d["table"], M, V, D, K, self.alpha,
                            self.beta, self.scale, **ws)
        for l in range(L, -1, -1):
            # what reached the stream behind this norm comes in through the residual
            add_rmsnorm_grad(self.dn, self.dr if l < L else None, self.r[l], p[f"norm.{l}"],
                             self.dr, d[f"norm.{l}"], M, D, self.eps, **ws)
            if l > 0:
                b = l - 1
                mlp_grad(self.dr, self.n[b], *self.kept[b], p[f"gate.{b}"], p[f"up.{b}"],
                         p[f"down.{b}"], self.dn, d[f"gate.{b}"], d[f"up.{b}"], d[f"down.{b}"],
                         M, D, F, self.act, **ws)
        # the table is tied: its rows' gradient as inputs on top of that as outputs
        embedding_grad(self.ids, self.dr, d["table"], M, V, D, 1.0, True, **ws)
        clip_grad_norm(self.grad_list, None, self.max_norm, self.norm, **ws)

    def step(self, ids, entries, logits, rate: float = 1.0):
        self.ids.copy_(ids)
        self.entries.copy_(entries)
        self.logits.copy_(logits)
        if self.graph is not None:
            self.graph.replay()
        else:
            self.launch()
        for k, v in self.master.items():
            v.add_(self.grads[k], alpha=-rate)
            self.parameters[k].copy_(v)
        return self.mean, self.norm


def main():
    V, D, F, M, K, clusters = 8192, 512, 1408, 4096, 16, 64
    model = Student(V, D, F, 2, M, K, alpha=8.0, temperature=2.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    # a teacher that expects the next token in the present one's cluster, a few of them
    # likelier than others
    liking = torch.randn(V, generator=g, device="cuda") * 2.0
    offsets = torch.arange(K, device="cuda") * clusters
    for i in range(201):
        ids = torch.randint(0, V, (M,), generator=g, device="cuda")
        entries = (ids % clusters)[:, None] + offsets
        mean, norm = model.step(ids, entries, 8.0 + liking[entries], rate=3.0)
        if i % 40 == 0:
            print(f"step {i:4d}  KL from the teacher {float(mean):.4f}  gradient norm {float(norm):.4f}")


if __name__ == "__main__":
    main()
