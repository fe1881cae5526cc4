"""A tied embedding table trained with the operators at a model's two ends:
lookup, linear cross entropy, its gradients, the lookup's gradient added to
them, and the clipped norm, in one captured chain.

``TiedTable`` is the smallest model that uses them all: the next token's
logits are the products of the table's rows with the scaled row of the present
token, l[v] = alpha * E[v] . (scale * E[prev]).  A larger model puts its blocks
between ``x`` and the loss.  ``python -m tcgen05_tmem_bf16_gb300.heads`` trains
one on made-up text.
"""
from __future__ import annotations

import torch

from . import (TensorList, clip_grad_norm, embedding_grad, embedding_lookup, gbf_workspace_size,
               linear_ce, linear_ce_grad)
from .graphs import CapturedChain


class TiedTable:
    """A table E [V][D] (fp32 master values and their bf16 rounding) and the
    buffers of training steps on ``tokens`` positions each.

    ``step(prev, target)`` copies the int64 ids in (``prev`` -1: a zero input;
    ``target`` outside [0, V): not scored), replays the captured chain, and
    takes one step down the clipped gradient.  It returns the mean loss and the
    gradient's norm as device tensors that the next step overwrites.
    ``graph=False`` issues the launches directly."""

    def __init__(self, V: int, D: int, tokens: int, alpha: float = 1.0, max_norm: float = 1.0,
                 seed: int = 0, graph: bool = True, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.V, self.D, self.M = V, D, tokens
        self.alpha, self.scale, self.max_norm = alpha, 1.0, max_norm
        self.master = torch.randn(V, D, generator=g, device=device) * D ** -0.5
        bf16 = dict(device=device, dtype=torch.bfloat16)
        f32 = dict(device=device, dtype=torch.float32)
        self.table = self.master.to(torch.bfloat16)
        self.prev = torch.zeros(tokens, device=device, dtype=torch.int64)
        self.target = torch.zeros(tokens, device=device, dtype=torch.int64)
        self.x, self.dx = torch.empty(tokens, D, **bf16), torch.empty(tokens, D, **bf16)
        self.dtable = torch.empty(V, D, **bf16)
        self.loss, self.lse = torch.empty(tokens, **f32), torch.empty(tokens, **f32)
        self.mean, self.norm = torch.empty(1, **f32), torch.empty(1, **f32)
        self.grads = TensorList([self.dtable])
        # one workspace: the calls of a step run one after another
        self.ws_bytes = max([gbf_workspace_size(op, tokens, V, D, True)
                             for op in ("linear_ce", "linear_ce_grad", "embedding_grad")]
                            + [gbf_workspace_size("clip_grad_norm", 1, 0, 0, True)])
        self.workspace = torch.empty(self.ws_bytes, device=device, dtype=torch.uint8)
        self.graph = CapturedChain(self.launch) if graph else None

    def launch(self, stream=None):
        """Loss, gradient and clipping of the present ids (no update)."""
        M, V, D = self.M, self.V, self.D
        ws = dict(workspace=self.workspace, workspace_bytes=self.ws_bytes, stream=stream)
        embedding_lookup(self.prev, self.table, self.x, M, V, D, self.scale, stream=stream)
        linear_ce(self.x, self.table, self.target, self.loss, self.lse, self.mean, M, V, D,
                  self.alpha, **ws)
        linear_ce_grad(self.x, self.table, self.target, self.lse, None, self.dx, self.dtable, M,
                       V, D, self.alpha, **ws)
        # the table is tied: its rows' gradient as inputs on top of that as outputs
        embedding_grad(self.prev, self.dx, self.dtable, M, V, D, self.scale, True, **ws)
        clip_grad_norm(self.grads, None, self.max_norm, self.norm, **ws)

    def step(self, prev, target, rate: float = 1.0):
        self.prev.copy_(prev)
        self.target.copy_(target)
        if self.graph is not None:
            self.graph.replay()
        else:
            self.launch()
        self.master.add_(self.dtable, alpha=-rate)
        self.table.copy_(self.master)
        return self.mean, self.norm


def clustered_text(n: int, V: int, clusters: int, generator, device="cuda"):
    """(present, next) ids: the next token is any of the present one's cluster."""
    prev = torch.randint(0, V, (n,), generator=generator, device=device)
    other = torch.randint(0, V // clusters, (n,), generator=generator, device=device)
    return prev, prev % clusters + clusters * other


def main():
    V, D, M, clusters = 8192, 512, 4096, 64
    model = TiedTable(V, D, M, alpha=8.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(201):
        mean, norm = model.step(*clustered_text(M, V, clusters, g), rate=30.0)
        if i % 40 == 0:
            print(f"step {i:4d}  loss {float(mean):.3f}  gradient norm {float(norm):.4f}")
    print(f"a uniform guess: {torch.log(torch.tensor(float(V))):.3f}, "
          f"the best there is: {torch.log(torch.tensor(float(V // clusters))):.3f}")


if __name__ == "__main__":
    main()
