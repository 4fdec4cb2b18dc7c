"""A training step that distils a teacher into an expert-parallel block with a tied
head, on emulated ranks: layer norm, balance loss and distillation with the
operators and collectives of expert_step, as a program uses them.

Every rank holds one range of the vocabulary's table, which embeds tokens and
gives their logits.  One step is

  expert_step's embedding                        x
  layer_norm, expert_step's expert layer         n = norm(x), y
  balance_loss, all_reduce, balance_join         the loss of all ranks' picks
  layer_norm with the residual                   t = x + y, m = norm(t)
  all_gather, the product with the own range     every token's logits for the range
  distil_parts, all_gather, distil_join          the loss over the whole vocabulary

and the same backwards: distil_loss_grad in the logits' place, the products,
reduce_scatter, layer_norm_grad, expert_step's backward pass with
balance_loss_grad added to the router's, layer_norm_grad with the residual's
gradient, and the embedding's gradient added to the head's.

    python -m collective_datapath_reduce_gb300.distil_step
"""

from __future__ import annotations

import dataclasses

import torch

from . import expert_step
from . import torch_api as purlin


@dataclasses.dataclass
class Shape(expert_step.Shape):
    balance: float = 0.01    # the balance loss of experts that are alike
    temperature: float = 2.0


class DistilStep(expert_step.ExpertStep):
    def __init__(self, shape: Shape, device="cuda", dtype=torch.float32, seed=0):
        super().__init__(shape, device, dtype, seed)
        one, zero = self._new(shape.width).fill_(1), self._new(shape.width).zero_()
        self.norms = [one, zero, one.clone(), zero.clone()]    # weight and bias, before the experts and before the head

    def parameters(self):
        return [*super().parameters(), *self.norms]

    # ------------------------------------------------------------ forward

    def _norm(self, x, which, residual=None):
        """(normalised rows, the sums with the residual, statistics) of every rank."""
        weight, bias = self.norms[2 * which:2 * which + 2]
        y = [torch.empty_like(t) for t in x]
        totals = [torch.empty_like(t) for t in x] if residual else x
        stats = [self._new(t.shape[0], 2, dtype=torch.float32) for t in x]
        for r, t in enumerate(x):
            purlin.layer_norm(t, weight, bias, y[r], self.handle, residual=residual[r] if residual else None,
                              total=totals[r] if residual else None, stats=stats[r])
        return y, totals, stats

    def _gather(self, parts):
        out = [p.new_empty(len(parts) * p.shape[0], *p.shape[1:]) for p in parts]
        purlin.all_gather(parts, out, self.handle)
        return out

    def _balance(self, f):
        s, h = self.shape, self.handle
        f["sums"] = [self._new(2 * s.experts + 1, dtype=torch.float32) for _ in f["ids"]]
        f["counts_of"] = [self._new(s.experts, dtype=torch.int32) for _ in f["ids"]]
        for r, sums in enumerate(f["sums"]):
            purlin.balance_loss(f["logits"][r], f["ids"][r], f["counts_of"][r], sums, None, h)
        purlin.all_reduce(f["sums"], f["sums"], h)
        loss = self._new(1, dtype=torch.float32)
        purlin.balance_join(f["sums"][0], loss, h, scale=s.balance)
        return loss

    def forward(self, tokens, words, teacher):
        """(loss, what the backward pass needs).  words (int64) and teacher (float32): of
        every rank, tokens x picks, the teacher's best words and their logits."""
        s, h = self.shape, self.handle
        everyone, x = self._embed(tokens)
        n, _, stats_n = self._norm(x, 0)
        y, f = self._layer(n)
        balance = self._balance(f)
        m, t, stats_m = self._norm(y, 1, x)
        rows, words, teacher = self._gather(m), self._gather(words), self._gather(teacher)
        logits, parts = [], []
        for r, table in enumerate(self.tables):
            logits.append(rows[r] @ table.t())
            parts.append(self._new(rows[r].shape[0], 4, dtype=torch.float32))
            purlin.distil_parts(logits[r], words[r], teacher[r], parts[r], h, first=r * table.shape[0],
                                vocabulary=s.vocabulary, temperature=s.temperature)
        parts = self._gather(parts)
        loss = [self._new(p.shape[0], dtype=torch.float32) for p in rows]
        stats = [self._new(p.shape[0], 2, dtype=torch.float32) for p in rows]
        for r in range(s.world):
            purlin.distil_join(parts[r], loss[r], stats[r], h, temperature=s.temperature, scale=s.temperature ** 2)
        f.update(everyone=everyone, x=x, n=n, stats_n=stats_n, t=t, stats_m=stats_m, rows=rows, words=words,
                 teacher=teacher, logits_of=logits, stats=stats)
        return loss[0].mean() + balance[0], f

    # ----------------------------------------------------------- backward

    def _route_grad(self, f, r, grad_weights):
        grad = super()._route_grad(f, r, grad_weights)
        purlin.balance_loss_grad(f["logits"][r], f["ids"][r], f["sums"][r], None, grad, self.handle,
                                 scale=self.shape.balance, base=grad)
        return grad

    def _norm_grad(self, grad_y, x, stats, which, grad_total=None):
        """(gradients of x, of the weight and of the bias, these two of all ranks)."""
        grad_x = [torch.empty_like(t) for t in x]
        of_weight, of_bias = ([torch.empty_like(self.norms[0]) for _ in x] for _ in range(2))
        for r, g in enumerate(grad_y):
            purlin.layer_norm_grad(g, x[r], stats[r], self.norms[2 * which], grad_x[r], of_weight[r], of_bias[r],
                                   self.handle, grad_total=grad_total[r] if grad_total else None)
        for side in (of_weight, of_bias):
            purlin.all_reduce(side, side, self.handle)
        return grad_x, of_weight[0], of_bias[0]

    def backward(self, f):
        """Gradients in the order of parameters(), given forward's second result, once: the logits,
        the largest of what it holds, become their gradients in place."""
        s, h = self.shape, self.handle
        logits = f.pop("logits_of", None)
        if logits is None:
            raise RuntimeError("backward: this forward's logits are gradients by now; run forward again")
        count = s.world * s.tokens
        grad_loss = self._new(count, dtype=torch.float32).fill_(1 / count)
        grad_rows, grad_tables = [], []
        for r, table in enumerate(self.tables):
            dz = logits[r]
            purlin.distil_loss_grad(dz, f["words"][r], f["teacher"][r], f["stats"][r], grad_loss, dz, h,
                                    first=r * table.shape[0], vocabulary=s.vocabulary, temperature=s.temperature,
                                    scale=s.temperature ** 2)
            grad_rows.append(dz @ table)
            grad_tables.append(dz.t() @ f["rows"][r])
        grad_m = [self._new(s.tokens, s.width) for _ in grad_rows]
        purlin.reduce_scatter(grad_rows, grad_m, h)
        grad_t, *of_m = self._norm_grad(grad_m, f["t"], f["stats_m"], 1)
        layer = dict(f, x=f["n"])
        grad_n, *rest = self._layer_grad(grad_t, layer)
        grad_x, *of_n = self._norm_grad(grad_n, f["x"], f["stats_n"], 0, grad_t)
        return [*self._embed_grad(grad_x, f["everyone"], grad_tables), *rest, *of_n, *of_m]

    def step(self, tokens, words, teacher):
        """One step: (loss, gradients' norm)."""
        s = self.shape
        loss, saved = self.forward(tokens, words, teacher)
        grads = [g.contiguous() for g in self.backward(saved)]
        norm = self._new(1, dtype=torch.float32)
        purlin.clip_grad_norm(grads, grads, s.max_norm, norm, self.handle)
        for p, g in zip(self.parameters(), grads):
            p -= s.rate * g
        return loss, norm[0]


def main():
    shape = Shape(rate=1.0, scale=1.0)
    model = DistilStep(shape)
    g = torch.Generator(device="cuda").manual_seed(1)
    W, T, V, K = shape.world, shape.tokens, shape.vocabulary, 16
    tokens = [torch.randint(0, V, (T,), generator=g, device="cuda") for _ in range(W)]
    words = [torch.rand(T, V, generator=g, device="cuda").topk(K, 1).indices for _ in range(W)]
    teacher = [2 * torch.randn(T, K, generator=g, device="cuda") for _ in range(W)]
    for i in range(10):
        loss, norm = model.step(tokens, words, teacher)
        print(f"step {i}: loss {loss.item():.4f}, gradient norm {norm.item():.4f}")
    model.close()


if __name__ == "__main__":
    main()
