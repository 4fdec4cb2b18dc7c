"""A training step of an expert-parallel layer on emulated ranks: the operators
around the collectives and the collectives together, as a program uses them.

Every rank holds one range of the vocabulary's embedding table, some of the
experts, a copy of the router and its own tokens.  One step is

  all_gather (tokens), embed, reduce_scatter     the tokens' embeddings
  route_experts, expert_plan, dispatch_rows      rows packed by expert
  all_to_all_v                                   to the experts' ranks
  expert_plan, dispatch_rows, the experts' products, combine_rows
  all_to_all_v, combine_rows                     back, and the weighted sum

and the same backwards (combine_rows_grad, route_experts_grad, embed_grad),
then all_reduce for the router's gradient, one clip_grad_norm over the
gradients of all ranks, and the update.  The experts' and the router's products
are torch's.

    python -m collective_datapath_reduce_gb300.expert_step
"""

from __future__ import annotations

import dataclasses

import torch

from . import torch_api as purlin


@dataclasses.dataclass
class Shape:
    world: int = 4
    tokens: int = 256        # of each rank
    vocabulary: int = 4096
    width: int = 256
    hidden: int = 512
    experts: int = 16
    top_k: int = 4
    scale: float = 8.0       # of the embeddings
    max_norm: float = 1.0
    rate: float = 0.05


class ExpertStep:
    def __init__(self, shape: Shape, device="cuda", dtype=torch.float32, seed=0):
        s, self.shape, self.dtype = shape, shape, dtype
        if s.vocabulary % s.world or s.experts % s.world:
            raise ValueError("the vocabulary and the experts must split into world equal parts")
        self.device = torch.device(device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        g = torch.Generator(device=self.device).manual_seed(seed)

        def normal(*size, std):
            return (torch.randn(size, generator=g, device=self.device) * std).to(dtype)
        W, local = range(s.world), s.experts // s.world
        self.tables = [normal(s.vocabulary // s.world, s.width, std=0.1) for _ in W]
        self.router = normal(s.experts, s.width, std=s.width ** -0.5)
        self.up = [normal(local, s.width, s.hidden, std=s.width ** -0.5) for _ in W]
        self.down = [normal(local, s.hidden, s.width, std=s.hidden ** -0.5) for _ in W]
        self.handle = purlin.initialize(s.world, self.device)

    def close(self):
        purlin.finalize(self.handle)

    def _new(self, *size, dtype=None):
        return torch.empty(size, dtype=dtype or self.dtype, device=self.device)

    def parameters(self):
        return [*self.tables, self.router, *self.up, *self.down]

    # ------------------------------------------------------------ forward

    def _embed(self, tokens):
        """Every rank looks all tokens up in its range; the sum of the parts is scattered."""
        s, h = self.shape, self.handle
        everyone = [self._new(s.world * s.tokens, dtype=torch.int64) for _ in tokens]
        purlin.all_gather(tokens, everyone, h)
        parts = [self._new(s.world * s.tokens, s.width) for _ in tokens]
        for r, part in enumerate(parts):
            purlin.embed(self.tables[r], everyone[r], part, h, first=r * self.tables[r].shape[0], scale=s.scale)
        x = [self._new(s.tokens, s.width) for _ in tokens]
        purlin.reduce_scatter(parts, x, h)
        return everyone, x

    def _exchange(self, rows, counts):
        """Rows to their ranks: counts[s][d] rows of width elements from s to d."""
        D = self.shape.width
        out = [self._new(sum(c[d] for c in counts), D) for d in range(self.shape.world)]
        purlin.all_to_all_v([t[:sum(c)] for t, c in zip(rows, counts)], out, [[n * D for n in c] for c in counts],
                            self.handle)
        return out

    def forward(self, tokens):
        """(outputs of every rank, what the backward pass needs)."""
        s, h, local = self.shape, self.handle, self.shape.experts // self.shape.world
        everyone, x = self._embed(tokens)
        ids, weights, places, logits, offsets, rows = [], [], [], [], [], []
        for r in range(s.world):
            logits.append((x[r].float() @ self.router.float().t()).contiguous())
            ids.append(self._new(s.tokens, s.top_k, dtype=torch.int32))
            weights.append(self._new(s.tokens, s.top_k, dtype=torch.float32))
            places.append(self._new(s.tokens, s.top_k, dtype=torch.int32))
            offsets.append(self._new(s.experts + 1, dtype=torch.int32))
            rows.append(self._new(s.tokens * s.top_k, s.width))
            purlin.route_experts(logits[r], ids[r], weights[r], h)
            purlin.expert_plan(ids[r], offsets[r], places[r], h)
            purlin.dispatch_rows(x[r], places[r], rows[r], h)
        # the exchange is described on the host: one small copy
        per_expert = torch.stack(offsets).diff(dim=1).cpu()
        counts = per_expert.view(s.world, s.world, local).sum(2).tolist()
        arrived = self._exchange(rows, counts)
        regrouped, groups, back = [], [], []
        for d in range(s.world):
            mine = per_expert[:, d * local:(d + 1) * local]
            which = torch.arange(local, dtype=torch.int32).repeat(s.world).repeat_interleave(mine.reshape(-1))
            which = which.to(self.device).view(-1, 1)
            groups.append(self._new(*which.shape, dtype=torch.int32))
            purlin.expert_plan(which, self._new(local + 1, dtype=torch.int32), groups[d], h)
            regrouped.append(torch.empty_like(arrived[d]))
            purlin.dispatch_rows(arrived[d], groups[d], regrouped[d], h)
            out = self._experts(d, regrouped[d], mine.sum(0).tolist())
            back.append(torch.empty_like(out))
            purlin.combine_rows(out, groups[d], None, back[d], h)
        returned = self._exchange(back, [list(c) for c in zip(*counts)])
        y = [self._new(s.tokens, s.width) for _ in tokens]
        for r in range(s.world):
            purlin.combine_rows(returned[r], places[r], weights[r], y[r], h)
        return y, dict(everyone=everyone, x=x, logits=logits, ids=ids, weights=weights, places=places, counts=counts,
                       per_expert=per_expert, groups=groups, regrouped=regrouped, returned=returned)

    def _experts(self, d, rows, sizes):
        out = [torch.relu(part @ up) @ down for part, up, down in zip(rows.split(sizes), self.up[d], self.down[d])]
        return torch.cat(out)

    # ----------------------------------------------------------- backward

    def _experts_grad(self, d, rows, grad, sizes):
        grad_rows, grad_up, grad_down = [], [], []
        for part, g, up, down in zip(rows.split(sizes), grad.split(sizes), self.up[d], self.down[d]):
            hidden = torch.relu(part @ up)
            grad_hidden = (g @ down.t()) * (hidden > 0)
            grad_rows.append(grad_hidden @ up.t())
            grad_up.append(part.t() @ grad_hidden)
            grad_down.append(hidden.t() @ g)
        return torch.cat(grad_rows), torch.stack(grad_up), torch.stack(grad_down)

    def backward(self, grad_y, f):
        """Gradients in the order of parameters(), given the outputs' and forward's second result."""
        s, h, local = self.shape, self.handle, self.shape.experts // self.shape.world
        W = range(s.world)
        grad_rows = [torch.empty_like(f["returned"][r]) for r in W]
        grad_weights = [torch.empty_like(f["weights"][r]) for r in W]
        for r in W:
            purlin.combine_rows_grad(f["returned"][r], f["places"][r], f["weights"][r], grad_y[r], grad_rows[r],
                                     grad_weights[r], h)
        arrived = self._exchange(grad_rows, f["counts"])
        grad_up, grad_down, back = [], [], []
        for d in W:
            regrouped = torch.empty_like(arrived[d])
            purlin.dispatch_rows(arrived[d], f["groups"][d], regrouped, h)     # the gradient of its inverse
            sizes = f["per_expert"][:, d * local:(d + 1) * local].sum(0).tolist()
            g, up, down = self._experts_grad(d, f["regrouped"][d], regrouped, sizes)
            grad_up.append(up)
            grad_down.append(down)
            back.append(torch.empty_like(g))
            purlin.combine_rows(g, f["groups"][d], None, back[d], h)
        returned = self._exchange(back, [list(c) for c in zip(*f["counts"])])
        grad_x, grad_router = [], []
        for r in W:
            grad_x.append(self._new(s.tokens, s.width))
            purlin.combine_rows(returned[r], f["places"][r], None, grad_x[r], h)
            grad_logits = torch.empty_like(f["logits"][r])
            purlin.route_experts_grad(f["logits"][r], f["ids"][r], grad_weights[r], grad_logits, h)
            grad_x[r] += (grad_logits @ self.router.float()).to(self.dtype)
            grad_router.append((grad_logits.t() @ f["x"][r].float()).to(self.dtype).contiguous())
        purlin.all_reduce(grad_router, grad_router, h)
        everyone = [self._new(s.world * s.tokens, s.width) for _ in W]
        purlin.all_gather(grad_x, everyone, h)
        grad_tables = [torch.empty_like(t) for t in self.tables]
        for r in W:
            purlin.embed_grad(everyone[r], f["everyone"][r], grad_tables[r], h, first=r * self.tables[r].shape[0],
                              scale=s.scale)
        return [*grad_tables, grad_router[0], *grad_up, *grad_down]

    def step(self, tokens, targets):
        """One step on half the mean squared distance to the targets: (loss, gradients' norm)."""
        s = self.shape
        y, saved = self.forward(tokens)
        off = [a - b for a, b in zip(y, targets)]
        count = s.world * s.tokens
        loss = sum((d.float() ** 2).sum() for d in off) / (2 * count)
        grads = self.backward([d / count for d in off], saved)
        norm = self._new(1, dtype=torch.float32)
        purlin.clip_grad_norm(grads, grads, s.max_norm, norm, self.handle)
        for p, g in zip(self.parameters(), grads):
            p -= s.rate * g
        return loss, norm[0]


def main():
    shape = Shape(rate=2.0)
    model = ExpertStep(shape)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = [torch.randint(0, shape.vocabulary, (shape.tokens,), generator=g, device="cuda") for _ in range(shape.world)]
    targets = [torch.randn(shape.tokens, shape.width, generator=g, device="cuda") for _ in range(shape.world)]
    for i in range(10):
        loss, norm = model.step(tokens, targets)
        print(f"step {i}: loss {loss.item():.4f}, gradient norm {norm.item():.4f}")
    model.close()


if __name__ == "__main__":
    main()
