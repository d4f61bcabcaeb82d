"""QueryHead: the learned side of an index, from a model's hidden states to its queries.

A frozen linear layer in int8 (the last layer of an encoder) makes features; a
router sends each feature vector to its best leaves (the centroid scoring that a
partitioned search starts with); every leaf has its own projection, and a query is
the sum of its leaves' projections weighted by the softmax of their scores.  The
projections are trained against answers that an index gave, (ids, scores) as every
search here returns them: the head's own scores of all items, the int8 score plane
of the flat search, are pulled towards the teacher's by the distillation loss.

All products, the routing, the loss and the gradients are the C-ABI calls
ah_i8_linear, ah_partition_score, ah_group_rows, ah_grouped_matmul (_dx, _dw) and
ah_distill_topk; torch keeps the memory and does the elementwise arithmetic.
"""
from __future__ import annotations

import torch

from . import ahlib


class QueryHead:
    def __init__(self, trunk: torch.Tensor, router: torch.Tensor, dim: int, fan: int = 2, seed: int = 0):
        """trunk: float32 [k, h], the frozen layer's weights (h: the hidden width); router: float32
        [L, k], one centroid a leaf; dim: the index's dimension; fan: leaves a query goes through."""
        self.trunk8, self.trunk_scale = ahlib.ah_i8_quantize_rows(trunk)
        self.router = router.contiguous()
        L, k = router.shape
        if trunk.shape[0] != k or not 1 <= fan <= L:
            raise ValueError("trunk and router differ in width, or fan is not in 1..leaves")
        self.fan = int(fan)
        g = torch.Generator(device=router.device)
        g.manual_seed(seed)
        self.weights = torch.randn(L, dim, k, generator=g, device=router.device) * k ** -0.5  # float32 master copy
        self.w = self.weights.bfloat16()
        self._kept = None

    def queries(self, hidden: torch.Tensor, keep: bool = False) -> torch.Tensor:
        """Queries float32 [m, dim] of hidden states (bfloat16 or float32 [m, h]); keep: hold this
        pass's features, order and gates."""
        q, x, _, offsets, order, gate, _ = self._forward(hidden)
        if keep:
            self._kept = (x, offsets, order, gate)
        return q

    def _forward(self, hidden):
        """Queries, features bfloat16 [m, k], leaves [m, fan], the slots' order, gates float32 [m, fan] and
        the slots' projections float32 [m, fan, dim]."""
        x = ahlib.ah_i8_linear(hidden, self.trunk8, self.trunk_scale, out_dtype=torch.bfloat16)
        leaves, scores = ahlib.ah_partition_score(x.float(), self.router, self.fan)
        offsets, order = ahlib.ah_group_rows(leaves, self.router.shape[0])
        y = ahlib.ah_grouped_matmul(x, self.w, offsets, order=order, fan=self.fan, out_dtype=torch.float32)
        gate = torch.softmax(scores, dim=1)
        y = y.view(*gate.shape, self.w.shape[1])
        return (y * gate[:, :, None]).sum(1), x, leaves, offsets, order, gate, y

    def step(self, hidden, items, ids, scores, tau: float = 1.0, lr: float = 0.1, want_dx: bool = False):
        """One step of training on a batch: items is an `Items`, ids / scores the teacher's answers
        (int32 / float32 [m, k]).  Returns (losses float32 [m], gradient of the features or None).

        The gradient (bfloat16 [m, k], of the mean loss) is that of the features x in
        q = sum_f softmax(router x)_f W_f x: through the projections and through the gates, with the choice
        of leaves held.  The rounding of queries to int8 codes in the score plane counts as
        the identity."""
        m = hidden.shape[0]
        q, x, leaves, offsets, order, gate, y = self._forward(hidden)
        # bfloat16 scores: the gradient that leaves the loss is the next product's operand
        z = ahlib.ah_i8_linear(q, items.codes, items.step, out_dtype=torch.bfloat16)
        weight = torch.full((m,), 1.0 / max(m, 1), device=q.device)
        loss, dz = ahlib.ah_distill_topk(z, ids, scores, tau=tau, row_weight=weight, grad_out=z)
        one = torch.full((2,), m, dtype=torch.int64, device=q.device)  # one leaf, [0, m); made on the device,
        one[:1].zero_()                                                # so that a graph can hold the step
        dq = None
        for a, part in items.parts():  # a product sums at most 2^20 items; more are added up in order
            d = ahlib.ah_grouped_matmul(dz[:, a:a + part.shape[1]], part[None], one, out_dtype=torch.float32)
            dq = d if dq is None else dq.add_(d)
        dy = (gate[:, :, None] * dq[:, None, :]).to(torch.bfloat16).reshape(m * self.fan, q.shape[1])
        dw = ahlib.ah_grouped_matmul_dw(dy, x, offsets, order=order, fan=self.fan)
        dx = None
        if want_dx:
            dx = ahlib.ah_grouped_matmul_dx(dy, self.w, offsets, order=order, fan=self.fan, out_dtype=torch.float32)
            # the gates: d gate_f / d score_g = gate_f ([f = g] - gate_g), score_f = router[leaf_f] . x
            along = (y * dq[:, None, :]).sum(2)
            dscore = gate * (along - (gate * along).sum(1, keepdim=True))
            dscore = torch.where(leaves >= 0, dscore, torch.zeros_like(dscore))  # no leaf, no score
            dx += (dscore[:, :, None] * self.router[leaves.clamp(min=0).long()]).sum(1)
            dx = dx.to(torch.bfloat16)
        self.weights.add_(dw, alpha=-lr)
        self.w.copy_(self.weights)
        return loss, dx


class Items:
    """What a head is trained to score: rows float32 [n, d] as int8 codes and steps, and their
    values by column (bfloat16, [d, at most 2^20] a part) for the gradient.  A step on m queries keeps
    their scores of all items, m n bfloat16 values."""

    MOST = ahlib.AH_MAX_WIDTH  # items of a part

    def __init__(self, rows: torch.Tensor):
        self.codes, self.step = ahlib.ah_i8_quantize_rows(rows)
        n, d = rows.shape
        self._parts = []
        for a in range(0, max(n, 1), self.MOST):
            b = min(n, a + self.MOST)
            columns = torch.empty(d, b - a, dtype=torch.bfloat16, device=rows.device)
            for c in range(a, b, 1 << 16):
                part = slice(c, min(b, c + (1 << 16)))
                columns[:, c - a:part.stop - a] = (self.codes[part].float() * self.step[part, None]).t().to(torch.bfloat16)
            self._parts.append(columns)

    def parts(self):
        """(first item, values by column) of each part."""
        return [(i * self.MOST, columns) for i, columns in enumerate(self._parts)]

    @property
    def columns(self) -> torch.Tensor:
        """The values of all items by column, bfloat16 [d, n] (put together where there are several parts)."""
        return self._parts[0] if len(self._parts) == 1 else torch.cat(self._parts, dim=1)
