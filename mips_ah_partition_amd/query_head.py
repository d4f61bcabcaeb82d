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

Options: a leaf's projection can be a gated feed-forward block (inner; ah_grouped_gated and
its gradient), trained with dropout (drop; also of the features, ah_dropout), and the linear layer can be in
8-bit floats instead of int8 (trunk_type; ah_f8_linear), which can be trained too.
"""
from __future__ import annotations

import torch

from . import ahlib


class QueryHead:
    ROWS = ahlib.AH_MAX_WIDTH  # rows that a product of the trunk's gradient sums (a multiple of 128)

    def __init__(self, trunk: torch.Tensor, router: torch.Tensor, dim: int, fan: int = 2, seed: int = 0,
                 inner: int = 0, act: str = "silu", drop: float = 0.0, trunk_type: str = "i8"):
        """trunk: float32 [k, h], the linear layer's weights (h: the hidden width); router: float32
        [L, k], one centroid a leaf; dim: the index's dimension; fan: leaves a query goes through.
        inner: 0, a leaf has one matrix [dim, k]; else the hidden width of its gated block, W_out (act(W_gate x) *
        (W_up x)).  drop: dropout in `step`, of the features that go to the leaves and of the blocks' hidden values.
        trunk_type: "i8" (frozen) or "f8" (e4m3; `step` can train it)."""
        if trunk_type not in ("i8", "f8"):
            raise ValueError("trunk_type must be i8 or f8")
        ahlib._act_code(act)
        if inner < 0 or not 0.0 <= drop < 1.0:
            raise ValueError("inner must not be negative, and drop in [0, 1)")
        self.trunk_type, self.inner, self.act, self.drop = trunk_type, int(inner), act, float(drop)
        if trunk_type == "i8":
            self.trunk8, self.trunk_scale = ahlib.ah_i8_quantize_rows(trunk)
        else:
            self.trunk = torch.clone(trunk.float(), memory_format=torch.contiguous_format)  # master copy
            self._codes = ahlib.ah_f8_quantize(self.trunk, want_columns=True)
        self.router = router.contiguous()
        L, k = router.shape
        if trunk.shape[0] != k or not 1 <= fan <= L:
            raise ValueError("trunk and router differ in width, or fan is not in 1..leaves")
        self.fan = int(fan)
        g = torch.Generator(device=router.device)
        g.manual_seed(seed)
        rnd = lambda rows, width: torch.randn(L, rows, width, generator=g, device=router.device) * width ** -0.5  # noqa: E731
        self.weights = rnd(dim, self.inner or k)  # float32 master copy
        self.w = self.weights.bfloat16()
        if self.inner:
            self.weights_in = rnd(2 * self.inner, k)
            self.w_in = self.weights_in.bfloat16()
        self.seed = int(seed)
        self.steps = torch.zeros(1, dtype=torch.int64, device=router.device)  # on the device: a graph counts on
        self._kept = None

    def queries(self, hidden: torch.Tensor, keep: bool = False) -> torch.Tensor:
        """Queries float32 [m, dim] of hidden states (bfloat16 or float32 [m, h]); keep: hold this
        pass's features, order and gates."""
        q, x, _, offsets, order, gate, _ = self._forward(hidden)
        if keep:
            self._kept = (x, offsets, order, gate)
        return q

    def _features(self, hidden):
        if self.trunk_type == "i8":
            return ahlib.ah_i8_linear(hidden, self.trunk8, self.trunk_scale, out_dtype=torch.bfloat16)
        return ahlib.ah_f8_linear(hidden, self._codes[0], self._codes[1], out_dtype=torch.bfloat16)

    def _forward(self, hidden, train=None):
        """Queries, features bfloat16 [m, k], leaves [m, fan], the slots' order, gates float32 [m, fan] and
        the slots' projections float32 [m, fan, dim].  train: a dict that receives what the backward pass needs more."""
        x = self._features(hidden)
        leaves, scores = ahlib.ah_partition_score(x.float(), self.router, self.fan)
        offsets, order = ahlib.ah_group_rows(leaves, self.router.shape[0])
        drop = self.drop if train is not None else 0.0
        into = ahlib.ah_dropout(x, drop, 2 * self.seed, step=self.steps) if drop else x  # the leaves' input
        pre = None
        if self.inner:
            h, pre = ahlib.ah_grouped_gated(into, self.w_in, offsets, order=order, fan=self.fan, act=self.act, drop=drop,
                                            seed=2 * self.seed + 1, step=self.steps, want_pre=train is not None)
            y = ahlib.ah_grouped_matmul(h, self.w, offsets, order=order, out_dtype=torch.float32)
        else:
            y = ahlib.ah_grouped_matmul(into, self.w, offsets, order=order, fan=self.fan, out_dtype=torch.float32)
        if train is not None:
            train["into"], train["pre"] = into, pre
        gate = torch.softmax(scores, dim=1)
        y = y.view(*gate.shape, self.w.shape[1])
        return (y * gate[:, :, None]).sum(1), x, leaves, offsets, order, gate, y

    def step(self, hidden, items, ids, scores, tau: float = 1.0, lr: float = 0.1, want_dx=False,
             trunk_lr: float = 0.0):
        """One step of training on a batch: items is an `Items`, ids / scores the teacher's answers
        (int32 / float32 [m, k]).  Returns (losses float32 [m], gradient of the features or None).

        The gradient (bfloat16 [m, k], of the mean loss) is that of the features x in
        q = sum_f softmax(router x)_f W_f x: through the projections and through the gates, with the choice
        of leaves held.  The rounding of queries to int8 codes in the score plane counts as
        the identity.  With dropout the masks are those of this step (seed and steps), and the gates see the
        features without it.  want_dx="hidden" (8-bit float trunk): the gradient of the hidden states, bfloat16 [m, h],
        in its place; trunk_lr: the trunk's own rate.  Both are products of 8-bit codes like the trunk's, whose
        roundings count as the identity."""
        if isinstance(want_dx, str) and want_dx != "hidden":
            raise ValueError(f'want_dx must be a truth value or "hidden", got {want_dx!r}')
        if self.trunk_type != "f8" and (want_dx == "hidden" or trunk_lr):
            raise ValueError("only an 8-bit float trunk has gradients")
        m = hidden.shape[0]
        more = {}
        q, x, leaves, offsets, order, gate, y = self._forward(hidden, more)
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
        into, dw_in = more["into"], None
        if self.inner:
            dpre, h = ahlib.ah_grouped_gated_grad(dy, self.w, more["pre"], offsets, order=order, act=self.act,
                                                  drop=self.drop, seed=2 * self.seed + 1, step=self.steps,
                                                  dpre_out=more["pre"])
            dw = ahlib.ah_grouped_matmul_dw(dy, h, offsets, order=order)
            dw_in = ahlib.ah_grouped_matmul_dw(dpre, into, offsets, order=order, fan=self.fan)
        else:
            dw = ahlib.ah_grouped_matmul_dw(dy, into, offsets, order=order, fan=self.fan)
        dx = None
        if want_dx or trunk_lr:
            dslot, wide = (dpre, self.w_in) if self.inner else (dy, self.w)
            dx = ahlib.ah_grouped_matmul_dx(dslot, wide, offsets, order=order, fan=self.fan, out_dtype=torch.float32)
            # the gates: d gate_f / d score_g = gate_f ([f = g] - gate_g), score_f = router[leaf_f] . x
            along = (y * dq[:, None, :]).sum(2)
            dscore = gate * (along - (gate * along).sum(1, keepdim=True))
            dscore = torch.where(leaves >= 0, dscore, torch.zeros_like(dscore))  # no leaf, no score
            gates = (dscore[:, :, None] * self.router[leaves.clamp(min=0).long()]).sum(1)
            if self.drop:
                dx = ahlib.ah_dropout(dx, self.drop, 2 * self.seed, step=self.steps, residual=gates, out=dx)
            else:
                dx += gates
            dx = dx.to(torch.bfloat16)
        if want_dx == "hidden" or trunk_lr:
            dx = self._trunk_back(dx, hidden, want_dx, trunk_lr)
        self.weights.add_(dw, alpha=-lr)
        self.w.copy_(self.weights)
        if dw_in is not None:
            self.weights_in.add_(dw_in, alpha=-lr)
            self.w_in.copy_(self.weights_in)
        if self.drop:
            self.steps.add_(1)
        return loss, dx

    def _trunk_back(self, dx, hidden, want_dx, trunk_lr):
        """Gradients through the 8-bit float layer x = W hidden: dx W and dx^T hidden, both sums over blocks of 128 with
        their own scales (so the transposed operands are quantised along the other side).  A product sums at most
        2^20 rows; more are added up in order."""
        m, dw = dx.shape[0], None
        back = torch.empty((m, hidden.shape[1]), dtype=torch.bfloat16, device=dx.device) if want_dx == "hidden" else dx
        for a in range(0, max(m, 1), self.ROWS):
            part = slice(a, a + self.ROWS)
            codes, scale, codes_t, scale_t = ahlib.ah_f8_quantize(dx[part], want_rows=want_dx == "hidden",
                                                                  want_columns=bool(trunk_lr))
            if want_dx == "hidden":
                ahlib.ah_f8_matmul(codes, scale, self._codes[2], self._codes[3], out=back[part])
            if trunk_lr:
                _, _, h8, hs = ahlib.ah_f8_quantize(hidden[part], want_rows=False, want_columns=True)
                d = ahlib.ah_f8_matmul(codes_t, scale_t, h8, hs, out_dtype=torch.float32)
                dw = d if dw is None else dw.add_(d)
        if trunk_lr:
            self.trunk.add_(dw, alpha=-trunk_lr)
            ahlib.ah_f8_quantize(self.trunk, want_columns=True, codes_out=self._codes[0], scale_out=self._codes[1],
                                 codes_t_out=self._codes[2], scale_t_out=self._codes[3])
        return back if want_dx else None


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
