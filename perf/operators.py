"""The operators of a learned query side, at sizes they meet: what a measurement runs.

int8 products with a scale for each token and channel (an encoder's linear layers, and
the score plane of int8 queries against int8 documents), products grouped by leaf (a
router's leaves as experts, rows in ragged groups) with their gradients, and the
distillation loss against a search's (ids, scores) with its gradient.

``own`` false: plain torch forms in 32 bits.  ``own`` true: the framework's calls.
"""
from __future__ import annotations

import math

import torch

own = False

BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one query through one linear layer of an encoder of 1,536-d embeddings: latency
        {"name": "i8_one_token", "op": "i8_linear", "m": 1, "k": 1536, "n": 4096, "bias": True},
        # a small batch of queries, no size a multiple of anything
        {"name": "i8_few_odd", "op": "i8_linear", "m": 37, "k": 1001, "n": 4003, "bias": True},
        # documents being embedded: a long prompt's worth of tokens through a wide layer
        {"name": "i8_prompt", "op": "i8_linear", "m": 8192, "k": 4096, "n": 16384, "bias": True},
        # 1,000 queries against a shard of 1,536-d int8 documents: the whole float32 score plane
        {"name": "i8_scores", "op": "i8_scores", "m": 1000, "k": 1536, "n": 100003, "bias": False},
        # serving step: 16 queries, each through the projections of its 4 best leaves
        {"name": "routed_step", "op": "routed", "rows": 16, "fan": 4, "leaves": 64, "k": 1536, "n": 1536,
         "out": "bf16"},
        # 100-d queries, odd output width, an empty leaf, some slots without a leaf
        {"name": "routed_odd", "op": "routed", "rows": 333, "fan": 3, "leaves": 37, "k": 100, "n": 385, "out": "f32"},
        # a batch of tokens routed to 4 of 64 leaves, wide output
        {"name": "routed_batch", "op": "routed", "rows": 8192, "fan": 4, "leaves": 64, "k": 1536, "n": 4096,
         "out": "bf16"},
        # gradients of the small, odd projection
        {"name": "routed_grad_odd", "op": "routed_grad", "rows": 500, "fan": 3, "leaves": 21, "k": 200, "n": 77,
         "out": "f32"},
        # gradients of a training batch: 2 of 16 leaves a query
        {"name": "routed_grad_batch", "op": "routed_grad", "rows": 8192, "fan": 2, "leaves": 16, "k": 1536,
         "n": 1536, "out": "f32"},
        # three rows over a large vocabulary: few rows, a long axis
        {"name": "distill_few", "op": "distill", "rows": 3, "vocab": 250001, "top": 20, "dtype": "bf16", "tau": 1.0},
        # a router learning the 200 best of 4,000 leaves for 1,000 queries
        {"name": "distill_leaves", "op": "distill", "rows": 1000, "vocab": 4000, "top": 200, "dtype": "f32",
         "tau": 2.0},
        # a training batch against the 64 best of 65,536 documents
        {"name": "distill_batch", "op": "distill", "rows": 4096, "vocab": 65536, "top": 64, "dtype": "bf16",
         "tau": 1.5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    caps = {"i8_linear": 8192 * 4096 * 16384, "i8_scores": 1000 * 1536 * 100003, "routed": 8192 * 4 * 1536 * 4096,
            "routed_grad": 8192 * 2 * 1536 * 1536, "distill": 4096 * 65536}
    op = rng.choice(sorted(caps))
    while True:
        if op == "i8_linear":
            c = {"op": op, "m": _log_int(rng, 1, 8192), "k": _log_int(rng, 64, 4096), "n": _log_int(rng, 64, 16384),
                 "bias": rng.random() < 0.5}
            size = c["m"] * c["k"] * c["n"]
        elif op == "i8_scores":
            c = {"op": op, "m": _log_int(rng, 1, 1000), "k": _log_int(rng, 64, 1536),
                 "n": _log_int(rng, 1000, 100003), "bias": False}
            size = c["m"] * c["k"] * c["n"]
        elif op in ("routed", "routed_grad"):
            leaves = _log_int(rng, 2, 64)
            fan = rng.randint(1, min(4, leaves))
            c = {"op": op, "rows": _log_int(rng, 1, 8192), "fan": fan, "leaves": leaves,
                 "k": _log_int(rng, 32, 1536), "n": _log_int(rng, 32, 4096 if op == "routed" else 1536),
                 "out": rng.choice(["bf16", "f32"])}
            if rng.random() < 0.5:  # widths of a model are mostly multiples of 64
                c["k"], c["n"] = max(64, c["k"] // 64 * 64), max(64, c["n"] // 64 * 64)
            size = c["rows"] * fan * c["k"] * c["n"]
        else:
            c = {"op": op, "rows": _log_int(rng, 1, 4096), "vocab": _log_int(rng, 500, 250001),
                 "top": _log_int(rng, 1, 200), "dtype": rng.choice(["bf16", "f32"]),
                 "tau": rng.choice([0.5, 1.0, 1.5, 2.0, 4.0])}
            size = c["rows"] * c["vocab"] * (2 if c["dtype"] == "f32" else 1)
        if size <= caps[op]:
            return c


def work(case):
    op = case["op"]
    if op in ("i8_linear", "i8_scores"):
        m, k, n = case["m"], case["k"], case["n"]
        act, out = (2 * m * k, 2) if op == "i8_linear" else (m * k + 4 * m, 4)
        return {"bytes": act + n * k + 4 * n + (4 * n if case["bias"] else 0) + out * m * n, "flops": 2 * m * n * k}
    if op in ("routed", "routed_grad"):
        T, L, k, n = case["rows"] * case["fan"], case["leaves"], case["k"], case["n"]
        hit = L * (1.0 - (1.0 - 1.0 / L) ** T)  # leaves that some slot goes to
        ob = 2 if case["out"] == "bf16" else 4
        if op == "routed":  # queries, the hit leaves' weights, leaves in and order out, the slots' outputs
            return {"bytes": 2 * case["rows"] * k + int(2 * hit * n * k) + 8 * T + ob * T * n, "flops": 2 * T * n * k}
        # slot gradients and queries in, hit weights in, both gradients out (weights' for every leaf)
        return {"bytes": 2 * T * n + 2 * 2 * case["rows"] * k + int(2 * hit * n * k) + ob * L * n * k + 4 * T,
                "flops": 4 * T * n * k}
    e = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": 2 * e * case["rows"] * case["vocab"] + 8 * case["rows"] * case["top"] + 8 * case["rows"],
            "flops": 6 * case["rows"] * case["vocab"]}


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape, dtype=F32, scale=1.0):
    t = torch.randn(*shape, generator=g, device="cuda", dtype=F32)
    return (t * scale).to(dtype) if dtype != F32 else t.mul_(scale)


def _activations(g, m, k):
    """Unit-variance activations with a few channels some times larger, as hidden states have."""
    x = _randn(g, m, k)
    ch = torch.randint(0, k, (max(1, k // 100),), generator=g, device="cuda")
    x[:, ch] *= 6.0
    return x.to(BF)


def _int8_rows(g, n, k):
    """Int8 rows with their steps, as weights and documents are stored."""
    codes = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    scale = (0.5 + torch.rand(n, generator=g, device="cuda")) * (1.7 / (127.0 * math.sqrt(k)))
    return codes, scale


def _routing(g, rows, fan, L):
    """Distinct leaves for each query, some leaves more popular, one (if it can be) without a
    row, and one slot in fifty without a leaf (-1)."""
    s = _randn(g, rows, L) + _randn(g, 1, L, scale=0.5)
    if fan < L:
        s[:, L // 2] = -1e30
    leaves = s.topk(fan, dim=1).indices.to(torch.int32)
    drop = torch.rand(rows, fan, generator=g, device="cuda") < 0.02
    return torch.where(drop, torch.full_like(leaves, -1), leaves).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op in ("i8_linear", "i8_scores"):
        m, k, n = case["m"], case["k"], case["n"]
        if op == "i8_linear":
            st["x"] = _activations(g, m, k)
        else:
            st["x8"], st["xs"] = _int8_rows(g, m, k)
        st["w8"], st["ws"] = _int8_rows(g, n, k)
        st["bias"] = _randn(g, n, scale=0.2) if case["bias"] else None
        st["out"] = torch.empty(m, n, dtype=BF if op == "i8_linear" else F32, device="cuda")
        return st
    if op in ("routed", "routed_grad"):
        rows, fan, L, k, n = (case[f] for f in ("rows", "fan", "leaves", "k", "n"))
        st["x"] = _randn(g, rows, k, dtype=BF)
        st["w"] = torch.empty(L, n, k, dtype=BF, device="cuda")
        for l in range(L):
            st["w"][l] = _randn(g, n, k, dtype=BF, scale=1.0 / math.sqrt(k))
        st["leaves"] = _routing(g, rows, fan, L)
        if op == "routed_grad":  # a backward pass has the forward's order in hand
            st["offsets"], st["order"] = _plain_group(st["leaves"], L)
            st["dy"] = _randn(g, rows * fan, n, dtype=BF, scale=0.1)
        return st
    rows, V, top = case["rows"], case["vocab"], min(case["top"], case["vocab"])
    dt = BF if case["dtype"] == "bf16" else F32
    z = _randn(g, rows, V, scale=2.0)
    ids = torch.empty(rows, top, dtype=torch.int32, device="cuda")
    sc = torch.empty(rows, top, dtype=F32, device="cuda")
    for r0 in range(0, rows, 512):  # a teacher that agrees with the student in part
        t = z[r0:r0 + 512] * 0.7 + _randn(g, min(512, rows - r0), V, scale=2.0)
        v, i = t.topk(top, dim=1)
        ids[r0:r0 + 512], sc[r0:r0 + 512] = i.to(torch.int32), v
    length = torch.randint(1, top + 1, (rows, 1), generator=g, device="cuda")  # some lists are short, some empty
    full = torch.rand(rows, 1, generator=g, device="cuda") < 0.8
    none = torch.rand(rows, 1, generator=g, device="cuda") < 0.01
    length = torch.where(full, torch.full_like(length, top), length)
    length = torch.where(none, torch.zeros_like(length), length)
    past = torch.arange(top, device="cuda")[None, :] >= length
    st["ids"] = ids.masked_fill_(past, -1)
    st["scores"] = sc.masked_fill_(past, -math.inf)
    st["z"] = z.to(dt)
    st["weight"] = torch.rand(rows, generator=g, device="cuda") / rows
    return st


# ------------------------------------------------------------------------------- plain forms
def _plain_quantize(x):
    xf = x.float()
    s = xf.abs().amax(dim=1) / 127.0
    c = torch.where(s[:, None] > 0, (xf / s[:, None]).round().clamp(-127, 127), torch.zeros_like(xf))
    return c, s


def _plain_i8(a, sa, b, sb, bias, dtype):
    y = (a.float() @ b.float().t()) * sa[:, None] * sb[None, :]
    if bias is not None:
        y = y + bias[None, :]
    return y.to(dtype)


def _plain_group(leaves, L):
    """(offsets int64 [L + 1], order int32 [slots]): slots by (leaf, slot), those without a leaf last."""
    lf = leaves.reshape(-1).long()
    lf = torch.where((lf < 0) | (lf >= L), torch.full_like(lf, L), lf)
    order = torch.sort(lf, stable=True).indices.to(torch.int32)
    count = (lf[:, None] == torch.arange(L, device=lf.device)[None, :]).sum(0)
    offsets = torch.zeros(L + 1, dtype=torch.int64, device=lf.device)
    offsets[1:] = count.cumsum(0)
    return offsets, order


def _plain_routed(x, w, offsets, order, fan, dtype):
    y = torch.zeros(order.numel(), w.shape[1], dtype=dtype, device=x.device)
    off = offsets.tolist()
    for l in range(w.shape[0]):
        if off[l + 1] > off[l]:
            s = order[off[l]:off[l + 1]].long()
            y[s] = (x[s // fan].float() @ w[l].float().t()).to(dtype)
    return y


def _plain_routed_grad(dy, x, w, offsets, order, fan, dtype):
    T, (L, n, k) = order.numel(), w.shape
    dx = torch.zeros(T, k, dtype=F32, device=x.device)
    dw = torch.zeros(L, n, k, dtype=dtype, device=x.device)
    off = offsets.tolist()
    for l in range(L):
        if off[l + 1] > off[l]:
            s = order[off[l]:off[l + 1]].long()
            d = dy[s].float()
            dx[s] = d @ w[l].float()
            dw[l] = (d.t() @ x[s // fan].float()).to(dtype)
    return dx.view(-1, fan, k).sum(1).to(x.dtype), dw


def _plain_distill(z, ids, scores, tau, weight):
    zf = z.float() / tau
    valid = (ids >= 0) & (ids < z.shape[1])
    some = (valid & (scores > -math.inf)).any(1, keepdim=True)
    t = torch.where(valid, scores / tau, torch.full_like(scores, -math.inf))
    t = torch.where(some, t, torch.zeros_like(t))
    e = (t - t.amax(1, keepdim=True)).exp()
    p = torch.where(some, e / e.sum(1, keepdim=True), torch.zeros_like(e))
    zmax = zf.amax(1, keepdim=True)
    ez = (zf - zmax).exp()
    sz = ez.sum(1, keepdim=True)
    at = ids.clamp(0, z.shape[1] - 1).long()
    logq = zf.gather(1, at) - zmax - sz.log()
    loss = torch.where(p > 0, p * (p.log() - logq), torch.zeros_like(p)).sum(1) * (tau * tau)
    g = ez.div_(sz).mul_(some.float())
    g.scatter_add_(1, at, -p)
    return loss, g.mul_(weight[:, None] * tau).to(z.dtype)


# ------------------------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        from mips_ah_partition_amd import ahlib as ah
        if op == "i8_linear":
            return ah.ah_i8_linear(state["x"], state["w8"], state["ws"], bias=state["bias"], out=state["out"])
        if op == "i8_scores":
            return ah.ah_i8_matmul(state["x8"], state["xs"], state["w8"], state["ws"], out=state["out"])
        if op == "routed":
            offsets, order = ah.ah_group_rows(state["leaves"], c["leaves"])
            y = ah.ah_grouped_matmul(state["x"], state["w"], offsets, order=order, fan=c["fan"],
                                     out_dtype=BF if c["out"] == "bf16" else F32)
            return offsets, order, y
        if op == "routed_grad":
            dx = ah.ah_grouped_matmul_dx(state["dy"], state["w"], state["offsets"], order=state["order"],
                                         fan=c["fan"], out_dtype=BF)
            dw = ah.ah_grouped_matmul_dw(state["dy"], state["x"], state["offsets"], order=state["order"],
                                         fan=c["fan"], out_dtype=BF if c["out"] == "bf16" else F32)
            return dx, dw
        return ah.ah_distill_topk(state["z"], state["ids"], state["scores"], tau=c["tau"],
                                  row_weight=state["weight"])
    if op == "i8_linear":
        a, sa = _plain_quantize(state["x"])
        return _plain_i8(a, sa, state["w8"], state["ws"], state["bias"], BF)
    if op == "i8_scores":
        return _plain_i8(state["x8"], state["xs"], state["w8"], state["ws"], None, F32)
    if op == "routed":
        offsets, order = _plain_group(state["leaves"], c["leaves"])
        return offsets, order, _plain_routed(state["x"], state["w"], offsets, order, c["fan"],
                                             BF if c["out"] == "bf16" else F32)
    if op == "routed_grad":
        return _plain_routed_grad(state["dy"], state["x"], state["w"], state["offsets"], state["order"], c["fan"],
                                  BF if c["out"] == "bf16" else F32)
    return _plain_distill(state["z"], state["ids"], state["scores"], c["tau"], state["weight"])


# ------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, D = case["op"], torch.float64
    if op in ("i8_linear", "i8_scores"):
        if op == "i8_linear":
            x = st["x"].to(D)
            step = x.abs().max(dim=1, keepdim=True).values / 127
            a = torch.nan_to_num(torch.round(x / step)) * step
        else:
            a = st["x8"].to(D) * st["xs"].to(D)[:, None]
        y = torch.empty(case["m"], case["n"], dtype=D, device="cuda")
        for j in range(0, case["n"], 8192):
            b = st["w8"][j:j + 8192].to(D) * st["ws"][j:j + 8192].to(D)[:, None]
            y[:, j:j + 8192] = torch.mm(a, b.t())
        return y if st["bias"] is None else y.add_(st["bias"].to(D))
    if op in ("routed", "routed_grad"):
        L, fan, k, n, rows = (case[f] for f in ("leaves", "fan", "k", "n", "rows"))
        flat = st["leaves"].flatten()
        x, T = st["x"].to(D), rows * fan
        if op == "routed":
            y = torch.zeros(T, n, dtype=D, device="cuda")
            for l in range(L):
                at = torch.nonzero(flat == l).flatten()
                y[at] = torch.mm(x[torch.div(at, fan, rounding_mode="floor")], st["w"][l].to(D).t())
            return None, None, y
        dx = torch.zeros(rows, k, dtype=D, device="cuda")
        dw = torch.zeros(L, n, k, dtype=D, device="cuda")
        for l in range(L):
            at = torch.nonzero(flat == l).flatten()
            q = torch.div(at, fan, rounding_mode="floor")  # distinct: a query's leaves are
            d = st["dy"][at].to(D)
            dx[q] += torch.mm(d, st["w"][l].to(D))
            dw[l] = torch.mm(d.t(), x[q])
        return dx, dw
    rows, tau = case["rows"], case["tau"]
    loss = torch.zeros(rows, dtype=D, device="cuda")
    grad = torch.zeros(rows, case["vocab"], dtype=D, device="cuda")
    for r0 in range(0, rows, 256):
        sl = slice(r0, r0 + 256)
        logq = torch.log_softmax(st["z"][sl].to(D) / tau, dim=1)
        ok = st["ids"][sl] >= 0
        has = ok.any(dim=1).to(D)
        logp = torch.log_softmax(st["scores"][sl].to(D).masked_fill(~ok, -1e300) / tau, dim=1)
        p = logp.exp() * ok * has[:, None]
        at = st["ids"][sl].long() * ok
        loss[sl] = (tau ** 2) * (p * (logp.masked_fill(~ok, 0.0) - logq.gather(1, at))).sum(dim=1)
        grad[sl] = (logq.exp() * has[:, None]).scatter_add(1, at, -p) * (st["weight"][sl].to(D) * tau)[:, None]
    return loss, grad
