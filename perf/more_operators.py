"""The operators of a query encoder that is trained and served, at sizes it meets: what a measurement runs.

A gated feed-forward block for each leaf (both projections, the activation and their product,
with dropout) and its backward pass, linear layers in 8-bit floating point with a power-of-two
scale for each block of 128 along the sum, their gradients, and dropout from a
counter-based generator with the addition of a residual.

``own`` false: plain torch forms in 32 bits.  ``own`` true: the framework's calls.
"""
from __future__ import annotations

import math

import torch

own = False

BF, F32, I64, D = torch.bfloat16, torch.float32, torch.int64, torch.float64
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
BLOCK = 128


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one query's features through a gated layer: latency, all time in the two weight matrices
        {"name": "gated_one_token", "op": "gated", "rows": 1, "fan": 1, "leaves": 1, "k": 1536, "n": 4096,
         "act": "silu", "drop": 0.0, "train": False, "out": "bf16"},
        # 100-d queries, odd width, an empty leaf, slots without a leaf, float32 results
        {"name": "gated_odd", "op": "gated", "rows": 333, "fan": 3, "leaves": 37, "k": 100, "n": 385, "act": "gelu",
         "drop": 0.1, "train": True, "out": "f32"},
        # a training batch: 2 of 16 leaves a query, pre-activations kept for the backward pass
        {"name": "gated_batch", "op": "gated", "rows": 8192, "fan": 2, "leaves": 16, "k": 1536, "n": 4096,
         "act": "silu", "drop": 0.1, "train": True, "out": "bf16"},
        # backward of the small, odd block
        {"name": "gated_grad_odd", "op": "gated_grad", "rows": 500, "fan": 3, "leaves": 21, "k": 77, "n": 200,
         "act": "relu", "drop": 0.25},
        # backward of the training batch: from the output's gradient to both projections' gradients
        {"name": "gated_grad_batch", "op": "gated_grad", "rows": 8192, "fan": 2, "leaves": 16, "k": 1536, "n": 4096,
         "act": "silu", "drop": 0.1},
        # one query through one linear layer of an encoder: latency
        {"name": "f8_one_token", "op": "f8_linear", "m": 1, "k": 1536, "n": 4096, "bias": True},
        # a small batch of queries, no size a multiple of anything
        {"name": "f8_few_odd", "op": "f8_linear", "m": 37, "k": 1001, "n": 4003, "bias": True},
        # documents being embedded: a long prompt's worth of tokens through a wide layer
        {"name": "f8_prompt", "op": "f8_linear", "m": 8192, "k": 4096, "n": 16384, "bias": True},
        # gradients of a small layer at odd sizes, the output's gradient in the wide-range type
        {"name": "f8_grad_odd", "op": "f8_grad", "m": 500, "k": 200, "n": 77, "dy": "e5m2"},
        # gradients of a layer over a training batch
        {"name": "f8_grad_batch", "op": "f8_grad", "m": 8192, "k": 1536, "n": 4096, "dy": "e4m3"},
        # dropout of a few queries' features: latency
        {"name": "dropout_few", "op": "dropout", "rows": 16, "n": 1536, "dtype": "bf16", "p": 0.1, "residual": False},
        # dropout and residual of a training batch's hidden states
        {"name": "dropout_batch", "op": "dropout", "rows": 32768, "n": 4096, "dtype": "bf16", "p": 0.1,
         "residual": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    caps = {"gated": 8192 * 2 * 1536 * 4096, "gated_grad": 8192 * 2 * 1536 * 4096, "f8_linear": 8192 * 4096 * 16384,
            "f8_grad": 8192 * 1536 * 4096, "dropout": 32768 * 4096 * 2}
    op = rng.choice(sorted(caps))
    while True:
        if op in ("gated", "gated_grad"):
            leaves = 1 if rng.random() < 0.25 else _log_int(rng, 2, 64)
            fan = rng.randint(1, min(4, leaves))
            c = {"op": op, "rows": _log_int(rng, 1, 8192), "fan": fan, "leaves": leaves, "k": _log_int(rng, 32, 1536),
                 "n": _log_int(rng, 32, 4096), "act": rng.choice(["silu", "gelu", "relu"]),
                 "drop": rng.choice([0.0, 0.1, 0.25])}
            if op == "gated":
                c["train"], c["out"] = rng.random() < 0.5, rng.choice(["bf16", "f32"])
            if rng.random() < 0.5:  # widths of a model are mostly multiples of 64
                c["k"], c["n"] = max(64, c["k"] // 64 * 64), max(64, c["n"] // 64 * 64)
            size = c["rows"] * fan * c["k"] * c["n"]
        elif op == "f8_linear":
            c = {"op": op, "m": _log_int(rng, 1, 8192), "k": _log_int(rng, 64, 4096), "n": _log_int(rng, 64, 16384),
                 "bias": rng.random() < 0.5}
            size = c["m"] * c["k"] * c["n"]
        elif op == "f8_grad":
            c = {"op": op, "m": _log_int(rng, 1, 8192), "k": _log_int(rng, 32, 1536), "n": _log_int(rng, 32, 4096),
                 "dy": rng.choice(["e4m3", "e5m2"])}
            size = c["m"] * c["k"] * c["n"]
        else:
            c = {"op": op, "rows": _log_int(rng, 1, 32768), "n": _log_int(rng, 32, 4096),
                 "dtype": rng.choice(["bf16", "f32"]), "p": rng.choice([0.05, 0.1, 0.3, 0.5]),
                 "residual": rng.random() < 0.5}
            size = c["rows"] * c["n"] * (2 if c["dtype"] == "bf16" else 4)
        if size <= caps[op]:
            return c


def work(case):
    op = case["op"]
    if op in ("gated", "gated_grad"):
        T, L, k, n = case["rows"] * case["fan"], case["leaves"], case["k"], case["n"]
        hit = L * (1.0 - (1.0 - 1.0 / L) ** T)  # leaves that some slot goes to
        if op == "gated":  # queries, order, the hit leaves' two matrices in; the product and pre-activations out
            ob = 2 if case["out"] == "bf16" else 4
            return {"bytes": 2 * case["rows"] * k + 4 * T + int(4 * hit * n * k) + ob * T * n
                    + (4 * T * n if case["train"] else 0), "flops": 4 * T * n * k}
        # the output's gradient, order, hit weights, pre-activations in; their gradients and the hidden values out
        return {"bytes": 2 * T * k + 4 * T + int(2 * hit * n * k) + (4 + 4 + 2) * T * n, "flops": 2 * T * n * k}
    if op == "f8_linear":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * m * k + n * k + n * _blocks(k) + (4 * n if case["bias"] else 0) + 2 * m * n,
                "flops": 2 * m * n * k}
    if op == "f8_grad":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": 2 * m * n + 2 * m * k + k * n + k * _blocks(n) + 2 * m * k + 2 * n * k,
                "flops": 4 * m * n * k}
    e = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": (3 if case["residual"] else 2) * e * case["rows"] * case["n"], "flops": 2 * case["rows"] * case["n"]}


def _blocks(k):
    return (k + BLOCK - 1) // BLOCK


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6271 + 29)
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


def _order(g, rows, fan, L):
    """A forward pass's order: slots by leaf, some leaves more popular, one (if it can be) without a
    row, one slot in fifty without a leaf (last).  (offsets int64 [L + 1], order int32 [slots])."""
    s = _randn(g, rows, L) + _randn(g, 1, L, scale=0.5)
    if fan < L:
        s[:, L // 2] = -1e30
    leaf = s.topk(fan, dim=1).indices.reshape(-1)
    if L > 1:
        leaf = torch.where(torch.rand(rows * fan, generator=g, device="cuda") < 0.02, torch.full_like(leaf, L), leaf)
    order = torch.sort(leaf, stable=True).indices.to(torch.int32)
    offsets = torch.zeros(L + 1, dtype=I64, device="cuda")
    offsets[1:] = (leaf[:, None] == torch.arange(L, device="cuda")[None, :]).sum(0).cumsum(0)
    return offsets, order


def _weights(g, L, n, k):
    w = torch.empty(L, n, k, dtype=BF, device="cuda")
    for l in range(L):
        w[l] = _randn(g, n, k, dtype=BF, scale=1.0 / math.sqrt(k))
    return w


def _pow2(e, dtype):
    """2^e for whole e in -300 .. 300, exactly (float32: 0 and infinity outside its range)."""
    return torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=D).to(dtype).to(e.device)[e.long() + 300]


def _f8_rows(x, dtype=E4M3):
    """Rows in 8 bits along the sum: codes [n, d to whole blocks of 128] and, block by block, the rows' scales
    2^(byte - 127): bytes [blocks, n to a multiple of 16].  The scale is the smallest power of two that keeps
    the block's largest value in range."""
    n, d = x.shape
    kb = _blocks(d)
    xf = torch.zeros(n, kb * BLOCK, dtype=F32, device=x.device)
    xf[:, :d] = x.float()
    xf = xf.view(n, kb, BLOCK)
    mant, exp = torch.frexp(xf.abs().amax(2))  # amax = mant 2^exp, mant in [0.5, 1); the types' largest: 0.875 2^9 or 2^16
    top = 9 if dtype is E4M3 else 16
    e = torch.where(mant > 0, exp - top + (mant > 0.875).to(exp.dtype), torch.zeros_like(exp)).clamp(min=-127)
    codes = (xf * _pow2(-e, F32)[:, :, None]).to(dtype).view(n, kb * BLOCK)
    scale = torch.full((kb, (n + 15) // 16 * 16), 127, dtype=torch.uint8, device=x.device)
    scale[:, :n] = (e + 127).t().to(torch.uint8)
    return codes, scale


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op in ("gated", "gated_grad"):
        rows, fan, L, k, n = (case[f] for f in ("rows", "fan", "leaves", "k", "n"))
        st["offsets"], st["order"] = _order(g, rows, fan, L)
        st["seed"] = int(seed) * 977 + 5
        if op == "gated":
            st["x"] = _randn(g, rows, k, dtype=BF)
            st["w"] = _weights(g, L, 2 * n, k)  # a leaf's gate rows, then its up rows
        else:
            st["dy"] = _randn(g, rows * fan, k, dtype=BF, scale=0.1)
            st["w"] = _weights(g, L, k, n)  # the block's second layer, [k, n] a leaf
            st["pre"] = _randn(g, rows * fan, 2 * n, dtype=BF)
        return st
    if op == "f8_linear":
        st["x"] = _activations(g, case["m"], case["k"])
        st["w8"], st["ws"] = _f8_rows(_randn(g, case["n"], case["k"], dtype=BF, scale=1.0 / math.sqrt(case["k"])))
        st["bias"] = _randn(g, case["n"], scale=0.2) if case["bias"] else None
        return st
    if op == "f8_grad":
        m, k, n = case["m"], case["k"], case["n"]
        st["x"] = _activations(g, m, k)
        st["dy"] = _randn(g, m, n, dtype=BF, scale=0.01)
        st["wt8"], st["wts"] = _f8_rows(_randn(g, k, n, dtype=BF, scale=1.0 / math.sqrt(k)))  # the weights' columns
        return st
    dt = BF if case["dtype"] == "bf16" else F32
    st["x"] = _randn(g, case["rows"], case["n"], dtype=dt)
    st["residual"] = _randn(g, case["rows"], case["n"], dtype=dt) if case["residual"] else None
    st["seed"] = int(seed) * 977 + 5
    st["step"] = torch.full((1,), 3 + int(seed), dtype=I64, device="cuda")
    return st


# ------------------------------------------------------------------------------- plain forms
def _plain_keep(rows, n, p, seed, step):
    """Which elements stay, [rows, n]: 16 bits each of Philox4x32-10 with key seed and counter
    (column / 8, row, step), kept where they are at least round(65536 p); and the factor of those that stay."""
    t = int(round(65536 * p))
    mask = 0xFFFFFFFF
    cols = torch.arange((n + 7) // 8, device="cuda", dtype=I64)[None, :].expand(rows, -1)
    c = [cols, torch.arange(rows, device="cuda", dtype=I64)[:, None].expand_as(cols),
         (step & mask).expand_as(cols), ((step >> 32) & mask).expand_as(cols)]
    key = [seed & mask, (seed >> 32) & mask]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # low 64 bits; the shifts below are masked
        c = [((b >> 32) & mask) ^ c[1] ^ key[0], b & mask, ((a >> 32) & mask) ^ c[3] ^ key[1], a & mask]
        key = [(key[0] + 0x9E3779B9) & mask, (key[1] + 0xBB67AE85) & mask]
    bits = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], 2).reshape(rows, -1)[:, :n]
    return bits >= t, 65536.0 / (65536 - t)


def _plain_act(a, act):
    """Activation and its derivative."""
    if act == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s))
    if act == "gelu":
        f = 0.5 * (1 + torch.erf(a * math.sqrt(0.5)))
        return a * f, f + a * torch.exp(-0.5 * a * a) * (1 / math.sqrt(2 * math.pi))
    return a.clamp(min=0), (a > 0).to(a.dtype)


def _plain_drop(h, p, seed):
    if p == 0:
        return h
    keep, f = _plain_keep(h.shape[0], h.shape[1], p, seed, torch.zeros(1, dtype=I64, device=h.device))
    return torch.where(keep, h * f, torch.zeros_like(h))


def _plain_gated(st):
    c = st["case"]
    T, n, dt = c["rows"] * c["fan"], c["n"], BF if c["out"] == "bf16" else F32
    pre = torch.zeros(T, 2 * n, dtype=F32, device="cuda")
    off = st["offsets"].tolist()
    for l in range(c["leaves"]):
        if off[l + 1] > off[l]:
            s = st["order"][off[l]:off[l + 1]].long()
            pre[s] = st["x"][s // c["fan"]].float() @ st["w"][l].float().t()
    h = _plain_drop(_plain_act(pre[:, :n], c["act"])[0] * pre[:, n:], c["drop"], st["seed"])
    return h.to(dt), pre.to(BF) if c["train"] else None


def _plain_gated_grad(st):
    c = st["case"]
    T, n = c["rows"] * c["fan"], c["n"]
    dh = torch.zeros(T, n, dtype=F32, device="cuda")
    off = st["offsets"].tolist()
    for l in range(c["leaves"]):
        if off[l + 1] > off[l]:
            s = st["order"][off[l]:off[l + 1]].long()
            dh[s] = st["dy"][s].float() @ st["w"][l].float()
    some = torch.zeros(T, 1, dtype=F32, device="cuda")
    some[st["order"][off[0]:off[-1]].long()] = 1.0  # rows of no leaf: zeros
    dh = _plain_drop(dh, c["drop"], st["seed"])
    a, b = st["pre"][:, :n].float(), st["pre"][:, n:].float()
    f, df = _plain_act(a, c["act"])
    h = _plain_drop(f * b * some, c["drop"], st["seed"])
    return torch.cat([dh * b * df, dh * f], 1).to(BF), h.to(BF)


def _plain_values(codes, scale):
    n, kp = codes.shape
    s = _pow2(scale[:, :n].t().int() - 127, F32)
    return (codes.float().view(n, kp // BLOCK, BLOCK) * s[:, :, None]).view(n, kp)


def _plain_f8(a, b, bias, dtype):
    y = a @ b.t()
    return (y if bias is None else y + bias[None, :]).to(dtype)


# ------------------------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        from mips_ah_partition_amd import ahlib as ah
        if op == "gated":
            return ah.ah_grouped_gated(state["x"], state["w"], state["offsets"], order=state["order"], fan=c["fan"],
                                       act=c["act"], drop=c["drop"], seed=state["seed"], want_pre=c["train"],
                                       out_dtype=BF if c["out"] == "bf16" else F32)
        if op == "gated_grad":
            return ah.ah_grouped_gated_grad(state["dy"], state["w"], state["pre"], state["offsets"],
                                            order=state["order"], act=c["act"], drop=c["drop"], seed=state["seed"],
                                            want_hidden=True)
        if op == "f8_linear":
            return ah.ah_f8_linear(state["x"], state["w8"], state["ws"], bias=state["bias"])
        if op == "f8_grad":
            d8, ds, dt8, dts = ah.ah_f8_quantize(state["dy"], dtype=E4M3 if c["dy"] == "e4m3" else E5M2,
                                                 want_columns=True)
            _, _, xt8, xts = ah.ah_f8_quantize(state["x"], want_rows=False, want_columns=True)
            dx = ah.ah_f8_matmul(d8, ds, state["wt8"], state["wts"], out_dtype=BF)
            return dx, ah.ah_f8_matmul(dt8, dts, xt8, xts, out_dtype=BF)
        return ah.ah_dropout(state["x"], c["p"], state["seed"], step=state["step"], residual=state["residual"])
    if op == "gated":
        return _plain_gated(state)
    if op == "gated_grad":
        return _plain_gated_grad(state)
    if op == "f8_linear":
        return _plain_f8(_plain_values(*_f8_rows(state["x"])), _plain_values(state["w8"], state["ws"]), state["bias"],
                         BF)
    if op == "f8_grad":
        t = E4M3 if c["dy"] == "e4m3" else E5M2
        d, dt = _plain_values(*_f8_rows(state["dy"], t)), _plain_values(*_f8_rows(state["dy"].t(), t))
        dx = _plain_f8(d, _plain_values(state["wt8"], state["wts"]), None, BF)
        return dx, _plain_f8(dt, _plain_values(*_f8_rows(state["x"].t())), None, BF)
    keep, f = _plain_keep(c["rows"], c["n"], c["p"], state["seed"], state["step"])
    y = torch.where(keep, state["x"].float() * f, torch.zeros((), device="cuda"))
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return y.to(state["x"].dtype)


# ------------------------------------------------------------------------------- in 64 bits
def _exact_factor(rows, n, p, seed, step):
    """0 or 1 / (1 - p'), element by element: Philox by 16-bit limbs, one row block at a time."""
    t = math.floor(65536 * p + 0.5)
    out = torch.empty(rows, n, dtype=D, device="cuda")

    def mul(v, m):  # (high, low) 32 bits of v m
        lo, mid = (v & 0xFFFF) * m, (v >> 16) * m
        s = mid + (lo >> 16)
        return s >> 16, ((s & 0xFFFF) << 16) | (lo & 0xFFFF)

    for r0 in range(0, rows, 4096):
        r1 = min(rows, r0 + 4096)
        w0, w1 = torch.meshgrid(torch.arange(r0, r1, device="cuda"), torch.arange((n + 7) // 8, device="cuda"),
                                indexing="ij")
        x0, x1 = w1, w0
        x2, x3 = torch.full_like(w0, step % 2 ** 32), torch.full_like(w0, step // 2 ** 32)
        for i in range(10):
            k0, k1 = (seed + i * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32
            h0, l0 = mul(x0, 0xD2511F53)
            h1, l1 = mul(x2, 0xCD9E8D57)
            x0, x1, x2, x3 = h1 ^ x1 ^ k0, l1, h0 ^ x3 ^ k1, l0
        for j in range(8):
            word = (x0, x1, x2, x3)[j // 2]
            col = ((word >> 16 if j % 2 else word) & 0xFFFF)[:, :(n - j + 7) // 8]
            out[r0:r1, j::8] = torch.where(col < t, 0.0, 1.0 / (1.0 - t / 65536.0)).to(D)
    return out


def _exact_act(a, act):
    if act == "silu":
        e = 1 / (1 + torch.exp(-a))
        return a * e, e + a * e * (1 - e)
    if act == "gelu":
        cdf = torch.special.ndtr(a)
        return a * cdf, cdf + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    return torch.relu(a), torch.where(a > 0, 1.0, 0.0).to(D)


def _exact_f8(x, dtype):
    """What the codes of a matrix's rows stand for."""
    x = x.to(D)
    out = torch.empty_like(x)
    most, bits, low = (448.0, 3, -6) if dtype is E4M3 else (57344.0, 2, -14)
    for a in range(0, x.shape[1], BLOCK):
        v = x[:, a:a + BLOCK]
        m = v.abs().max(1, keepdim=True).values
        e = torch.ceil(torch.log2(torch.where(m > 0, m, torch.full_like(m, most)) / most)).clamp(min=-127)
        u = v * _pow2(-e, D)
        step = _pow2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** low))) - bits, D)
        out[:, a:a + BLOCK] = torch.round(u / step) * step * _pow2(e, D)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("gated", "gated_grad"):
        rows, fan, L, n = (case[f] for f in ("rows", "fan", "leaves", "n"))
        T = rows * fan
        owner = torch.full((T,), -1, dtype=I64, device="cuda")
        for l in range(L):
            owner[st["order"][int(st["offsets"][l]):int(st["offsets"][l + 1])].long()] = l
        factor = _exact_factor(T, n, case["drop"], st["seed"], 0)
        if op == "gated":
            pre = torch.zeros(T, 2 * n, dtype=D, device="cuda")
            for l in range(L):
                at = torch.nonzero(owner == l).flatten()
                pre[at] = torch.mm(st["x"][torch.div(at, fan, rounding_mode="floor")].to(D), st["w"][l].to(D).t())
            gate, up = pre.chunk(2, 1)
            return _exact_act(gate, case["act"])[0] * up * factor, pre if case["train"] else None
        dh = torch.zeros(T, n, dtype=D, device="cuda")
        for l in range(L):
            at = torch.nonzero(owner == l).flatten()
            dh[at] = torch.mm(st["dy"][at].to(D), st["w"][l].to(D))
        gate, up = st["pre"].to(D).chunk(2, 1)
        f, df = _exact_act(gate, case["act"])
        dh *= factor
        return torch.cat([dh * up * df, dh * f], 1), f * up * factor * (owner >= 0)[:, None]
    if op == "f8_linear":
        a = _exact_f8(st["x"], E4M3)
        w = st["w8"].to(D)[:, :case["k"]] * _pow2(
            st["ws"][:, :case["n"]].t().int() - 127, D).repeat_interleave(BLOCK, 1)[:, :case["k"]]
        y = torch.mm(a, w.t())
        return y if st["bias"] is None else y.add_(st["bias"].to(D))
    if op == "f8_grad":
        t = E4M3 if case["dy"] == "e4m3" else E5M2
        n, k = case["n"], case["k"]
        wt = st["wt8"].to(D)[:, :n] * _pow2(st["wts"][:, :k].t().int() - 127, D).repeat_interleave(BLOCK, 1)[:, :n]
        dx = torch.mm(_exact_f8(st["dy"], t), wt.t())
        return dx, torch.mm(_exact_f8(st["dy"].t(), t), _exact_f8(st["x"].t(), E4M3).t())
    y = st["x"].to(D) * _exact_factor(case["rows"], case["n"], case["p"], st["seed"], int(st["step"]))
    return y if st["residual"] is None else y + st["residual"].to(D)
