"""QueryHead with gated blocks, dropout and an 8-bit float trunk: the operators together, forward and backward, against the
same formulas in float64 (autograd) on the features that the trunk's layer made.

Tolerances.  dy, the kept projections, their gradients and the hidden values are bfloat16: 2^-8 of their sizes each, and a
projection that is off by 2^-8 moves act' by at most 0.6 2^-8 |a| (second derivatives below 0.6).  So what a
product of these sums is off by at most 4 2^-8 of its terms' sizes, with 1.2 + 0.3 |a| in the place of |act'|.
"""
import numpy as np
import pytest

from philox_reference import factors

pytestmark = pytest.mark.gpu
EPS = 4 * 2.0 ** -8


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mips_ah_partition_amd import ahlib, query_head
    ahlib.lib()
    return torch, ahlib, query_head


def _setup(torch, qh, m, h=96, k=64, d=48, L=6, n=700, fan=2, **kw):
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n + fan)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    head = qh.QueryHead(rnd(k, h) * h ** -0.5, rnd(L, k) * 0.5, d, fan=fan, seed=1, **kw)
    rows = rnd(n, d)
    items = qh.Items(rows / rows.norm(dim=1, keepdim=True))
    hidden = rnd(m, h).bfloat16()
    s, i = torch.mm(rnd(m, d) * 4, items.columns.float()).topk(10, dim=1)
    return head, items, hidden, i.to(torch.int32), s.float()


def _act(torch, a, act):
    if act == "silu":
        return a * torch.sigmoid(a)
    if act == "gelu":
        return 0.5 * a * (1 + torch.erf(a / 2 ** 0.5))
    return a.clamp(min=0)


@pytest.mark.parametrize("m,fan,inner,act,drop,trunk", [
    (1, 2, 40, "silu", 0.0, "i8"), (50, 3, 56, "gelu", 0.2, "i8"), (900, 2, 64, "silu", 0.1, "f8"), (300, 1, 33, "relu", 0.5, "f8"),
    (400, 2, 0, "silu", 0.3, "f8"), (60, 2, 0, "silu", 0.0, "f8")])
def test_gradients(gpu, m, fan, inner, act, drop, trunk):
    torch, ah, qh = gpu
    D, tau = torch.float64, 2.0
    head, items, hidden, ids, sc = _setup(torch, qh, m, fan=fan, inner=inner, act=act, drop=drop, trunk_type=trunk)
    head.steps.fill_(4)
    head.queries(hidden, keep=True)
    x = head._kept[0]
    leaves = ah.ah_partition_score(x.float(), head.router, fan)[0].long()
    L, k = head.router.shape
    fx = torch.from_numpy(factors(m, k, drop, 2, 4)).cuda()
    fh = torch.from_numpy(factors(m * fan, max(inner, 1), drop, 3, 4)).cuda().view(m, fan, -1)
    # the features after dropout as the head's operands hold them (bfloat16), with the gradient of x f
    xd = (x.to(D) * fx).to(torch.bfloat16).to(D)
    router, w = head.router.to(D), head.w.to(D).clone().requires_grad_()
    win = head.w_in.to(D).clone().requires_grad_() if inner else None
    a_x, a_in = x.to(D).clone().requires_grad_(), xd.clone().requires_grad_()

    def project(v):  # [m, fan, dim], by leaf
        out = 0
        for l in range(L):
            on = (leaves == l).to(D)
            if inner:
                pre = v @ win[l].t()
                hid = (_act(torch, pre[:, :inner], act) * pre[:, inner:])[:, None, :] * fh
                y = hid @ w[l].t()
            else:
                y = (v @ w[l].t())[:, None, :]
            out = out + y * on[:, :, None]
        return out

    gate = torch.softmax((a_x[:, None, :] * router[leaves]).sum(2), 1)
    q64 = (gate[:, :, None] * project(a_in)).sum(1)
    before = head.weights.clone(), head.weights_in.clone() if inner else None
    # the head's own queries of this step: the loss and its gradient start from them
    q, *_ = head._forward(hidden, {})
    z = ah.ah_i8_linear(q, items.codes, items.step, out_dtype=torch.bfloat16).to(D)
    it = items.columns.to(D)
    p = torch.softmax(sc.to(D) / tau, 1)
    lq = torch.log_softmax(z / tau, 1)
    dz = (lq.exp().scatter_add(1, ids.long(), -p)) * tau / m
    dq, dqa = dz @ it.t(), dz.abs() @ it.abs().t()
    loss, dx = head.step(hidden, items, ids, sc, tau=tau, lr=1.0, want_dx=True)
    want = tau * tau * (p * (p.log() - lq.gather(1, ids.long()))).sum(1)
    assert ((loss.to(D) - want).abs() <= 1e-4 * (1 + want.abs())).all()
    assert int(head.steps) == (5 if drop else 4)
    grads = torch.autograd.grad((q64 * dq).sum(), [a_x, a_in, w] + ([win] if inner else []))
    # sizes of the terms
    with torch.no_grad():
        ya = torch.zeros(m, fan, w.shape[1], dtype=D, device="cuda")
        rx, rw, rwin, qa = torch.zeros_like(xd), torch.zeros_like(w), None if win is None else torch.zeros_like(win), 0
        for l in range(L):
            for f in range(fan):
                at = (leaves[:, f] == l).nonzero().flatten()
                if not len(at):
                    continue
                dya = gate[at, f, None] * dqa[at]
                if inner:
                    pre = xd[at] @ win[l].t()
                    a, b = pre[:, :inner].abs(), pre[:, inner:].abs()
                    pa = xd[at].abs() @ win[l].abs().t()  # the kept projections are off by their own rounding alone
                    fac = fh[at, f]
                    hid = (a * 1.2 * b + a * pa[:, inner:] * 2.0 ** -8) * fac
                    ya[at, f] = hid @ w[l].abs().t()
                    dh = (dya @ w[l].abs()) * fac
                    dpre = torch.cat([dh * b * (1.2 + 0.3 * a), dh * a * 1.2], 1)
                    rw[l] += dya.t() @ hid
                    rwin[l] += dpre.t() @ xd[at].abs()
                    rx[at] += dpre @ win[l].abs()
                else:
                    ya[at, f] = xd[at].abs() @ w[l].abs().t()
                    rw[l] += dya.t() @ xd[at].abs()
                    rx[at] += dya @ w[l].abs()
        qa = (gate[:, :, None] * ya).sum(1)
        assert ((q.to(D) - q64).abs() <= EPS * qa).all()
        along = (ya * dqa[:, None, :]).sum(2)
        dsc = gate * (along + (gate * along).sum(1, keepdim=True))
        ga = (dsc[:, :, None] * router[leaves].abs()).sum(1)
        want = grads[0] + grads[1] * fx
        assert ((dx.to(D) - want).abs() <= EPS * (rx * fx + ga) + 2.0 ** -8 * want.abs()).all()
        dw = (before[0] - head.weights).to(D)
        assert ((dw - grads[2]).abs() <= EPS * rw + 2.0 ** -22 * before[0].abs().to(D)).all()
        if inner:
            dwin = (before[1] - head.weights_in).to(D)
            assert ((dwin - grads[3]).abs() <= EPS * rwin + 2.0 ** -22 * before[1].abs().to(D)).all()
            assert torch.equal(head.w_in, head.weights_in.bfloat16())
    assert torch.equal(head.w, head.weights.bfloat16())


def test_trunk_gradients(gpu):
    """What the step does to the trunk and hands on: the two products of 8-bit codes of the features' gradient."""
    torch, ah, qh = gpu
    D = torch.float64
    head, items, hidden, ids, sc = _setup(torch, qh, 500, inner=40, drop=0.1, trunk_type="f8")
    twin, *_ = _setup(torch, qh, 500, inner=40, drop=0.1, trunk_type="f8")
    before = head.trunk.clone()
    _, dh = head.step(hidden, items, ids, sc, tau=2.0, want_dx="hidden", trunk_lr=0.5)
    _, dx = twin.step(hidden, items, ids, sc, tau=2.0, want_dx=True)
    assert dh.shape == hidden.shape and dx.shape == (500, 64)
    d, w, hx = dx.to(D), before.to(D), hidden.to(D)
    # each code is within 2^-4 of its value, or within 2^-17 of its block's largest
    size_h = d.abs() @ w.abs() + 2.0 ** -17 * (d.abs().amax(1, keepdim=True) * w.abs().sum(0) + d.abs().sum(1, keepdim=True) * w.abs().amax(0))
    assert ((dh.to(D) - d @ w).abs() <= 2.2 * 2.0 ** -4 * size_h).all()
    step = (before - head.trunk).to(D) / 0.5
    want = d.t() @ hx
    size_w = d.t().abs() @ hx.abs() + 500 * 2.0 ** -17 * d.abs().amax(0)[:, None] * hx.abs().amax(0) * 2
    assert ((step - want).abs() <= 2.2 * 2.0 ** -4 * size_w + 2.0 ** -22 * before.abs().to(D)).all()
    # the codes follow the master copy
    fresh = ah.ah_f8_quantize(head.trunk, want_columns=True)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(head._codes[::2], fresh[::2]))
    with pytest.raises(ValueError):
        _setup(torch, qh, 5)[0].step(hidden, items, ids, sc, trunk_lr=0.1)


def test_serving_has_no_dropout(gpu):
    torch, ah, qh = gpu
    a, items, hidden, ids, sc = _setup(torch, qh, 33, inner=40, drop=0.5, trunk_type="f8")
    b, *_ = _setup(torch, qh, 33, inner=40, drop=0.0, trunk_type="f8")
    assert torch.equal(a.queries(hidden), b.queries(hidden))
    assert torch.equal(a.queries(hidden), a.queries(hidden))
    one = torch.cat([a.queries(hidden[i:i + 1]) for i in range(33)])
    assert ((one - a.queries(hidden)).abs() <= 1e-2 * a.queries(hidden).abs().amax()).all()


def test_step_in_a_graph(gpu):
    torch, ah, qh = gpu
    kw = dict(inner=48, drop=0.2, trunk_type="f8")
    head, items, hidden, ids, sc = _setup(torch, qh, 256, **kw)
    other, *_ = _setup(torch, qh, 256, **kw)
    run = lambda h: h.step(hidden, items, ids, sc, tau=2.0, lr=0.5, want_dx="hidden", trunk_lr=0.2)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(head)
    torch.cuda.current_stream().wait_stream(s)
    run(other)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, dx = run(head)
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        want, wdx = run(other)
        assert torch.equal(loss, want) and torch.equal(dx, wdx), i
        assert torch.equal(head.weights, other.weights) and torch.equal(head.trunk, other.trunk)
    assert int(head.steps) == int(other.steps) == 4


def test_no_rows_and_bad_arguments(gpu):
    torch, ah, qh = gpu
    head, items, hidden, ids, sc = _setup(torch, qh, 8, inner=40, drop=0.1, trunk_type="f8")
    loss, dx = head.step(hidden[:0], items, ids[:0], sc[:0], want_dx="hidden", trunk_lr=0.1)
    assert loss.shape == (0,) and dx.shape == (0, 96) and torch.isfinite(head.trunk).all()
    for kw in (dict(trunk_type="f4"), dict(drop=1.0), dict(inner=-1), dict(act="tanh")):
        with pytest.raises(ValueError):
            _setup(torch, qh, 8, **kw)
