"""QueryHead.step on the GPU: the gradient of the features through projections and gates, and the
step's own edges.

Tolerance of the gradient: the scores' gradient, the slots' gradient and the result are rounded to
bfloat16 once each (2^-9 of the terms' sizes), the products and sums between them are float32; four times
2^-8 of the terms' absolute sizes covers them.
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mips_ah_partition_amd import ahlib, query_head
    ahlib.lib()
    return torch, ahlib, query_head


def _setup(torch, qh, m, h=96, k=64, d=48, L=6, n=700, fan=2, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n + fan + seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    head = qh.QueryHead(rnd(k, h) * h ** -0.5, rnd(L, k) * 0.5, d, fan=fan, seed=1)
    rows = rnd(n, d)
    items = qh.Items(rows / rows.norm(dim=1, keepdim=True))
    return head, items, rnd(m, h).bfloat16(), rnd


def _teacher(torch, items, rnd, m, d, k=10):
    s, i = torch.mm(rnd(m, d) * 4, items.columns.float()).topk(k, dim=1)
    return i.to(torch.int32), s.float()


@pytest.mark.parametrize("m,fan", [(1, 2), (50, 1), (50, 3), (900, 2)])
def test_gradient_of_the_features(gpu, m, fan):
    torch, ah, qh = gpu
    D, tau, d = torch.float64, 2.0, 48
    head, items, hidden, rnd = _setup(torch, qh, m, fan=fan)
    ids, sc = _teacher(torch, items, rnd, m, d)
    q = head.queries(hidden, keep=True)
    x = head._kept[0].to(D)
    leaves = ah.ah_partition_score(head._kept[0].float(), head.router, fan)[0].long()
    z = ah.ah_i8_linear(q, items.codes, items.step, out_dtype=torch.bfloat16).to(D)
    w, router, it = head.w.to(D), head.router.to(D), items.columns.to(D)
    dz = torch.softmax(z / tau, 1).scatter_add(1, ids.long(), -torch.softmax(sc.to(D) / tau, 1)) * tau / m
    dq, dqa = dz @ it.t(), dz.abs() @ it.abs().t()

    def parts(a, dirq, mat, r):  # sum over the slots of gate_f <W_f a, dirq>
        gate = torch.softmax((a[:, None, :] * r[leaves]).sum(2), 1)
        y = torch.stack([sum((mat[l] @ a.t()).t() * (leaves[:, f] == l)[:, None] for l in range(mat.shape[0]))
                         for f in range(fan)], 1)
        return gate, y, ((gate[:, :, None] * y).sum(1) * dirq).sum()

    a = x.clone().requires_grad_()
    gate, y, f = parts(a, dq, w, router)
    want, = torch.autograd.grad(f, a)
    with torch.no_grad():
        # the reference itself, along a direction, against a central difference
        way = rnd(m, x.shape[1]).to(D)
        h = 2.0 ** -12
        diff = (parts(x + h * way, dq, w, router)[2] - parts(x - h * way, dq, w, router)[2]) / (2 * h)
        assert abs(float(diff) - float((want * way).sum())) <= 1e-5 * float((want * way).abs().sum())
        ya = torch.stack([sum((w[l].abs() @ x.abs().t()).t() * (leaves[:, g] == l)[:, None] for l in range(w.shape[0]))
                          for g in range(fan)], 1)
        along = (ya * dqa[:, None, :]).sum(2)
        size = sum(((gate[:, g, None] * dqa) @ w[l].abs()) * (leaves[:, g] == l)[:, None]
                   for g in range(fan) for l in range(w.shape[0]))
        if fan > 1:
            dsc = gate * (along + (gate * along).sum(1, keepdim=True))
            size = size + (dsc[:, :, None] * router[leaves].abs()).sum(1)
    _, dx = head.step(hidden, items, ids, sc, tau=tau, want_dx=True)
    assert dx.dtype == torch.bfloat16 and dx.shape == x.shape
    assert ((dx.to(D) - want).abs() <= 4 * 2.0 ** -8 * size).all()
    # the roundings are independent of each other: in norm they stay near one bfloat16 step
    assert float((dx.to(D) - want).norm()) <= 0.05 * float(want.norm())
