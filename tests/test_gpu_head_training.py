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


def _weight_gradient(torch, ah, head, items, hidden, ids, sc, tau):
    """The weights' gradient in 64 bits from the head's own queries on, and the sizes of its terms."""
    D, m = torch.float64, hidden.shape[0]
    q = head.queries(hidden, keep=True)
    x, _, _, gate = head._kept
    leaves = ah.ah_partition_score(x.float(), head.router, head.fan)[0].long()
    z = ah.ah_i8_linear(q, items.codes, items.step, out_dtype=torch.bfloat16).to(D)
    dz = torch.softmax(z / tau, 1).scatter_add(1, ids.long(), -torch.softmax(sc.to(D) / tau, 1)) * tau / m
    it = items.columns.to(D)
    dq, dqa = torch.mm(dz, it.t()), torch.mm(dz.abs(), it.abs().t())
    want, size = (torch.zeros(head.w.shape, dtype=D, device="cuda") for _ in range(2))
    for f in range(head.fan):
        for l in range(head.w.shape[0]):
            at = (leaves[:, f] == l).nonzero().flatten()
            gf = gate[at, f, None].to(D)
            want[l] += torch.mm((gf * dq[at]).t(), x[at].to(D))
            size[l] += torch.mm((gf * dqa[at]).t(), x[at].to(D).abs())
    return want, size


def test_items_beyond_one_product(gpu):
    """More items than a product sums at once: 2^20."""
    torch, ah, qh = gpu
    m, d, n = 5, 16, (1 << 20) + 1000
    head, items, hidden, rnd = _setup(torch, qh, m, h=32, k=24, d=d, L=3, n=n)
    assert items.columns.shape == (d, n)
    ids, sc = _teacher(torch, items, rnd, m, d)
    ids[:, 0] = torch.arange(n - m, n, device="cuda", dtype=torch.int32)  # of the last part
    want, size = _weight_gradient(torch, ah, head, items, hidden, ids, sc, 2.0)
    before = head.weights.clone()
    loss, _ = head.step(hidden, items, ids, sc, tau=2.0, lr=1.0)
    got = (before - head.weights).double()
    assert torch.isfinite(loss).all()
    assert ((got - want).abs() <= 4 * 2.0 ** -8 * size + 2.0 ** -22 * before.abs()).all()
    assert float((got - want).norm()) <= 0.05 * float(want.norm())


@pytest.mark.parametrize("most", [64, 256, 696])
def test_items_in_parts_give_the_gradient_of_all(gpu, most, monkeypatch):
    torch, ah, qh = gpu
    m, d, n = 40, 48, 700
    head, items, hidden, rnd = _setup(torch, qh, m, d=d, n=n)
    ids, sc = _teacher(torch, items, rnd, m, d)
    monkeypatch.setattr(qh.Items, "MOST", most)
    again, cut, _, _ = _setup(torch, qh, m, d=d, n=n)
    assert len(cut.parts()) == -(-n // most) and torch.equal(cut.columns, items.columns)
    want, size = _weight_gradient(torch, ah, head, items, hidden, ids, sc, 2.0)
    before = head.weights.clone()
    l0, dx0 = head.step(hidden, items, ids, sc, tau=2.0, lr=1.0, want_dx=True)
    l1, dx1 = again.step(hidden, cut, ids, sc, tau=2.0, lr=1.0, want_dx=True)
    assert torch.equal(l0, l1)
    for h in (head, again):
        assert (((before - h.weights).double() - want).abs() <= 4 * 2.0 ** -8 * size + 2.0 ** -22 * before.abs()).all()
    assert float((dx0 - dx1).float().norm()) <= 0.02 * float(dx0.float().norm())


def test_step_in_a_graph(gpu):
    torch, ah, qh = gpu
    m, d = 70, 48
    head, items, hidden, rnd = _setup(torch, qh, m)
    other = _setup(torch, qh, m)[0]
    ids, sc = _teacher(torch, items, rnd, m, d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        head.step(hidden, items, ids, sc, lr=0.0, want_dx=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, dx = head.step(hidden, items, ids, sc, tau=2.0, lr=0.5, want_dx=True)
    for i in range(4):
        hidden.copy_(rnd(*hidden.shape))
        graph.replay()
        torch.cuda.synchronize()
        want, wdx = other.step(hidden, items, ids, sc, tau=2.0, lr=0.5, want_dx=True)
        assert torch.equal(loss, want) and torch.equal(dx, wdx)
        assert torch.equal(head.weights, other.weights) and torch.equal(head.w, other.w)


def test_step_without_a_row(gpu):
    torch, ah, qh = gpu
    head, items, hidden, _ = _setup(torch, qh, 4)
    before = head.weights.clone()
    loss, dx = head.step(hidden[:0], items, torch.empty((0, 5), dtype=torch.int32, device="cuda"),
                         torch.empty((0, 5), device="cuda"), want_dx=True)
    assert loss.shape == (0,) and dx.shape == (0, 64) and torch.equal(head.weights, before)


def test_a_head_learns_from_an_index(gpu):
    """The whole way: a partitioned index answers the teacher's queries, its leaves' centroids route the head, and the
    head's own queries, put to the same index, come to find what the teacher's found."""
    import numpy as np
    import synth
    from mips_ah_partition_amd import index as ixm
    from mips_ah_partition_amd.search import AHIndex
    torch, ah, qh = gpu
    w = synth.WORKLOADS["tiny"]
    n, m = 4000, 300
    X = synth.rows(w, 0, n)
    d = X.shape[1]
    host = ixm.build(X, w.dpb, w.eta, num_leaves=16, seed=1, iters=4)
    idx = AHIndex(host, X, num_leaves_to_search=8, reorder=100, final_num_neighbors=20)
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    head = qh.QueryHead(rnd(d, 96) * 96 ** -0.5, idx.centroids, d, fan=3, seed=1)
    hidden = rnd(m, 96).bfloat16()
    feats = ah.ah_i8_linear(hidden, head.trunk8, head.trunk_scale, out_dtype=torch.float32)
    ids, scores = idx.search_batched(torch.mm(feats, rnd(d, d) * d ** -0.5).contiguous())
    items = qh.Items(torch.from_numpy(np.ascontiguousarray(X)).cuda())

    def found():
        own, _ = idx.search_batched(head.queries(hidden).contiguous())
        return float((own[:, :, None] == ids[:, None, :]).any(2).float().mean())

    before, losses = found(), []
    for _ in range(41):
        losses.append(float(head.step(hidden, items, ids, scores, lr=4.0)[0].mean()))
    assert losses[-1] < 0.7 * losses[0] and found() > before + 0.05
