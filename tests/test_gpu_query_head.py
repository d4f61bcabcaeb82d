"""QueryHead on the GPU: its forward and its gradients against the same formulas in 64 bits
on the values that the int8 layer made, and training that brings the head's answers to the
teacher's.

Tolerances: the projections' inputs are bfloat16 (as given), their sums float32, so queries
are off by k 2^-23 of their terms; gradients pass through bfloat16 twice (scores' gradient, slot
gradient) and once through bfloat16 items, each 2^-8 of the terms' sizes.
"""
import numpy as np
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


def _setup(torch, qh, m, h=96, k=64, d=48, L=6, n=700, fan=2):
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    head = qh.QueryHead(rnd(k, h) * h ** -0.5, rnd(L, k), d, fan=fan, seed=1)
    rows = rnd(n, d)
    items = qh.Items(rows / rows.norm(dim=1, keepdim=True))
    return head, items, rnd(m, h).bfloat16(), rnd


@pytest.mark.parametrize("m", [1, 50, 900])
def test_forward_and_gradients(gpu, m):
    torch, ah, qh = gpu
    head, items, hidden, rnd = _setup(torch, qh, m)
    q = head.queries(hidden, keep=True)
    x, offsets, order, gate = head._kept
    D = torch.float64
    leaves, _ = ah.ah_partition_score(x.float(), head.router, head.fan)
    w, xd = head.w.to(D), x.to(D)
    ref = sum(gate[:, f, None].to(D) * torch.bmm(w[leaves[:, f].long()], xd[:, :, None])[:, :, 0]
              for f in range(head.fan))
    mag = sum(gate[:, f, None].to(D) * torch.bmm(w[leaves[:, f].long()].abs(), xd[:, :, None].abs())[:, :, 0]
              for f in range(head.fan))
    assert ((q.to(D) - ref).abs() <= 70 * 2.0 ** -23 * mag).all()
    # the teacher's answers: an exact search by other queries
    t = torch.mm(rnd(m, 48) * 4, items.columns.float())
    s, i = t.topk(10, dim=1)
    before = head.weights.clone()
    loss, dx = head.step(hidden, items, i.to(torch.int32), s.float(), tau=2.0, lr=1.0, want_dx=True)
    dw = before - head.weights
    # the same in 64 bits from the queries on
    z = ah.ah_i8_linear(q, items.codes, items.step, out_dtype=torch.bfloat16).to(D)
    p = torch.softmax(s.to(D) / 2, 1)
    lq = torch.log_softmax(z / 2, 1)
    want = 4 * (p * (p.log() - lq.gather(1, i))).sum(1)
    assert ((loss.to(D) - want).abs() <= 1e-4 * (1 + want.abs())).all()
    dz = (lq.exp().scatter_add(1, i, -p)) * 2 / m
    it = items.columns.to(D)
    dq, dqa = dz @ it.t(), dz.abs() @ it.abs().t()
    rw, rwa = torch.zeros_like(w), torch.zeros_like(w)
    rx, rxa = torch.zeros_like(xd), torch.zeros_like(xd)
    for f in range(head.fan):
        gf = gate[:, f, None].to(D)
        for l in range(w.shape[0]):
            at = (leaves[:, f] == l).nonzero().flatten()
            rw[l] += (gf * dq)[at].t() @ xd[at]
            rwa[l] += (gf * dqa)[at].t() @ xd[at].abs()
            rx[at] += (gf * dq)[at] @ w[l]
            rxa[at] += (gf * dqa)[at] @ w[l].abs()
    eps = 4 * 2.0 ** -8
    assert ((dw.to(D) - rw).abs() <= eps * rwa + 2.0 ** -22 * before.abs().to(D)).all()
    assert ((dx.to(D) - rx).abs() <= eps * rxa).all()


def test_training_brings_the_answers_together(gpu):
    torch, ah, qh = gpu
    m, d = 600, 48
    head, items, hidden, rnd = _setup(torch, qh, m)
    # a teacher that the head can learn: queries that are a linear map of the features
    feats = ah.ah_i8_linear(hidden, head.trunk8, head.trunk_scale, out_dtype=torch.bfloat16).float()
    t = torch.mm(torch.mm(feats, rnd(64, d) * 0.5), items.columns.float())
    s, i = t.topk(20, dim=1)
    ids, s = i.to(torch.int32), s.float()
    def hits():
        z = ah.ah_i8_linear(head.queries(hidden), items.codes, items.step, out_dtype=torch.float32)
        top = z.topk(20, dim=1).indices
        return float((top[:, :, None] == i[:, None, :]).any(2).float().mean())
    first, hit0 = None, hits()
    for _ in range(60):
        loss, _ = head.step(hidden, items, ids, s, tau=1.0, lr=4.0)
        first = float(loss.mean()) if first is None else first
    assert float(loss.mean()) < 0.5 * first and hits() > hit0 + 0.2
