"""The 8-bit float trunk's gradients of batches that one product does not sum: parts of QueryHead.ROWS rows, added up in order.

Tolerance of the weights' gradient dx^T hidden from its bfloat16 and 8-bit operands: a code is within 2^-4 of its value or within
2^-17 of its block's largest (half the smallest step, 2^-10 2^e, of a scale 2^e <= 2 max / 448), so a product of two within
2 2^-4 + 2^-8 of its size; the instruction cuts off 2^-10 and the float32 sum of m terms (m / 8 + 16) 2^-23 of the sizes.  The
gradient is read off the master copy, which rounds by 2^-24 of the weight, twice, over the rate.
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


def _setup(torch, qh, m, h=40, k=24, d=16, L=3, n=60, fan=2, **kw):
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    head = qh.QueryHead(rnd(k, h) * h ** -0.5, rnd(L, k) * 0.5, d, fan=fan, seed=1, trunk_type="f8", **kw)
    rows = rnd(n, d)
    items = qh.Items(rows / rows.norm(dim=1, keepdim=True))
    hidden = rnd(m, h).bfloat16()
    s, i = torch.mm(rnd(m, d) * 4, items.columns.float()).topk(5, dim=1)
    return head, items, hidden, i.to(torch.int32), s.float()


def _check(torch, before, head, dx, hidden, lr):
    """The update of the trunk against dx^T hidden in float64."""
    D, m = torch.float64, hidden.shape[0]
    d, x = dx.to(D), hidden.to(D)
    size = torch.mm(d.abs().t().contiguous(), x.abs())
    size = size + 2.0 ** -13 * (d.abs().amax(0)[:, None] * x.abs().sum(0) + d.abs().sum(0)[:, None] * x.abs().amax(0))
    eps = 2 * 2.0 ** -4 + 2.0 ** -8 + 2.0 ** -10 + (m / 8 + 16) * 2.0 ** -23
    got = (before - head.trunk).to(D) / lr
    assert ((got - torch.mm(d.t().contiguous(), x)).abs() <= eps * size + 2.0 ** -23 * before.abs().to(D) / lr).all()


def test_more_rows_than_one_product_sums(gpu):
    torch, ah, qh = gpu
    m, lr = ah.AH_MAX_WIDTH + 300, 32.0
    head, items, hidden, ids, sc = _setup(torch, qh, m)
    twin, *_ = _setup(torch, qh, m)
    before = head.trunk.clone()
    loss, dh = head.step(hidden, items, ids, sc, tau=2.0, lr=1.0, want_dx="hidden", trunk_lr=lr)
    want, dx = twin.step(hidden, items, ids, sc, tau=2.0, lr=1.0, want_dx=True)
    assert torch.equal(loss, want) and torch.equal(head.weights, twin.weights) and dh.shape == hidden.shape
    _check(torch, before, head, dx, hidden, lr)
    codes, scale, _, _ = ah.ah_f8_quantize(dx)  # rows have no such limit: the same product from all of them at once
    assert torch.equal(dh, ah.ah_f8_matmul(codes, scale, twin._codes[2], twin._codes[3]))


@pytest.mark.parametrize("most", [128, 384, 512])
def test_parts_give_the_gradients_of_all(gpu, most, monkeypatch):
    torch, ah, qh = gpu
    m, kw = 500, dict(inner=40, drop=0.1)
    head, items, hidden, ids, sc = _setup(torch, qh, m, **kw)
    cut, *_ = _setup(torch, qh, m, **kw)
    twin, *_ = _setup(torch, qh, m, **kw)
    before = head.trunk.clone()
    l0, dh0 = head.step(hidden, items, ids, sc, tau=2.0, lr=1.0, want_dx="hidden", trunk_lr=2.0)
    monkeypatch.setattr(qh.QueryHead, "ROWS", most)
    l1, dh1 = cut.step(hidden, items, ids, sc, tau=2.0, lr=1.0, want_dx="hidden", trunk_lr=2.0)
    _, dx = twin.step(hidden, items, ids, sc, tau=2.0, lr=1.0, want_dx=True)
    assert torch.equal(l0, l1) and torch.equal(dh0, dh1) and torch.equal(head.weights_in, cut.weights_in)
    for h in (head, cut):
        _check(torch, before, h, dx, hidden, 2.0)
    if most >= m:
        assert torch.equal(head.trunk, cut.trunk)
    fresh = ah.ah_f8_quantize(cut.trunk, want_columns=True)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cut._codes[::2], fresh[::2]))
