"""Gated products of thousands of rows: the large tile shapes (256 x 256, 192 x 256) with their ring of half-steps where the sum
is long enough, 128 x 128 where it is not, and rows of no leaf.  References and tolerances as in test_gpu_gated.
"""
import pytest

from philox_reference import factors
from test_gpu_gated import _act, _forward_reference, _half, _route, gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# m, L, k, n: one leaf and several with ragged ends, 2 to 32 steps of 64, whole and partial columns
CASES = [(16128, 1, 128, 512), (12096, 1, 128, 512), (15000, 3, 192, 500), (11300, 4, 320, 520), (12096, 1, 2048, 512), (16128, 1, 1600, 512),
         (40000, 5, 256, 136), (22000, 3, 1024, 136), (12096, 1, 1024, 512), (30000, 5, 1600, 132)]


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("m,L,k,n", CASES)
def test_forward(gpu, m, L, k, n, p):  # noqa: F811
    torch, ah = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(m + L + k + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    act = ["silu", "gelu", "relu"][(m + n) % 3]
    x, w = rnd(m, k).bfloat16(), (rnd(L, 2 * n, k) * k ** -0.5 * 2).bfloat16()
    leaves, offsets, order = _route(torch, ah, rnd, m, 1, L, none=0.02 if L > 1 else 0)
    factor = torch.from_numpy(factors(m, n, p, 77, 5)).cuda()
    step = torch.tensor([5], device="cuda")
    want, tol, wpre, epre = _forward_reference(torch, x, w, leaves, act, factor)
    for dt in (torch.bfloat16, torch.float32):
        big, bigp = torch.full((m + 1, n), 7.0, dtype=dt, device="cuda"), torch.full((m + 1, 2 * n), 7.0, device="cuda").bfloat16()
        h, pre = ah.ah_grouped_gated(x, w, offsets, order=order, act=act, drop=p, seed=77, step=step, out=big[:m], pre_out=bigp[:m])
        assert (big[m:] == 7).all() and (bigp[m:] == 7).all()
        assert ((h.double() - want).abs() <= tol + (want.abs() + tol) * _half(torch, dt)).all()
        assert ((pre.double() - wpre).abs() <= epre + (wpre.abs() + epre) * 2.0 ** -8).all()
        assert (h[leaves.flatten() < 0] == 0).all() and (pre[leaves.flatten() < 0] == 0).all() and (h[factor == 0] == 0).all()
        again, _ = ah.ah_grouped_gated(x, w, offsets, order=order, act=act, drop=p, seed=77, step=step, out_dtype=dt)
        assert torch.equal(again, h)


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("m,L,d,n", [(12096, 1, 128, 1024), (11300, 4, 320, 1000), (12096, 1, 1600, 1024), (30000, 5, 256, 264)])
def test_gradient(gpu, m, L, d, n, p):  # noqa: F811
    torch, ah = gpu
    D = torch.float64
    g = torch.Generator(device="cuda")
    g.manual_seed(m + L + d + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    act = ["silu", "gelu", "relu"][(m + d) % 3]
    dy, w, pre = rnd(m, d).bfloat16(), (rnd(L, d, n) * n ** -0.5).bfloat16(), (rnd(m, 2 * n) * 2).bfloat16()
    leaves, offsets, order = _route(torch, ah, rnd, m, 1, L, none=0.02 if L > 1 else 0)
    flat = leaves.flatten()
    factor = torch.from_numpy(factors(m, n, p, 3, 0)).cuda()
    dpre, h = ah.ah_grouped_gated_grad(dy, w, pre, offsets, order=order, act=act, drop=p, seed=3)
    over = pre.clone()
    ah.ah_grouped_gated_grad(dy, w, over, offsets, order=order, act=act, drop=p, seed=3, want_hidden=False, dpre_out=over)
    assert torch.equal(over, dpre)
    dh, size = torch.zeros(m, n, dtype=D, device="cuda"), torch.zeros(m, n, dtype=D, device="cuda")
    for l in range(L):
        at = (flat == l).nonzero().flatten()
        dh[at] = dy[at].to(D) @ w[l].to(D)
        size[at] = dy[at].to(D).abs() @ w[l].to(D).abs()
    a, b = pre.to(D).chunk(2, 1)
    f, df = _act(torch, a, act)
    e, ef, edf = (d + 16) * 2.0 ** -23 * size, (f.abs() * (a.abs() + 16) + a.abs()) * 2.0 ** -22, (a.abs() + 16) * 2.0 ** -22
    dh = dh * factor
    some = (flat >= 0)[:, None].to(D)
    for got, want, tol in ((dpre[:, :n], dh * b * df, (e * (df.abs() + edf) * factor + dh.abs() * edf) * b.abs()),
                           (dpre[:, n:], dh * f, e * (f.abs() + ef) * factor + dh.abs() * ef), (h, f * b * factor * some, ef * b.abs() * factor)):
        assert ((got.double() - want).abs() <= tol + (want.abs() + tol) * 2.0 ** -8).all()
    assert (dpre[flat < 0] == 0).all() and (h[flat < 0] == 0).all()


STARTS = [(60, 64, 40), (60, 400, 40), (900, 128, 64), (900, 100, 30), (12096, 128, 512)]


@pytest.mark.parametrize("m,k,n", STARTS)
def test_rows_before_the_first_leaf(gpu, m, k, n):  # noqa: F811
    """Rows before the first start and behind the last one belong to no leaf: zeros."""
    torch, ah = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(m + k)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, wo = rnd(m, k).bfloat16(), rnd(3, 2 * n, k).bfloat16(), rnd(3, k, n).bfloat16()
    offsets = torch.tensor([5, m // 3, m // 3, m - 7], device="cuda")  # the second leaf's rows: none
    h, pre = ah.ah_grouped_gated(x, w, offsets, want_pre=True)
    d, hid = ah.ah_grouped_gated_grad(x, wo, pre, offsets)
    for t in (h, pre, d, hid):
        assert (t[:5] == 0).all() and (t[m - 7:] == 0).all() and torch.isfinite(t).all()
    for a, b, l in ((5, m // 3, 0), (m // 3, m - 7, 2)):  # each leaf alone: other sizes, other orders of the sum
        p = x[a:b].double() @ w[l].double().t()
        e = (k + 16) * 2.0 ** -23 * (x[a:b].double().abs() @ w[l].double().abs().t())
        assert ((pre[a:b].double() - p).abs() <= e + (p.abs() + e) * 2.0 ** -8).all()


@pytest.mark.parametrize("m,k,n", STARTS)
def test_starts_out_of_order(gpu, m, k, n):  # noqa: F811
    """Starts have to ascend.  Others give rows of no meaning (leaves that overlap), and nothing outside the outputs."""
    torch, ah = gpu
    x, w, wo = (torch.ones(*s, device="cuda").bfloat16() for s in ((m, k), (3, 2 * n, k), (3, k, n)))
    outs = [torch.full((m + 2, c), 7.0, device="cuda").bfloat16() for c in (n, 2 * n, 2 * n, n)]
    offsets = torch.tensor([5, m // 2, m // 3, m - 7], device="cuda")
    ah.ah_grouped_gated(x, w, offsets, out=outs[0][1:-1], pre_out=outs[1][1:-1])
    ah.ah_grouped_gated_grad(x, wo, outs[1][1:-1], offsets, dpre_out=outs[2][1:-1], hidden_out=outs[3][1:-1])
    for t in outs:
        assert (t[0] == 7).all() and (t[-1] == 7).all()
