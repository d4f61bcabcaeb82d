"""Variants of the tiled kernels that the other files' sizes do not choose: gated products and their gradient at 128 x 128 with
operands through registers, sums that are no whole steps at that size, the ring of half-steps at its fewest steps, rows
that span 4 GB, and the wide-range type (e5m2) on either side of the 8-bit float product at every tile shape.  Beside
each case stands the tile it takes, in blocks of 64 (rows x columns).  References and tolerances as in test_gpu_gated and
test_gpu_f8.
"""
import pytest

from philox_reference import factors
from test_gpu_f8 import _values
from test_gpu_gated import _act, _forward_reference, _half, gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def _leaves(torch, ah, g, m, fan, L):
    """Leaves of a batch, one slot in fifty without one; all from g."""
    s = torch.randn(m, L, generator=g, device="cuda") + torch.randn(1, L, generator=g, device="cuda")
    leaves = s.topk(fan, dim=1).indices.to(torch.int32)
    if L > 1:
        leaves[torch.rand(m, fan, generator=g, device="cuda") < 0.02] = -1
    return (leaves,) + ah.ah_group_rows(leaves.contiguous(), L)


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("m,fan,L,k,n", [
    (20000, 1, 2, 100, 385),   # 2 x 2 through registers
    (9001, 2, 3, 77, 200),     # the same, rows of odd addresses, two slots a query
    (20000, 1, 3, 72, 300),    # 2 x 2, a last step of 8 elements
    (25000, 1, 1, 256, 200),   # bfloat16 4 x 4 with four steps, float32 2 x 2
    (9750, 2, 3, 256, 260),    # the same with two slots a query and columns that end inside a run of eight
    (11000, 2, 3, 1024, 136)])  # 3 x 4 in both types
def test_gated(gpu, m, fan, L, k, n, p):  # noqa: F811
    torch, ah = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(m + fan + L + k + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    act, T = ["silu", "gelu", "relu"][(m + n + k) % 3], m * fan
    x, w = rnd(m, k).bfloat16(), (rnd(L, 2 * n, k) * k ** -0.5 * 2).bfloat16()
    leaves, offsets, order = _leaves(torch, ah, g, m, fan, L)
    factor = torch.from_numpy(factors(T, n, p, 21, 2)).cuda()
    step = torch.tensor([2], device="cuda")
    want, tol, wpre, epre = _forward_reference(torch, x, w, leaves, act, factor)
    none = leaves.flatten() < 0
    for dt in (torch.bfloat16, torch.float32):
        big, bigp = torch.full((T + 1, n), 7.0, dtype=dt, device="cuda"), torch.full((T + 1, 2 * n), 7.0, device="cuda").bfloat16()
        h, pre = ah.ah_grouped_gated(x, w, offsets, order=order, fan=fan, act=act, drop=p, seed=21, step=step, out=big[:T], pre_out=bigp[:T])
        assert (big[T:] == 7).all() and (bigp[T:] == 7).all()
        assert ((h.double() - want).abs() <= tol + (want.abs() + tol) * _half(torch, dt)).all()
        assert ((pre.double() - wpre).abs() <= epre + (wpre.abs() + epre) * 2.0 ** -8).all()
        assert (h[none] == 0).all() and (pre[none] == 0).all() and (h[factor == 0] == 0).all()
        again, _ = ah.ah_grouped_gated(x, w, offsets, order=order, fan=fan, act=act, drop=p, seed=21, step=step, out_dtype=dt)
        assert torch.equal(again, h)


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("m,L,d,n", [
    (20000, 2, 77, 385),    # 2 x 2 through registers
    (18000, 3, 104, 390),   # the same, the rows whole chunks and the columns not
    (20000, 3, 72, 304),    # 2 x 2, a last step of 8 elements
    (33000, 5, 128, 160),   # 3 x 4 with two steps
    (33000, 1, 192, 166)])  # 2 x 2 through registers, one leaf
def test_gradient(gpu, m, L, d, n, p):  # noqa: F811
    torch, ah = gpu
    D = torch.float64
    g = torch.Generator(device="cuda")
    g.manual_seed(m + L + d + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    act = ["silu", "gelu", "relu"][(m + d + n) % 3]
    dy, w, pre = rnd(m, d).bfloat16(), (rnd(L, d, n) * n ** -0.5).bfloat16(), (rnd(m, 2 * n) * 2).bfloat16()
    leaves, offsets, order = _leaves(torch, ah, g, m, 1, L)
    flat = leaves.flatten()
    factor = torch.from_numpy(factors(m, n, p, 3, 0)).cuda()
    big, bigh = torch.full((m + 1, 2 * n), 7.0, device="cuda").bfloat16(), torch.full((m + 1, n), 7.0, device="cuda").bfloat16()
    dpre, h = ah.ah_grouped_gated_grad(dy, w, pre, offsets, order=order, act=act, drop=p, seed=3, dpre_out=big[:m], hidden_out=bigh[:m])
    assert (big[m:] == 7).all() and (bigh[m:] == 7).all()
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


@pytest.mark.parametrize("stride", [177536, 177544])
def test_rows_that_span_4_gb(gpu, stride):  # noqa: F811
    """12,096 rows whose last ones lie 4 GB behind the first: up to there the ring's 32-bit offsets reach (the first stride, the
    largest that they do), past it the general loads run.  The rows lie in the upper part of a larger block."""
    torch, ah = gpu
    m, k, n, lead = 12096, 1024, 512, 1100 * 1024 * 1024
    assert (m * stride * 2 < 2 ** 32) == (stride == 177536)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    block = torch.empty(lead + m * stride, dtype=torch.bfloat16, device="cuda")
    x, w = rnd(m, k).bfloat16(), (rnd(1, 2 * n, k) * k ** -0.5 * 2).bfloat16()
    far = block[lead:].view(m, stride)[:, :k]
    far.copy_(x)
    leaves = torch.zeros(m, 1, dtype=torch.int32, device="cuda")
    want, tol, wpre, epre = _forward_reference(torch, x, w, leaves, "silu", torch.ones(m, n, dtype=torch.float64, device="cuda"))
    for dt in (torch.bfloat16, torch.float32):
        h, pre = ah.ah_grouped_gated(far, w, want_pre=True, out_dtype=dt)
        assert ((h.double() - want).abs() <= tol + (want.abs() + tol) * _half(torch, dt)).all()
        assert ((pre.double() - wpre).abs() <= epre + (wpre.abs() + epre) * 2.0 ** -8).all()
    n = 1024  # (a gradient of 512 columns takes the smallest tile)
    wo, pre = (rnd(1, k, n) * n ** -0.5).bfloat16(), (rnd(m, 2 * n) * 2).bfloat16()
    near, hn = ah.ah_grouped_gated_grad(x, wo, pre)
    got, hf = ah.ah_grouped_gated_grad(far, wo, pre)
    assert torch.equal(hn, hf)
    if stride == 177536:
        assert torch.equal(got, near)
    # other loads, the sum in another order: both within its error, and a rounding apart
    size = (x.double().abs() @ wo[0].double().abs()) * (k + 16) * 2.0 ** -23
    a, b = pre.double().chunk(2, 1)
    f, df = _act(torch, a, "silu")
    sizes = torch.cat([size * (b * df).abs(), size * f.abs()], 1)
    assert ((got.double() - near.double()).abs() <= 2.1 * sizes + 2.1 * 2.0 ** -8 * near.double().abs()).all()


@pytest.mark.parametrize("out", ["bfloat16", "float32"])
@pytest.mark.parametrize("xt,wt", [("float8_e5m2", "float8_e4m3fn"), ("float8_e5m2", "float8_e5m2"), ("float8_e4m3fn", "float8_e5m2")])
@pytest.mark.parametrize("m,k,n", [
    (4100, 2000, 3001),   # 4 x 4
    (2700, 300, 3001),    # 3 x 4
    (8100, 300, 1501),    # 4 x 3
    (1300, 129, 3001),    # 2 x 3
    (1100, 300, 1000),    # 2 x 2
    (1000, 100, 1000),    # 1 x 1, two steps in LDS
    (1000, 2000, 1000)])  # 1 x 1, four
def test_wide_range_types(gpu, m, k, n, xt, wt, out):  # noqa: F811
    torch, ah = gpu
    D, dt, xt, wt = torch.float64, getattr(torch, out), getattr(torch, xt), getattr(torch, wt)
    g = torch.Generator(device="cuda")
    g.manual_seed(m + k + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rnd(m, k) * torch.exp2(torch.randint(-6, 7, (m, 1), generator=g, device="cuda").float()) \
        * torch.exp2((torch.arange(k, device="cuda") // 128 % 5 - 2).float())
    w = rnd(n, k) * torch.exp2(torch.randint(-6, 7, (n, 1), generator=g, device="cuda").float())
    bias = rnd(n) if n % 2 else None
    x8, xs, _, _ = ah.ah_f8_quantize(x, dtype=xt)
    w8, ws, _, _ = ah.ah_f8_quantize(w, dtype=wt)
    big = torch.full((m + 1, n), 7.0, dtype=dt, device="cuda")
    y = ah.ah_f8_matmul(x8, xs, w8, ws, bias=bias, out=big[:m])
    assert (big[m] == 7).all()
    a, b = _values(torch, x8, xs).cuda(), _values(torch, w8, ws).cuda()
    want, size = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
    if bias is not None:
        want, size = want + bias.to(D), size + bias.to(D).abs()
    tol = size * (2.0 ** -10 + (k / 8 + 16) * 2.0 ** -23)
    assert ((y.to(D) - want).abs() <= tol + (want.abs() + tol) * torch.finfo(dt).eps / 2).all()
    assert torch.equal(ah.ah_f8_matmul(x8, xs, w8, ws, bias=bias, out_dtype=dt), y)
    # whole numbers up to 8 are codes of both types: exact
    xi = torch.randint(-8, 9, (m, k), generator=g, device="cuda").float()
    wi = torch.randint(-8, 9, (n, k), generator=g, device="cuda").float()
    q, s, _, _ = ah.ah_f8_quantize(xi, dtype=xt)
    v, t, _, _ = ah.ah_f8_quantize(wi, dtype=wt)
    assert torch.equal(ah.ah_f8_matmul(q, s, v, t, out_dtype=torch.float32), xi @ wi.t())
