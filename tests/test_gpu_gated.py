"""The gated products on the GPU against their formulas in 64 bits.

Tolerances.  A sum of k bfloat16 products in float32 is off by at most (k + 16) 2^-23 of its terms' sizes: e.  With
a, b off by ea, eb, act(a) b is off by 1.2 ea (|b| + eb) + |act(a)| eb (the activations' slopes are below 1.2);
the activation itself by (|a| + 16) 2^-22 of |act(a)| and, in gelu's tail, |a| 2^-22.  Its derivative
likewise, (|a| + 16) 2^-22 (its values are below 1.2).  Results are rounded once, half a step of their type.
"""
import numpy as np
import pytest

from philox_reference import factors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mips_ah_partition_amd import ahlib
    ahlib.lib()
    return torch, ahlib


def _act(torch, a, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-a))
        return a * s, s * (1 + a * (1 - s))
    if act == "gelu":
        c = 0.5 * (1 + torch.erf(a / 2 ** 0.5))
        return a * c, c + a * torch.exp(-a * a / 2) / (2 * np.pi) ** 0.5
    return a.clamp(min=0), (a > 0).to(a.dtype)


def _half(torch, dtype):
    return torch.finfo(dtype).eps / 2


def _route(torch, ah, rnd, m, fan, L, none=0.05):
    """Leaves of a batch, one leaf (if there are more) without a row and some slots without a leaf."""
    if L == 1 and fan == 1:
        leaves = torch.zeros(m, 1, dtype=torch.int32, device="cuda")
    else:
        s = rnd(m, L) + rnd(1, L)
        if L > fan:
            s[:, L // 2] = -1e30
        leaves = s.topk(fan, dim=1).indices.to(torch.int32)
    if none:
        leaves[torch.rand(m, fan, device="cuda") < none] = -1
    return (leaves,) + ah.ah_group_rows(leaves.contiguous(), L)


def _forward_reference(torch, x, w, leaves, act, factor):
    D = torch.float64
    T, n = leaves.numel(), w.shape[1] // 2
    flat, fan = leaves.flatten(), leaves.shape[1]
    pre = torch.zeros(T, 2 * n, dtype=D, device="cuda")
    size = torch.zeros_like(pre)
    for l in range(w.shape[0]):
        at = (flat == l).nonzero().flatten()
        xs, ws = x[torch.div(at, fan, rounding_mode="floor")].to(D), w[l].to(D)
        pre[at] = xs @ ws.t()
        size[at] = xs.abs() @ ws.abs().t()
    a, b = pre.chunk(2, 1)
    e = (x.shape[1] + 16) * 2.0 ** -23 * size
    ea, eb = e.chunk(2, 1)
    f, _ = _act(torch, a, act)
    tol = 1.2 * ea * (b.abs() + eb) + f.abs() * eb + (f * b).abs() * (a.abs() + 16) * 2.0 ** -22 + (a * b).abs() * 2.0 ** -22
    return f * b * factor, tol * factor, pre, e


CASES = [  # m, fan, L, k, n: few rows and many, whole tiles and odd ends, one leaf and many
    (1, 1, 1, 64, 64), (1, 1, 1, 1536, 130), (1, 2, 3, 8, 1), (3, 1, 2, 1, 5), (7, 2, 5, 33, 17), (16, 4, 64, 256, 96),
    (40, 1, 1, 200, 72), (300, 2, 3, 64, 96), (333, 3, 37, 100, 385), (1000, 1, 1, 128, 256), (2000, 2, 4, 192, 320),
    (600, 1, 2, 72, 40), (513, 1, 1, 65, 129), (5000, 1, 3, 16, 8), (700, 2, 200, 48, 64)]


@pytest.mark.parametrize("out", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,fan,L,k,n", CASES)
def test_forward(gpu, m, fan, L, k, n, out):
    torch, ah = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(m + fan + L + k + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = getattr(torch, out)
    act, p = ["silu", "gelu", "relu"][(m + n) % 3], [0.0, 0.1, 0.5][(k + L) % 3]
    x, w = rnd(m, k).bfloat16(), (rnd(L, 2 * n, k) * k ** -0.5 * 2).bfloat16()
    leaves, offsets, order = _route(torch, ah, rnd, m, fan, L)
    T = m * fan
    factor = torch.from_numpy(factors(T, n, p, 77, 5)).cuda()
    step = torch.tensor([5], device="cuda")
    # outputs inside larger blocks: nothing behind the last row is written
    big, bigp = torch.full((T + 2, n), 7.0, dtype=dt, device="cuda"), torch.full((T + 2, 2 * n), 7.0, device="cuda").bfloat16()
    h, pre = ah.ah_grouped_gated(x, w, offsets, order=order, fan=fan, act=act, drop=p, seed=77, step=step, out=big[:T],
                                 pre_out=bigp[:T])
    assert (big[T:] == 7).all() and (bigp[T:] == 7).all()
    want, tol, wpre, epre = _forward_reference(torch, x, w, leaves, act, factor)
    assert ((h.double() - want).abs() <= tol + (want.abs() + tol) * _half(torch, dt)).all()
    assert ((pre.double() - wpre).abs() <= epre + (wpre.abs() + epre) * 2.0 ** -8).all()
    assert (h[leaves.flatten() < 0] == 0).all() and (pre[leaves.flatten() < 0] == 0).all()
    assert (h[factor == 0] == 0).all()
    # without the projections: the same h; again: the same bits
    h2, none = ah.ah_grouped_gated(x, w, offsets, order=order, fan=fan, act=act, drop=p, seed=77, step=step, out_dtype=dt)
    assert none is None and torch.equal(h2, h)


@pytest.mark.parametrize("hidden", [True, False])
@pytest.mark.parametrize("m,fan,L,d,n", CASES)
def test_gradient(gpu, m, fan, L, d, n, hidden):
    torch, ah = gpu
    D = torch.float64
    g = torch.Generator(device="cuda")
    g.manual_seed(m + fan + L + d + 2 * n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    act, p = ["silu", "gelu", "relu"][(m + d) % 3], [0.0, 0.1, 0.5][(n + L) % 3]
    T = m * fan
    dy, w, pre = rnd(T, d).bfloat16(), (rnd(L, d, n) * n ** -0.5).bfloat16(), (rnd(T, 2 * n) * 2).bfloat16()
    leaves, offsets, order = _route(torch, ah, rnd, m, fan, L)
    flat = leaves.flatten()
    factor = torch.from_numpy(factors(T, n, p, 3, 0)).cuda()
    big = torch.full((T + 2, 2 * n), 7.0, device="cuda").bfloat16()
    dpre, h = ah.ah_grouped_gated_grad(dy, w, pre, offsets, order=order, act=act, drop=p, seed=3, want_hidden=hidden,
                                       dpre_out=big[:T])
    assert (big[T:] == 7).all() and (h is None) == (not hidden)
    dh, size = torch.zeros(T, n, dtype=D, device="cuda"), torch.zeros(T, n, dtype=D, device="cuda")
    some = (flat >= 0)[:, None].to(D)
    for l in range(L):
        at = (flat == l).nonzero().flatten()
        dh[at] = dy[at].to(D) @ w[l].to(D)
        size[at] = dy[at].to(D).abs() @ w[l].to(D).abs()
    a, b = pre.to(D).chunk(2, 1)
    f, df = _act(torch, a, act)
    e = (d + 16) * 2.0 ** -23 * size
    ef = (f.abs() * (a.abs() + 16) + a.abs()) * 2.0 ** -22
    edf = (a.abs() + 16) * 2.0 ** -22
    dh = dh * factor
    for got, want, tol in ((dpre[:, :n], dh * b * df, (e * (df.abs() + edf) * factor + dh.abs() * edf) * b.abs()),
                           (dpre[:, n:], dh * f, e * (f.abs() + ef) * factor + dh.abs() * ef)):
        assert ((got.double() - want).abs() <= tol + (want.abs() + tol) * 2.0 ** -8).all()
    if hidden:
        want, tol = f * b * factor * some, ef * b.abs() * factor
        assert ((h.double() - want).abs() <= tol + (want.abs() + tol) * 2.0 ** -8).all()
        assert (h[flat < 0] == 0).all()
    assert (dpre[flat < 0] == 0).all()
    # in the projections' own memory
    over = pre.clone()
    ah.ah_grouped_gated_grad(dy, w, over, offsets, order=order, act=act, drop=p, seed=3, want_hidden=False, dpre_out=over)
    assert torch.equal(over, dpre)


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_gradient_against_differences(gpu, act):
    """The whole block, h = f(W x): <dh, h(pre + eps v) - h(pre - eps v)> / 2 eps is <dpre, v>, all in float64 from the
    kernel's dpre (its rounding: 2^-8 of each term)."""
    torch, ah = gpu
    D = torch.float64
    m, d, n = 60, 40, 56
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dy, w, pre = rnd(m, d).bfloat16(), rnd(1, d, n).bfloat16(), rnd(m, 2 * n).bfloat16()
    dpre, _ = ah.ah_grouped_gated_grad(dy, w, pre, act=act, drop=0.3, seed=9)
    fac = torch.from_numpy(factors(m, n, 0.3, 9, 0)).cuda()
    dh = dy.to(D) @ w[0].to(D)
    v, h = rnd(m, 2 * n).to(D), 2.0 ** -14

    def y(q):
        a, b = q.chunk(2, 1)
        return _act(torch, a, act)[0] * b * fac

    p = pre.to(D)
    terms = dh * (y(p + h * v) - y(p - h * v)) / (2 * h)
    got = dpre.to(D) * v
    # truncation of the difference: h^2 times third derivatives (below 10); relu: an element within h |v| of 0 (none here)
    assert act != "relu" or (p[:, :n].abs() > h * v[:, :n].abs()).all()
    assert abs(float(got.sum() - terms.sum())) <= 2.0 ** -7 * float(got.abs().sum()) + 10 * h * h * float(dh.abs().sum())


def test_strided_and_shifted_inputs(gpu):
    torch, ah = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    for m, k, n in ((5, 72, 24), (500, 72, 24)):
        w, wo, pre = rnd(2, 2 * n, k), rnd(2, k, n), rnd(m, 2 * n)
        leaves = torch.randint(0, 2, (m, 1), generator=g, device="cuda", dtype=torch.int32)
        offsets, order = ah.ah_group_rows(leaves, 2)
        for off, pad in ((0, 8), (8, 8), (1, 2), (3, 4)):
            wide = rnd(m, off + k + pad)
            x = wide[:, off:off + k]
            h, p = ah.ah_grouped_gated(x, w, offsets, order=order, want_pre=True)
            h2, p2 = ah.ah_grouped_gated(x.contiguous(), w, offsets, order=order, want_pre=True)
            d, hid = ah.ah_grouped_gated_grad(x, wo, pre, offsets, order=order)
            d2, hid2 = ah.ah_grouped_gated_grad(x.contiguous(), wo, pre, offsets, order=order)
            for a, b in ((h, h2), (p, p2), (d, d2), (hid, hid2)):  # other loads, other orders of the sum: rounding apart
                assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 2e-5).all()
        # weights and outputs at addresses that are no multiple of 16 bytes
        flat = torch.zeros(2 * 2 * n * k + 1, device="cuda").bfloat16()
        flat[1:] = w.flatten()
        out = torch.zeros(m * n + 1, device="cuda").bfloat16()[1:].view(m, n)
        pout = torch.zeros(m * 2 * n + 1, device="cuda").bfloat16()[1:].view(m, 2 * n)
        h3, p3 = ah.ah_grouped_gated(x.contiguous(), flat[1:].view(2, 2 * n, k), offsets, order=order, out=out, pre_out=pout)
        assert ((h3.float() - h2.float()).abs() <= 2.0 ** -7 * h2.float().abs() + 2e-5).all()
        assert ((p3.float() - p2.float()).abs() <= 2.0 ** -7 * p2.float().abs() + 2e-5).all()


def test_no_offsets_is_one_leaf(gpu):
    torch, ah = gpu
    for m in (1, 9, 200, 1000):
        x, w = torch.randn(m, 64, device="cuda").bfloat16(), torch.randn(1, 48, 64, device="cuda").bfloat16()
        wo, dy = torch.randn(1, 40, 24, device="cuda").bfloat16(), torch.randn(m, 40, device="cuda").bfloat16()
        offsets = torch.tensor([0, m], device="cuda")
        h, pre = ah.ah_grouped_gated(x, w, want_pre=True)
        h2, pre2 = ah.ah_grouped_gated(x, w, offsets, want_pre=True)
        assert torch.equal(h, h2) and torch.equal(pre, pre2)
        for a, b in zip(ah.ah_grouped_gated_grad(dy, wo, pre), ah.ah_grouped_gated_grad(dy, wo, pre, offsets)):
            assert torch.equal(a, b)


def test_bad_values_stay_in_their_rows(gpu):
    torch, ah = gpu
    for m in (6, 400):
        x, w = torch.randn(m, 64, device="cuda").bfloat16(), torch.randn(1, 64, 64, device="cuda").bfloat16()
        want, wpre = ah.ah_grouped_gated(x, w, want_pre=True)
        y = x.clone()
        y[2, 5], y[4, 0] = float("nan"), float("inf")
        h, pre = ah.ah_grouped_gated(y, w, want_pre=True)
        ok = torch.ones(m, dtype=torch.bool, device="cuda")
        ok[[2, 4]] = False
        assert torch.equal(h[ok], want[ok]) and torch.equal(pre[ok], wpre[ok])
        assert torch.isnan(h[2]).all() and not torch.isfinite(pre[4]).any()
        h, _ = ah.ah_grouped_gated(y, w, drop=0.5, seed=1)
        f = torch.from_numpy(factors(m, 32, 0.5, 1, 0)).cuda()
        assert (h[f == 0] == 0).all() and torch.isnan(h[2][f[2] > 0]).all()


def test_large_activations(gpu):
    """Gates from -3e4 to 3e4: the logistic function's exponential overflows and underflows without a NaN."""
    torch, ah = gpu
    x = torch.linspace(-3e4, 3e4, 257, device="cuda")[:, None].bfloat16()
    w = torch.ones(1, 2, 1, device="cuda").bfloat16()
    w[0, 1] = 2.0 ** -14
    a = x.double()
    for act in ("silu", "gelu", "relu"):
        h, _ = ah.ah_grouped_gated(x, w, act=act, out_dtype=torch.float32)
        want = torch.where(a > 0, a, torch.zeros_like(a)) * (a * 2.0 ** -14)  # the nearest gates are 234 from 0
        assert ((h.double() - want).abs() <= want.abs() * 2.0 ** -20 + 1e-30).all()
        pre = torch.cat([x, x * 2.0 ** -14], 1)
        d, _ = ah.ah_grouped_gated_grad(torch.ones(257, 1, device="cuda").bfloat16(), torch.ones(1, 1, 1, device="cuda").bfloat16(), pre, act=act)
        assert torch.isfinite(d).all()


def test_orders_and_starts_out_of_range(gpu):
    """Entries of order outside the slots and starts outside the rows are not followed."""
    torch, ah = gpu
    for m in (20, 600):
        x, w = torch.randn(m, 32, device="cuda").bfloat16(), torch.randn(2, 32, 32, device="cuda").bfloat16()
        order = torch.arange(m, dtype=torch.int32, device="cuda")
        order[3], order[m - 1] = -5, 2 ** 31 - 1
        offsets = torch.tensor([-7, m // 2, m + 1000], device="cuda")
        out, pre = torch.full((m, 16), 5.0, device="cuda").bfloat16(), torch.full((m, 32), 5.0, device="cuda").bfloat16()
        ah.ah_grouped_gated(x, w, offsets, order=order, out=out, pre_out=pre)
        torch.cuda.synchronize()
        assert (out[3] == 5).all() and (out[m - 1] == 5).all()  # slots that the order does not hold
        good = torch.tensor([0, m // 2, m], device="cuda")
        want, wp = ah.ah_grouped_gated(x, w, good, order=torch.arange(m, dtype=torch.int32, device="cuda"), want_pre=True)
        ok = torch.ones(m, dtype=torch.bool, device="cuda")
        ok[[3, m - 1]] = False
        assert torch.equal(out[ok], want[ok]) and torch.equal(pre[ok], wp[ok])
        wo = torch.randn(2, 8, 16, device="cuda").bfloat16()
        d, h = ah.ah_grouped_gated_grad(x[:, :8], wo, pre, offsets, order=order)
        d2, h2 = ah.ah_grouped_gated_grad(x[:, :8], wo, pre, good, order=torch.arange(m, dtype=torch.int32, device="cuda"))
        assert torch.equal(d[ok], d2[ok]) and torch.equal(h[ok], h2[ok])


def test_streams_and_graph(gpu):
    torch, ah = gpu
    x, w = torch.randn(700, 64, device="cuda").bfloat16(), torch.randn(1, 128, 64, device="cuda").bfloat16()
    wo, dy = torch.randn(1, 64, 64, device="cuda").bfloat16(), torch.randn(700, 64, device="cuda").bfloat16()
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def block(stream=None):
        h, pre = ah.ah_grouped_gated(x, w, drop=0.25, seed=6, step=step, want_pre=True, stream=stream)
        return (h, pre) + ah.ah_grouped_gated_grad(dy, wo, pre, drop=0.25, seed=6, step=step, stream=stream)

    want = block()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = block(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = block()
        step.add_(1)
    step.zero_()
    for i in range(3):
        step.fill_(i)
        want = block()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want)), i


def test_bindings_check_shapes(gpu):
    torch, ah = gpu
    b = lambda *s: torch.zeros(*s, device="cuda").bfloat16()  # noqa: E731
    off, order = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad, err in (
            (lambda: ah.ah_grouped_gated(b(4, 8), b(1, 5, 8)), ValueError), (lambda: ah.ah_grouped_gated(b(4, 8), b(1, 6, 9)), ValueError),
            (lambda: ah.ah_grouped_gated(b(4, 8), b(2, 6, 8)), ValueError), (lambda: ah.ah_grouped_gated(b(4, 8), b(1, 6, 8), fan=2), ValueError),
            (lambda: ah.ah_grouped_gated(b(4, 8), b(1, 6, 8), act="tanh"), ValueError),
            (lambda: ah.ah_grouped_gated(b(4, 8), b(1, 6, 8), drop=1.0), ah.AHError),
            (lambda: ah.ah_grouped_gated(b(4, 8).float(), b(1, 6, 8)), TypeError),
            (lambda: ah.ah_grouped_gated(b(4, 8), b(2, 6, 8), off, order=order[:3]), ValueError),
            (lambda: ah.ah_grouped_gated(b(4, 8), b(1, 6, 8), out=b(4, 4)), ValueError),
            (lambda: ah.ah_grouped_gated_grad(b(4, 8), b(1, 8, 3), b(4, 5)), ValueError),
            (lambda: ah.ah_grouped_gated_grad(b(4, 8), b(1, 7, 3), b(4, 6)), ValueError),
            (lambda: ah.ah_grouped_gated_grad(b(4, 8), b(1, 8, 3), b(3, 6)), ValueError)):
        with pytest.raises(err):
            bad()
    h, pre = ah.ah_grouped_gated(b(0, 8), b(1, 6, 8), want_pre=True)
    assert h.shape == (0, 3) and pre.shape == (0, 6)
    d, h = ah.ah_grouped_gated_grad(b(0, 8), b(1, 8, 3), b(0, 6))
    assert d.shape == (0, 6) and h.shape == (0, 3)
