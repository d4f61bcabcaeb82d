"""8-bit float products on the GPU: codes and scales bit for bit, products against float64.

Tolerance of a product: the matrix instruction cuts the products of each eight elements off at 2^-13 of the power
of two below the largest, so eight are off by at most 8 2^-13 of the largest of them, in all 2^-10 of the sum of
sizes; adding up in float32, (k / 8 + 16) 2^-23 of it; the result half a step of its type.  Small whole numbers
(products below 2^12) are exact.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
TOP = {"float8_e4m3fn": 448.0, "float8_e5m2": 57344.0}


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mips_ah_partition_amd import ahlib
    ahlib.lib()
    return torch, ahlib


def _pow2(torch, e):
    return torch.from_numpy(np.ldexp(1.0, e.cpu().numpy().astype(np.int32)))


def _reference(torch, x, name):
    """(values that the codes stand for, float64 [n, d]; scale bytes [kb, n]; rows' bad blocks [n, kb]) on the CPU."""
    x = x.double().cpu()
    n, d = x.shape
    kb = (d + 127) // 128
    p = torch.zeros(n, kb * 128, dtype=torch.float64)
    p[:, :d] = x
    p = p.view(n, kb, 128)
    bad = ~torch.isfinite(p).all(2)
    p = torch.where(bad[:, :, None], torch.zeros_like(p), p)
    top, bits, low = TOP[name], 3 if "e4m3" in name else 2, -6 if "e4m3" in name else -14
    m = p.abs().amax(2).numpy()
    f, e = np.frexp(m / top)  # smallest power of two that is >= m / top
    e = np.where(m > 0, np.maximum(np.where(f == 0.5, e - 1, e), -127), 0)
    u = p.numpy() * np.ldexp(1.0, -e)[:, :, None]
    _, ue = np.frexp(np.maximum(np.abs(u), 2.0 ** low))
    step = np.ldexp(1.0, ue - 1 - bits)
    v = np.round(u / step) * step * np.ldexp(1.0, e)[:, :, None]
    return torch.from_numpy(v).view(n, -1), torch.from_numpy((e + 127).T.astype(np.uint8)), bad


def _values(torch, codes, scale):
    n, kp = codes.shape
    s = _pow2(torch, scale[:, :n].t().int() - 127)
    return (codes.cpu().float().double().view(n, kp // 128, 128) * s[:, :, None]).view(n, kp)


def _check(torch, codes, scale, x, name):
    v, s, bad = _reference(torch, x, name)
    n, d = x.shape
    kb = (d + 127) // 128
    assert codes.shape == (n, kb * 128) and scale.shape == (kb, (n + 15) // 16 * 16)
    assert torch.equal(scale[:, :n].cpu(), s)
    got = _values(torch, codes, scale)
    wide = bad[:, :, None].expand(n, kb, 128).reshape(n, -1)
    assert torch.equal(got[~wide], v[~wide])
    assert (got[:, d:][~wide[:, d:]] == 0).all() and torch.isnan(got[:, :d][wide[:, :d]]).all()


@pytest.mark.parametrize("name", list(TOP))
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n,d", [(1, 1), (1, 128), (3, 129), (16, 64), (17, 300), (128, 128), (129, 1001), (300, 77), (1000, 256),
                                 (5, 4096), (2, 20001)])
def test_codes(gpu, n, d, dtype, name):
    torch, ah = gpu
    dt = getattr(torch, dtype)
    g = torch.Generator(device="cuda")
    g.manual_seed(n + d)
    x = torch.randn(n, d, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-8, 9, (n, 1), generator=g, device="cuda").float())  # rows of different sizes
    x[:, torch.randint(0, d, (max(1, d // 50),), generator=g, device="cuda")] *= 20
    x = x.to(dt)
    if n > 2:
        x[1] = 0
    for rows, cols in ((True, False), (False, True), (True, True)):
        c, s, ct, st = ah.ah_f8_quantize(x, dtype=getattr(torch, name), want_rows=rows, want_columns=cols)
        assert (c is None) == (not rows) and (ct is None) == (not cols)
        if rows:
            _check(torch, c, s, x, name)
        if cols:
            _check(torch, ct, st, x.t(), name)


@pytest.mark.parametrize("name", list(TOP))
def test_ends_of_the_range(gpu, name):
    """Largest values at and next to a power of two times the type's largest, denormal, huge and bad blocks."""
    torch, ah = gpu
    top = TOP[name]
    heads = [top, np.nextafter(np.float32(top), np.float32(np.inf)), np.nextafter(np.float32(top), np.float32(0)), top / 2,
             top * 2.0 ** 40, 3e38, 1e-38, 1e-44, 2.0 ** -149, 2.0 ** -140, 0.0, 1.0, float("nan"), float("inf"), -float("inf"), -top]
    x = torch.randn(len(heads), 384, device="cuda") * 0.2
    for i, h in enumerate(heads):
        if np.isfinite(h):
            x[i] = x[i].clamp(-1, 1) * abs(float(h))
        x[i, 130] = float(h)
    for y in (x, x.bfloat16(), x[:, 100:300]):
        c, s, ct, st = ah.ah_f8_quantize(y, dtype=getattr(torch, name), want_columns=True)
        _check(torch, c, s, y, name)
        _check(torch, ct, st, y.t(), name)
    # every value of the type and the middles between neighbours: ties to even
    allv = torch.arange(256, dtype=torch.uint8).view(getattr(torch, name)).float()
    allv = allv[torch.isfinite(allv)].sort().values
    x = torch.cat([allv, (allv[1:] + allv[:-1]) / 2])
    x = torch.nn.functional.pad(x, (0, -len(x) % 127)).view(-1, 127)
    x = torch.cat([x, torch.full((len(x), 1), top)], 1).cuda()  # every block's scale is 1
    c, s, _, _ = ah.ah_f8_quantize(x, dtype=getattr(torch, name))
    assert (s[:, :len(x)] == 127).all()
    _check(torch, c, s, x, name)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_codes_of_strided_rows(gpu, dtype):
    torch, ah = gpu
    for n, d, off, pad in ((5, 128, 8, 8), (200, 200, 1, 3), (130, 64, 3, 0), (7, 1000, 0, 1)):
        wide = torch.randn(n, off + d + pad, device="cuda").to(getattr(torch, dtype))
        x = wide[:, off:off + d]
        got = ah.ah_f8_quantize(x, want_columns=True)
        want = ah.ah_f8_quantize(x.contiguous(), want_columns=True)
        for a, b, r in zip(got, want, (n, n, d, d)):
            a, b = (a.view(torch.uint8), b.view(torch.uint8)) if a.dtype != torch.uint8 else (a[:, :r], b[:, :r])
            assert torch.equal(a, b)


CASES = [(1, 1, 1), (1, 1536, 130), (3, 128, 16), (16, 64, 64), (16, 1000, 200), (17, 100, 33), (37, 1001, 403), (64, 256, 64), (100, 512, 100),
         (300, 384, 520), (1000, 128, 256), (513, 1100, 700), (2000, 300, 129), (129, 3000, 1), (600, 5000, 260)]


@pytest.mark.parametrize("out", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,k,n", CASES)
def test_products(gpu, m, k, n, out):
    torch, ah = gpu
    D, dt = torch.float64, getattr(torch, out)
    names = list(TOP)
    xt, wt = getattr(torch, names[(m + k) % 2]), getattr(torch, names[(k + n) % 2])
    g = torch.Generator(device="cuda")
    g.manual_seed(m + k + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    # blocks of very different sizes, so that a scale in a wrong place shows
    x = (rnd(m, k) * torch.exp2(torch.randint(-6, 7, (m, 1), generator=g, device="cuda").float())
         * torch.exp2((torch.arange(k, device="cuda") // 128 % 5 - 2).float())).bfloat16()
    w = rnd(n, k) * torch.exp2(torch.randint(-6, 7, (n, 1), generator=g, device="cuda").float())
    bias = rnd(n) * k ** 0.5 if (m + n) % 3 else None
    x8, xs, _, _ = ah.ah_f8_quantize(x, dtype=xt)
    w8, ws, _, _ = ah.ah_f8_quantize(w, dtype=wt)
    big = torch.full((m + 1, n), 7.0, dtype=dt, device="cuda")
    y = ah.ah_f8_matmul(x8, xs, w8, ws, bias=bias, out=big[:m])
    assert (big[m] == 7).all()
    a, b = _values(torch, x8, xs).cuda(), _values(torch, w8, ws).cuda()
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    if bias is not None:
        want, size = want + bias.to(D), size + bias.to(D).abs()
    tol = size * (2.0 ** -10 + (k / 8 + 16) * 2.0 ** -23)
    assert ((y.to(D) - want).abs() <= tol + (want.abs() + tol) * torch.finfo(dt).eps / 2).all()
    # the layer: the same codes, so the same sums up to their order
    z = ah.ah_f8_linear(x, w8, ws, bias=bias, x_type=xt, out_dtype=dt)
    assert ((z.to(D) - want).abs() <= tol + (want.abs() + tol) * torch.finfo(dt).eps / 2).all()
    assert torch.equal(ah.ah_f8_linear(x, w8, ws, bias=bias, x_type=xt, out_dtype=dt), z)


@pytest.mark.parametrize("m,k,n", CASES)
def test_whole_numbers_are_exact(gpu, m, k, n):
    torch, ah = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(m * k + n)
    x = torch.randint(-8, 9, (m, k), generator=g, device="cuda").bfloat16()
    w = torch.randint(-8, 9, (n, k), generator=g, device="cuda").float()
    bias = torch.randint(-50, 50, (n,), generator=g, device="cuda").float()
    w8, ws, _, _ = ah.ah_f8_quantize(w)
    want = x.double() @ w.double().t() + bias.double()
    assert torch.equal(ah.ah_f8_linear(x, w8, ws, bias=bias, out_dtype=torch.float32).double(), want)
    assert torch.equal(ah.ah_f8_linear(x.float(), w8, ws, bias=bias, out_dtype=torch.float32).double(), want)
    x8, xs, _, _ = ah.ah_f8_quantize(x)
    assert torch.equal(ah.ah_f8_matmul(x8, xs, w8, ws, bias=bias, out_dtype=torch.float32).double(), want)


@pytest.mark.parametrize("m", [1, 9, 40, 300, 1000])
def test_bad_values_stay_in_their_rows(gpu, m):
    torch, ah = gpu
    k, n = 300, 150
    x, w = torch.randn(m, k, device="cuda"), torch.randn(n, k, device="cuda")
    w8, ws, _, _ = ah.ah_f8_quantize(w)
    want = ah.ah_f8_linear(x, w8, ws)
    y = x.clone()
    y[m // 2, 200], y[0, 299] = float("nan"), float("inf")
    got = ah.ah_f8_linear(y, w8, ws)
    ok = torch.ones(m, dtype=torch.bool, device="cuda")
    ok[[0, m // 2]] = False
    assert torch.equal(got[ok], want[ok]) and torch.isnan(got[~ok]).all()
    w[7, 3] = float("nan")
    w8, ws, _, _ = ah.ah_f8_quantize(w)
    got = ah.ah_f8_linear(x, w8, ws)
    cols = torch.arange(n, device="cuda") != 7
    assert torch.equal(got[:, cols], want[:, cols]) and torch.isnan(got[:, 7]).all()


@pytest.mark.parametrize("m,k,n", [(1, 40, 30), (130, 100, 77), (500, 200, 300)])
def test_gradients(gpu, m, k, n):
    """dx = dy w and dw = dy^T x of codes along the other side, against the products of what the codes stand for, and
    those against the unquantised gradients: each code is off by at most 2^-4 (e4m3) or 2^-3 (e5m2) of its value or
    by half the smallest step of its block, 2^-10 (2^-17) 2^e, where 2^e <= 2 max / 448 (2 max / 57344)."""
    torch, ah = gpu
    D = torch.float64
    for dyt, eps in ((torch.float8_e4m3fn, 2.0 ** -4), (torch.float8_e5m2, 2.0 ** -3)):
        x, w, dy = torch.randn(m, k, device="cuda").bfloat16(), torch.randn(n, k, device="cuda"), torch.randn(m, n, device="cuda").bfloat16()
        d8, ds, dt8, dts = ah.ah_f8_quantize(dy, dtype=dyt, want_columns=True)
        _, _, xt8, xts = ah.ah_f8_quantize(x, want_rows=False, want_columns=True)
        _, _, wt8, wts = ah.ah_f8_quantize(w, want_rows=False, want_columns=True)
        dx = ah.ah_f8_matmul(d8, ds, wt8, wts, out_dtype=torch.float32)
        dw = ah.ah_f8_matmul(dt8, dts, xt8, xts, out_dtype=torch.float32)
        assert dx.shape == (m, k) and dw.shape == (n, k)
        for got, a, b, pa, pb in ((dx, d8, wt8, ds, wts), (dw, dt8, xt8, dts, xts)):
            va, vb = _values(torch, a, pa).cuda(), _values(torch, b, pb).cuda()
            size = va.abs() @ vb.abs().t()
            assert ((got.to(D) - va @ vb.t()).abs() <= size * (2.0 ** -10 + (va.shape[1] / 8 + 16) * 2.0 ** -23)).all()

        def off(t, e):  # how far a code may be from the value it stands for
            t = t.to(D)
            p = torch.nn.functional.pad(t, (0, -t.shape[1] % 128)).view(t.shape[0], -1, 128).abs().amax(2)
            return t.abs() * e + (p * 2.0 ** -17).repeat_interleave(128, 1)[:, :t.shape[1]]

        for got, a, b, ea, eb in ((dx, dy, w.t(), eps, 2.0 ** -4), (dw, dy.t(), x.t(), eps, 2.0 ** -4)):
            va, vb, oa, ob = a.to(D), b.to(D), off(a, ea), off(b, eb)
            tol = oa @ vb.abs().t() + va.abs() @ ob.t() + oa @ ob.t()
            size = va.abs() @ vb.abs().t() + tol
            assert ((got.to(D) - va @ vb.t()).abs() <= tol + size * (2.0 ** -10 + (va.shape[1] / 8 + 16) * 2.0 ** -23)).all()


def test_streams_and_graph(gpu):
    torch, ah = gpu
    for m in (4, 300):
        x, w = torch.randn(m, 256, device="cuda").bfloat16(), torch.randn(128, 256, device="cuda")
        w8, ws, _, _ = ah.ah_f8_quantize(w)
        want = ah.ah_f8_linear(x, w8, ws)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        got = ah.ah_f8_linear(x, w8, ws, stream=s)
        s.synchronize()
        assert torch.equal(got, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept = ah.ah_f8_linear(x, w8, ws)
        for i in range(3):
            x.copy_(torch.randn(m, 256, device="cuda"))
            want = ah.ah_f8_linear(x, w8, ws)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(kept, want)


def test_bindings_check_shapes(gpu):
    torch, ah = gpu
    x = torch.randn(5, 200, device="cuda")
    x8, xs, _, _ = ah.ah_f8_quantize(x)
    w8, ws, _, _ = ah.ah_f8_quantize(torch.randn(9, 300, device="cuda"))
    for bad, err in ((lambda: ah.ah_f8_matmul(x8, xs, w8, ws), ValueError), (lambda: ah.ah_f8_linear(x, w8, ws), ValueError),
                     (lambda: ah.ah_f8_matmul(x8, xs[:1], x8, xs), ValueError), (lambda: ah.ah_f8_matmul(x8[:, :64].contiguous(), xs, x8, xs), ValueError),
                     (lambda: ah.ah_f8_matmul(x8, xs, x8, xs, bias=torch.zeros(4, device="cuda")), ValueError),
                     (lambda: ah.ah_f8_matmul(x8.view(torch.uint8), xs, x8, xs), TypeError),
                     (lambda: ah.ah_f8_quantize(x, dtype=torch.float16), TypeError), (lambda: ah.ah_f8_quantize(x.half()), TypeError),
                     (lambda: ah.ah_f8_quantize(x, want_rows=False), ah.AHError)):
        with pytest.raises(err):
            bad()
    e8, es, et8, ets = ah.ah_f8_quantize(x[:0], want_columns=True)
    assert e8.shape == (0, 256) and es.shape == (2, 0) and et8.shape == (200, 0) and ets.shape == (0, 208)
    assert ah.ah_f8_matmul(e8, es, x8, xs).shape == (0, 5)
    assert (ah.ah_f8_matmul(et8, ets, et8, ets, out_dtype=torch.float32) == 0).all()  # a sum over no rows
