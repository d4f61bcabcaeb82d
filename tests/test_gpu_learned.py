"""The learned query side on the GPU against plain forms in 64 bits.

Tolerances.  int8: codes, steps and products bit for bit (the dot is exact, the float32
operations are the stated ones).  Grouped products: a float32 sum of t exact products
is off by at most t 2^-23 sum |a||b| (whatever its order), and its one rounding by
2^-8 (bfloat16) or 2^-23 relative.  Distillation: float32 exponentials of x = z / tau are
off by a few (1 + |x|) 2^-23, sums of V terms by (V / 256 + 32) 2^-23 relative.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

E = 2.0 ** -23


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mips_ah_partition_amd import ahlib
    ahlib.lib()
    return torch, ahlib


def _t(torch, a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _np(t):
    return t.float().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


def _f64(t):
    return _np(t).astype(np.float64)


# --------------------------------------------------------------------------- int8
def _quantize(x):
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        s = np.abs(x).max(1) / np.float32(127)
        s[~np.isfinite(np.abs(x).max(1))] = np.nan
        c = np.clip(np.rint(x / s[:, None]), -127, 127)
    return np.where(s[:, None] > 0, c, 0).astype(np.int8), s


@pytest.mark.parametrize("n,d", [(1, 1), (3, 17), (70, 128), (5, 1001), (2, 16384), (300, 96)])
@pytest.mark.parametrize("bf16", [True, False])
def test_i8_quantize_rows(gpu, n, d, bf16):
    torch, ah = gpu
    rng = np.random.default_rng(n * 31 + d)
    X = (rng.standard_normal((n, d)) * np.exp(rng.standard_normal((n, 1)) * 3)).astype(np.float32)
    if n > 2:
        X[1] = 0.0
        X[2] *= np.float32(1e-42)  # a step that is not a normal number
    x = _t(torch, X, torch.bfloat16 if bf16 else torch.float32)
    c, s = ah.ah_i8_quantize_rows(x)
    rc, rs = _quantize(_np(x))
    assert np.array_equal(_np(s), rs) and np.array_equal(_np(c), rc)


@pytest.mark.parametrize("bf16", [True, False])
def test_i8_quantize_nonfinite_rows_and_strides(gpu, bf16):
    torch, ah = gpu
    big = torch.randn(9, 300, device="cuda", dtype=torch.bfloat16 if bf16 else torch.float32)
    x = big[:, 7:250]
    x[1, 242], x[3, 0], x[5, 100] = float("nan"), float("inf"), -float("inf")
    c, s = ah.ah_i8_quantize_rows(x)
    rc, rs = _quantize(_np(x))
    assert np.isnan(_np(s)[[1, 3, 5]]).all()
    assert np.array_equal(_np(s), rs, equal_nan=True) and np.array_equal(_np(c), rc)


def _i8_ref(torch, c, s, w, ws, bias, dtype):
    acc = (c.astype(np.float64) @ w.astype(np.float64).T).astype(np.int64).astype(np.float32)
    with np.errstate(all="ignore"):
        y = (acc * s[:, None]) * ws[None, :]
        if bias is not None:
            y = y + bias[None, :]
    return _np(torch.from_numpy(y).to(dtype))


I8_SIZES = [(1, 1, 1), (1, 16, 4096), (1, 1536, 100), (2, 17, 33), (5, 100, 16), (16, 64, 64), (17, 128, 130),
            (33, 144, 257), (64, 4096, 70), (65, 1001, 403), (128, 256, 128), (200, 80, 515), (300, 512, 1),
            (129, 16384, 48), (513, 272, 300), (1030, 640, 520), (2100, 272, 7001), (3333, 1104, 4000)]


@pytest.mark.parametrize("m,k,n", I8_SIZES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_i8_matmul(gpu, m, k, n, out):
    torch, ah = gpu
    rng = np.random.default_rng(m + 3 * k + 7 * n)
    c, w = rng.integers(-128, 128, (m, k), dtype=np.int8), rng.integers(-128, 128, (n, k), dtype=np.int8)
    s, ws = rng.random(m).astype(np.float32), rng.random(n).astype(np.float32)
    bias = rng.standard_normal(n).astype(np.float32) * 100 if (m + n) % 2 else None
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    y = ah.ah_i8_matmul(_t(torch, c), _t(torch, s), _t(torch, w), _t(torch, ws),
                        bias=None if bias is None else _t(torch, bias), out_dtype=dt)
    assert y.dtype == dt and np.array_equal(_np(y), _i8_ref(torch, c, s, w, ws, bias, dt))


def test_i8_matmul_at_odd_addresses(gpu):
    torch, ah = gpu
    rng = np.random.default_rng(5)
    m, k, n = 40, 96, 50
    buf = torch.randint(-127, 128, (m * k + 3,), device="cuda", dtype=torch.int8)
    wbuf = torch.randint(-127, 128, (n * k + 5,), device="cuda", dtype=torch.int8)
    x8, w8 = buf[3:].view(m, k), wbuf[5:].view(n, k)
    s, ws = rng.random(m).astype(np.float32), rng.random(n).astype(np.float32)
    obuf = torch.full((m * n + 1,), 7.0, device="cuda", dtype=torch.bfloat16)
    y = ah.ah_i8_matmul(x8, _t(torch, s), w8, _t(torch, ws), out=obuf[1:].view(m, n))
    assert np.array_equal(_np(y), _i8_ref(torch, _np(x8), s, _np(w8), ws, None, torch.bfloat16))
    assert float(obuf[0]) == 7.0


@pytest.mark.parametrize("m,k,n", I8_SIZES)
@pytest.mark.parametrize("bf16", [True, False])
def test_i8_linear(gpu, m, k, n, bf16):
    torch, ah = gpu
    rng = np.random.default_rng(11 * m + k + n)
    x = _t(torch, rng.standard_normal((m, k)).astype(np.float32) * 3, torch.bfloat16 if bf16 else torch.float32)
    if m > 4:
        x[1] = 0
        x[2, k - 1] = float("nan")
        x[4, 0] = float("inf")
    w, ws = rng.integers(-127, 128, (n, k), dtype=np.int8), rng.random(n).astype(np.float32)
    bias = rng.standard_normal(n).astype(np.float32)
    y = _np(ah.ah_i8_linear(x, _t(torch, w), _t(torch, ws), bias=_t(torch, bias)))
    c, s = _quantize(_np(x))
    assert np.array_equal(y, _i8_ref(torch, c, s, w, ws, bias, torch.bfloat16), equal_nan=True)
    if m > 4:
        assert np.isnan(y[[2, 4]]).all() and np.array_equal(y[1], _np(torch.from_numpy(bias).bfloat16()))


def test_i8_linear_takes_strided_tokens_and_nothing_at_all(gpu):
    torch, ah = gpu
    big = torch.randn(20, 200, device="cuda", dtype=torch.bfloat16)
    w8 = torch.randint(-127, 128, (30, 64), device="cuda", dtype=torch.int8)
    ws = torch.rand(30, device="cuda")
    x = big[::2, 8:72]
    assert torch.equal(ah.ah_i8_linear(x, w8, ws), ah.ah_i8_linear(x.contiguous(), w8, ws))
    assert ah.ah_i8_linear(x[:0], w8, ws).shape == (0, 30)
    assert ah.ah_i8_linear(x, w8[:0], ws[:0]).shape == (10, 0)


def test_i8_output_beyond_32_bits(gpu):
    torch, ah = gpu
    m, n, k = 66000, 66000, 16  # 4.36e9 outputs
    x8 = torch.randint(-127, 128, (m, k), device="cuda", dtype=torch.int8)
    w8 = torch.randint(-127, 128, (n, k), device="cuda", dtype=torch.int8)
    y = ah.ah_i8_matmul(x8, torch.ones(m, device="cuda"), w8, torch.ones(n, device="cuda"), out_dtype=torch.bfloat16)
    for rows in (slice(0, 3), slice(32500, 32503), slice(m - 3, m)):
        ref = torch.mm(x8[rows].float(), w8.float().t()).to(torch.bfloat16)
        assert torch.equal(y[rows], ref)


# --------------------------------------------------------------------------- grouped
def _order(leaves, L):
    lf = leaves.reshape(-1).astype(np.int64)
    lf = np.where((lf < 0) | (lf >= L), L, lf)
    return np.searchsorted(np.sort(lf, kind="stable"), np.arange(L + 1)), np.argsort(lf, kind="stable"), lf


@pytest.mark.parametrize("n,L", [(0, 3), (1, 1), (63, 2), (64, 4096), (4096, 7), (4097, 1), (9000, 64), (70000, 4096),
                                 (300001, 1000)])
def test_group_rows(gpu, n, L):
    torch, ah = gpu
    rng = np.random.default_rng(n + L)
    leaves = (rng.random(n) ** 2 * (L + 2)).astype(np.int32) - 1  # -1 and L stand for no leaf
    off, order = ah.ah_group_rows(_t(torch, leaves), L)
    ro, rr, _ = _order(leaves, L)
    assert np.array_equal(_np(off), ro) and np.array_equal(_np(order), rr)


def _grouped_ref(x, w, dy, lf, fan):
    """Forward, both gradients, and the sums of absolute products that bound their rounding."""
    L, n, k = w.shape
    T = lf.size
    y, ya = np.zeros((T, n)), np.zeros((T, n))
    dxs, dxa = np.zeros((T, k)), np.zeros((T, k))
    dw, dwa = np.zeros((L, n, k)), np.zeros((L, n, k))
    for l in range(L):
        s = np.nonzero(lf == l)[0]
        xs, ds = x[s // fan], dy[s]
        y[s], ya[s] = xs @ w[l].T, np.abs(xs) @ np.abs(w[l]).T
        dxs[s], dxa[s] = ds @ w[l], np.abs(ds) @ np.abs(w[l])
        dw[l], dwa[l] = ds.T @ xs, np.abs(ds).T @ np.abs(xs)
    m = T // fan
    return (y, ya), (dxs.reshape(m, fan, k).sum(1), dxa.reshape(m, fan, k).sum(1)), (dw, dwa)


def _close(got, ref, mag, terms, dtype_bits):
    tol = terms * E * mag + 2.0 ** -dtype_bits * np.abs(ref) + 1e-30
    err = np.abs(got - ref)
    assert (err <= tol).all(), float((err - tol).max())


GROUPED_SIZES = [  # rows, fan, leaves, k, n
    (1, 1, 1, 8, 8), (1, 3, 5, 64, 64), (4, 2, 300, 128, 72), (16, 4, 64, 256, 128), (33, 3, 7, 100, 77),
    (40, 1, 3, 1, 1), (150, 2, 2, 136, 264), (257, 1, 1, 520, 129), (100, 3, 9, 65, 48), (500, 4, 11, 192, 192),
    (700, 2, 600, 40, 24), (1500, 2, 5, 320, 328), (3000, 2, 6, 264, 1288), (4000, 2, 10, 1104, 1096)]


def _grouped_case(torch, rows, fan, L, k, n, seed=0):
    rng = np.random.default_rng(rows + 10 * fan + 100 * L + k + n + seed)
    x = _t(torch, rng.standard_normal((rows, k)).astype(np.float32), torch.bfloat16)
    w = _t(torch, rng.standard_normal((L, n, k)).astype(np.float32), torch.bfloat16)
    dy = _t(torch, rng.standard_normal((rows * fan, n)).astype(np.float32), torch.bfloat16)
    leaves = (rng.random((rows, fan)) ** 1.5 * L).astype(np.int32)
    leaves[rng.random((rows, fan)) < 0.1] = -1
    if L > 2:
        leaves[leaves == L // 2] = L + 5  # an empty leaf in the middle, ids outside the range
    return x, w, dy, leaves


@pytest.mark.parametrize("rows,fan,L,k,n", GROUPED_SIZES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_grouped_products(gpu, rows, fan, L, k, n, out):
    torch, ah = gpu
    x, w, dy, leaves = _grouped_case(torch, rows, fan, L, k, n)
    dt, bits = (torch.bfloat16, 8) if out == "bf16" else (torch.float32, 23)
    off, order = ah.ah_group_rows(_t(torch, leaves), L)
    y = ah.ah_grouped_matmul(x, w, off, order=order, fan=fan, out_dtype=dt)
    dx = ah.ah_grouped_matmul_dx(dy, w, off, order=order, fan=fan, out_dtype=dt)
    dw = ah.ah_grouped_matmul_dw(dy, x, off, order=order, fan=fan, out_dtype=dt)
    ro, rr, lf = _order(leaves, L)
    (ry, ya), (rdx, dxa), (rdw, dwa) = _grouped_ref(_f64(x), _f64(w), _f64(dy), lf, fan)
    _close(_f64(y), ry, ya, k + 2, bits)
    _close(_f64(dx), rdx, dxa, n + fan + 2, bits)
    _close(_f64(dw), rdw, dwa, rows + 2, bits)
    none = lf == L
    assert (_np(y)[none] == 0).all()
    for l in range(L):
        if not (lf == l).any():
            assert (_np(dw)[l] == 0).all()
    # the same calls again give the same bits
    assert torch.equal(y, ah.ah_grouped_matmul(x, w, off, order=order, fan=fan, out_dtype=dt))
    assert torch.equal(dx, ah.ah_grouped_matmul_dx(dy, w, off, order=order, fan=fan, out_dtype=dt))
    assert torch.equal(dw, ah.ah_grouped_matmul_dw(dy, x, off, order=order, fan=fan, out_dtype=dt))


@pytest.mark.parametrize("rows,k,n", [(90, 64, 96), (300, 100, 33)])
def test_grouped_rows_already_in_order(gpu, rows, k, n):
    """An index's leaf_offsets without an order; rows before the first and after the last leaf are of no leaf."""
    torch, ah = gpu
    L = 4
    x, w, dy, _ = _grouped_case(torch, rows, 1, L, k, n, seed=1)
    off = np.array([5, 5, rows // 2, rows // 2 + 1, rows - 9], dtype=np.int64)
    lf = np.full(rows, L)
    for l in range(L):
        lf[off[l]:off[l + 1]] = l
    o = _t(torch, off)
    (ry, ya), (rdx, dxa), (rdw, dwa) = _grouped_ref(_f64(x), _f64(w), _f64(dy), lf, 1)
    _close(_f64(ah.ah_grouped_matmul(x, w, o, out_dtype=torch.float32)), ry, ya, k + 2, 23)
    _close(_f64(ah.ah_grouped_matmul_dx(dy, w, o, out_dtype=torch.float32)), rdx, dxa, n + 2, 23)
    _close(_f64(ah.ah_grouped_matmul_dw(dy, x, o)), rdw, dwa, rows + 2, 23)


@pytest.mark.parametrize("k,n", [(64, 64), (37, 50)])
def test_grouped_rows_without_any_leaf(gpu, k, n):
    torch, ah = gpu
    x, w, dy, _ = _grouped_case(torch, 20, 2, 3, k, n)
    off, order = ah.ah_group_rows(torch.full((20, 2), -1, device="cuda", dtype=torch.int32), 3)
    nan = torch.full((40, n), float("nan"), device="cuda", dtype=torch.float32)
    assert (ah.ah_grouped_matmul(x, w, off, order=order, fan=2, out=nan) == 0).all()
    assert (ah.ah_grouped_matmul_dx(dy, w, off, order=order, fan=2) == 0).all()
    assert (ah.ah_grouped_matmul_dw(dy, x, off, order=order, fan=2) == 0).all()
    off, order = ah.ah_group_rows(torch.empty((0, 2), device="cuda", dtype=torch.int32), 3)
    assert ah.ah_grouped_matmul(x[:0], w, off, order=order, fan=2).shape == (0, n)
    assert ah.ah_grouped_matmul_dx(dy[:0], w, off, order=order, fan=2).shape == (0, k)
    assert (ah.ah_grouped_matmul_dw(dy[:0], x[:0], off, order=order, fan=2) == 0).all()


def test_grouped_nan_stays_in_its_leaf_and_row(gpu):
    torch, ah = gpu
    rows, L, k, n = 60, 3, 72, 40
    x, w, dy, _ = _grouped_case(torch, rows, 1, L, k, n)
    leaves = np.arange(rows, dtype=np.int32) % L
    leaves[7] = -1
    w[1] = float("nan")
    x[0, 3], dy[3, 5] = float("nan"), float("inf")
    x[7], dy[7] = float("nan"), float("nan")  # of no leaf: touches nothing
    off, order = ah.ah_group_rows(_t(torch, leaves), L)
    y = _np(ah.ah_grouped_matmul(x, w, off, order=order))
    bad = np.isnan(y).any(1)
    assert np.array_equal(bad, (leaves == 1) | (np.arange(rows) == 0))
    assert (y[7] == 0).all()
    dx = _np(ah.ah_grouped_matmul_dx(dy, w, off, order=order))
    assert np.array_equal(~np.isfinite(dx).all(1), (leaves == 1) | (np.arange(rows) == 3))
    assert (dx[7] == 0).all()
    dw = _np(ah.ah_grouped_matmul_dw(dy, x, off, order=order))
    assert np.isfinite(dw[1:]).all() and np.isnan(dw[0][:, 3]).all() and not np.isfinite(dw[0][5]).any()
    clean = np.delete(np.delete(dw[0], 5, 0), 3, 1)
    assert np.isfinite(clean).all()


def test_grouped_takes_strided_and_unaligned_rows(gpu):
    torch, ah = gpu
    rows, fan, L, k, n = 70, 2, 4, 96, 88
    big = torch.randn(rows, 300, device="cuda", dtype=torch.bfloat16)
    dbig = torch.randn(rows * fan, 200, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(L, n, k, device="cuda", dtype=torch.bfloat16)
    off, order = ah.ah_group_rows(torch.randint(0, L, (rows, fan), device="cuda", dtype=torch.int32), L)
    for o in (8, 3):
        x, dy = big[:, o:o + k], dbig[:, o:o + n]
        xc, dc = x.contiguous(), dy.contiguous()
        f32 = torch.float32
        assert torch.equal(ah.ah_grouped_matmul(x, w, off, order=order, fan=fan, out_dtype=f32),
                           ah.ah_grouped_matmul(xc, w, off, order=order, fan=fan, out_dtype=f32))
        assert torch.equal(ah.ah_grouped_matmul_dx(dy, w, off, order=order, fan=fan, out_dtype=f32),
                           ah.ah_grouped_matmul_dx(dc, w, off, order=order, fan=fan, out_dtype=f32))
        assert torch.equal(ah.ah_grouped_matmul_dw(dy, x, off, order=order, fan=fan),
                           ah.ah_grouped_matmul_dw(dc, xc, off, order=order, fan=fan))


def test_grouped_rows_beyond_32_bits(gpu):
    torch, ah = gpu
    k, n, stride = 64, 48, (1 << 31) + 64  # element offsets past 2^32 bytes from the second row on
    buf = torch.empty(2 * stride + 64, device="cuda", dtype=torch.bfloat16)
    x = buf.as_strided((3, k), (stride, 1))
    xs = torch.randn(3, k, device="cuda", dtype=torch.bfloat16)
    x.copy_(xs)
    w = torch.randn(2, n, k, device="cuda", dtype=torch.bfloat16)
    leaves = torch.tensor([[0, 1], [1, 0], [1, -1]], device="cuda", dtype=torch.int32)
    off, order = ah.ah_group_rows(leaves, 2)
    assert torch.equal(ah.ah_grouped_matmul(x, w, off, order=order, fan=2),
                       ah.ah_grouped_matmul(xs, w, off, order=order, fan=2))
    dys = torch.randn(6, n, device="cuda", dtype=torch.bfloat16)
    assert torch.equal(ah.ah_grouped_matmul_dw(dys, x, off, order=order, fan=2),
                       ah.ah_grouped_matmul_dw(dys, xs, off, order=order, fan=2))


def test_grouped_bad_offsets_and_order_stay_inside(gpu):
    """Values outside their ranges: no output is promised, but nothing outside the arrays is touched."""
    torch, ah = gpu
    x, w, dy, _ = _grouped_case(torch, 50, 2, 3, 64, 64)
    off = torch.tensor([-5, 1 << 40, 7, 1000], device="cuda", dtype=torch.int64)
    order = torch.arange(100, device="cuda", dtype=torch.int32) * 977 - 500
    guard = torch.full((102, 64), 3.0, device="cuda", dtype=torch.float32)
    ah.ah_grouped_matmul(x, w, off, order=order, fan=2, out=guard[1:101])
    ah.ah_grouped_matmul_dx(dy, w, off, order=order, fan=2)
    ah.ah_grouped_matmul_dw(dy, x, off, order=order, fan=2)
    torch.cuda.synchronize()
    assert (guard[0] == 3).all() and (guard[101] == 3).all()


def test_grouped_gradients_against_differences(gpu):
    """y is linear in x and in w: with small whole numbers every product and sum is exact, and a
    central difference along a direction equals the gradient's dot with it exactly."""
    torch, ah = gpu
    rng = np.random.default_rng(3)
    rows, fan, L, k, n = 45, 2, 4, 48, 56
    ints = lambda *s: _t(torch, rng.integers(-3, 4, s).astype(np.float32), torch.bfloat16)  # noqa: E731
    x, w, dy, dirx, dirw = ints(rows, k), ints(L, n, k), ints(rows * fan, n), ints(rows, k), ints(L, n, k)
    off, order = ah.ah_group_rows(_t(torch, rng.integers(-1, L, (rows, fan)).astype(np.int32)), L)
    f = lambda a, b: float((ah.ah_grouped_matmul(a, b, off, order=order, fan=fan, out_dtype=torch.float32).double()  # noqa: E731
                            * dy.double()).sum())
    dx = ah.ah_grouped_matmul_dx(dy, w, off, order=order, fan=fan, out_dtype=torch.float32)
    dw = ah.ah_grouped_matmul_dw(dy, x, off, order=order, fan=fan)
    assert (f(x + dirx, w) - f(x - dirx, w)) / 2 == float((dx.double() * dirx.double()).sum())
    assert (f(x, w + dirw) - f(x, w - dirw)) / 2 == float((dw.double() * dirw.double()).sum())


# --------------------------------------------------------------------------- distillation
def _distill_ref(z, ids, sc, tau, weight):
    n, V = z.shape
    loss, grad = np.zeros(n), np.zeros((n, V))
    with np.errstate(all="ignore"):
        for r in range(n):
            ok = (ids[r] >= 0) & (ids[r] < V) & (sc[r] != -np.inf)
            if not ok.any():
                continue
            t = sc[r][ok].astype(np.float64) / tau
            lp = t - t.max()
            lp = lp - np.log(np.exp(lp).sum())
            x = z[r].astype(np.float64) / tau
            mx = x.max() if x.max() > -np.inf else 0.0
            S = np.exp(x - mx).sum()
            lq = x - mx - np.log(S)
            q = np.zeros(V) if S == 0 else np.exp(x - mx) / S
            p = np.exp(lp)
            for j, i in enumerate(ids[r][ok]):
                if p[j] != 0:
                    loss[r] += tau * tau * p[j] * (lp[j] - (-np.inf if z[r, i] == -np.inf else lq[i]))
                q[i] -= p[j]
            grad[r] = q * tau * (1.0 if weight is None else weight[r])
    return loss, grad


def _distill_check(torch, ah, z, ids, sc, tau, weight, **kw):
    loss, grad = ah.ah_distill_topk(z, ids, sc, tau=tau, row_weight=weight, **kw)
    zn = _np(z)
    rl, rg = _distill_ref(zn, _np(ids), _np(sc), tau, None if weight is None else _np(weight))
    V = z.shape[1]
    with np.errstate(all="ignore"):
        fin = np.where(np.isfinite(zn), np.abs(zn), 0).max(1)
        tin = np.where(np.isfinite(_np(sc)), np.abs(_np(sc)), 0).max(1)
        unit = (V / 256 + 32) * E * (1 + (fin + tin) / tau)
        w = tau if weight is None else np.abs(_np(weight)) * tau
        l, g = _f64(loss), _f64(grad)
        same = np.isnan(rl) & np.isnan(l) | (rl == l)
        assert (same | (np.abs(l - rl) <= unit * tau * tau * (1 + (fin + tin) / tau + np.log(V)))).all()
        bits = 8 if z.dtype == torch.bfloat16 else 23
        # q and p apart: their difference may cancel
        tol = (unit * w)[:, None] * np.ones((1, V))
        tol = np.minimum(tol, unit[:, None] * (np.abs(rg) + 2 * w * 1.0 if np.isscalar(w) else
                                               np.abs(rg) + 2 * w[:, None])) + 2.0 ** -bits * np.abs(rg)
        gs = np.isnan(rg) & np.isnan(g) | (np.abs(g - rg) <= tol + 1e-37)
        assert gs.all(), float(np.nanmax(np.abs(g - rg) - tol))
    # away from the teacher's entries nothing cancels: relative accuracy even of small q
    far = np.ones_like(rg, dtype=bool)
    idn = _np(ids)
    for r in range(zn.shape[0]):
        far[r, idn[r][(idn[r] >= 0) & (idn[r] < V)]] = False
    far &= np.abs(rg) > 1e-30
    rel = np.abs(g - rg)[far] / np.abs(rg)[far]
    lim = np.broadcast_to((unit * 2 + 2.0 ** -bits)[:, None], rg.shape)[far]
    ok = ~(rel > lim)
    assert ok.all()
    return loss, grad


def _distill_case(torch, n, V, k, dtype, seed=0):
    rng = np.random.default_rng(n + V + k + seed)
    z = _t(torch, rng.standard_normal((n, V)).astype(np.float32) * 3, dtype)
    ids = np.stack([rng.permutation(V)[:min(k, V)] for _ in range(n)]).astype(np.int32) if n else np.zeros((0, k), np.int32)
    sc = -np.sort(-rng.standard_normal(ids.shape).astype(np.float32) * 4, axis=1)
    return z, ids, sc


DISTILL_SIZES = [(1, 1, 1), (2, 7, 3), (5, 64, 64), (3, 1000, 10), (40, 4000, 200), (300, 513, 5), (2, 70001, 33),
                 (1, 250001, 20), (7, 9000, 4096), (600, 65, 9), (33, 16384, 64), (4, 32768, 16), (260, 12000, 50)]


@pytest.mark.parametrize("n,V,k", DISTILL_SIZES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("tau", [1.0, 3.0])
def test_distill(gpu, n, V, k, bf16, tau):
    torch, ah = gpu
    z, ids, sc = _distill_case(torch, n, V, k, torch.bfloat16 if bf16 else torch.float32)
    w = _t(torch, np.random.default_rng(1).random(n).astype(np.float32)) if tau != 1.0 else None
    loss, grad = _distill_check(torch, ah, z, _t(torch, ids), _t(torch, sc), tau, w)
    only, none = ah.ah_distill_topk(z, _t(torch, ids), _t(torch, sc), tau=tau, row_weight=w, want_grad=False)
    assert none is None and torch.equal(only, loss)


@pytest.mark.parametrize("V", [37, 5000, 150000])
@pytest.mark.parametrize("bf16", [True, False])
def test_distill_masks(gpu, V, bf16):
    """Short and empty lists, ids out of range, repeated ids, scores of -inf, masked and spoilt logits."""
    torch, ah = gpu
    k = 12
    z, ids, sc = _distill_case(torch, 14, V, k, torch.bfloat16 if bf16 else torch.float32)
    ids[0] = -1
    ids[1, 5:] = -1
    sc[2] = -np.inf
    sc[3, 1:] = -np.inf
    ids[4, :3] = [V, V + 100, -7]
    ids[5] = ids[5, 0]
    ids[6, 4], ids[6, 9] = ids[6, 1], ids[6, 1]
    sc[7] = -3.0e38
    z[8, :] = -float("inf")
    z[9, ::2] = -float("inf")
    ids[9] = (ids[9] | 1) % V
    ids[9] = np.where(ids[9] % 2 == 0, 1, ids[9])
    z[10, int(ids[10, 0])] = -float("inf")
    z[11, V // 2] = float("nan")
    z[12, 0] = float("inf")
    z[0, 3] = float("nan")  # of a row without a teacher: loss 0, gradient 0
    z[13, :] = torch.finfo(z.dtype).min
    loss, grad = _distill_check(torch, ah, z, _t(torch, ids), _t(torch, sc), 1.0, None)
    l, g = _np(loss), _np(grad)
    assert l[0] == 0 and l[2] == 0 and (g[[0, 2]] == 0).all()
    assert l[8] == np.inf and l[10] == np.inf and np.isfinite(g[[8, 9, 10]]).all()
    assert np.isnan(l[[11, 12]]).all() and np.isfinite(l[[1, 3, 4, 5, 6, 7, 9, 13]]).all()


@pytest.mark.parametrize("n,V", [(6, 1003), (3, 100003)])
@pytest.mark.parametrize("bf16", [True, False])
def test_distill_strided_and_in_place(gpu, n, V, bf16):
    torch, ah = gpu
    dt = torch.bfloat16 if bf16 else torch.float32
    z, ids, sc = _distill_case(torch, n, V, 8, dt)
    ids, sc = _t(torch, ids), _t(torch, sc)
    loss, grad = ah.ah_distill_topk(z, ids, sc)
    pad = torch.full((n, V + 41), 99.0, device="cuda", dtype=dt)
    pad[:, 5:5 + V] = z
    gpad = torch.full((n, V + 10), 7.0, device="cuda", dtype=dt)
    l2, g2 = ah.ah_distill_topk(pad[:, 5:5 + V], ids, sc, grad_out=gpad[:, 3:3 + V])
    assert torch.allclose(l2, loss, rtol=1e-5) and torch.allclose(g2.float(), grad.float(), rtol=2 ** -7, atol=1e-6)
    assert (gpad[:, :3] == 7).all() and (gpad[:, 3 + V:] == 7).all()
    zc = z.clone()
    l3, g3 = ah.ah_distill_topk(zc, ids, sc, grad_out=zc)
    assert torch.equal(l3, loss) and torch.equal(g3, grad) and g3.data_ptr() == zc.data_ptr()
    assert ah.ah_distill_topk(z[:0], ids[:0], sc[:0])[1].shape == (0, V)


def test_distill_rows_beyond_32_bits(gpu):
    torch, ah = gpu
    V, stride = 5000, (1 << 31) + 40
    z, ids, sc = _distill_case(torch, 3, V, 6, torch.bfloat16)
    buf = torch.empty(2 * stride + V, device="cuda", dtype=torch.bfloat16)
    far = buf.as_strided((3, V), (stride, 1))
    far.copy_(z)
    loss, grad = ah.ah_distill_topk(z, _t(torch, ids), _t(torch, sc))
    l2, g2 = ah.ah_distill_topk(far, _t(torch, ids), _t(torch, sc), grad_out=far)
    assert torch.allclose(l2, loss, rtol=1e-5) and torch.allclose(g2.float(), grad.float(), rtol=2 ** -7, atol=1e-6)


@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_distill_gradient_against_differences(gpu, tau):
    """Central differences of the call's own float32 loss: off by the loss's rounding (16 units of
    2^-23 for a loss of order 10) over h, plus h^2 / 6 times a third derivative below 1 / tau."""
    torch, ah = gpu
    z, ids, sc = _distill_case(torch, 1, 40, 6, torch.float32)
    ids, sc = _t(torch, ids), _t(torch, sc)
    g = _np(ah.ah_distill_topk(z, ids, sc, tau=tau)[1])[0]
    h = 2.0 ** -5
    zz = z.repeat(80, 1)
    for v in range(40):
        zz[2 * v, v] += h
        zz[2 * v + 1, v] -= h
    l = _f64(ah.ah_distill_topk(zz, ids.repeat(80, 1), sc.repeat(80, 1), tau=tau, want_grad=False)[0])
    d = (l[0::2] - l[1::2]) / (2 * h)
    assert (np.abs(d - g) <= 16 * E * 10 * tau * tau / h + h * h / 6 / tau).all()


# --------------------------------------------------------------------------- streams and graphs
def _all_calls(torch, ah, x, leaves, w, w8, ws, ids, sc, **kw):
    off, order = ah.ah_group_rows(leaves, w.shape[0], **kw)
    y = ah.ah_grouped_matmul(x, w, off, order=order, fan=2, **kw)
    z = ah.ah_i8_linear(y, w8, ws, **kw)
    loss, dz = ah.ah_distill_topk(z, ids, sc, **kw)
    dy = dz[:, :w.shape[1]]
    dx = ah.ah_grouped_matmul_dx(dy, w, off, order=order, fan=2, **kw)
    dw = ah.ah_grouped_matmul_dw(dy, x, off, order=order, fan=2, **kw)
    return y, z, loss, dz, dx, dw


def _chain(torch, rows):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    L, k, n, V = 5, 96, 80, 600
    x = torch.randn(rows, k, generator=g, device="cuda").bfloat16()
    leaves = torch.randint(-1, L, (rows, 2), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn(L, n, k, generator=g, device="cuda").bfloat16()
    w8 = torch.randint(-127, 128, (V, n), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(V, generator=g, device="cuda") * 0.01
    ids = torch.randint(-1, V, (2 * rows, 5), generator=g, device="cuda", dtype=torch.int32)
    sc = torch.randn(2 * rows, 5, generator=g, device="cuda")
    return x, leaves, w, w8, ws, ids, sc


@pytest.mark.parametrize("rows", [1, 90, 3000])
def test_calls_on_another_stream(gpu, rows):
    torch, ah = gpu
    args = _chain(torch, rows)
    want = _all_calls(torch, ah, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _all_calls(torch, ah, *args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [1, 90, 3000])
def test_calls_in_a_graph(gpu, rows):
    torch, ah = gpu
    args = _chain(torch, rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _all_calls(torch, ah, *args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _all_calls(torch, ah, *args)
    for i in range(4):
        args[0].copy_(torch.randn(args[0].shape, device="cuda"))
        args[1].copy_(torch.randint(-1, 5, args[1].shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = _all_calls(torch, ah, *args)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
