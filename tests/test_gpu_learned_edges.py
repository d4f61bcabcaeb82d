"""The learned query side's calls at the ends of the sizes that they accept, and in the kernel variants that only
larger products reach, against plain forms in 64 bits.

Tolerances as for the other tests of these calls.  int8: bit for bit.  Grouped products: a float32 sum of t
exact products is off by at most t 2^-23 sum |a||b|, its rounding by 2^-8 (bfloat16) or 2^-23
relative.  Distillation: a few (1 + |z / tau|) 2^-23 for the exponentials, 2^-8 for a bfloat16 gradient.
"""
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
    yield torch, ahlib
    torch.cuda.empty_cache()


# --------------------------------------------------------------------------- more workgroups than a launch can have
@pytest.mark.parametrize("m", [1, 20])
def test_int8_rows_against_more_columns_than_a_row_launch_has(gpu, m):
    """16 columns a workgroup of 512 threads would be 2^32 work-items from 2^27 columns on."""
    torch, ah = gpu
    k, n = 16, (1 << 27) + 1000
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    w8 = torch.randint(-127, 128, (n, k), device="cuda", dtype=torch.int8, generator=g)
    ws = torch.rand(n, device="cuda", generator=g)
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    c, s = ah.ah_i8_quantize_rows(x)
    y = ah.ah_i8_linear(x, w8, ws)
    z = ah.ah_i8_matmul(c, s, w8, ws, out_dtype=torch.bfloat16)
    for j in range(0, n, 1 << 24):
        part = slice(j, j + (1 << 24))
        dot = torch.mm(c.float(), w8[part].float().t())  # whole numbers below 2^24
        ref = ((dot * s[:, None]) * ws[None, part]).bfloat16()
        assert torch.equal(y[:, part], ref) and torch.equal(z[:, part], ref)


def test_distillation_of_more_rows_than_a_launch_has(gpu):
    """A workgroup of 256 threads a row would be 2^32 work-items from 2^24 rows on."""
    torch, ah = gpu
    n, V, k = (1 << 24) + 9, 16, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    z = torch.randn(n, V, device="cuda", generator=g).bfloat16()
    ids = torch.randint(-1, V, (n, k), device="cuda", dtype=torch.int32, generator=g)
    sc = torch.randn(n, k, device="cuda", generator=g)
    w = torch.rand(n, device="cuda", generator=g)
    loss, grad = ah.ah_distill_topk(z, ids, sc, row_weight=w)
    for r in range(0, n, 1 << 21):
        part = slice(r, r + (1 << 21))
        zd, ok = z[part].double(), ids[part] >= 0
        lq = torch.log_softmax(zd, 1)
        some = ok.any(1)
        t = torch.where(ok, sc[part].double(), torch.full_like(sc[part].double(), -float("inf")))
        lp = torch.log_softmax(torch.where(some[:, None], t, torch.zeros_like(t)), 1)
        p = torch.where(ok, lp.exp(), torch.zeros_like(lp))
        at = ids[part].clamp(min=0).long()
        want = torch.where(ok, p * (lp - lq.gather(1, at)), torch.zeros_like(p)).sum(1)
        dz = (lq.exp() * some[:, None]).scatter_add(1, at, -p) * w[part].double()[:, None]
        size = 1 + zd.abs().amax(1) + sc[part].double().abs().amax(1)
        assert ((loss[part].double() - want).abs() <= 40 * E * size * (size + 3)).all()
        assert ((grad[part].double() - dz).abs() <= 40 * E * size[:, None] + 2.0 ** -8 * dz.abs()).all()


def test_weight_gradients_of_more_tiles_than_a_launch_has(gpu):
    """65,536 leaves of 256 tiles each: a workgroup of 256 threads a tile would be 2^32 work-items."""
    torch, ah = gpu
    L, n, k, rows = 1 << 16, 1 << 15, 1, 300
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    leaf = torch.randint(0, L, (rows,), device="cuda", generator=g)
    leaf[:3], leaf[3:40] = torch.tensor([0, L - 1, L - 1], device="cuda"), 777
    order = torch.sort(leaf, stable=True).indices.to(torch.int32)
    off = torch.searchsorted(torch.sort(leaf).values, torch.arange(L + 1, device="cuda"))
    x, dy = (torch.randn(rows, c, device="cuda", generator=g).bfloat16() for c in (k, n))
    dw = ah.ah_grouped_matmul_dw(dy, x, off, order=order, out_dtype=torch.bfloat16)
    left = sum(int(torch.count_nonzero(part)) for part in dw.split(4096))
    for l in leaf.unique().tolist():
        at = (leaf == l).nonzero().flatten()
        terms = dy[at].double() * x[at].double()
        want, got = terms.sum(0), dw[l, :, 0].double()
        assert ((got - want).abs() <= (rows + 2) * E * terms.abs().sum(0) + 2.0 ** -8 * want.abs()).all()
        left -= int(torch.count_nonzero(dw[l]))
    assert left == 0  # leaves without a row


# --------------------------------------------------------------------------- leaf starts that are not in order
def test_grouped_starts_out_of_order_walk_no_more_tiles_than_rows_have(gpu):
    """Starts 0, T, 0, T, ...: 32,768 leaves of all T rows each, 2^31 row tiles by their count.  No output is
    promised, but nothing outside the arrays is touched and the call ends."""
    torch, ah = gpu
    T, L, w = 1 << 23, 1 << 16, 8
    off = torch.zeros(L + 1, device="cuda", dtype=torch.int64)
    off[1::2] = T
    x = torch.ones(T, w, device="cuda", dtype=torch.bfloat16)
    mats = torch.ones(L, w, w, device="cuda", dtype=torch.bfloat16)
    guard = torch.full((T + 2, w), 3.0, device="cuda", dtype=torch.float32)
    ah.ah_grouped_matmul(x, mats, off, out=guard[1:T + 1])
    ah.ah_grouped_matmul_dx(x, mats, off, dx_out=guard[1:T + 1])
    torch.cuda.synchronize()
    assert (guard[0] == 3).all() and (guard[T + 1] == 3).all()
    # and in order again, every leaf 128 rows
    off = torch.arange(L + 1, device="cuda", dtype=torch.int64) * (T // L)
    y = ah.ah_grouped_matmul(x, mats, off, out_dtype=torch.float32)
    assert (y == w).all()


# --------------------------------------------------------------------------- distillation: the exponents' scale
@pytest.mark.parametrize("tau", [1.5625, 3.875, 6.6875])
@pytest.mark.parametrize("V", [4000, 100003])
def test_distillation_scales_exponents_by_the_nearest_factor(gpu, tau, V):
    """q_v = 2^((z_v - M) c) with c = log2(e) / tau: an error d of c turns a small q_v by x ln2 d, x the exponent.
    Over many values the other roundings average out, so the mean shows d: that of the float32 nearest to log2(e) / tau
    (a quarter of 2^-24 covers the mean's own error: the factors 1 / s and tau add at most 2^-23 over exponents of 57
    and more)."""
    import numpy as np
    torch, ah = gpu
    n = 20
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    z = -tau * (40 + 40 * torch.rand(n, V, device="cuda", generator=g))
    z[:, 0] = 0
    ids = torch.zeros(n, 1, device="cuda", dtype=torch.int32)
    _, grad = ah.ah_distill_topk(z, ids, torch.zeros(n, 1, device="cuda"), tau=tau)
    far = z[:, 1:].double() / tau
    s = 1 + far.exp().sum(1, keepdim=True)
    rel = grad[:, 1:].double() / (tau * far.exp() / s) - 1
    exact = np.log2(np.e) / tau
    d = float(np.float32(exact)) / exact - 1
    assert abs(float((rel / far).mean()) - d) <= 0.25 * 2.0 ** -24


# --------------------------------------------------------------------------- every tile, and few rows of each kind
def _close(torch, got, want, size, terms, dt):
    tol = terms * E * size + (2.0 ** -8 if dt == torch.bfloat16 else E) * want.abs() + 1e-30
    assert bool(((got.double() - want).abs() <= tol).all())


def _gen(torch, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _grouped_order(torch, leaf, L):
    """Order and starts of any number of leaves (leaf in [0, L], L: none)."""
    s, order = torch.sort(leaf, stable=True)
    return torch.searchsorted(s, torch.arange(L + 1, device="cuda")), order.to(torch.int32)


def _products(torch, ah, x, w, dy, leaf, fan, dt):
    """All three products against 64 bits, leaf by leaf."""
    L, n, k = w.shape
    T, m = leaf.numel(), x.shape[0]
    off, order = _grouped_order(torch, leaf, L)
    y = ah.ah_grouped_matmul(x, w, off, order=order, fan=fan, out_dtype=dt)
    dx = ah.ah_grouped_matmul_dx(dy, w, off, order=order, fan=fan, out_dtype=dt)
    dw = ah.ah_grouped_matmul_dw(dy, x, off, order=order, fan=fan, out_dtype=dt)
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    ry, ya, rx, xa = z(T, n), z(T, n), z(T, k), z(T, k)
    for l in range(L):
        at = (leaf == l).nonzero().flatten()
        xs, ds, wl = x[at // fan].double(), dy[at].double(), w[l].double()
        ry[at], ya[at] = torch.mm(xs, wl.t()), torch.mm(xs.abs(), wl.abs().t())
        rx[at], xa[at] = torch.mm(ds, wl), torch.mm(ds.abs(), wl.abs())
        _close(torch, dw[l], torch.mm(ds.t(), xs), torch.mm(ds.abs().t(), xs.abs()), T + 2, dt)
    _close(torch, y, ry, ya, k + 2, dt)
    _close(torch, dx, rx.view(m, fan, k).sum(1), xa.view(m, fan, k).sum(1), n + fan + 2, dt)


# rows, fan, leaves, k, n: 256 x 256 tiles forward; in dx; in dx with shared rows; 192 x 256 in both; then few rows a leaf,
# of whole 16-byte chunks and not, 1, 2 and 4 fragments of 16 rows
TILES = [(2500, 1, 3, 264, 5000), (2500, 1, 3, 5000, 264), (8192, 2, 16, 1536, 1536), (9000, 1, 3, 1032, 2056),
         (10, 1, 3, 33, 20), (30, 2, 6, 64, 64), (20, 2, 4, 33, 20), (60, 2, 4, 72, 64), (60, 2, 4, 73, 41)]


@pytest.mark.parametrize("rows,fan,L,k,n", TILES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_grouped_tiles(gpu, rows, fan, L, k, n, out):
    torch, ah = gpu
    g = _gen(torch, rows + k + n)
    x, dy = (torch.randn(r, c, device="cuda", generator=g).bfloat16() for r, c in ((rows, k), (rows * fan, n)))
    w = torch.randn(L, n, k, device="cuda", generator=g).bfloat16()
    leaf = torch.randint(0, L + 1, (rows * fan,), device="cuda", generator=g)  # L: no leaf
    _products(torch, ah, x, w, dy, leaf, fan, torch.bfloat16 if out == "bf16" else torch.float32)


# 192 x 256 tiles; few rows at widths that are not whole chunks
@pytest.mark.parametrize("m,k,n", [(1800, 272, 5000), (1800, 272, 5001), (20, 33, 70), (50, 100, 90), (64, 1001, 33)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_int8_tiles(gpu, m, k, n, out):
    torch, ah = gpu
    g = _gen(torch, m + k + n)
    x8, w8 = (torch.randint(-128, 128, (r, k), device="cuda", dtype=torch.int8, generator=g) for r in (m, n))
    s, ws, bias = (torch.rand(r, device="cuda", generator=g) for r in (m, n, n))
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    y = ah.ah_i8_matmul(x8, s, w8, ws, bias=bias, out_dtype=dt)
    ref = torch.mm(x8.double(), w8.double().t()).float() * s[:, None]
    ref = ref * ws[None, :]
    assert torch.equal(y, (ref + bias[None, :]).to(dt))


@pytest.mark.parametrize("L,T,w", [(4000, 12000, 64), (4000, 260000, 64), (65534, 70000, 16), (65536, 70000, 16),
                                   (65536, 3000000, 16)])
def test_grouped_thousands_of_leaves(gpu, L, T, w):
    """Few and many rows a leaf, up to the most leaves; every fourth leaf is empty, one slot in nine has none."""
    torch, ah = gpu
    g = _gen(torch, L + T)
    x, dy = (torch.randn(T, w, device="cuda", generator=g).bfloat16() for _ in range(2))
    mats = torch.randn(L, w, w, device="cuda", generator=g).bfloat16()
    leaf = torch.randint(0, L, (T,), device="cuda", generator=g)
    leaf[leaf % 4 == 3] -= 1
    leaf[:2] = torch.tensor([0, L - 1], device="cuda")
    leaf[5::9] = L
    off, order = _grouped_order(torch, leaf, L)
    if L <= 4096:
        o2, r2 = ah.ah_group_rows(leaf.to(torch.int32), L)
        assert torch.equal(o2, off) and torch.equal(r2, order)
    y = ah.ah_grouped_matmul(x, mats, off, order=order, out_dtype=torch.float32)
    dx = ah.ah_grouped_matmul_dx(dy, mats, off, order=order, out_dtype=torch.float32)
    dw = ah.ah_grouped_matmul_dw(dy, x, off, order=order)
    assert (y[leaf == L] == 0).all() and (dx[leaf == L] == 0).all()
    rw, wa = (torch.zeros(L + 1, w, w, dtype=torch.float64, device="cuda") for _ in range(2))
    step = (1 << 28) // (w * w)
    for a in range(0, T, step):
        lf, xs, ds = leaf[a:a + step], x[a:a + step].double(), dy[a:a + step].double()
        m = mats[lf.clamp(max=L - 1)].double() * (lf < L)[:, None, None]
        _close(torch, y[a:a + step], (m * xs[:, None, :]).sum(2), (m * xs[:, None, :]).abs().sum(2), w + 2, torch.float32)
        _close(torch, dx[a:a + step], (m * ds[:, :, None]).sum(1), (m * ds[:, :, None]).abs().sum(1), w + 3, torch.float32)
        m = ds[:, :, None] * xs[:, None, :]
        rw.index_add_(0, lf, m)
        wa.index_add_(0, lf, m.abs_())
    _close(torch, dw, rw[:L], wa[:L], int(torch.bincount(leaf, minlength=L + 1)[:L].max()) + 2, torch.float32)


def test_grouped_one_leaf_takes_all(gpu):
    """4,000 leaves, nearly every slot in one of them."""
    torch, ah = gpu
    g = _gen(torch, 9)
    rows, L, k, n = 5000, 4000, 40, 24
    x, dy = (torch.randn(rows, c, device="cuda", generator=g).bfloat16() for c in (k, n))
    w = torch.randn(L, n, k, device="cuda", generator=g).bfloat16()
    leaf = torch.full((rows,), 17, device="cuda")
    leaf[::1000] = torch.tensor([0, 16, 18, 3999, 4000], device="cuda")
    _products(torch, ah, x, w, dy, leaf, 1, torch.float32)


def test_grouped_weights_beyond_32_bits(gpu):
    """5.3 GB of matrices, 50 rows a leaf: read by tiles forward and in dx, written in dw."""
    torch, ah = gpu
    L, w, rows = 70, 6144, 3500
    g = _gen(torch, 10)
    mats = torch.empty(L, w, w, device="cuda", dtype=torch.bfloat16)
    for l in range(L):
        mats[l] = torch.randn(w, w, device="cuda", generator=g)
    x, dy = (torch.randn(rows, w, device="cuda", generator=g).bfloat16() for _ in range(2))
    leaf = torch.randint(0, L, (rows,), device="cuda", generator=g)
    off, order = _grouped_order(torch, leaf, L)
    bf = torch.bfloat16
    y = ah.ah_grouped_matmul(x, mats, off, order=order)
    dx = ah.ah_grouped_matmul_dx(dy, mats, off, order=order)
    dw = ah.ah_grouped_matmul_dw(dy, x, off, order=order, out_dtype=bf)
    for l in (0, 55, 56, 57, 58, L - 1):  # 4 GB end inside matrix 56
        at = (leaf == l).nonzero().flatten()
        xs, ds, m = x[at].double(), dy[at].double(), mats[l].double()
        _close(torch, y[at], torch.mm(xs, m.t()), torch.mm(xs.abs(), m.abs().t()), w + 2, bf)
        _close(torch, dx[at], torch.mm(ds, m), torch.mm(ds.abs(), m.abs()), w + 2, bf)
        _close(torch, dw[l], torch.mm(ds.t(), xs), torch.mm(ds.abs().t(), xs.abs()), rows + 2, bf)


@pytest.mark.parametrize("k,n", [(64, 72), (33, 41)])
def test_grouped_tiles_of_rows_beyond_32_bits(gpu, k, n):
    torch, ah = gpu
    rows, L, stride = 200, 2, (1 << 24) + 8
    g = _gen(torch, k)
    buf = torch.empty((rows - 1) * stride + (1 << 13), device="cuda", dtype=torch.bfloat16)  # 6.7 GB
    far = lambda c, at: buf[at:].as_strided((rows, c), (stride, 1))  # noqa: E731
    xs, ds = (torch.randn(rows, c, device="cuda", generator=g).bfloat16() for c in (k, n))
    x, dy = far(k, 0).copy_(xs), far(n, 1 << 12).copy_(ds)  # in one buffer, side by side
    w = torch.randn(L, n, k, device="cuda", generator=g).bfloat16()
    off, order = ah.ah_group_rows(torch.randint(0, L, (rows,), device="cuda", dtype=torch.int32, generator=g), L)
    f32 = torch.float32
    assert torch.equal(ah.ah_grouped_matmul(x, w, off, order=order, out_dtype=f32),
                       ah.ah_grouped_matmul(xs, w, off, order=order, out_dtype=f32))
    assert torch.equal(ah.ah_grouped_matmul_dx(dy, w, off, order=order, out_dtype=f32),
                       ah.ah_grouped_matmul_dx(ds, w, off, order=order, out_dtype=f32))
    assert torch.equal(ah.ah_grouped_matmul_dw(dy, x, off, order=order), ah.ah_grouped_matmul_dw(ds, xs, off, order=order))


@pytest.mark.parametrize("m,n", [(270000, 20), (70, 270000), (3, 270000)])
def test_int8_operands_beyond_32_bits(gpu, m, n):
    torch, ah = gpu
    k = 16384  # 4.4 GB on one side
    g = _gen(torch, m)
    x8, w8 = (torch.randint(-127, 128, (r, k), device="cuda", dtype=torch.int8, generator=g) for r in (m, n))
    s, ws = (torch.rand(r, device="cuda", generator=g) for r in (m, n))
    y = ah.ah_i8_matmul(x8, s, w8, ws)
    for r in (slice(0, 70), slice(262100, 262200), slice(269930, 270000)):
        a, b = (r, slice(None)) if m > n else (slice(None), r)
        dot = torch.mm(x8[a].double(), w8[b].double().t()).float()
        assert torch.equal(y[a, b], (dot * s[a, None]) * ws[None, b])
