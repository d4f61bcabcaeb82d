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
