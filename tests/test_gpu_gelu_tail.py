"""gelu's tail on the GPU: gates from -12.5 to 12, held to a share of the value itself, also where the value is 10^-35.

Tolerance.  The gates are exact.  The kernels compute c = erfc(t) / 2 at t = -a / sqrt(2) in float32, whose product
and constant are off by at most 1.5 2^-24 of t; |t erfc'(t) / erfc(t)| <= 2 t^2 + 1 = a^2 + 1, so c moves by at
most (a^2 + 1) 1.5 2^-24; the library's erfc itself by 16 units in the last place, 16 2^-23; the products behind it
by 2^-24 each.  In all less than (a^2 + 20) 2^-23: E.  The density d = exp(-a^2 / 2) / sqrt(2 pi): its
exponent's three roundings 0.5 a^2 3 2^-24, the exponential 2^-23, constant and products 3 2^-24: also below E.  So gelu
is off by E of its value, its derivative c + a d by E of |c| + |a d|; results by half a step of their type.
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mips_ah_partition_amd import ahlib
    ahlib.lib()
    return torch, ahlib


def _gates(torch, m):
    """m gates, bfloat16: the range from end to end, and 0."""
    a = torch.linspace(-12.5, 12.0, m, device="cuda").bfloat16()
    a[m // 2] = 0
    return a


def _parts(torch, a):
    """c and d of the docstring, float64."""
    a = a.double()
    return 0.5 * torch.special.erfc(-a * 0.5 ** 0.5), torch.exp(-a * a / 2) / (2 * torch.pi) ** 0.5


# m, k, n: the kernel for few rows (short and long sums), small and large tiles by each way of loading
SIZES = [(48, 8, 5), (40, 320, 24), (300, 7, 33), (300, 64, 40), (3000, 72, 300), (20000, 100, 160), (16128, 1600, 512)]


@pytest.mark.parametrize("m,k,n", SIZES)
def test_forward(gpu, m, k, n):
    torch, ah = gpu
    a = _gates(torch, m)
    x = torch.zeros(m, k, device="cuda").bfloat16()
    x[:, 0], x[:, 1] = a, 1
    w = torch.zeros(1, 2 * n, k, device="cuda").bfloat16()  # gates a, the other projection 1
    w[:, :n, 0], w[:, n:, 1] = 1, 1
    c, _ = _parts(torch, a)
    want, e = (a.double() * c)[:, None], ((a.double() ** 2 + 20) * 2.0 ** -23)[:, None]
    for dt in (torch.float32, torch.bfloat16):
        h, _ = ah.ah_grouped_gated(x, w, act="gelu", out_dtype=dt)
        assert ((h.double() - want).abs() <= want.abs() * (e + (1 + e) * torch.finfo(dt).eps / 2)).all(), dt


@pytest.mark.parametrize("m,d,n", [(40, 8, 16), (300, 7, 33), (3000, 72, 304), (20000, 100, 300), (16128, 1600, 1024)])
def test_gradient(gpu, m, d, n):
    torch, ah = gpu
    a = _gates(torch, m)
    dy, w = torch.zeros(m, d, device="cuda").bfloat16(), torch.zeros(1, d, n, device="cuda").bfloat16()
    dy[:, 0], w[:, 0] = 1, 1  # the hidden values' gradient is 1
    pre = torch.ones(m, 2 * n, device="cuda").bfloat16()
    pre[:, :n] = a[:, None]
    dpre, h = ah.ah_grouped_gated_grad(dy, w, pre, act="gelu")
    c, dens = _parts(torch, a)
    e = (a.double() ** 2 + 20) * 2.0 ** -23
    g, slope, size = a.double() * c, c + a.double() * dens, c + a.double().abs() * dens
    half = 2.0 ** -8
    for got, want, tol in ((dpre[:, :n], slope, size * e), (dpre[:, n:], g, g.abs() * e), (h, g, g.abs() * e)):
        assert ((got.double() - want[:, None]).abs() <= (tol + (want.abs() + tol) * half)[:, None]).all()
