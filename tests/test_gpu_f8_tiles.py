"""The 8-bit float product's tile shapes, chosen by how they fill the chip, and blocks at the ends of the scales' range.
Tolerances as in test_gpu_f8.
"""
import pytest

from test_gpu_f8 import _values, gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# m, k, n: 256 x 256, 192 x 256, 256 x 192, 128 x 192, 128 x 128 and 64 x 64 tiles; one step of the sum (k <= 128), two, three and more; ragged ends
CASES = [(8192, 256, 2048), (8192, 100, 2048), (8192, 1000, 2000), (8064, 256, 1536), (8000, 60, 1530), (8192, 512, 1536), (8190, 128, 1500),
         (4096, 384, 1536), (4001, 700, 1531), (4096, 256, 1536), (900, 120, 900),
         (8200, 2048, 1500), (4000, 1300, 4000), (5400, 300, 1500), (8100, 300, 1500),
         # 64 x 64 tiles of long sums, four steps in LDS, and the kernel for few rows at more than its rows: 16, 32 and 64 a workgroup
         (1000, 4100, 400), (333, 2000, 1001), (900, 1025, 900), (100, 3000, 100), (500, 200, 77), (1500, 300, 20), (40, 4096, 2000),
         (500, 2048, 500), (200, 4090, 1000), (64, 4096, 9000), (33, 700, 33)]


@pytest.mark.parametrize("out", ["bfloat16", "float32"])
@pytest.mark.parametrize("m,k,n", CASES)
def test_shapes(gpu, m, k, n, out):  # noqa: F811
    torch, ah = gpu
    D, dt = torch.float64, getattr(torch, out)
    g = torch.Generator(device="cuda")
    g.manual_seed(m + k + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rnd(m, k) * torch.exp2(torch.randint(-6, 7, (m, 1), generator=g, device="cuda").float()) \
        * torch.exp2((torch.arange(k, device="cuda") // 128 % 5 - 2).float())
    w = rnd(n, k) * torch.exp2(torch.randint(-6, 7, (n, 1), generator=g, device="cuda").float())
    bias = rnd(n) if n % 2 else None
    x8, xs, _, _ = ah.ah_f8_quantize(x)
    w8, ws, _, _ = ah.ah_f8_quantize(w, dtype=torch.float8_e5m2 if k % 3 == 0 else torch.float8_e4m3fn)
    big = torch.full((m + 1, n), 7.0, dtype=dt, device="cuda")
    y = ah.ah_f8_matmul(x8, xs, w8, ws, bias=bias, out=big[:m])
    assert (big[m] == 7).all()
    a, b = _values(torch, x8, xs).cuda(), _values(torch, w8, ws).cuda()
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    if bias is not None:
        want, size = want + bias.to(D), size + bias.to(D).abs()
    tol = size * (2.0 ** -10 + (k / 8 + 16) * 2.0 ** -23)
    assert ((y.to(D) - want).abs() <= tol + (want.abs() + tol) * torch.finfo(dt).eps / 2).all()
    assert torch.equal(ah.ah_f8_matmul(x8, xs, w8, ws, bias=bias, out_dtype=dt), y)
    # whole numbers are exact
    xi = torch.randint(-8, 9, (m, k), generator=g, device="cuda").bfloat16()
    wi = torch.randint(-8, 9, (n, k), generator=g, device="cuda").bfloat16()
    q, s, _, _ = ah.ah_f8_quantize(xi)
    v, t, _, _ = ah.ah_f8_quantize(wi)
    assert torch.equal(ah.ah_f8_matmul(q, s, v, t, out_dtype=torch.float32), xi.float() @ wi.float().t())


@pytest.mark.parametrize("m", [3, 40, 700])
def test_scales_far_apart(gpu, m):  # noqa: F811
    """Scales down to 2^-127 and up to 2^119 against their opposites: their sum decides, not either of them."""
    torch, ah = gpu
    k, n = 256, 80
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    x = torch.randn(m, k, generator=g, device="cuda")
    w = torch.randn(n, k, generator=g, device="cuda")
    w8, ws, _, _ = ah.ah_f8_quantize(w)
    want = ah.ah_f8_linear(x, w8, ws, out_dtype=torch.float32)
    for e in (-110, -60, 60, 110):
        v8, vs, _, _ = ah.ah_f8_quantize(torch.ldexp(w, torch.tensor(-e, device="cuda")))
        got = ah.ah_f8_linear(torch.ldexp(x, torch.tensor(e, device="cuda")), v8, vs, out_dtype=torch.float32)
        assert torch.equal(got, want), e


def test_any_rows_of_few(gpu):  # noqa: F811
    """Up to 16 rows at any alignment and width are quantised in the product: the codes are ah_f8_quantize's."""
    torch, ah = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for k in (1, 7, 130, 1001):
        w8, ws, _, _ = ah.ah_f8_quantize(torch.randn(50, k, generator=g, device="cuda"))
        for dt in (torch.float32, torch.bfloat16):
            for off in (0, 1, 3):
                for m in (1, 5, 16):
                    x = torch.randn(m, off + k + 2, generator=g, device="cuda").to(dt)[:, off:off + k]
                    x8, xs, _, _ = ah.ah_f8_quantize(x)
                    assert torch.equal(ah.ah_f8_linear(x, w8, ws, out_dtype=torch.float32),
                                       ah.ah_f8_matmul(x8, xs, w8, ws, out_dtype=torch.float32))
