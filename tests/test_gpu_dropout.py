"""Dropout on the GPU: the generator against published outputs and numpy, every mask bit, strides and steps.

An element that stays is x f (+ residual) in float32, rounded once to the type: f is rounded (2^-24), the product
and the sum too; the result by half a step of its type.
"""
import numpy as np
import pytest

from philox_reference import factors, numbers, philox

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mips_ah_partition_amd import ahlib
    ahlib.lib()
    return torch, ahlib


def _half_step(torch, dtype):
    return torch.finfo(dtype).eps / 2


def test_known_answers(gpu):
    # published outputs of Philox4x32-10 for the counter and key of zeros and of ones
    assert [int(v) for v in philox([0] * 4, [0] * 2)] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert [int(v) for v in philox([2 ** 32 - 1] * 4, [2 ** 32 - 1] * 2)] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    torch, ah = gpu
    x = torch.ones(1, 8, device="cuda")
    for j, u in enumerate([0xE8D5, 0x6627, 0xC58D, 0xE169, 0xAC4C, 0xBC57, 0xDBD8, 0x9B00]):
        assert float(ah.ah_dropout(x, u / 65536, 0)[0, j]) != 0 and float(ah.ah_dropout(x, (u + 1) / 65536, 0)[0, j]) == 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("rows,n,p,residual", [
    (1, 1, 0.5, False), (1, 7, 0.5, True), (3, 8, 0.1, True), (5, 9, 0.3, False), (17, 100, 0.1, True), (2, 4096, 0.25, True),
    (300, 385, 0.05, False), (1000, 64, 0.9, True), (70000, 3, 0.5, False), (1, 100001, 0.2, True)])
def test_values(gpu, rows, n, p, residual, dtype):
    torch, ah = gpu
    dt = getattr(torch, dtype)
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + n)
    x = torch.randn(rows, n, generator=g, device="cuda").to(dt)
    r = torch.randn(rows, n, generator=g, device="cuda").to(dt) if residual else None
    for seed, step in ((0, None), (12345678901234567, 0), (-1, 2 ** 40 + 17)):
        st = None if step is None else torch.tensor([step], device="cuda")
        y = ah.ah_dropout(x, p, seed, step=st, residual=r)
        f = torch.from_numpy(factors(rows, n, p, seed, step or 0)).cuda()
        want = x.double() * f + (r.double() if residual else 0)
        size = (x.double() * f).abs() + (r.double().abs() if residual else 0)
        assert y.dtype == dt and ((y.double() - want).abs() <= size * 2.0 ** -22 + want.abs() * _half_step(torch, dt)).all()
        if not residual:
            assert torch.equal(y == 0, (f == 0) | (x == 0))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n,off,pad", [(64, 0, 8), (64, 1, 8), (61, 3, 5), (9, 0, 0), (40, 2, 1)])
def test_strides_and_places(gpu, dtype, n, off, pad):
    torch, ah = gpu
    dt, rows, p = getattr(torch, dtype), 33, 0.4
    wide = lambda: torch.randn(rows, off + n + pad, device="cuda").to(dt)  # noqa: E731
    a, b, o = wide(), wide(), wide()
    want = ah.ah_dropout(a[:, off:off + n].contiguous(), p, 7, residual=b[:, off:off + n].contiguous())
    before = o.clone()
    y = ah.ah_dropout(a[:, off:off + n], p, 7, residual=b[:, off:off + n], out=o[:, off:off + n])
    assert torch.equal(y, want) and torch.equal(o[:, off:off + n], want)
    before[:, off:off + n] = o[:, off:off + n]
    assert torch.equal(o, before)  # nothing beside the rows is written
    ah.ah_dropout(a[:, off:off + n], p, 7, residual=b[:, off:off + n], out=b[:, off:off + n])
    assert torch.equal(b[:, off:off + n], want)
    want = ah.ah_dropout(a[:, off:off + n].contiguous(), p, 7)
    ah.ah_dropout(a[:, off:off + n], p, 7, out=a[:, off:off + n])
    assert torch.equal(a[:, off:off + n], want)


def test_zero_probability_and_no_rows(gpu):
    torch, ah = gpu
    x = torch.randn(5, 20, device="cuda").bfloat16()
    assert torch.equal(ah.ah_dropout(x, 0.0, 3), x)
    assert torch.equal(ah.ah_dropout(x, 2.0 ** -18, 3), x)  # below the generator's resolution
    assert ah.ah_dropout(x[:0], 0.5, 3).shape == (0, 20)
    y = ah.ah_dropout(x, 1 - 2.0 ** -20, 3)  # all but one number in 2^16 is dropped
    assert (y == 0).all() or float((y != 0).float().mean()) < 0.1


def test_dropped_elements_are_zero_whatever_they_were(gpu):
    torch, ah = gpu
    x = torch.full((64, 64), float("nan"), device="cuda")
    x[::2] = float("inf")
    y = ah.ah_dropout(x, 0.5, 1)
    f = torch.from_numpy(factors(64, 64, 0.5, 1, 0)).cuda()
    assert (y[f == 0] == 0).all() and not torch.isfinite(y[f > 0]).any()


def test_gradient_is_the_same_mask(gpu):
    torch, ah = gpu
    x, dy = torch.randn(40, 50, device="cuda"), torch.randn(40, 50, device="cuda")
    dx = ah.ah_dropout(dy, 0.3, 11)
    # y is linear in x: <dy, y(x + d) - y(x)> = <dx, d>
    d = torch.randn(40, 50, device="cuda")
    with_d = ah.ah_dropout(d, 0.3, 11).double()
    assert abs(float((dy.double() * with_d).sum() - (dx.double() * d.double()).sum())) <= 2.0 ** -22 * float((dy * d).abs().sum()) * 2
    assert torch.equal(ah.ah_dropout(x, 0.3, 11) == 0, dx == 0)


def test_share_of_dropped_elements(gpu):
    torch, ah = gpu
    n = 1 << 22
    for p in (0.1, 0.5):
        y = ah.ah_dropout(torch.ones(1024, n // 1024, device="cuda"), p, 99)
        t = round(65536 * p) / 65536
        assert abs(float((y == 0).double().mean()) - t) <= 6 * (t * (1 - t) / n) ** 0.5
    assert len(np.unique(numbers(64, 64, 99, 0))) > 3900  # 4,096 draws of 65,536


def test_graph_with_a_counted_step(gpu):
    torch, ah = gpu
    x, step = torch.randn(30, 70, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    out = torch.empty_like(x)
    ah.ah_dropout(x, 0.5, 5, step=step, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ah.ah_dropout(x, 0.5, 5, step=step, out=out)
        step.add_(1)
    for i in range(4):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ah.ah_dropout(x, 0.5, 5, step=torch.tensor([i], device="cuda")))


def test_another_stream(gpu):
    torch, ah = gpu
    x = torch.randn(500, 600, device="cuda")
    want = ah.ah_dropout(x, 0.2, 8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ah.ah_dropout(x, 0.2, 8, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_bindings_check_shapes(gpu):
    torch, ah = gpu
    x = torch.zeros(4, 8, device="cuda")
    for bad, err in ((lambda: ah.ah_dropout(x, 0.1, 1, residual=x[:2]), ValueError),
                     (lambda: ah.ah_dropout(x, 0.1, 1, residual=x.bfloat16()), TypeError),
                     (lambda: ah.ah_dropout(x, 0.1, 1, out=x[:, :4]), ValueError),
                     (lambda: ah.ah_dropout(x, 0.1, 1, step=torch.zeros(2, dtype=torch.int64, device="cuda")), ValueError),
                     (lambda: ah.ah_dropout(x, 0.1, 1, step=torch.zeros(1, device="cuda")), TypeError),
                     (lambda: ah.ah_dropout(x.t(), 0.1, 1), ValueError), (lambda: ah.ah_dropout(x.half(), 0.1, 1), TypeError),
                     (lambda: ah.ah_dropout(x, 1.0, 1), ah.AHError)):
        with pytest.raises(err):
            bad()
