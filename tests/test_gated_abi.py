"""Refusals of the gated products, the 8-bit float products and dropout: every bad argument is turned away on the host,
before anything is enqueued (no GPU needed, no pointer is dereferenced)."""
import ctypes as C

import pytest

vp = C.c_void_p
NULL, SHAPE, UNSUPPORTED, WORKSPACE = -1, -2, -3, -4
F, ODD = vp(4096), vp(4097)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from mips_ah_partition_amd import ahlib
    return ahlib.lib()


def _with(base, **kw):
    a = dict(base)
    a.update(kw)
    return list(a.values())


GATED = dict(x=F, xs=8, w=F, L=4, n=6, k=8, offsets=F, order=F, slots=10, fan=2, act=0, drop=0.1, seed=1, step=None,
             pre=F, out=F, odt=1, stream=None)
BOTH = [(dict(L=0), SHAPE), (dict(n=0), SHAPE), (dict(L=65537), UNSUPPORTED), (dict(n=(1 << 19) + 1), UNSUPPORTED),
        (dict(act=3), UNSUPPORTED), (dict(act=-1), UNSUPPORTED), (dict(drop=1.0), SHAPE), (dict(drop=-0.1), SHAPE),
        (dict(drop=float("nan")), SHAPE), (dict(step=ODD), UNSUPPORTED), (dict(offsets=None), NULL), (dict(w=None), NULL),
        (dict(slots=1 << 31), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(slots=9), SHAPE), (dict(slots=-2), SHAPE), (dict(fan=0), SHAPE), (dict(k=0), SHAPE), (dict(xs=7), SHAPE),
    (dict(order=None), SHAPE), (dict(odt=3), UNSUPPORTED), (dict(x=None), NULL), (dict(out=None), NULL),
    (dict(slots=0, x=None, out=None), 0)])
def test_grouped_gated(lib, kw, want):
    assert lib.ah_grouped_gated(*_with(GATED, **kw)) == want


GRAD = dict(dy=F, ds=8, w=F, L=4, d=8, n=6, offsets=F, order=F, slots=10, pre=F, act=0, drop=0.1, seed=1, step=None,
            dpre=F, hidden=F, stream=None)


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(slots=-1), SHAPE), (dict(d=0), SHAPE), (dict(ds=7), SHAPE), (dict(dy=None), NULL), (dict(pre=None), NULL),
    (dict(dpre=None), NULL), (dict(slots=0, dy=None), 0)])
def test_grouped_gated_grad(lib, kw, want):
    assert lib.ah_grouped_gated_grad(*_with(GRAD, **kw)) == want


QUANT = dict(x=F, dt=1, n=3, d=8, xs=8, type=0, codes=F, scale=F, codes_t=F, scale_t=F, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), SHAPE), (dict(d=0), SHAPE), (dict(xs=7), SHAPE), (dict(dt=2), UNSUPPORTED), (dict(type=2), UNSUPPORTED),
    (dict(d=(1 << 20) + 1, xs=1 << 21), UNSUPPORTED), (dict(n=(1 << 20) + 1), UNSUPPORTED),
    (dict(n=(1 << 30) + 1, codes_t=None), UNSUPPORTED), (dict(x=None), NULL), (dict(codes=None, codes_t=None), NULL),
    (dict(scale=None), NULL), (dict(scale_t=None), NULL), (dict(codes=ODD), UNSUPPORTED), (dict(scale_t=ODD), UNSUPPORTED),
    (dict(n=0, x=None, codes=None), 0)])
def test_f8_quantize(lib, kw, want):
    assert lib.ah_f8_quantize(*_with(QUANT, **kw)) == want


MATMUL = dict(x8=F, xs=F, xt=0, m=2, w8=F, ws=F, wt=0, n=5, k=16, bias=None, out=F, odt=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), SHAPE), (dict(n=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=(1 << 20) + 1), UNSUPPORTED),
    (dict(xt=2), UNSUPPORTED), (dict(wt=-1), UNSUPPORTED), (dict(odt=5), UNSUPPORTED), (dict(m=1 << 31), UNSUPPORTED),
    (dict(n=1 << 31), UNSUPPORTED), (dict(x8=None), NULL), (dict(xs=None), NULL), (dict(w8=None), NULL),
    (dict(ws=None), NULL), (dict(out=None), NULL), (dict(x8=ODD), UNSUPPORTED), (dict(ws=ODD), UNSUPPORTED),
    (dict(m=0, x8=None, out=None), 0), (dict(n=0, w8=None), 0)])
def test_f8_matmul(lib, kw, want):
    assert lib.ah_f8_matmul(*_with(MATMUL, **kw)) == want


LINEAR = dict(x=F, dt=1, m=20, k=16, xs=16, xt=0, w8=F, ws=F, wt=0, n=5, bias=None, out=F, odt=1, work=F, bytes=BIG,
              stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), SHAPE), (dict(xs=15), SHAPE), (dict(dt=7), UNSUPPORTED), (dict(xt=3), UNSUPPORTED),
    (dict(wt=3), UNSUPPORTED), (dict(odt=-1), UNSUPPORTED), (dict(k=(1 << 20) + 1, xs=1 << 21), UNSUPPORTED),
    (dict(x=None), NULL), (dict(w8=None), NULL), (dict(out=None), NULL), (dict(work=None), WORKSPACE),
    (dict(bytes=2591), WORKSPACE), (dict(work=ODD), UNSUPPORTED), (dict(w8=ODD), UNSUPPORTED), (dict(m=0, x=None), 0)])
def test_f8_linear(lib, kw, want):
    assert lib.ah_f8_linear_workspace_bytes(20, 16) == 2592  # rows of 128 codes, 32 scale bytes
    assert lib.ah_f8_linear_workspace_bytes(16, 16) == 0  # few rows need none
    assert lib.ah_f8_linear(*_with(LINEAR, **kw)) == want


DROP = dict(x=F, dt=1, rows=3, n=8, xs=8, p=0.1, seed=1, step=None, res=F, rs=8, out=F, os=8, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), SHAPE), (dict(n=0), SHAPE), (dict(xs=7), SHAPE), (dict(rs=7), SHAPE), (dict(os=7), SHAPE),
    (dict(p=1.0), SHAPE), (dict(p=-1e-9), SHAPE), (dict(p=float("nan")), SHAPE), (dict(dt=2), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(n=1 << 31, xs=1 << 31, rs=1 << 31, os=1 << 31), UNSUPPORTED),
    (dict(step=ODD), UNSUPPORTED), (dict(x=None), NULL), (dict(out=None), NULL), (dict(rows=0, x=None), 0)])
def test_dropout(lib, kw, want):
    assert lib.ah_dropout(*_with(DROP, **kw)) == want


def test_bindings_refuse_host_tensors():
    import torch
    from mips_ah_partition_amd import ahlib as ah
    x = torch.zeros(2, 8)
    b = x.bfloat16()
    c = torch.zeros(2, 128).to(torch.float8_e4m3fn)
    s = torch.zeros(1, 16, dtype=torch.uint8)
    for call in (lambda: ah.ah_grouped_gated(b, b[None]), lambda: ah.ah_grouped_gated_grad(b, b[None], b),
                 lambda: ah.ah_f8_quantize(x), lambda: ah.ah_f8_matmul(c, s, c, s), lambda: ah.ah_f8_linear(x, c, s),
                 lambda: ah.ah_dropout(x, 0.5, 1), lambda: ah.ah_f8_matmul(x, s, c, s)):
        with pytest.raises(TypeError):
            call()
