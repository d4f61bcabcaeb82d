"""Refusals of the learned query side's calls: every bad argument is turned away on the
host, before anything is enqueued (no GPU needed, no pointer is dereferenced)."""
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


QUANT = dict(x=F, dt=1, n=3, d=8, xs=8, codes=F, scale=F, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), SHAPE), (dict(d=0), SHAPE), (dict(xs=7), SHAPE), (dict(dt=2), UNSUPPORTED),
    (dict(d=16385, xs=16385), UNSUPPORTED), (dict(x=None), NULL), (dict(codes=None), NULL), (dict(scale=None), NULL),
    (dict(n=0, x=None, codes=None, scale=None), 0)])
def test_i8_quantize_rows(lib, kw, want):
    assert lib.ah_i8_quantize_rows(*_with(QUANT, **kw)) == want


MATMUL = dict(x8=F, xs=F, m=2, w8=F, ws=F, n=5, k=16, bias=None, out=F, odt=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), SHAPE), (dict(n=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=16385), UNSUPPORTED),
    (dict(odt=5), UNSUPPORTED), (dict(m=1 << 31), UNSUPPORTED), (dict(n=1 << 31), UNSUPPORTED), (dict(x8=None), NULL),
    (dict(xs=None), NULL), (dict(w8=None), NULL), (dict(ws=None), NULL), (dict(out=None), NULL),
    (dict(m=0, x8=None, out=None), 0), (dict(n=0, w8=None, out=None), 0)])
def test_i8_matmul(lib, kw, want):
    assert lib.ah_i8_matmul(*_with(MATMUL, **kw)) == want


LINEAR = dict(x=F, dt=1, m=2, k=16, xs=16, w8=F, ws=F, n=5, bias=None, out=F, odt=1, work=F, bytes=BIG, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), SHAPE), (dict(xs=15), SHAPE), (dict(dt=7), UNSUPPORTED), (dict(odt=-1), UNSUPPORTED),
    (dict(k=16385, xs=16385), UNSUPPORTED), (dict(x=None), NULL), (dict(w8=None), NULL), (dict(out=None), NULL),
    (dict(work=None), WORKSPACE), (dict(bytes=39), WORKSPACE), (dict(work=ODD), UNSUPPORTED), (dict(m=0, x=None), 0)])
def test_i8_linear(lib, kw, want):
    assert lib.ah_i8_linear_workspace_bytes(2, 16) == 40  # two rows of codes and their steps
    assert lib.ah_i8_linear(*_with(LINEAR, **kw)) == want


GROUP = dict(leaves=F, n=100, L=4, offsets=F, order=F, work=None, bytes=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), SHAPE), (dict(L=0), SHAPE), (dict(L=4097), UNSUPPORTED), (dict(n=1 << 31), UNSUPPORTED),
    (dict(leaves=None), NULL), (dict(offsets=None), NULL), (dict(order=None), NULL), (dict(n=5000), WORKSPACE),
    (dict(n=5000, work=F, bytes=39), WORKSPACE)])
def test_group_rows(lib, kw, want):
    assert lib.ah_group_rows_workspace_bytes(4096, 4) == 0
    assert lib.ah_group_rows_workspace_bytes(5000, 4) >= 40  # two slices' counts at least, five bins each
    assert lib.ah_group_rows(*_with(GROUP, **kw)) == want


FWD = dict(x=F, xs=8, w=F, L=4, n=6, k=8, offsets=F, order=F, slots=10, fan=2, out=F, odt=1, stream=None)
GROUPED = [
    (dict(slots=-2), SHAPE), (dict(slots=9), SHAPE), (dict(fan=0), SHAPE), (dict(L=0), SHAPE), (dict(n=0), SHAPE),
    (dict(k=0), SHAPE), (dict(order=None), SHAPE), (dict(odt=3), UNSUPPORTED), (dict(L=65537), UNSUPPORTED),
    (dict(slots=1 << 31), UNSUPPORTED), (dict(offsets=None), NULL)]


@pytest.mark.parametrize("kw,want", GROUPED + [
    (dict(xs=7), SHAPE), (dict(n=(1 << 20) + 1), UNSUPPORTED), (dict(x=None), NULL), (dict(w=None), NULL),
    (dict(out=None), NULL), (dict(slots=0, x=None), 0)])
def test_grouped_matmul(lib, kw, want):
    assert lib.ah_grouped_matmul(*_with(FWD, **kw)) == want


DX = dict(dy=F, ds=6, w=F, L=4, n=6, k=8, offsets=F, order=F, slots=10, fan=2, dx=F, odt=1, work=F, bytes=BIG,
          stream=None)


@pytest.mark.parametrize("kw,want", GROUPED + [
    (dict(ds=5), SHAPE), (dict(dy=None), NULL), (dict(w=None), NULL), (dict(dx=None), NULL),
    (dict(work=None), WORKSPACE), (dict(bytes=319), WORKSPACE), (dict(work=ODD), UNSUPPORTED),
    (dict(slots=0, dy=None), 0)])
def test_grouped_matmul_dx(lib, kw, want):
    assert lib.ah_grouped_dx_workspace_bytes(10, 8, 2) == 320  # float32 terms of the shared rows
    assert lib.ah_grouped_dx_workspace_bytes(10, 8, 1) == 0
    assert lib.ah_grouped_matmul_dx(*_with(DX, **kw)) == want


DW = dict(dy=F, ds=6, x=F, xs=8, L=4, n=6, k=8, offsets=F, order=F, slots=10, fan=2, dw=F, odt=0, stream=None)


@pytest.mark.parametrize("kw,want", GROUPED + [
    (dict(ds=5), SHAPE), (dict(xs=7), SHAPE), (dict(dy=None), NULL), (dict(x=None), NULL), (dict(dw=None), NULL)])
def test_grouped_matmul_dw(lib, kw, want):
    assert lib.ah_grouped_matmul_dw(*_with(DW, **kw)) == want


DISTILL = dict(z=F, dt=1, n=3, V=50, zs=50, ids=F, sc=F, k=4, tau=C.c_float(1.0), w=None, loss=F, grad=F, gs=50, work=F,
               bytes=BIG, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), SHAPE), (dict(V=0), SHAPE), (dict(zs=49), SHAPE), (dict(k=0), SHAPE), (dict(gs=49), SHAPE),
    (dict(tau=C.c_float(0.0)), SHAPE), (dict(tau=C.c_float(-1.0)), SHAPE), (dict(tau=C.c_float(float("nan"))), SHAPE),
    (dict(tau=C.c_float(float("inf"))), SHAPE), (dict(tau=C.c_float(1e-31)), UNSUPPORTED), (dict(dt=9), UNSUPPORTED),
    (dict(k=4097), UNSUPPORTED), (dict(V=1 << 31, zs=1 << 31, gs=1 << 31), UNSUPPORTED), (dict(z=None), NULL),
    (dict(ids=None), NULL), (dict(sc=None), NULL), (dict(loss=None), NULL), (dict(n=0, z=None), 0)])
def test_distill_topk(lib, kw, want):
    assert lib.ah_distill_topk(*_with(DISTILL, **kw)) == want


def test_bindings_refuse_host_tensors():
    import torch
    from mips_ah_partition_amd import ahlib as ah
    x = torch.zeros(2, 8)
    for call in (lambda: ah.ah_i8_quantize_rows(x), lambda: ah.ah_group_rows(torch.zeros(4, dtype=torch.int32), 2),
                 lambda: ah.ah_distill_topk(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)),
                 lambda: ah.ah_grouped_matmul(x.bfloat16(), x.bfloat16()[None], torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(TypeError):
            call()
