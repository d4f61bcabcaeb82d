"""Status codes of the learned query side's calls at the ends of their accepted ranges (checked on the host,
before anything is enqueued; no GPU needed, no pointer is dereferenced)."""
import ctypes as C

import pytest

vp = C.c_void_p
SHAPE, UNSUPPORTED, WORKSPACE = -2, -3, -4
F = vp(4096)


@pytest.fixture(scope="module")
def lib():
    from mips_ah_partition_amd import ahlib
    return ahlib.lib()


@pytest.mark.parametrize("tau,want", [
    (1e30, UNSUPPORTED), (3e38, UNSUPPORTED), (1e-31, UNSUPPORTED), (1e-45, UNSUPPORTED),
    (9.9e29, WORKSPACE), (1.1e-30, WORKSPACE), (1.0, WORKSPACE),  # in range: the next check, a missing workspace
    (float("inf"), SHAPE), (float("nan"), SHAPE), (-float("inf"), SHAPE), (0.0, SHAPE), (-1e30, SHAPE)])
def test_distillation_temperature(lib, tau, want):
    n, V, k = 3, 50000, 4
    assert lib.ah_distill_workspace_bytes(n, V, k) > 0
    assert lib.ah_distill_topk(F, 1, n, V, V, F, F, k, C.c_float(tau), None, F, F, V, None, 0, None) == want
