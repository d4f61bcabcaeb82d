"""Dropout's probability at its ends: t = min(rint(65536 p), 65535) numbers of 65,536 are dropped, whatever p below 1 asks for,
and what stays is multiplied by 65536 / (65536 - t).  Bit by bit against the numbers themselves."""
import pytest

from philox_reference import numbers

pytestmark = pytest.mark.gpu
# p and its t: halves go to the even number, and no p below 1 drops everything
ENDS = [(0.0, 0), (0.5 / 65536, 0), (0.51 / 65536, 1), (1.5 / 65536, 2), (2.5 / 65536, 2), (65533.5 / 65536, 65534), (65534.5 / 65536, 65534),
        (65534.51 / 65536, 65535), (65535 / 65536, 65535), (65535.5 / 65536, 65535), (1 - 2.0 ** -20, 65535), (1 - 2.0 ** -53, 65535)]


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mips_ah_partition_amd import ahlib
    ahlib.lib()
    return torch, ahlib


@pytest.mark.parametrize("p,t", ENDS)
def test_dropout(gpu, p, t):
    torch, ah = gpu
    rows, n = 1024, 1025  # 16 of a million numbers are 65535
    keep = torch.from_numpy(numbers(rows, n, 12, 0) >= t).cuda()
    assert keep.any()
    for dt in (torch.float32, torch.bfloat16):
        y = ah.ah_dropout(torch.ones(rows, n, device="cuda", dtype=dt), p, 12)
        want = torch.where(keep, 65536.0 / (65536 - t), 0.0).to(torch.float32).to(dt)
        assert torch.equal(y, want)


@pytest.mark.parametrize("m,k,n", [(40, 64, 1000), (700, 72, 260), (12096, 1024, 512)])
def test_gated(gpu, m, k, n):
    """The gated products drop by the same rule: projections of exactly 2 and 3, relu, hidden values of 6 times the factor."""
    torch, ah = gpu
    x, w = torch.zeros(m, k, device="cuda").bfloat16(), torch.zeros(1, 2 * n, k, device="cuda").bfloat16()
    x[:, 0], w[:, :n, 0], w[:, n:, 0] = 1, 2, 3
    dy, wo = torch.zeros(m, k, device="cuda").bfloat16(), torch.zeros(1, k, n, device="cuda").bfloat16()
    dy[:, 0], wo[:, 0] = 1, 1
    u = torch.from_numpy(numbers(m, n, 5, 0)).cuda()
    for p, t in ((65533.5 / 65536, 65534), (1 - 2.0 ** -20, 65535)):
        f = torch.where(u >= t, 65536.0 / (65536 - t), 0.0)
        for dt in (torch.float32, torch.bfloat16):
            h, pre = ah.ah_grouped_gated(x, w, act="relu", drop=p, seed=5, want_pre=True, out_dtype=dt)
            assert torch.equal(h, (6 * f).to(dt))
        d, h = ah.ah_grouped_gated_grad(dy, wo, pre, act="relu", drop=p, seed=5)
        assert torch.equal(d, torch.cat([3 * f, 2 * f], 1).bfloat16()) and torch.equal(h, (6 * f).bfloat16())
