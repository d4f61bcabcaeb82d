"""A NaN among the kept projections reaches every gradient made from it, with each activation; the elements beside it, and
dropped ones, do not change."""
import pytest

from philox_reference import factors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mips_ah_partition_amd import ahlib
    ahlib.lib()
    return torch, ahlib


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("drop", [0.0, 0.5])
@pytest.mark.parametrize("m,d,n", [(6, 64, 24), (300, 7, 33), (12096, 128, 1024)])
def test_gradient(gpu, m, d, n, drop, act):
    torch, ah = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    dy, w, pre = rnd(m, d), rnd(1, d, n), rnd(m, 2 * n)
    want, wh = ah.ah_grouped_gated_grad(dy, w, pre, act=act, drop=drop, seed=8)
    bad = pre.clone()
    bad[1, 3], bad[4, 17], bad[m - 1, n + 5] = float("nan"), float("nan"), float("nan")  # two gates, one up
    got, h = ah.ah_grouped_gated_grad(dy, w, bad, act=act, drop=drop, seed=8)
    keep = torch.from_numpy(factors(m, n, drop, 8, 0)).cuda() > 0
    nan = torch.zeros(m, 2 * n, dtype=torch.bool, device="cuda")
    for r, c in ((1, 3), (4, 17)):  # da = dh b act'(a), db = dh act(a)
        nan[r, c] = nan[r, n + c] = keep[r, c]
    nan[m - 1, 5] = keep[m - 1, 5]  # da alone: db has no b
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])
    hnan = nan[:, :n]
    assert torch.equal(torch.isnan(h), hnan) and torch.equal(h[~hnan], wh[~hnan])


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("m", [6, 300])
def test_forward(gpu, m, act):
    torch, ah = gpu
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    x, w = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((m, 16), (1, 20, 16)))
    want, _ = ah.ah_grouped_gated(x, w, act=act)
    x[3, 2] = float("nan")
    h, pre = ah.ah_grouped_gated(x, w, act=act, want_pre=True)
    others = torch.arange(m, device="cuda") != 3
    assert torch.isnan(h[3]).all() and torch.isnan(pre[3]).all() and torch.equal(h[others], want[others])
