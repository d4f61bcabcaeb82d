"""What QueryHead.step refuses before it looks at its batch (no GPU needed)."""
import pytest


def _head(trunk_type):
    from mips_ah_partition_amd.query_head import QueryHead
    head = QueryHead.__new__(QueryHead)
    head.trunk_type = trunk_type
    return head


@pytest.mark.parametrize("trunk_type", ["i8", "f8"])
@pytest.mark.parametrize("want_dx", ["Hidden", "features", "", "x"])
def test_unknown_gradient(trunk_type, want_dx):
    with pytest.raises(ValueError, match="want_dx"):
        _head(trunk_type).step(None, None, None, None, want_dx=want_dx)


@pytest.mark.parametrize("kw", [dict(want_dx="hidden"), dict(trunk_lr=0.1), dict(want_dx=True, trunk_lr=-0.1)])
def test_int8_trunk_has_no_gradient(kw):
    with pytest.raises(ValueError, match="8-bit float"):
        _head("i8").step(None, None, None, None, **kw)
