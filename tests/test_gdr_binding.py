"""CPU checks of the binding of the gated delta rule that need no call."""
import pytest
import torch

from gated_delta_rule_31_amd.gdr import _input


@pytest.mark.parametrize("first", range(1, 8))
def test_only_wide_loads_need_a_border_of_16(first):
    """A tensor on the border that its reader needs is taken as it is, any other copied to one."""
    base = torch.arange(16, dtype=torch.float32)
    assert base.data_ptr() % 16 == 0
    x = base[first : first + 5]
    assert _input(x, "x", base, torch.float32, 4).data_ptr() == x.data_ptr()
    wide = _input(x, "x", base, torch.float32)
    assert wide.data_ptr() % 16 == 0 and torch.equal(wide, x) and (wide.data_ptr() == x.data_ptr()) == (first % 4 == 0)
