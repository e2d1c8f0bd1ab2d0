"""What the 8-bit calls say when they refuse."""
import pytest

import ternary_weight_only_amd as tq
from ternary_weight_only_amd import binding


@pytest.mark.parametrize("bad", ["tanh", 2, True, ["silu"]])
def test_every_activation_is_named(bad):
    """An unknown activation: the message has all that the call takes."""
    with pytest.raises(tq.TQError) as e:
        binding._act_i8(bad)
    for name in binding.ACTS_I8:
        assert repr(name) in str(e.value), name
