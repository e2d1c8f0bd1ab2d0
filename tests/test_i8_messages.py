"""What the 8-bit calls say when they refuse."""
import pytest

import ternary_weight_only_amd as tq
from ternary_weight_only_amd import binding
from tests.test_i8_args import _lib


@pytest.mark.parametrize("bad", ["tanh", 2, True, ["silu"]])
def test_every_activation_is_named(bad):
    """An unknown activation: the message has all that the call takes."""
    with pytest.raises(tq.TQError) as e:
        binding._act_i8(bad)
    for name in binding.ACTS_I8:
        assert repr(name) in str(e.value), name


def test_an_act_that_another_call_takes():
    """The gated calls refuse two values that are activations: the text of the
    status does not say that they are none."""
    lib = _lib()
    fake, big = 0x100000, 1 << 40  # never dereferenced
    rc = lib.tq_glu(fake, fake, fake, fake, fake, 3, 5, 128, 64, binding.ACTS_I8["relu2"], fake, fake, big, None, None)
    text = lib.tq_status_string(rc).decode()
    assert text.startswith("TQ_ERR_ACT") and "not a tq_act value that the call takes" in text
