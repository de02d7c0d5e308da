"""CPU checks of what the Python side of gift_mx_* refuses before it looks at
a device: anything but an MxOperand where an operand is asked for."""

import pytest
import torch

import fac_whitening_gift_amd as fg

STREAM = object()   # never reached


@pytest.mark.parametrize("stream", [None, STREAM])
@pytest.mark.parametrize("bad", [None, 3, torch.zeros(64, 128)])
def test_operands_are_operands(bad, stream):
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError, match="w must be an MxOperand"):
        fg.gift_mx_linear(x, bad, stream=stream)
    with pytest.raises(ValueError, match="a must be an MxOperand"):
        fg.gift_mx_matmul(bad, bad, stream=stream)
    with pytest.raises(ValueError, match="a must be an MxOperand"):
        fg.gift_mx_dequantize(bad, stream=stream)


def test_an_operand_lives_on_a_device():
    """A host buffer behind an operand would reach the kernels as an address."""
    x = torch.zeros(64, 128)
    with pytest.raises(ValueError, match="device tensor"):
        fg.MxOperand(64, 128, like=x)
    with pytest.raises(ValueError, match="device tensor"):
        fg.MxOperand(64, 128, device="cpu")
    with pytest.raises(ValueError, match="device tensor"):
        fg.MxOperand(64, 128, data=torch.zeros(4352, dtype=torch.uint8))
