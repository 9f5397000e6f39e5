"""Checks of the e4m3 layers that come before any kernel."""
import pytest
import torch

import int8_quantized_matmul_outlier_b200 as m


@pytest.mark.parametrize("shape", [(3, 2, 256), (3, 1, 2, 256), (2, 4, 256)])
def test_a_residual_of_another_shape_is_refused(shape):
    """The rows would be added in storage order: (3, 2) to (2, 3) is a wrong sum, not an error further down."""
    norm = m.RMSNormBlock8bit(256, device="cpu")
    with pytest.raises(ValueError, match="residual of shape"):
        norm(torch.zeros(2, 3, 256, dtype=torch.float16), torch.zeros(*shape, dtype=torch.float16))
