"""What the binding of the serving calls takes for a tensor (no GPU needed)."""
import numpy as np
import pytest

import hybrid_attention_ssm_hymba_b200 as H

P = 1 << 20   # an aligned address that nothing may read


@pytest.mark.parametrize("thing", [b"0123456789abcdef", "0123456789abcdef", bytearray(16), np.zeros(4), [1, 2], 1.0])
def test_only_tensors_and_addresses_are_pointers(thing):
    """bytes and str would pass as pointers to host memory, which a kernel would read."""
    with pytest.raises(AttributeError):
        H.hymba_rmsnorm(thing, P, 1, 16, 1e-5, H.HYMBA_BF16, stream=0)
    with pytest.raises(AttributeError):
        H.hymba_quantize_w4(P, thing, P, 16, 128, 64, H.HYMBA_BF16, stream=0)
    with pytest.raises(AttributeError):
        H.hymba_workspace_status(thing, stream=0)
