"""CPU: sizes at the ends of their types, refused by the 16-bit operators before a device is touched."""
import pytest

from quantized_moe_gb300 import ds4moe as api
from test_mm16_refusals import linear_grad, loss, loss_grad


@pytest.mark.parametrize("call", [linear_grad, loss, loss_grad])
@pytest.mark.parametrize("size", [-2 ** 63, -2 ** 63 + 1, -2 ** 62, -1, 0])
def test_no_negative_workspace_passes(call, size):
    with pytest.raises(api.Ds4MoeError) as ei:
        call(workspace_bytes=size)
    assert ei.value.code == api.DS4MOE_ERR_CAPACITY and "workspace_bytes" in str(ei.value)
