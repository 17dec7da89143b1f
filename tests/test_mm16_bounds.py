"""CPU: sizes at the ends of their types and tensors that the call does not describe, refused by the 16-bit operators
before a device is touched."""
import pytest
import torch

from quantized_moe_gb300 import ds4moe as api
from test_mm16_refusals import grouped, grouped_dw, linear, linear_grad, loss, loss_grad


@pytest.mark.parametrize("call", [linear_grad, loss, loss_grad])
@pytest.mark.parametrize("size", [-2 ** 63, -2 ** 63 + 1, -2 ** 62, -1, 0])
def test_no_negative_workspace_passes(call, size):
    with pytest.raises(api.Ds4MoeError) as ei:
        call(workspace_bytes=size)
    assert ei.value.code == api.DS4MOE_ERR_CAPACITY and "workspace_bytes" in str(ei.value)


A = torch.zeros((3, 8, 8), dtype=torch.bfloat16)
WIDE = torch.zeros((6, 8, 16), dtype=torch.bfloat16)


@pytest.mark.parametrize("call,kw", [
    (linear, dict(w=A[0].T)), (linear, dict(x=WIDE[0, :4, ::2])), (linear, dict(x=WIDE[0, :4, :8])),
    (linear, dict(x=WIDE[0, :4, :8], ldx=8)), (linear, dict(y=WIDE[0, :4, 8:], ldy=17)), (linear, dict(bias=WIDE[0, 0, ::2])),
    (linear, dict(bias=WIDE[0, 0, :1].expand(8))), (linear, dict(residual=A[0, :4].expand(4, 8)[:, ::2])),
    (linear, dict(zout=WIDE[0, :4, :8])), (grouped, dict(w=WIDE[:2, :, :8])), (grouped, dict(w=WIDE[::2, :, :8], ldw=16)),
    (grouped, dict(w=WIDE[::2, :, :8], ldw=16, w_stride=128)), (grouped, dict(w=A[:1].expand(2, 8, 8))),
    (grouped, dict(w=A.transpose(1, 2)[:2])), (grouped_dw, dict(dw=A[::2])), (grouped_dw, dict(dy=A[0, :4].T)),
    (linear_grad, dict(db=WIDE[0, 0, ::2])), (linear_grad, dict(z=A[0].T)), (loss, dict(x=A[0].T)),
    (loss_grad, dict(dloss=torch.ones(1).expand(4))), (loss_grad, dict(dw=WIDE[0, :, :8])),
])
def test_views_whose_strides_the_call_does_not_give_are_refused(call, kw):
    with pytest.raises(ValueError, match="strides"):
        call(**kw)


@pytest.mark.parametrize("call,kw", [
    (linear, dict(x=WIDE[0, :4, 8:], ldx=16)), (linear, dict(x=WIDE[:2, :2, :8].contiguous())), (linear, dict(w=WIDE[0, :, :8], ldw=16)),
    (linear, dict(x=WIDE[:2, :, 8:], ldx=16)), (linear, dict(x=A[0, :1].expand(1, 8))), (linear, dict(y=A.flatten())),
    (grouped, dict(w=WIDE[::2, :, :8], ldw=16, w_stride=256)), (grouped, dict(w=WIDE[:2, :, :8], ldw=16)), (grouped_dw, dict(dw=A[::2], dw_stride=128)),
    (linear, dict(w=torch.zeros((1, 8)).T[:8], k=1, x=torch.zeros((4, 1)), n=8)), (linear_grad, dict(db=torch.zeros(8))),
])
def test_views_that_the_call_describes_pass(call, kw):
    """They reach the library, which refuses host memory (or the lack of a device)."""
    with pytest.raises(api.Ds4MoeError) as ei:
        call(**kw)
    assert ei.value.code in (api.DS4MOE_ERR_INVALID_ARG, api.DS4MOE_ERR_CUDA)
    assert "device" in str(ei.value).lower() or "driver" in str(ei.value).lower()
