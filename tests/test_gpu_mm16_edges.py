"""GPU: the 16-bit operators at their edges, against 64 bits: no rows with the smallest workspace, gradients of rows
that are not finite, closed vocabularies, activations' tails and slopes, sums of many terms."""
import pytest
import torch

from quantized_moe_gb300 import ds4moe as api
from test_gpu_mm16 import ULP, gen, normal, stream

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,act", [(1000, "silu"), (1000, "none"), (8, "gelu"), (1, "relu"), (40001, "silu")])
def test_gradients_of_no_rows_stay_inside_the_workspace(n, act):
    """The documented workspace, exactly, at the front of a larger buffer: the bytes after it are not touched, nor are
    those after the results."""
    k = 24
    size = api.ds4moe_linear_grad_workspace(0, n, act)
    buf = torch.full((size + (1 << 20),), 255, dtype=torch.uint8, device="cuda")
    dw, db = torch.ones(n * k + 64, dtype=torch.bfloat16, device="cuda"), torch.ones(n + 64, dtype=torch.bfloat16, device="cuda")
    api.ds4moe_linear_grad(None, None, None, None, None, dw, db, 0, n, k, act, workspace=buf, workspace_bytes=size, stream=stream())
    assert bool((buf[size:] == 255).all())
    assert not bool(dw[:n * k].any()) and bool((dw[n * k:] == 1).all())
    assert not bool(db[:n].any()) and bool((db[n:] == 1).all())
    assert api.ds4moe_ops_status() == 0
