"""GPU: 16-bit products whose operands start at any element, with everything that can be done to their results: whole numbers,
whose sums fp32 holds exactly, must come out as the rounded 64-bit ones."""
import pytest
import torch

from quantized_moe_gb300 import ds4moe as api
from test_gpu_mm16 import DT, NAN, groups_of, offsets, stream, strided, whole

pytestmark = pytest.mark.gpu


def at(t, cols, pad, skew):
    """(buffer, address) of a matrix with rows cols + pad apart that starts skew elements into its buffer."""
    buf, _ = strided(t, cols + pad, skew=skew)
    return buf, buf.data_ptr() + skew * t.element_size()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("counts,n,k", [([7] * 6, 40, 72), ([9, 0, 3, 140, 1], 136, 77), ([1500, 17, 0, 515], 33, 129), ([64, 16], 300, 1001), ([2], 1, 1)])
@pytest.mark.parametrize("gap", [0, 3])
def test_weight_gradients(dtype, out, accumulate, counts, n, k, gap):
    rows, g = sum(counts) + 5, len(counts)
    dy, x = whole((rows, n), dtype, 1), whole((rows, k), dtype, 2)
    dy[sum(counts):], x[sum(counts):] = NAN, NAN
    (db, pdy), (xb, px) = at(dy, n, 1, 1), at(x, k, 1, 1)
    old = whole((g, n, k), "bf16", 3, 1).to(torch.float32 if out == "fp32" else DT[dtype])
    buf, dw = strided(old, k + gap, fill=7.0)
    api.ds4moe_grouped_mm_dw(pdy, px, offsets(counts), buf, rows, n, k, g, dtype, "fp32" if out == "fp32" else None, accumulate, n + 1, k + 1, k + gap, 0, stream())
    for e, lo, hi in groups_of(counts):
        want = dy[lo:hi].double().T @ x[lo:hi].double() + (old[e].double() if accumulate else 0)
        assert torch.equal(dw[e], want.to(dw.dtype)), e
    dw.fill_(7.0)
    assert bool((buf == 7.0).all()) and api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n,k", [(1, 64, 63), (33, 72, 199), (200, 264, 65), (300, 1000, 575), (129, 77, 129), (2, 513, 1023), (16, 2048, 1023), (260, 1, 9)])
@pytest.mark.parametrize("bias,residual,z,gap", [(True, False, True, 0), (False, True, False, 0), (True, True, True, 0), (False, False, False, 0), (True, True, True, 5)])
def test_dense_products(dtype, rows, n, k, bias, residual, z, gap):
    x, w, b, r = whole((rows, k), dtype, 1), whole((n, k), dtype, 2), whole((n,), dtype, 3), whole((rows, n), dtype, 4)
    (xb, px), (wb, pw) = at(x, k, 1, 1), at(w, k, 2, 1)
    (yb, y), (zb, zv) = (strided(torch.full_like(r, 7.0), n + gap, fill=7.0) for _ in range(2))
    rb, _ = strided(r, n + gap)
    api.ds4moe_linear(px, pw, b if bias else None, rb if residual else None, yb, rows, n, k, "relu", dtype, zb if z else None, k + 1, k + 2, n + gap, n + gap,
                      n + gap, stream())
    want = x.double() @ w.double().T + (b.double() if bias else 0)
    assert torch.equal(y, (want.clamp(min=0) + (r.double() if residual else 0)).to(y.dtype))
    if z:
        assert torch.equal(zv, want.to(zv.dtype))
    y.fill_(7.0), zv.fill_(7.0)
    assert bool((yb == 7.0).all()) and bool((zb == 7.0).all()) and api.ds4moe_ops_status() == 0
