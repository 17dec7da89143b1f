"""GPU: the 16-bit operators at their edges, against 64 bits: no rows with the smallest workspace, gradients of rows
that are not finite, closed vocabularies, activations' tails and slopes, sums of many terms."""
import pytest
import torch

from quantized_moe_gb300 import ds4moe as api
from test_gpu_mm16 import DT, ULP, _ce, _ce_check, gen, normal, stream

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


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("pad", [0, 3])
def test_a_weight_that_is_not_finite_stays_in_its_row(dtype, bad, pad):
    """dx[t] depends on row t alone: the other rows' are what they are without the bad one, bit for bit."""
    rows, vocab, d = 37, 600, 72
    x, w = normal((rows, d), dtype, 1, 0.2), normal((vocab, d), dtype, 2, d ** -0.5)
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    dloss = 1.0 + 60000.0 * torch.rand(rows, generator=gen(4), device="cuda")  # (times 2^13, far past fp16)
    dloss[0], dloss[5], dloss[11] = 61001.0, 1e-3, 0.0
    want = _ce(x, w, labels, dloss, dtype, pad=pad)
    _ce_check(x, w, labels, dloss, dtype, want)
    dloss[8] = 0.0
    want = _ce(x, w, labels, dloss, dtype, pad=pad)[2]
    dloss[8] = bad
    loss, lse, dx, dw = _ce(x, w, labels, dloss, dtype, pad=pad)
    others = torch.arange(rows, device="cuda") != 8
    assert torch.equal(dx[others], want[others])
    assert not bool(dx[8].isfinite().any()) and not bool(dw.isfinite().any())
    labels[8] = -100  # without a label it is read by nothing
    loss, lse, dx, dw = _ce(x, w, labels, dloss, dtype, pad=pad)
    assert torch.equal(dx[others], want[others]) and not bool(dx[8].any()) and bool(dw.isfinite().all())


@pytest.mark.parametrize("rows,pad", [(5, 0), (5, 3), (300, 0)])
def test_a_row_of_closed_words_only(rows, pad):
    """A row whose every logit is -inf has lse -inf (the logarithm of an empty sum); NaN logits stay NaN, whatever else
    the row holds; the rows beside them are what they are without them."""
    vocab, d = 700, 72
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    x[:, 0], w[:, 0] = 0.0, 1.0
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    labels[3] = -100
    one = torch.ones(rows, device="cuda")
    clean = _ce(x, w, labels, one, "bf16", pad=pad)
    x[1, 0], x[3, 0] = -float("inf"), -float("inf")  # every word's logit of the row
    x[2, 0] = float("nan")
    loss, lse, dx, dw = _ce(x, w, labels, one, "bf16", pad=pad)
    fine = torch.ones(rows, dtype=torch.bool, device="cuda")
    fine[1:4] = False
    assert torch.equal(lse[fine], clean[1][fine]) and torch.equal(loss[fine], clean[0][fine]) and torch.equal(dx[fine], clean[2][fine])
    assert lse[1] == -float("inf") and lse[3] == -float("inf") and bool(lse[2].isnan())
    assert loss[3] == 0 and not bool(dx[3].any()) and bool(loss[2].isnan())
    assert bool(loss[1].isnan())  # -inf less the label's -inf: no word has a probability


def _dz(z, dy, act, dtype):
    """dy * act'(z), through the gradient's column sums: one row, so that db is dz."""
    n = z.numel()
    size = api.ds4moe_linear_grad_workspace(1, n, act)
    ws, db, dx = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty_like(z), torch.empty((1, 8), dtype=z.dtype, device="cuda")
    w = torch.zeros((n, 8), dtype=z.dtype, device="cuda")
    api.ds4moe_linear_grad(dy, None, w, z, dx, None, db, 1, n, 8, act, dtype, ws, size, stream=stream())
    kept = ws[:2 * n].view(z.dtype)  # dz as the products read it
    assert torch.equal(kept.isnan(), db.isnan()) and torch.equal(kept.nan_to_num(), db.nan_to_num())
    return db


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [8, 13])  # by 16-byte loads, and one by one
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_slopes_where_the_kept_sums_are_not_finite(dtype, act, n):
    """z overflows its type long before the forward's fp32 does: at -inf the slope is 0, at +inf 1, as it is for every
    large z; at NaN it is NaN, as the forward's value is."""
    inf, nan = float("inf"), float("nan")
    z = torch.zeros(n, dtype=torch.float32, device="cuda")
    z[:6] = torch.tensor([inf, -inf, nan, 6e4, -6e4, 1.0])
    dy = torch.full((n,), 0.75, device="cuda").to(z.dtype)
    got = _dz(z.to(DT[dtype]), dy.to(DT[dtype]), act, dtype).float()
    assert got[0] == 0.75 and got[1] == 0 and bool(got[2].isnan()) and got[3] == 0.75 and got[4] == 0
    assert bool(got[5:].isfinite().all())


@pytest.mark.parametrize("n", [8, 13])
def test_relu_passes_nothing_through_a_closed_place(n):
    """Where z <= 0 the gradient is 0 whatever dy holds; where z > 0 it is dy."""
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([-1.0, 0.0, -0.0, -inf, 2.0, 2.0, 2.0, -3.0] + [1.0] * (n - 8), device="cuda").to(torch.bfloat16)
    dy = torch.tensor([inf, -inf, nan, nan, inf, nan, 3.0, 3.0] + [1.0] * (n - 8), device="cuda").to(torch.bfloat16)
    got = _dz(z, dy, "relu", "bf16").float().tolist()
    assert got[:5] == [0.0, 0.0, 0.0, 0.0, inf] and got[5] != got[5] and got[6:] == [3.0, 0.0] + [1.0] * (n - 8)


# exp(-z^2 / 2) by an fp32 exponent: z^2, its way to base 2 and that base's constant are each rounded, 2.5 * 2^-24 of 84.5
# at z = -13, 2^-16.2 of the result; the rest of the arithmetic, 5e-7 and a few units, is less
TAIL = 2.0 ** -15


def _tail(dtype):
    """-13 to 3 in bf16's steps, less what the type cannot hold as a normal result."""
    z = torch.linspace(-13.0, 3.0, 4001, device="cuda").to(torch.bfloat16).unique().to(DT[dtype])
    z = z[z.abs() > 2.0 ** -9]
    return z if dtype == "bf16" else z[z > -3.8]  # gelu(-3.8) = 2^-11.8, and fp16 is normal from 2^-14


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_the_tail_of_gelu(dtype):
    """gelu is relatively exact far into its negative tail, where 1 + erf cancels."""
    z = _tail(dtype)
    n = z.numel()
    one, y, y32 = torch.ones((1, 1), dtype=z.dtype, device="cuda"), torch.empty_like(z), torch.empty_like(z)
    api.ds4moe_linear(z, one, None, None, y, n, 1, 1, "gelu", dtype, stream=stream())
    want = 0.5 * z.double() * torch.special.erfc(-z.double() * 0.5 ** 0.5)
    assert bool(((y.double() - want).abs() <= (ULP[dtype] + TAIL) * want.abs()).all())
    wide, ones = z.repeat(16, 1), torch.eye(16, dtype=z.dtype, device="cuda")  # results by rows: 16 lanes
    out = torch.empty((n, 16), dtype=z.dtype, device="cuda")
    api.ds4moe_linear(wide.T.contiguous(), ones, None, None, out, n, 16, 16, "gelu", dtype, stream=stream())
    assert torch.equal(out, y[:, None].expand(n, 16))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_the_tail_of_gelus_slope(dtype):
    """0.5 erfc(-z / sqrt 2) + z phi(z): the two terms are z^2 times the result's size apart and cancel by it where z is
    far below zero; each is relatively exact."""
    z = _tail(dtype)
    got = _dz(z, torch.ones_like(z), "gelu", dtype).double()
    phi = torch.exp(-0.5 * z.double() ** 2) / (2 * 3.141592653589793) ** 0.5
    cdf = 0.5 * torch.special.erfc(-z.double() * 0.5 ** 0.5)
    want = cdf + z.double() * phi
    off = TAIL * (cdf + (z.double() * phi).abs()) + 2.0 ** -23 * want.abs()
    sub = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -133
    assert bool(((got - want).abs() <= ULP[dtype] * want.abs() + off + sub).all())
