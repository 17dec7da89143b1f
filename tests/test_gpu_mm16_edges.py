"""GPU: the 16-bit operators at their edges, against 64 bits: no rows with the smallest workspace, gradients of rows
that are not finite, closed vocabularies, activations' tails and slopes, sums of many terms."""
import pytest
import torch

from quantized_moe_gb300 import ds4moe as api
from test_gpu_mm16 import DT, ULP, _ce, _ce_check, gen, normal, stream, whole

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


# The tensor cores' fp32 sums cut what they cannot hold instead of rounding: a step of 16 terms loses up to a unit, 2^-23
# of the sum so far. A result may have collected that over 2^14 terms, 2^10 steps of half the sum on average, 2^-14 in
# all; what is added up beyond them is rounded, 2^-24 for each of at most 2^10 additions. On top comes the one rounding
# of the result, and the inputs of these sums are positive, so that the loss cannot average out.
CUT = 2.0 ** -14 + 2.0 ** -14


def _positive(shape, dtype, seed, scale=1.0):
    return ((torch.rand(shape, generator=gen(seed), device="cuda") + 0.5) * scale).to(DT[dtype])


def _check_long(got, a, b, dtype, extra=0.0):
    want = torch.zeros(got.shape, dtype=torch.float64, device="cuda") + extra
    for i in range(0, a.shape[1], 1 << 16):
        want += a[:, i:i + (1 << 16)].double() @ b[:, i:i + (1 << 16)].double().T
    # rounding is monotone: the result lies between the rounded ends of what the fp32 sum may be (the few rounded additions
    # may also lie above, 2^-25 for each of at most 2^8)
    low, high = (want * (1 - CUT)).to(DT[dtype]), (want * (1 + 2.0 ** -17)).to(DT[dtype])
    assert bool(((got >= low) & (got <= high)).all()), float(((got.double() - want) / want).abs().max())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n,k,skew", [((1 << 20) + 21, 72, 136, 0),    # a cluster shares the sum
                                           ((1 << 18) + 5, 72, 136, 1),     # unaligned operands
                                           ((1 << 17) + 100, 1024, 1032, 0)])  # pairs of CTAs
def test_weight_gradients_of_many_rows(dtype, rows, n, k, skew):
    dy, x = _positive((rows * n + skew,), dtype, 1, 2.0 ** -10), _positive((rows * k + skew,), dtype, 2, 2.0 ** -4)
    dyv, xv = dy[skew:].view(rows, n), x[skew:].view(rows, k)
    dw, db = torch.empty((n, k), dtype=x.dtype, device="cuda"), torch.empty(n, dtype=x.dtype, device="cuda")
    size = api.ds4moe_linear_grad_workspace(rows, n)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    api.ds4moe_linear_grad(dy.data_ptr() + 2 * skew, x.data_ptr() + 2 * skew, None, None, None, dw, db, rows, n, k, "none", dtype, ws, size, stream=stream())
    _check_long(dw, dyv.T, xv.T, dtype)
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("skew", [0, 1])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,k", [(136, 72), (520, 264)])
def test_experts_with_many_rows_beside_experts_with_few(dtype, skew, accumulate, n, k):
    counts = [5, (1 << 18) + 37, 0, 130, 16384, 16385, 1, 40000, 64, 300, 0, 33000, 2]
    rows, g = sum(counts), len(counts)
    dy, x = _positive((rows * n + skew,), dtype, 1, 2.0 ** -5), _positive((rows * k + skew,), dtype, 2, 2.0 ** -4)
    dyv, xv = dy[skew:].view(rows, n), x[skew:].view(rows, k)
    dw = torch.full((g, n, k), 1.0, dtype=x.dtype, device="cuda")
    again = dw.clone()
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    for out in (dw, again):
        api.ds4moe_grouped_mm_dw(dy.data_ptr() + 2 * skew, x.data_ptr() + 2 * skew, off, out, rows, n, k, g, dtype, accumulate=accumulate, stream=stream())
    assert torch.equal(dw, again)
    lo = 0
    for e, c in enumerate(counts):
        if c or accumulate:
            _check_long(dw[e], dyv[lo:lo + c].T, xv[lo:lo + c].T, dtype, 1.0 if accumulate else 0.0)
        else:
            assert not bool(dw[e].any())
        lo += c
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("rows,n,skew", [(1, 72, 0), (64, 200, 0), (300, 2056, 0), (33, 72, 1), (600, 1032, 1)])
def test_products_of_long_rows(rows, n, skew):
    """y over k, and dx over n."""
    k, dtype = (1 << 18) + 24, "fp16"
    x, w = _positive((rows * k + skew,), dtype, 1, 2.0 ** -8), _positive((n * k + skew,), dtype, 2, 2.0 ** -6)
    xv, wv = x[skew:].view(rows, k), w[skew:].view(n, k)
    y, z, bias, r = (torch.empty((rows, n), dtype=x.dtype, device="cuda") for _ in range(4))
    bias, r = torch.full((n,), 0.5, dtype=x.dtype, device="cuda"), torch.full((rows, n), 0.25, dtype=x.dtype, device="cuda")
    api.ds4moe_linear(x.data_ptr() + 2 * skew, w.data_ptr() + 2 * skew, bias, r, y, rows, n, k, "relu", dtype, z, stream=stream())
    _check_long(z, xv, wv, dtype, 0.5)
    _check_long(y, xv, wv, dtype, 0.75)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    api.ds4moe_grouped_mm(x.data_ptr() + 2 * skew, w.data_ptr() + 2 * skew, off, y, rows, n, k, 1, dtype, stream=stream())
    _check_long(y, xv, wv, dtype)
    # the same matrices the other way round: w as the gradient [n, k] of n rows, x as weights [k, rows] read across
    wt = torch.empty(k * rows + skew, dtype=x.dtype, device="cuda")
    wt[skew:].view(k, rows).copy_(xv.T)
    dx = torch.empty((n, rows), dtype=x.dtype, device="cuda")
    off = torch.tensor([0, n // 3, n], dtype=torch.int32, device="cuda")
    both = torch.cat([wt[skew:], wt[skew:]])
    src = both if skew == 0 else torch.cat([both[:1], both])
    api.ds4moe_grouped_mm_dx(w.data_ptr() + 2 * skew, src.data_ptr() + 2 * skew, off, dx, n, k, rows, 2, dtype, stream=stream())
    _check_long(dx, wv, xv, dtype)
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("rows,pad", [(3, 0), (130, 0), (20, 1)])
def test_losses_over_long_rows(rows, pad):
    """The logits of a long d, of one sign: a logit may have lost what 2^14 terms cut, and half as much in the loss's own
    shorter sums. The labels' probability and the gradients follow within that error of the exponent."""
    vocab, d = 300, (1 << 17) + 8
    x, w = _positive((rows, d), "bf16", 1, 2.0 ** -8), _positive((vocab, d), "bf16", 2, 2.0 ** -6)
    w *= torch.linspace(0.98, 1.0, vocab, device="cuda")[:, None].to(w.dtype)
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    dloss = torch.ones(rows, device="cuda")
    loss, lse, dx, dw = _ce(x, w, labels, dloss, "bf16", pad=pad)
    z = x.double() @ w.double().T
    want = torch.logsumexp(z, 1)
    # accumulators of 2^11 to 2^12 terms: 2^-17 to 2^-16 of a logit (about 8), rounded additions 2^-24 * 64 more
    tol = (2.0 ** -16 + 2.0 ** -18) * z.max() + 2.0 ** -21 * (1 + want.abs().max())
    assert float((lse - want).abs().max()) <= float(tol)
    own = z.gather(1, labels.long()[:, None])[:, 0]
    assert float((loss - (want - own)).abs().max()) <= 2 * float(tol)
    p = torch.softmax(z, 1)
    dz = p.scatter_add(1, labels.long()[:, None], -torch.ones((rows, 1), dtype=torch.float64, device="cuda"))
    for got, ref, terms in ((dx, dz @ w.double(), dz.abs() @ w.double()), (dw, dz.T @ x.double(), dz.abs().T @ x.double())):
        # the exponents are off by the logit's and the lse's error, dz is rounded (2^-9), the result too
        assert bool(((got.double() - ref).abs() <= ULP["bf16"] * ref.abs() + (2.0 ** -9 + CUT * z.max() + tol + 2.0 ** -14) * terms + 1e-30).all())
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("n,k", [(1024, 1024), (2304, 512), (1000, 520), (4096, 256), (2056, 1544)])
@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
def test_weight_gradients_of_one_group(n, k, out_dtype):
    """One group's last round of tiles is not split as a dense product's is, whatever width its tiles have."""
    rows, used = 300, 287
    x, dy = whole((rows, k), "bf16", 1), whole((rows, n), "bf16", 2)
    x[used:], dy[used:] = float("nan"), float("nan")
    dw = torch.full((n * k + 64,), 7.0, dtype=DT[out_dtype], device="cuda")
    off = torch.tensor([0, used], dtype=torch.int32, device="cuda")
    api.ds4moe_grouped_mm_dw(dy, x, off, dw, rows, n, k, 1, "bf16", out_dtype, stream=stream())
    assert torch.equal(dw[:n * k].view(n, k), (dy[:used].double().T @ x[:used].double()).to(DT[out_dtype]))
    assert bool((dw[n * k:] == 7.0).all()) and api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("rows,vocab,d,pad,dtype", [
    (16, 80001, 2056, 0, "bf16"), (1, 45000, 4096, 0, "fp16"), (128, 45000, 4096, 0, "bf16"), (16, 80001, 4104, 0, "bf16"),
    (100, 41000, 6200, 0, "fp16"), (20, 45000, 2100, 3, "bf16"), (200, 41000, 4200, 3, "fp16")])
def test_losses_of_few_rows_over_a_wide_model(rows, vocab, d, pad, dtype):
    """A token's logits take two accumulators side by side (d above 2048) or one after the other (above 4096), on
    single CTAs, and there are more tiles of the vocabulary than SMs: both accumulators are used again."""
    x, w = normal((rows, d), dtype, 1), normal((vocab, d), dtype, 2, 2.0 * d ** -0.5)
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    if rows > 1:
        labels[::7] = -100
        labels[1], labels[rows - 1] = vocab - 1, 0
    dloss = torch.rand(rows, generator=gen(4), device="cuda") / rows
    got = _ce(x, w, labels, dloss, dtype, pad=pad)
    _ce_check(x, w, labels, dloss, dtype, got)
    again = _ce(x, w, labels, dloss, dtype, pad=pad)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("rows,d,pad", [(16, 512, 0), (40, 520, 0), (9, 136, 3), (33, 1000, 0)])
@pytest.mark.parametrize("piece", [768, 1024, 2560])
def test_pieces_that_split_their_sums_over_a_cluster(rows, d, pad, piece):
    """dx of few rows, piece after piece of the vocabulary: each piece's sum is shared out over the CTAs of a cluster and
    added to the one before it in fp32."""
    vocab = 10007
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    labels[::5] = -100
    dloss = torch.rand(rows, generator=gen(4), device="cuda")
    size = 16 + (4 * rows * d + 15) // 16 * 16 + 2 * ((rows + 7) // 8 * 8) * piece
    _ce_check(x, w, labels, dloss, "bf16", _ce(x, w, labels, dloss, "bf16", ws_bytes=size, pad=pad))
    assert api.ds4moe_ops_status() == 0


def test_graphs_whose_calls_follow_fills_and_copies():
    """Captured behind a fill and a copy, which are no kernels: each call still sees what they wrote."""
    rows, n, k = 40, 136, 72
    x, w, dy = whole((rows, k), "bf16", 1), whole((n, k), "bf16", 2), whole((rows, n), "bf16", 3)
    src, y, dw, db, dw0, db0 = torch.zeros_like(x), torch.empty_like(dy), torch.empty_like(w), torch.empty_like(w[:, 0].contiguous()), torch.ones_like(w), torch.ones_like(w[:, 0].contiguous())
    size = api.ds4moe_linear_grad_workspace(rows, n)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    acc = torch.empty((1, n, k), device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")

    def calls():
        s = stream()
        src.copy_(x)
        api.ds4moe_linear(src, w, None, None, y, rows, n, k, stream=s)
        src.zero_()
        src[1:].copy_(x[1:])
        api.ds4moe_linear_grad(dy, src, w, None, None, dw, db, rows, n, k, workspace=ws, workspace_bytes=size, stream=s)
        acc.zero_()
        api.ds4moe_grouped_mm_dw(dy, x, off, acc, rows, n, k, 1, dw_dtype="fp32", accumulate=True, stream=s)
        api.ds4moe_linear_grad(None, None, None, None, None, dw0, db0, 0, n, k, workspace=ws, workspace_bytes=16, stream=s)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        for t in (src, y, dw, db, dw0, db0, acc):
            t.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, (x.double() @ w.double().T).to(y.dtype))
        assert torch.equal(dw, (dy[1:].double().T @ x[1:].double()).to(dw.dtype)) and torch.equal(db, dy.double().sum(0).to(db.dtype))
        assert torch.equal(acc[0].double(), dy.double().T @ x.double())
        assert not bool(dw0.any()) and not bool(db0.any())
    assert api.ds4moe_ops_status() == 0
