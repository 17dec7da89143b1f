"""GPU: the operators on 16-bit matrices against plain 64-bit forms.

Two kinds of comparison. With small whole numbers as inputs every partial sum is a whole number
below 2^24, exact in fp32 whatever the order, so a result must equal the correctly rounded 64-bit
one bit for bit. With ordinary inputs an element may be off by the rounding of its type
(2^-8 |v| in bf16, 2^-11 |v| in fp16: half a unit in the last of 8 or 11 bits, doubled for a value
that sits next to a rounding boundary) plus the fp32 sum's error, at most 2^-23 of the sum of the
terms' magnitudes for each of the r additions.
"""
import math

import pytest
import torch

from quantized_moe_gb300 import ds4moe as api

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ULP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
NAN = float("nan")


def stream():
    return torch.cuda.current_stream().cuda_stream


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(shape, dtype, seed, most=2):
    return torch.randint(-most, most + 1, shape, generator=gen(seed), device="cuda").to(DT[dtype])


def normal(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(DT[dtype])


def strided(t, ld, fill=NAN, skew=0):
    """t's values in a buffer of row distance ld, `skew` elements into it, everything else `fill`."""
    rows, cols = t.shape[-2], t.shape[-1]
    n = t.numel() // max(1, rows * cols) if t.dim() == 3 else 1
    buf = torch.full((skew + n * rows * ld + 64,), fill, dtype=t.dtype, device="cuda")
    view = buf[skew:skew + n * rows * ld].view(*t.shape[:-1], ld)[..., :cols]
    view.copy_(t)
    return buf, view


def offsets(counts):
    return torch.tensor([0] + list(counts), dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def groups_of(counts):
    lo = 0
    for g, c in enumerate(counts):
        yield g, lo, lo + c
        lo += c


COUNTS = {"one": [1], "eights": [0, 1, 0, 1, 1, 0, 0, 1], "ragged": [0, 1, 130, 0, 257, 16, 15, 17, 0],
          "long": [700, 0, 3], "none": [0, 0, 0]}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("direction", ["y", "dx", "dw"])
@pytest.mark.parametrize("pattern,n,k,pad,skew", [
    ("one", 64, 64, 0, 0), ("one", 1, 1, 0, 0), ("eights", 136, 72, 8, 0), ("ragged", 264, 200, 0, 0),
    ("ragged", 129, 77, 0, 0), ("ragged", 40, 328, 24, 8), ("ragged", 40, 328, 3, 1), ("long", 128, 128, 0, 0),
    ("long", 300, 72, 5, 0), ("none", 64, 72, 0, 0)])
def test_grouped_products_of_whole_numbers_are_exact(dtype, direction, pattern, n, k, pad, skew):
    counts = COUNTS[pattern]
    used = sum(counts)
    rows, g = used + 5, len(counts)  # five rows at the end belong to no group: NaN there, untouched outputs
    off = offsets(counts)
    x, dy, w = whole((rows, k), dtype, 1), whole((rows, n), dtype, 2), whole((g, n, k), dtype, 3)
    x[used:], dy[used:] = NAN, NAN
    (xb, xv), (db, dyv), (wb, wv) = strided(x, k + pad, skew=skew), strided(dy, n + pad, skew=skew), strided(w, k + pad, skew=skew)
    es = x.element_size()
    ptr = lambda b: b.data_ptr() + skew * es
    if direction == "dw":
        for out_dtype in (dtype, "fp32"):
            for accumulate in (False, True):
                start = whole((g, n, k), out_dtype, 4)
                ob, ov = strided(start, k + pad, fill=7.0)
                api.ds4moe_grouped_mm_dw(ptr(db), ptr(xb), off, ob, rows, n, k, g, dtype, out_dtype, accumulate,
                                         lddy=n + pad, ldx=k + pad, lddw=k + pad, stream=stream())
                want = torch.stack([dy[lo:hi].double().T @ x[lo:hi].double() for _, lo, hi in groups_of(counts)])
                want = want + start.double() if accumulate else want
                assert torch.equal(ov, want.to(DT[out_dtype]))
                ov.fill_(7.0)
                assert bool((ob == 7.0).all())  # nothing was written between the rows
    else:
        cols, wid, src = (n, k, ptr(xb)) if direction == "y" else (k, n, ptr(db))
        ob, ov = strided(torch.full((rows, cols), 7.0, dtype=DT[dtype], device="cuda"), cols + pad, fill=7.0)
        fn = api.ds4moe_grouped_mm if direction == "y" else api.ds4moe_grouped_mm_dx
        fn(src, ptr(wb), off, ob, rows, n, k, g, dtype, wid + pad, k + pad, 0, cols + pad, stream=stream())
        for e, lo, hi in groups_of(counts):
            want = x[lo:hi].double() @ w[e].double().T if direction == "y" else dy[lo:hi].double() @ w[e].double()
            assert torch.equal(ov[lo:hi], want.to(DT[dtype])), (e, lo, hi)
        assert bool((ov[used:] == 7.0).all())
        ov.fill_(7.0)
        assert bool((ob == 7.0).all())
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("direction", ["y", "dx", "dw"])
def test_a_row_that_is_not_finite_stays_in_its_row_or_group(direction):
    counts, n, k = [30, 3, 0, 131], 136, 200
    rows, g = sum(counts), len(counts)
    x, dy, w = normal((rows, k), "bf16", 1), normal((rows, n), "bf16", 2), normal((g, n, k), "bf16", 3, k ** -0.5)
    x[31, 5], dy[31, 5] = math.inf, NAN  # the middle row of group 1
    out = {"y": torch.empty((rows, n), dtype=x.dtype, device="cuda"), "dx": torch.empty_like(x),
           "dw": torch.empty_like(w)}[direction]
    if direction == "y":
        api.ds4moe_grouped_mm(x, w, offsets(counts), out, rows, n, k, g, stream=stream())
    elif direction == "dx":
        api.ds4moe_grouped_mm_dx(dy, w, offsets(counts), out, rows, n, k, g, stream=stream())
    else:
        api.ds4moe_grouped_mm_dw(dy, x, offsets(counts), out, rows, n, k, g, stream=stream())
    bad = ~torch.isfinite(out.float()).flatten(1).all(1)
    assert bad.nonzero().flatten().tolist() == ([1] if direction == "dw" else [31])


def test_offsets_out_of_order_or_range_reach_nothing_outside():
    n, k, rows = 72, 64, 40
    x, w = whole((rows, k), "bf16", 1), whole((4, n, k), "bf16", 2)
    y = torch.full((rows, n), 7.0, dtype=x.dtype, device="cuda")
    off = torch.tensor([-5, 10, 3, 90, 2 ** 31 - 1], dtype=torch.int32, device="cuda")  # clamped: 0-10, -, 3-40, -
    api.ds4moe_grouped_mm(x, w, off, y, rows, n, k, 4, stream=stream())
    assert torch.equal(y[10:], (x[10:].double() @ w[2].double().T).to(x.dtype))
    dw = torch.empty_like(w)
    api.ds4moe_grouped_mm_dw(y, x, off, dw, rows, n, k, 4, stream=stream())
    assert bool((dw[1] == 0).all()) and bool((dw[3] == 0).all())


def _tolerance(ref, terms, r, dtype):
    return ULP[dtype] * ref.abs() + (r + 8) * 2.0 ** -23 * terms + 1e-30


ACTS64 = {"none": lambda z: z, "relu": torch.nn.functional.relu, "silu": torch.nn.functional.silu,
          "gelu": torch.nn.functional.gelu}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("rows,n,k,pad,bias,residual,keep", [
    (1, 64, 128, 0, True, True, True), (1, 1, 1, 0, True, False, True), (2, 1000, 520, 0, False, True, False),
    (16, 136, 200, 8, True, True, True), (17, 129, 77, 0, True, True, True), (130, 264, 72, 3, False, False, True),
    (300, 128, 64, 0, True, True, False), (513, 40, 264, 0, True, False, True)])
def test_linear(dtype, act, rows, n, k, pad, bias, residual, keep):
    x, w = normal((rows, k), dtype, 1), normal((n, k), dtype, 2, k ** -0.5)
    b = normal((n,), dtype, 3) if bias else None
    r = normal((rows, n), dtype, 4) if residual else None
    xb, _ = strided(x, k + pad)
    wb, _ = strided(w, k + pad)
    rb = strided(r, n + pad)[0] if residual else None
    y, yv = strided(torch.full((rows, n), 7.0, dtype=x.dtype, device="cuda"), n + pad, fill=7.0)
    z, zv = strided(torch.full((rows, n), 7.0, dtype=x.dtype, device="cuda"), n + pad, fill=7.0)
    api.ds4moe_linear(xb, wb, b, rb, y, rows, n, k, act, dtype, z if keep else None, ldx=k + pad, ldw=k + pad,
                      ldr=n + pad, ldy=n + pad, ldz=n + pad, stream=stream())
    ref = x.double() @ w.double().T + (b.double() if bias else 0)
    terms = x.double().abs() @ w.double().abs().T + (b.double().abs() if bias else 0)
    want = ACTS64[act](ref) + (r.double() if residual else 0)
    # |act'| <= 1.13; silu and gelu are evaluated to a few units of 2^-22 of their terms
    slack = 1.13 * _tolerance(0 * ref, terms, k, dtype) + 2.0 ** -20 * (ref.abs() + (r.double().abs() if residual else 0))
    assert bool(((yv.double() - want).abs() <= ULP[dtype] * want.abs() + slack + 2.0 ** -25).all())
    if keep:
        assert bool(((zv.double() - ref).abs() <= _tolerance(ref, terms, k, dtype) + 2.0 ** -25).all())
    yv.fill_(7.0), zv.fill_(7.0)
    assert bool((y == 7.0).all()) and bool((z == 7.0).all())
    assert api.ds4moe_ops_status() == 0


def test_linear_adds_into_the_residual_in_place():
    x, w, r = whole((33, 72), "bf16", 1), whole((80, 72), "bf16", 2), whole((33, 80), "bf16", 3)
    want = (x.double() @ w.double().T + r.double()).to(x.dtype)
    api.ds4moe_linear(x, w, None, r, r, 33, 80, 72, stream=stream())
    assert torch.equal(r, want)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_linear_of_extreme_values(act):
    """Large and infinite pre-activations saturate as the activation does; NaN stays NaN."""
    z = torch.tensor([0.0, -0.0, 88.0, -88.0, 1e4, -1e4, 3e38, math.inf, NAN], device="cuda").to(torch.bfloat16)
    one = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((9, 1), dtype=torch.bfloat16, device="cuda")
    api.ds4moe_linear(z.reshape(9, 1), one, None, None, y, 9, 1, 1, act, stream=stream())
    want = ACTS64[act](z.double())
    got = y.flatten().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert bool(((got - want)[fine & want.isfinite()].abs() <= 2.0 ** -8 * want[fine & want.isfinite()].abs() + 1e-30).all())
    assert torch.equal(got[fine & want.isinf()], want[fine & want.isinf()])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("rows,n,k,pad,want", [(1, 64, 72, 0, "xwb"), (5, 1, 3, 0, "xwb"), (130, 136, 264, 8, "xwb"),
                                               (257, 77, 129, 0, "xwb"), (300, 200, 64, 3, "xwb"),
                                               (700, 64, 128, 0, "b"), (64, 72, 80, 0, "x"), (64, 72, 80, 0, "w")])
def test_linear_gradients(dtype, act, rows, n, k, pad, want):
    dy, x, w, z = normal((rows, n), dtype, 1), normal((rows, k), dtype, 2), normal((n, k), dtype, 3, k ** -0.5), normal((rows, n), dtype, 4)
    new = lambda *s: strided(torch.full(s, 7.0, dtype=x.dtype, device="cuda"), s[1] + pad, fill=7.0)
    (dxb, dxv), (dwb, dwv) = new(rows, k), new(n, k)
    db = torch.full((n,), 7.0, dtype=x.dtype, device="cuda")
    size = api.ds4moe_linear_grad_workspace(rows, n, act)
    ws = torch.full((size + 16,), 255, dtype=torch.uint8, device="cuda")
    api.ds4moe_linear_grad(strided(dy, n + pad)[0], strided(x, k + pad)[0], strided(w, k + pad)[0],
                           None if act == "none" else strided(z, n + pad)[0], dxb if "x" in want else None,
                           dwb if "w" in want else None, db if "b" in want else None, rows, n, k, act, dtype, ws, size,
                           lddy=n + pad, ldx=k + pad, ldw=k + pad, ldz=n + pad, lddx=k + pad, lddw=k + pad,
                           stream=stream())
    assert bool((ws[size:] == 255).all())
    z64 = z.double().requires_grad_()
    dz = dy.double() if act == "none" else torch.autograd.grad(ACTS64[act](z64), z64, dy.double())[0]
    # dz is rounded to 16 bits before the products (2^-8 or 2^-11 of each term; fp16 also loses what
    # lies below half its smallest subnormal, 2^-25) and its slope carries a few units of 2^-22
    u = 0.0 if act == "none" else ULP[dtype]
    sub = 2.0 ** -25 if dtype == "fp16" and act != "none" else 0.0
    err = lambda a, b: u * (a.abs() @ b.abs()) + 2.0 ** -18 * (dy.double().abs().T.max() * torch.ones_like(a).abs() @ b.abs() if act != "none" else 0) + sub * (torch.ones_like(a) @ b.abs())
    if "x" in want:
        ref = dz @ w.double()
        tol = _tolerance(ref, dz.abs() @ w.double().abs(), n, dtype) + err(dz, w.double()) + 2.0 ** -25
        assert bool(((dxv.double() - ref).abs() <= tol).all())
    if "w" in want:
        ref = dz.T @ x.double()
        tol = _tolerance(ref, dz.T.abs() @ x.double().abs(), rows, dtype) + err(dz.T, x.double()) + 2.0 ** -25
        assert bool(((dwv.double() - ref).abs() <= tol).all())
    if "b" in want:
        ref = dz.sum(0)
        tol = _tolerance(ref, dz.abs().sum(0), rows, dtype) + 2.0 ** -18 * dy.double().abs().sum(0) + 2.0 ** -25
        assert bool(((db.double() - ref).abs() <= tol).all())
    dxv.fill_(7.0), dwv.fill_(7.0)
    assert bool((dxb == 7.0).all()) and bool((dwb == 7.0).all())


def test_linear_gradients_of_no_rows_are_zero():
    dw, db = torch.ones((8, 16), dtype=torch.bfloat16, device="cuda"), torch.ones(8, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 12, dtype=torch.uint8, device="cuda")
    api.ds4moe_linear_grad(None, None, None, None, None, dw, db, 0, 8, 16, "silu", workspace=ws, workspace_bytes=ws.numel(), stream=stream())
    assert not bool(dw.any()) and not bool(db.any())
    dw.fill_(1)
    api.ds4moe_grouped_mm_dw(None, None, offsets([0, 0]), dw, 0, 4, 16, 2, stream=stream())
    assert not bool(dw.any())


def test_linear_gradients_against_differences():
    """The loss sum(c * y) moved along a direction of x, w and bias: a central difference of the 64-bit
    forward (its error is h^2 f''' / 6, about 1e-8 at h = 1e-4) against the kernels' gradients."""
    rows, n, k = 24, 40, 56
    x, w, b, c = normal((rows, k), "bf16", 1), normal((n, k), "bf16", 2, k ** -0.5), normal((n,), "bf16", 3), normal((rows, n), "bf16", 4)
    y, z = torch.empty((rows, n), dtype=x.dtype, device="cuda"), torch.empty((rows, n), dtype=x.dtype, device="cuda")
    api.ds4moe_linear(x, w, b, None, y, rows, n, k, "gelu", zout=z, stream=stream())
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    size = api.ds4moe_linear_grad_workspace(rows, n, "gelu")
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    api.ds4moe_linear_grad(c, x, w, z, dx, dw, db, rows, n, k, "gelu", workspace=ws, workspace_bytes=size, stream=stream())
    f = lambda x, w, b: (c.double() * torch.nn.functional.gelu(x @ w.T + b)).sum()
    at, h = [x.double(), w.double(), b.double()], 1e-4
    for i, got in enumerate((dx, dw, db)):
        v = torch.randn(at[i].shape, generator=gen(9 + i), device="cuda", dtype=torch.float64)
        hi, lo = [t + h * v if j == i else t for j, t in enumerate(at)], [t - h * v if j == i else t for j, t in enumerate(at)]
        want, have = (f(*hi) - f(*lo)) / (2 * h), (got.double() * v).sum()
        # the kept z, dz and the results are each rounded to bf16: 3 * 2^-9 of each term on average;
        # the terms' errors are independent, four of their standard deviations are allowed
        assert abs(have - want) <= 4 * 3 * 2.0 ** -9 * (got.double() * v).norm() + 1e-6


def _ce(x, w, labels, dloss, dtype, ignore=-100, ws_bytes=None, pad=0, want="xw"):
    (rows, d), vocab = x.shape, w.shape[0]
    loss, lse = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    size = api.ds4moe_cross_entropy_workspace(rows, vocab, d)
    ws = torch.full((size + 16,), 255, dtype=torch.uint8, device="cuda")
    xb, wb = strided(x, d + pad)[0], strided(w, d + pad)[0]
    api.ds4moe_cross_entropy(xb, wb, labels, loss, lse, rows, vocab, d, dtype, ignore, ws, size, d + pad, d + pad, stream=stream())
    dxb, dx = strided(torch.full((rows, d), 7.0, dtype=x.dtype, device="cuda"), d + pad, fill=7.0)
    dwb, dw = strided(torch.full((vocab, d), 7.0, dtype=x.dtype, device="cuda"), d + pad, fill=7.0)
    api.ds4moe_cross_entropy_grad(xb, wb, labels, lse, dloss, dxb if "x" in want else None, dwb if "w" in want else None,
                                  rows, vocab, d, dtype, ignore, ws, ws_bytes or size, d + pad, d + pad, d + pad, d + pad,
                                  stream=stream())
    assert bool((ws[size:] == 255).all())
    out = (loss, lse, dx.clone(), dw.clone())
    dx.fill_(7.0), dw.fill_(7.0)
    assert bool((dxb == 7.0).all()) and bool((dwb == 7.0).all())
    return out


def _ce_check(x, w, labels, dloss, dtype, got, ignore=-100):
    loss, lse, dx, dw = got
    d, vocab = x.shape[1], w.shape[0]
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    z = x64 @ w64.T
    kept = (labels != ignore) & (labels >= 0) & (labels < vocab)
    at = torch.where(kept, labels, 0).long()[:, None]
    want_lse = torch.logsumexp(z, 1)
    want = torch.where(kept, want_lse - z.gather(1, at)[:, 0], 0.0)
    # a logit's error: d additions; the lse's: the largest logit's and the sum's, a few units of 2^-22
    zerr = (d + 8) * 2.0 ** -23 * (x64.abs() @ w64.abs().T).max(1).values.detach()
    tol = 2 * zerr + 2.0 ** -21 * (1 + want_lse.abs() + z.abs().max(1).values).detach()
    assert bool(((lse - want_lse).abs() <= tol).all())
    assert bool(((loss - want).abs() <= 2 * tol).all())
    assert bool((loss[~kept] == 0).all())
    g = torch.where(kept, dloss.double(), 0.0)
    gx, gw = torch.autograd.grad((want * g).sum(), (x64, w64))
    p = torch.softmax(z, 1).detach()
    hot = torch.zeros_like(p).scatter_(1, at, 1.0)
    dz = ((p - hot) * g[:, None]).abs()
    # each dz: its rounding, the exponential of a logit and an lse that are off (by tol in all), and in
    # fp16, scaled to max |g| = 2^13, half the smallest subnormal
    gmax = g.abs().max()
    off = ULP[dtype] * dz + (2 * tol[:, None] + 2.0 ** -20) * p * g.abs()[:, None] + 2.0 ** -21 * dz + (2.0 ** -25 * 2.0 ** -13 * gmax if dtype == "fp16" else 0)
    sub = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -130
    if dx is not None:
        lim = _tolerance(gx, dz @ w64.abs().detach(), vocab, dtype) + off @ w64.abs().detach() + sub
        assert bool(((dx.double() - gx).abs() <= lim).all())
        assert not bool(dx[~kept].any())
    if dw is not None:
        lim = _tolerance(gw, dz.T @ x64.abs().detach(), x.shape[0], dtype) + off.T @ x64.abs().detach() + sub
        assert bool(((dw.double() - gw).abs() <= lim).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,d,pad", [(1, 1, 1, 0), (1, 1000, 64, 0), (16, 1003, 72, 0), (3, 257, 129, 0),
                                              (130, 777, 200, 8), (129, 640, 77, 3), (300, 9001, 64, 0)])
def test_cross_entropy(dtype, rows, vocab, d, pad):
    x, w = normal((rows, d), dtype, 1), normal((vocab, d), dtype, 2, 2.0 * d ** -0.5)
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    labels[::7] = -100
    if rows > 1:
        labels[1], labels[rows - 1] = vocab - 1, 0
    dloss = torch.rand(rows, generator=gen(4), device="cuda") / rows
    _ce_check(x, w, labels, dloss, dtype, _ce(x, w, labels, dloss, dtype, pad=pad))
    assert api.ds4moe_ops_status() == 0


def test_cross_entropy_in_small_pieces_of_the_vocabulary():
    rows, vocab, d = 70, 2000, 136
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    dloss = torch.ones(rows, device="cuda")
    small = 16 + 4 * rows * d + 2 * ((rows + 7) // 8 * 8) * 256  # the documented smallest size: 256 words a piece
    _ce_check(x, w, labels, dloss, "bf16", _ce(x, w, labels, dloss, "bf16", ws_bytes=small))
    with pytest.raises(api.Ds4MoeError) as ei:
        _ce(x, w, labels, dloss, "bf16", ws_bytes=small - 600)
    assert ei.value.code == api.DS4MOE_ERR_CAPACITY


def test_cross_entropy_ignored_and_foreign_labels():
    rows, vocab, d = 40, 500, 64
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    dloss = torch.ones(rows, device="cuda")
    labels = torch.full((rows,), 7, device="cuda", dtype=torch.int32)  # every row ignored, by a label in range
    loss, lse, dx, dw = _ce(x, w, labels, dloss, "bf16", ignore=7)
    assert not bool(loss.any()) and not bool(dx.any()) and not bool(dw.any()) and bool(lse.isfinite().all())
    assert api.ds4moe_ops_status() == 0
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    labels[4], labels[5] = vocab, -1
    _ce_check(x, w, labels, dloss, "bf16", _ce(x, w, labels, dloss, "bf16"))
    assert api.ds4moe_ops_status() == 1
    assert api.ds4moe_ops_status() == 0


def test_cross_entropy_of_large_logits_and_closed_words():
    """Logits in the thousands do not overflow; words closed by an infinitely negative logit add nothing."""
    rows, vocab, d = 20, 700, 64
    x = normal((rows, d), "bf16", 1).abs() + 0.1
    w = normal((vocab, d), "bf16", 2, 60.0)
    w[64:300, 3] = -math.inf  # whole tiles of the vocabulary
    labels = torch.randint(300, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    loss, lse, dx, dw = _ce(x, w, labels, torch.ones(rows, device="cuda"), "bf16", want="w")
    z = x.double() @ torch.where(w.isinf(), 0, w).double().T
    z[:, 64:300] = -math.inf
    want = torch.logsumexp(z, 1)
    assert bool(((lse - want).abs() <= 2.0 ** -14 * want.abs()).all())
    assert bool(loss.isfinite().all())
    assert not bool(dw[64:300].any()) and bool(dw.isfinite().all())


def test_cross_entropy_small_gradients_do_not_vanish_in_fp16():
    rows, vocab, d = 64, 4000, 64
    x, w = normal((rows, d), "fp16", 1), normal((vocab, d), "fp16", 2, 0.5 * d ** -0.5)
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    loss, lse, dx, dw = _ce(x, w, labels, torch.full((rows,), 1.0, device="cuda"), "fp16")
    few = _ce(x, w, labels, torch.full((rows,), 2.0 ** -30, device="cuda"), "fp16")
    # dz keeps the same bits under a power of two; only the results round (to zero, here)
    assert torch.equal(few[2], (dx.double() * 2.0 ** -30).to(torch.float16))
    other = _ce(x, w, labels, torch.full((rows,), 2.0 ** -9, device="cuda"), "fp16")[3].double() * 2.0 ** 9
    assert bool(((other - dw.double()).abs() <= 2.0 ** -11 * dw.double().abs() + 2.0 ** -25 * 2 ** 9).all())


def test_cross_entropy_gradient_against_differences():
    rows, vocab, d = 12, 300, 40
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    c = torch.rand(rows, generator=gen(4), device="cuda")
    _, _, dx, dw = _ce(x, w, labels, c, "bf16")
    f = lambda x, w: (c.double() * torch.nn.functional.cross_entropy(x @ w.T, labels.long(), reduction="none")).sum()
    at, h = [x.double(), w.double()], 1e-4
    for i, got in enumerate((dx, dw)):
        v = torch.randn(at[i].shape, generator=gen(9 + i), device="cuda", dtype=torch.float64)
        hi, lo = [t + h * v if j == i else t for j, t in enumerate(at)], [t - h * v if j == i else t for j, t in enumerate(at)]
        want, have = (f(*hi) - f(*lo)) / (2 * h), (got.double() * v).sum()
        # dz and the result are each rounded to bf16 (2^-9 of a term on average); four deviations
        assert abs(have - want) <= 4 * 2 * 2.0 ** -9 * (got.double() * v).norm() + 1e-6


def test_results_repeat_bit_for_bit_on_other_streams_and_in_graphs():
    rows, n, k, vocab = 200, 520, 328, 3000
    counts = [0, 3, 150, 47]
    x, w, dy = normal((rows, k), "bf16", 1), normal((4, n, k), "bf16", 2, k ** -0.5), normal((rows, n), "bf16", 3)
    head = normal((vocab, k), "bf16", 4, k ** -0.5)
    labels = torch.randint(0, vocab, (rows,), generator=gen(5), device="cuda", dtype=torch.int32)
    g = torch.ones(rows, device="cuda")
    off = offsets(counts)
    size = api.ds4moe_cross_entropy_workspace(rows, vocab, k)
    lsize = api.ds4moe_linear_grad_workspace(rows, n, "silu")

    def buffers():
        e = lambda *s, dt=torch.bfloat16: torch.full(s, 9.0, dtype=dt, device="cuda")
        return [e(rows, n), e(rows, k), e(4, n, k), e(rows, n), e(rows, k), e(n, k), e(n), e(rows, dt=torch.float32),
                e(rows, dt=torch.float32), e(rows, k), e(vocab, k)], [torch.empty(s, dtype=torch.uint8, device="cuda") for s in (size, lsize)]

    def calls(o, ws):
        s = stream()
        api.ds4moe_grouped_mm(x, w, off, o[0], rows, n, k, 4, stream=s)
        api.ds4moe_grouped_mm_dx(dy, w, off, o[1], rows, n, k, 4, stream=s)
        api.ds4moe_grouped_mm_dw(dy, x, off, o[2], rows, n, k, 4, stream=s)
        api.ds4moe_linear(x, w[0], None, dy, o[3], rows, n, k, "gelu", stream=s)
        api.ds4moe_linear_grad(dy, x, w[1], dy, o[4], o[5], o[6], rows, n, k, "silu", workspace=ws[1], workspace_bytes=lsize, stream=s)
        api.ds4moe_cross_entropy(x, head, labels, o[7], o[8], rows, vocab, k, workspace=ws[0], workspace_bytes=size, stream=s)
        api.ds4moe_cross_entropy_grad(x, head, labels, o[8], g, o[9], o[10], rows, vocab, k, workspace=ws[0], workspace_bytes=size, stream=s)

    first, ws = buffers()
    calls(first, ws)
    torch.cuda.synchronize()
    sets = [buffers() for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for st, (o, ws) in zip(streams, sets):
            with torch.cuda.stream(st):
                calls(o, ws)
    torch.cuda.synchronize()
    for o, _ in sets:
        for a, b in zip(first, o):
            assert torch.equal(a, b)
    o, ws = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(o, ws)
    for _ in range(2):
        for t in o:
            t.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, o):
            assert torch.equal(a, b)


def test_pointers_that_are_not_this_devices_memory_are_refused():
    x = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")
    host = torch.zeros((8, 8), dtype=torch.bfloat16)
    for bad in (host, host.pin_memory()):
        with pytest.raises(api.Ds4MoeError) as ei:
            api.ds4moe_linear(x, bad, None, None, x, 4, 8, 8, stream=stream())
        assert ei.value.code == api.DS4MOE_ERR_INVALID_ARG and "w is not device memory" in str(ei.value)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n,k,pad", [(1, 4096, 4096, 0), (3, 256, 2048, 0), (32, 384, 1096, 8), (33, 200, 4104, 0),
                                          (64, 1000, 520, 0), (7, 130, 1001, 0), (64, 513, 2001, 0)])
def test_few_rows_split_over_the_reduction(dtype, rows, n, k, pad):
    """Few tiles share out the reduction among the CTAs of a cluster; whole numbers stay exact."""
    x, w, b, r = whole((rows, k), dtype, 1), whole((n, k), dtype, 2), whole((n,), dtype, 3), whole((rows, n), dtype, 4)
    y, z = torch.empty((rows, n), dtype=x.dtype, device="cuda"), torch.empty((rows, n), dtype=x.dtype, device="cuda")
    api.ds4moe_linear(strided(x, k + pad)[0], strided(w, k + pad)[0], b, r, y, rows, n, k, "relu", dtype, z, ldx=k + pad, ldw=k + pad, stream=stream())
    ref = x.double() @ w.double().T + b.double()
    assert torch.equal(z, ref.to(x.dtype))
    assert torch.equal(y, (ref.clamp(min=0) + r.double()).to(x.dtype))
    counts = [0, rows // 2, 0, rows - rows // 2]
    wg = whole((4, n, k), dtype, 5)
    api.ds4moe_grouped_mm(x, wg, offsets(counts), y, rows, n, k, 4, dtype, stream=stream())
    want = torch.cat([x[lo:hi].double() @ wg[g].double().T for g, lo, hi in groups_of(counts)])
    assert torch.equal(y, want.to(x.dtype))
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("counts,n,k", [([128] * 40, 1024, 1024), ([5, 0, 64, 200, 0, 33] * 12, 520, 1304), ([700] * 9, 2048, 640)])
def test_many_small_weight_gradients(counts, n, k):
    """Enough output tiles that the two halves of the epilogue take whole tiles in turn, empty groups among them."""
    rows, g = sum(counts), len(counts)
    x, dy = whole((rows, k), "bf16", 1), whole((rows, n), "bf16", 2)
    for out_dtype in ("bf16", "fp32"):
        dw = torch.full((g, n, k), 7.0, dtype=DT[out_dtype], device="cuda")
        api.ds4moe_grouped_mm_dw(dy, x, offsets(counts), dw, rows, n, k, g, "bf16", out_dtype, stream=stream())
        for e, lo, hi in groups_of(counts):
            assert torch.equal(dw[e], (dy[lo:hi].double().T @ x[lo:hi].double()).to(DT[out_dtype])), e
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("rows,n,k", [(1100, 4000, 264), (2500, 2056, 64), (4096, 520, 200)])
def test_uneven_schedules(rows, n, k):
    """Sizes whose last round of tiles is partial, so that it is split over its columns."""
    x, w, dy = whole((rows, k), "bf16", 1), whole((n, k), "bf16", 2), whole((rows, n), "bf16", 3)
    y = torch.empty((rows, n), dtype=x.dtype, device="cuda")
    api.ds4moe_linear(x, w, None, None, y, rows, n, k, stream=stream())
    assert torch.equal(y, (x.double() @ w.double().T).to(x.dtype))
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(n, dtype=x.dtype, device="cuda")
    size = api.ds4moe_linear_grad_workspace(rows, n)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    api.ds4moe_linear_grad(dy, x, w, None, dx, dw, db, rows, n, k, workspace=ws, workspace_bytes=size, stream=stream())
    assert torch.equal(dx, (dy.double() @ w.double()).to(x.dtype))
    assert torch.equal(dw, (dy.double().T @ x.double()).to(x.dtype))
    assert torch.equal(db, dy.double().sum(0).to(x.dtype))


@pytest.mark.parametrize("rows,n,k", [(3100, 1536, 3400), (2600, 4096, 2312)])
def test_larger_gradients(rows, n, k):
    """Several rounds of tiles over the SMs, whole numbers exact."""
    x, w, dy = whole((rows, k), "bf16", 1), whole((n, k), "bf16", 2), whole((rows, n), "bf16", 3)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    size = api.ds4moe_linear_grad_workspace(rows, n)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    api.ds4moe_linear_grad(dy, x, w, None, dx, dw, None, rows, n, k, workspace=ws, workspace_bytes=size, stream=stream())
    assert torch.equal(dx, (dy.double() @ w.double()).to(x.dtype))
    assert torch.equal(dw, (dy.double().T @ x.double()).to(x.dtype))
    assert api.ds4moe_ops_status() == 0


def test_larger_cross_entropy_gradients_in_pieces():
    rows, vocab, d = 2100, 5000, 2304
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    dloss = torch.full((rows,), 1.0 / rows, device="cuda")
    small = 16 + 4 * rows * d + 2 * ((rows + 7) // 8 * 8) * 2048  # several pieces
    _ce_check(x, w, labels, dloss, "bf16", _ce(x, w, labels, dloss, "bf16", ws_bytes=small))


def test_offsets_past_32_bits():
    """Rows and matrices that lie further apart than 2^31 elements."""
    rows, n, k, ld = 2200, 72, 64, 1 << 20
    x = whole((rows, k), "bf16", 1)
    far = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    far.view(rows, ld)[:, :k] = x
    w = whole((2, n, k), "bf16", 2)
    counts = [1000, rows - 1000]
    out = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    want = torch.cat([x[lo:hi].double() @ w[g].double().T for g, lo, hi in groups_of(counts)]).to(x.dtype)
    for skew in (0, 1):  # by the TMA unit, and by ordinary loads and stores
        src = far if skew == 0 else torch.cat([far[:skew], far])[:rows * ld]
        api.ds4moe_grouped_mm(src.data_ptr() + 2 * skew, w, offsets(counts), out.data_ptr() + 2 * skew, rows - skew, n, k, 2, ldx=ld, ldy=ld, stream=stream())
        got = out[skew:skew + (rows - skew - 1) * ld + n].as_strided((rows - skew, n), (ld, 1))
        assert torch.equal(got, want[:rows - skew])
    del far, out
    stride = (1 << 31) + 64
    wide = torch.empty(stride + n * k, dtype=torch.bfloat16, device="cuda")
    wide[:n * k], wide[stride:] = w[0].flatten(), w[1].flatten()
    y = torch.empty((rows, n), dtype=x.dtype, device="cuda")
    api.ds4moe_grouped_mm(x, wide, offsets(counts), y, rows, n, k, 2, w_stride=stride, stream=stream())
    assert torch.equal(y, want)
    dw = torch.empty(stride + n * k, dtype=torch.bfloat16, device="cuda")
    api.ds4moe_grouped_mm_dw(y, x, offsets(counts), dw, rows, n, k, 2, dw_stride=stride, stream=stream())
    for g, lo, hi in groups_of(counts):
        assert torch.equal(dw[g * stride:g * stride + n * k].view(n, k), (y[lo:hi].double().T @ x[lo:hi].double()).to(x.dtype))


@pytest.mark.parametrize("direction", ["y", "dw"])
def test_a_thousand_groups(direction):
    g, n, k = 1024, 40, 72
    counts = torch.randint(0, 4, (g,), generator=torch.Generator().manual_seed(1)).tolist()
    rows = sum(counts)
    x, dy, w = whole((rows, k), "fp16", 1), whole((rows, n), "fp16", 2), whole((g, n, k), "fp16", 3)
    if direction == "y":
        y = torch.empty((rows, n), dtype=x.dtype, device="cuda")
        api.ds4moe_grouped_mm(x, w, offsets(counts), y, rows, n, k, g, "fp16", stream=stream())
        of = torch.repeat_interleave(torch.arange(g), torch.tensor(counts)).cuda()
        assert torch.equal(y, torch.einsum("tk,tnk->tn", x.double(), w[of].double()).to(x.dtype))
    else:
        dw = torch.empty_like(w)
        api.ds4moe_grouped_mm_dw(dy, x, offsets(counts), dw, rows, n, k, g, "fp16", stream=stream())
        want = torch.stack([dy[lo:hi].double().T @ x[lo:hi].double() for _, lo, hi in groups_of(counts)])
        assert torch.equal(dw, want.to(x.dtype))


def test_cross_entropy_of_no_rows():
    dw = torch.ones((30, 16), dtype=torch.bfloat16, device="cuda")
    api.ds4moe_cross_entropy_grad(None, None, None, None, None, None, dw, 0, 30, 16, stream=stream())
    assert not bool(dw.any())


def test_a_chain_of_calls_sees_each_others_results():
    """Launches may overlap their set-up; every one still reads what the one before it wrote, in place too."""
    rows, n = 96, 256
    w = (torch.eye(n, device="cuda") * 2).to(torch.bfloat16)
    a, b = whole((rows, n), "bf16", 1), torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")
    want = a.clone()
    for _ in range(8):
        api.ds4moe_linear(a, w, None, None, b, rows, n, n, stream=stream())  # b = 2 a
        api.ds4moe_linear(b, w, None, a, a, rows, n, n, stream=stream())     # a = 4 a + a
        want = (want.double() * 5).to(torch.bfloat16)
    # (5^8 times small whole numbers is rounded on the way, by both alike)
    assert torch.equal(a, want)
