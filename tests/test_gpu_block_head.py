"""GPU: the gated block, the scores and the distillation against plain 64-bit forms.

Whole numbers, or 8-bit numbers on a grid, have products and sums that fp32 holds exactly: results must equal the
correctly rounded 64-bit ones, and the order of logits, ties among them, is known. Ordinary numbers: a result may be off
by half a step of its type (2^-8 |v| in bf16, 2^-11 |v| in fp16) plus the fp32 sums' errors, at most 2^-23 of the terms'
magnitudes for each addition.
"""
import math

import pytest
import torch

from quantized_moe_gb300 import ds4moe as api
from test_gpu_mm16 import ACTS64, COUNTS, DT, NAN, ULP, _tolerance, gen, groups_of, normal, offsets, strided, stream, whole

pytestmark = pytest.mark.gpu


def full(shape, dtype="fp32", v=7.0):
    return torch.full(shape, v, dtype=DT[dtype], device="cuda")


# ------------------------------------------------------------------------------------------ gated block


def block(x, w, off, n, act, dtype, pad=0, skew=0, keep=True, rows=None):
    """(h, z, whether anything beside the results was written) through buffers with gaps."""
    (g, n2, k), rows = w.shape, x.shape[0]
    xb, _ = strided(x, k + pad, skew=skew)
    wb, _ = strided(w, k + pad, skew=skew)
    hb, h = strided(full((rows, n), dtype), n + pad, fill=7.0)
    zb, z = strided(full((rows, n2), dtype), n2 + pad, fill=7.0)
    es = x.element_size()
    api.ds4moe_grouped_glu(xb.data_ptr() + skew * es, wb.data_ptr() + skew * es, off, hb, rows, n, k, g, act, dtype,
                           zb if keep else None, k + pad, k + pad, 0, n + pad, n2 + pad, stream())
    out = h.clone(), z.clone()
    h.fill_(7.0), z.fill_(7.0)
    return out + (bool((hb == 7.0).all()) and bool((zb == 7.0).all()),)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("pattern,n,k,pad,skew", [
    ("one", 64, 64, 0, 0), ("one", 1, 1, 0, 0), ("eights", 72, 72, 8, 0), ("ragged", 264, 200, 0, 0), ("ragged", 129, 77, 0, 0),
    ("ragged", 40, 328, 24, 8), ("ragged", 40, 328, 3, 1), ("long", 128, 128, 0, 0), ("long", 300, 72, 5, 0), ("long", 17, 64, 0, 0),
    ("none", 64, 72, 0, 0), ("dense", 96, 136, 0, 0), ("dense", 257, 65, 3, 1), ("dense", 1000, 72, 0, 0)])
def test_blocks_of_whole_numbers_are_exact(dtype, act, pattern, n, k, pad, skew):
    counts = COUNTS.get(pattern, [333])
    used, g = sum(counts), len(counts)
    rows = used + (0 if pattern == "dense" else 5)  # five rows at the end belong to no group
    x, w = whole((rows, k), dtype, 1), whole((g, 2 * n, k), dtype, 3)
    x[used:] = NAN
    h, z, clean = block(x, w, None if pattern == "dense" else offsets(counts), n, act, dtype, pad, skew)
    assert clean
    for e, lo, hi in groups_of(counts):
        ref = x[lo:hi].double() @ w[e].double().T
        assert torch.equal(z[lo:hi], ref.to(DT[dtype])), (e, lo, hi)
        assert torch.equal(h[lo:hi], (ACTS64[act](ref[:, :n]) * ref[:, n:]).to(DT[dtype])), (e, lo, hi)
    assert bool((h[used:] == 7.0).all()) and bool((z[used:] == 7.0).all())
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("counts,n,k,pad", [([1], 256, 2048, 0), ([0, 7, 120, 1], 136, 520, 0), ([300], 1000, 72, 0), ([31, 33], 77, 129, 0),
                                            ([64, 0, 5], 24, 4104, 8)])
def test_blocks(dtype, act, counts, n, k, pad):
    rows, g = sum(counts), len(counts)
    x, w = normal((rows, k), dtype, 1), normal((g, 2 * n, k), dtype, 2, 2 * k ** -0.5)
    h, _, clean = block(x, w, offsets(counts), n, act, dtype, pad, keep=False)
    assert clean
    for e, lo, hi in groups_of(counts):
        ref, terms = x[lo:hi].double() @ w[e].double().T, x[lo:hi].double().abs() @ w[e].double().abs().T
        a, b = ref[:, :n], ref[:, n:]
        want = ACTS64[act](a) * b
        # |act'| <= 1.13; each factor's sum is off by so much, act by a few units of 2^-22 of its argument
        ea, eb = 1.13 * (k + 8) * 2.0 ** -23 * terms[:, :n] + 2.0 ** -20 * a.abs(), (k + 8) * 2.0 ** -23 * terms[:, n:]
        lim = ULP[dtype] * want.abs() + ea * b.abs() + eb * ACTS64[act](a).abs() + ea * eb + 2.0 ** -22 * want.abs() + 2.0 ** -25
        assert bool(((h[lo:hi].double() - want).abs() <= lim).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("counts,n,k,pad,dense", [
    ([1], 64, 72, 0, True), ([130], 136, 264, 8, True), ([257], 77, 129, 0, True), ([300], 200, 64, 3, True), ([0, 3, 150, 0, 17], 72, 136, 0, False),
    ([5, 260], 33, 65, 0, False), ([40, 1, 0], 1, 8, 5, False), ([0, 0], 24, 40, 0, False)])
def test_block_gradients(dtype, act, counts, n, k, pad, dense):
    used, g = sum(counts), len(counts)
    rows = used + (0 if dense else 3)
    dh, x, z, w = normal((rows, n), dtype, 1), normal((rows, k), dtype, 2), normal((rows, 2 * n), dtype, 3), normal((g, 2 * n, k), dtype, 4, k ** -0.5)
    dh[used:], x[used:], z[used:] = NAN, NAN, NAN
    (dzb, dz), (dxb, dx), (dwb, dw) = (strided(full(s, dtype), s[-1] + pad, fill=7.0) for s in ((rows, 2 * n), (rows, k), (g, 2 * n, k)))
    off = None if dense else offsets(counts)
    api.ds4moe_grouped_glu_grad(strided(dh, n + pad)[0], strided(x, k + pad)[0], strided(w, k + pad)[0], off, strided(z, 2 * n + pad)[0], dzb, dxb,
                                dwb, rows, n, k, g, act, dtype, n + pad, k + pad, k + pad, 0, 2 * n + pad, 2 * n + pad, k + pad, k + pad, 0, stream())
    assert bool((dz[used:] == 7.0).all()) and bool((dx[used:] == 7.0).all())
    z64 = z[:used].double().requires_grad_()
    a, b = z64.chunk(2, 1)
    (want,) = torch.autograd.grad(ACTS64[act](a) * b, z64, dh[:used].double())
    d64, zd = dh[:used].double().abs(), z64.detach().abs()
    # a slope is off by a few units of 2^-22 of 1 and of its argument, act by as much of its argument
    slack = 2.0 ** -18 * torch.cat([d64 * zd[:, n:] * (1 + zd[:, :n]), d64 * zd[:, :n]], 1)
    assert bool(((dz[:used].double() - want).abs() <= ULP[dtype] * want.abs() + slack + 2.0 ** -25).all())
    got = dz[:used].double()  # what the products read
    for e, lo, hi in groups_of(counts):
        ref, terms = got[lo:hi] @ w[e].double(), got[lo:hi].abs() @ w[e].double().abs()
        assert bool(((dx[lo:hi].double() - ref).abs() <= _tolerance(ref, terms, 2 * n, dtype) + 2.0 ** -25).all())
        ref, terms = got[lo:hi].T @ x[lo:hi].double(), got[lo:hi].abs().T @ x[lo:hi].double().abs()
        assert bool(((dw[e].double() - ref).abs() <= _tolerance(ref, terms, hi - lo, dtype) + 2.0 ** -25).all())
    for v in (dz, dx, dw):
        v.fill_(7.0)
    assert all(bool((v == 7.0).all()) for v in (dzb, dxb, dwb))
    assert api.ds4moe_ops_status() == 0


def test_block_gradients_one_at_a_time_and_in_place():
    counts, n, k, g = [20, 0, 45], 64, 136, 3
    rows = sum(counts)
    dh, x, z, w = normal((rows, n), "bf16", 1), normal((rows, k), "bf16", 2), normal((rows, 2 * n), "bf16", 3), normal((g, 2 * n, k), "bf16", 4, k ** -0.5)
    new = lambda like: torch.full_like(like, 7.0)  # noqa: E731
    dz, dx, dw = new(z), new(x), new(w)
    sizes = dict(rows=rows, n=n, k=k, n_groups=g, act="silu", stream=stream())
    api.ds4moe_grouped_glu_grad(dh, x, w, offsets(counts), z, dz, dx, dw, **sizes)
    dz1, dx1, dw1 = new(z), new(x), new(w)
    api.ds4moe_grouped_glu_grad(dh, None, w, offsets(counts), z, dz1, dx1, None, **sizes)
    assert torch.equal(dz, dz1) and torch.equal(dx, dx1)
    z2 = z.clone()
    api.ds4moe_grouped_glu_grad(dh, x, None, offsets(counts), z2, z2, None, dw1, **sizes)  # dz in z's place
    assert torch.equal(dz, z2) and torch.equal(dw, dw1)
    # dz serves the grouped product's gradient, in fp32 and added to an older one
    old = torch.randn((g, 2 * n, k), generator=gen(5), device="cuda")
    acc = old.clone()
    api.ds4moe_grouped_mm_dw(dz, x, offsets(counts), acc, rows, 2 * n, k, g, dw_dtype="fp32", accumulate=True, stream=stream())
    want = torch.stack([dz[lo:hi].double().T @ x[lo:hi].double() for _, lo, hi in groups_of(counts)]) + old.double()
    assert bool(((acc.double() - want).abs() <= 2.0 ** -16 * (1 + want.abs())).all())


def test_block_gradients_of_no_rows_are_zero():
    for off in (None, offsets([0])):
        dw = full((1, 16, 24), "bf16")
        api.ds4moe_grouped_glu_grad(None, None, None, off, None, None, None, dw, 0, 8, 24, stream=stream())
        assert not bool(dw.any())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_block_gradients_against_differences(act):
    """sum(c * h) moved along a direction of x and w: a central difference of the 64-bit forward (error about 1e-8 at
    h = 1e-4) against the kernels' gradients."""
    rows, n, k = 24, 40, 56
    x, w, c = normal((rows, k), "bf16", 1), normal((1, 2 * n, k), "bf16", 2, k ** -0.5), normal((rows, n), "bf16", 4)
    h, z = full((rows, n), "bf16"), full((rows, 2 * n), "bf16")
    api.ds4moe_grouped_glu(x, w, None, h, rows, n, k, act=act, zout=z, stream=stream())
    dz, dx, dw = torch.empty_like(z), torch.empty_like(x), torch.empty_like(w)
    api.ds4moe_grouped_glu_grad(c, x, w, None, z, dz, dx, dw, rows, n, k, act=act, stream=stream())

    def f(x, w):
        a, b = (x @ w[0].T).chunk(2, 1)
        return (c.double() * ACTS64[act](a) * b).sum()

    at, step = [x.double(), w.double()], 1e-4
    for i, got in enumerate((dx, dw)):
        v = torch.randn(at[i].shape, generator=gen(9 + i), device="cuda", dtype=torch.float64)
        hi, lo = [t + step * v if j == i else t for j, t in enumerate(at)], [t - step * v if j == i else t for j, t in enumerate(at)]
        want, have = (f(*hi) - f(*lo)) / (2 * step), (got.double() * v).sum()
        # the kept z (both factors), dz and the result are rounded to bf16: 4 * 2^-9 of a term on average; four deviations
        assert abs(have - want) <= 4 * 4 * 2.0 ** -9 * (got.double() * v).norm() + 1e-6


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_block_gradients_where_z_overflowed(act):
    """z = +-inf of a narrower type: act and act' are at their limits; a closed place passes nothing."""
    z = torch.tensor([[-math.inf, 3.0], [-math.inf, math.inf], [math.inf, 2.0], [-1e4, math.inf], [NAN, 1.0]], device="cuda").to(torch.float16)
    dh = torch.ones((5, 1), dtype=torch.float16, device="cuda")
    dz = torch.empty_like(z)
    api.ds4moe_grouped_glu_grad(dh, None, None, None, z, dz, None, None, 5, 1, 8, act=act, dtype="fp16", stream=stream())
    got = dz.float().tolist()
    if act == "none":
        assert got[0] == [3.0, -math.inf] and got[2] == [2.0, math.inf] and got[4][0] == 1.0  # (dh b, whatever a is)
    else:
        assert got[0] == [0.0, 0.0] and got[1] == [0.0, 0.0] and got[3][0] == 0.0 and got[2] == [2.0, math.inf]
        assert math.isnan(got[4][0])
    assert math.isnan(got[4][1])


def test_a_block_row_that_is_not_finite_stays_in_its_row():
    counts, n, k = [30, 3, 0, 131], 72, 200
    rows, g = sum(counts), len(counts)
    x, w = normal((rows, k), "bf16", 1), normal((g, 2 * n, k), "bf16", 3, k ** -0.5)
    x[31, 5] = math.inf
    h, z, _ = block(x, w, offsets(counts), n, "silu", "bf16")
    for t in (h, z):
        bad = ~torch.isfinite(t.float()).all(1)
        assert bad.nonzero().flatten().tolist() == [31]


@pytest.mark.parametrize("rows,n,k,groups", [(2600, 1160, 264, 0), (4096, 520, 136, 0), (700, 264, 1304, 3), (64, 1000, 520, 0), (3, 2048, 4096, 0),
                                             (8, 512, 4096, 8)])
def test_larger_blocks(rows, n, k, groups):
    """Several rounds of tiles, and few tiles that share out the reduction; whole numbers stay exact."""
    g = max(1, groups)
    counts = [rows // g + (rows % g if e == 0 else 0) for e in range(g)]
    x, w = whole((rows, k), "bf16", 1), whole((g, 2 * n, k), "bf16", 2, 1)
    h, z, clean = block(x, w, offsets(counts) if groups else None, n, "relu", "bf16")
    assert clean
    for e, lo, hi in groups_of(counts):
        ref = x[lo:hi].double() @ w[e].double().T
        assert torch.equal(z[lo:hi], ref.to(z.dtype)) and torch.equal(h[lo:hi], (ref[:, :n].clamp(min=0) * ref[:, n:]).to(h.dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("counts", [[300, 257, 256, 420, 255, 0, 310, 400], [288, 1, 512, 513, 33, 320, 257, 900, 100, 230], [256 + 31 * (i % 3) for i in range(12)]])
def test_groups_around_the_width_of_an_accumulator(dtype, counts):
    """Tiles of up to 512 columns take both accumulators, narrower ones in between take turns: blocks, and both products that
    share the kernel. Whole numbers stay exact."""
    rows, g, n, k = sum(counts), len(counts), 1288, 200
    x, w = whole((rows, k), dtype, 1), whole((g, 2 * n, k), dtype, 2)
    off = offsets(counts)
    h, z, clean = block(x, w, off, n, "relu", dtype)
    y, dx = full((rows, 2 * n), dtype), full((rows, 2 * n), dtype)
    api.ds4moe_grouped_mm(x, w, off, y, rows, 2 * n, k, g, dtype, stream=stream())
    wt = w.transpose(1, 2).contiguous()  # [k x 2n]: dx = W^T dy has 2n features
    api.ds4moe_grouped_mm_dx(x, wt, off, dx, rows, k, 2 * n, g, dtype, stream=stream())
    assert clean and torch.equal(z, y) and torch.equal(z, dx)
    for e, lo, hi in groups_of(counts):
        ref = x[lo:hi].double() @ w[e].double().T
        assert torch.equal(z[lo:hi], ref.to(z.dtype)), e
        assert torch.equal(h[lo:hi], (ref[:, :n].clamp(min=0) * ref[:, n:]).to(h.dtype)), e
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("counts,n,k", [([300, 257, 256, 420, 255, 0, 310, 400], 1289, 136), ([3], 129, 4096), ([2, 0, 5], 17, 1024), ([1], 2500, 8),
                                        ([40] * 30, 16, 64), ([300, 290, 280], 3333, 72)])
def test_blocks_of_odd_widths(counts, n, k):
    """Aligned operands with results that are not: wide tiles and split sums stored a lane at a time."""
    rows, g = sum(counts), len(counts)
    x, w = whole((rows, k), "fp16", 1), whole((g, 2 * n, k), "fp16", 2, 1)
    h, z, clean = block(x, w, offsets(counts), n, "relu", "fp16")
    assert clean
    for e, lo, hi in groups_of(counts):
        ref = x[lo:hi].double() @ w[e].double().T
        assert torch.equal(z[lo:hi], ref.to(z.dtype)), e
        assert torch.equal(h[lo:hi], (ref[:, :n].clamp(min=0) * ref[:, n:]).to(h.dtype)), e
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("counts,n", [([3], 960), ([1], 1024), ([40], 1280), ([5], 1536), ([2], 1664), ([64], 2432), ([4, 4, 4, 4], 700), ([1, 0, 7], 800)])
@pytest.mark.parametrize("k", [2048, 2001])
def test_blocks_whose_sums_are_shared_out(counts, n, k):
    """Few rows: clusters that fit the device at once or would not, forward and dx, with the shares' sums exact."""
    rows, g = sum(counts), len(counts)
    x, w, dz = whole((rows, k), "bf16", 1), whole((g, 2 * n, k), "bf16", 3), full((rows, 2 * n), "bf16")
    off = None if g == 1 else offsets(counts)
    h, z, clean = block(x, w, off, n, "none", "bf16")
    assert clean
    dx = full((rows, k), "bf16")
    up = whole((rows, 2 * n), "bf16", 5)
    api.ds4moe_grouped_glu_grad(whole((rows, n), "bf16", 6), x, w, off, up, dz, dx, None, rows, n, k, g, "none", "bf16", stream=stream())
    for e, lo, hi in groups_of(counts):
        ref = x[lo:hi].double() @ w[e].double().T
        assert torch.equal(z[lo:hi], ref.to(torch.bfloat16)) and torch.equal(h[lo:hi], (ref[:, :n] * ref[:, n:]).to(torch.bfloat16))
        ref, terms = dz[lo:hi].double() @ w[e].double(), dz[lo:hi].double().abs() @ w[e].double().abs()
        assert bool(((dx[lo:hi].double() - ref).abs() <= _tolerance(ref, terms, 2 * n, "bf16")).all())
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("counts", [[20005, 17, 0, 300], [1, 16384, 16385]])
def test_long_ragged_weight_gradients(counts):
    """Sums of more terms than an accumulator takes, on pairs of CTAs, with ragged ends: rows of other groups that are not finite stay out."""
    n, k, g = 152, 264, len(counts)
    rows = sum(counts) + 7
    dh, x, z = whole((rows, n), "bf16", 1), whole((rows, k), "bf16", 2), whole((rows, 2 * n), "bf16", 3, 1)
    dh[sum(counts):], x[sum(counts):] = NAN, NAN
    if counts[1] > 1:
        x[counts[0] + 1, 3] = math.inf  # in the second group
    dz, dw = torch.empty_like(z), full((g, 2 * n, k), "bf16")
    api.ds4moe_grouped_glu_grad(dh, x, None, offsets(counts), z, dz, None, dw, rows, n, k, g, "none", stream=stream())
    for e, lo, hi in groups_of(counts):
        if e == 1 and counts[1] > 1:
            assert bool(dw[e][:, [c for c in range(k) if c != 3]].isfinite().all()) and not bool(dw[e][:, 3].isfinite().all())
            continue
        assert torch.equal(dw[e], (dz[lo:hi].double().T @ x[lo:hi].double()).to(dw.dtype)), e
    assert api.ds4moe_ops_status() == 0


def test_block_offsets_out_of_order_or_range_reach_nothing_outside():
    n, k, rows = 40, 64, 40
    x, w, dh, z = whole((rows, k), "bf16", 1), whole((4, 2 * n, k), "bf16", 2), whole((rows, n), "bf16", 3), whole((rows, 2 * n), "bf16", 4)
    off = torch.tensor([-5, 10, 3, 90, 2 ** 31 - 1], dtype=torch.int32, device="cuda")  # clamped: 0-10, -, 3-40, -
    h, _, clean = block(x, w, off, n, "none", "bf16")
    ref = x[10:].double() @ w[2].double().T
    assert clean and torch.equal(h[10:], (ref[:, :n] * ref[:, n:]).to(h.dtype))
    dz, dw = torch.zeros_like(z), torch.ones_like(w)
    api.ds4moe_grouped_glu_grad(dh, x, None, off, z, dz, None, dw, rows, n, k, 4, act="none", stream=stream())
    assert not bool(dw[1].any()) and not bool(dw[3].any())


def test_block_rows_past_32_bits():
    """Rows, kept factors and matrices that lie further apart than 2^31 elements."""
    rows, n, k, ld = 2200, 40, 64, 1 << 20
    x, w, counts = whole((rows, k), "bf16", 1), whole((2, 2 * n, k), "bf16", 2), [1000, 1200]
    far = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    far.view(rows, ld)[:, :k] = x
    out = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    stride = (1 << 31) + 64
    wide = torch.empty(stride + 2 * n * k, dtype=torch.bfloat16, device="cuda")
    wide[:2 * n * k], wide[stride:] = w[0].flatten(), w[1].flatten()
    ref = torch.cat([x[lo:hi].double() @ w[g].double().T for g, lo, hi in groups_of(counts)])
    want, zw = (ref[:, :n].clamp(min=0) * ref[:, n:]).to(x.dtype), ref.to(x.dtype)
    for skew in (0, 1):
        src = far if skew == 0 else torch.cat([far[:skew], far])[:rows * ld]
        # h in the first columns of each far row, z further on
        api.ds4moe_grouped_glu(src.data_ptr() + 2 * skew, wide, offsets(counts), out.data_ptr() + 2 * skew, rows - skew, n, k, 2, "relu",
                               zout=out.data_ptr() + 2 * skew + 512, ldx=ld, w_stride=stride, ldh=ld, ldz=ld, stream=stream())
        at = lambda off, wid: out[skew + off:].as_strided((rows - skew, wid), (ld, 1))  # noqa: E731
        assert torch.equal(at(0, n), want[:rows - skew]) and torch.equal(at(256, 2 * n), zw[:rows - skew])
        dz = torch.empty((rows - skew, 2 * n), dtype=x.dtype, device="cuda")
        api.ds4moe_grouped_glu_grad(out.data_ptr() + 2 * skew, None, None, None, out.data_ptr() + 2 * skew + 512, dz, None, None, rows - skew, n, k, 1, "none",
                                    lddh=ld, ldz=ld, stream=stream())
        a, b = zw[:rows - skew].double().chunk(2, 1)
        dh = want[:rows - skew].double()
        assert torch.equal(dz, torch.cat([dh * b, dh * a], 1).float().to(x.dtype))


# ----------------------------------------------------------------------------------------------- scores


def grid(shape, dtype, seed, scale, step):
    """8-bit whole numbers times a power of two."""
    return ((torch.randn(shape, generator=gen(seed), device="cuda") * scale).round().clamp(-127, 127) * step).to(DT[dtype])


def score(x, w, tokens, top, dtype="bf16", temperature=1.0, pad=0, skew=0, ws_bytes=None):
    (rows, d), vocab, n = x.shape, w.shape[0], tokens.shape[1]
    size = api.ds4moe_logprobs_workspace(rows, vocab, n, top) if ws_bytes is None else ws_bytes
    ws = torch.full((size + 16,), 255, dtype=torch.uint8, device="cuda")
    out = dict(logprob=full((rows + 1, n)), lse=full((rows + 1,)), entropy=full((rows + 1,)), top_logprob=full((rows + 1, max(1, top))),
               top_index=torch.full((rows + 1, max(1, top)), -7, dtype=torch.int32, device="cuda"))
    xb, wb = strided(x, d + pad, skew=skew)[0], strided(w, d + pad, skew=skew)[0]
    api.ds4moe_logprobs(xb.data_ptr() + 2 * skew, wb.data_ptr() + 2 * skew, tokens if n else None, out["logprob"] if n else None, out["lse"],
                        out["entropy"], out["top_index"] if top else None, out["top_logprob"] if top else None, rows, vocab, d, n, top, dtype,
                        temperature, ws, size, d + pad, d + pad, stream())
    assert bool((ws[size:] == 255).all())
    for name, t in out.items():
        assert bool((t[rows] == (-7 if name == "top_index" else 7)).all()), name
    if not top:
        assert bool((out["top_index"] == -7).all())
    return {name: t[:rows] for name, t in out.items()}


def score_check(x, w, tokens, top, dtype, temperature, got, order=True):
    d, vocab = x.shape[1], w.shape[0]
    z = x.double() @ w.double().T
    logp = z / temperature
    lse = torch.logsumexp(logp, 1, keepdim=True)
    # a logit's error: d additions; lse's: the largest logit's and the sum's, a few units of 2^-22
    zerr = (d + 8) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T).max(1, keepdim=True).values / temperature
    tol = 2 * zerr + 2.0 ** -21 * (1 + lse.abs() + logp.abs().max(1, keepdim=True).values)
    assert bool(((got["lse"][:, None] - lse).abs() <= tol).all())
    logp = logp - lse
    p = logp.exp()
    entropy = -(torch.where(p > 0, p * logp, 0.0)).sum(1, keepdim=True)
    # sum p |log p + H| <= 2 H times the logits' error, and each exponential's and the sums' 2^-17
    assert bool(((got["entropy"][:, None] - entropy).abs() <= (2 * entropy + 1) * (2 * zerr + 2.0 ** -17)).all())
    there = (tokens >= 0) & (tokens < vocab)
    want = torch.where(there, logp.gather(1, torch.where(there, tokens, 0).long()), 0.0)
    if tokens.shape[1]:
        assert bool(((got["logprob"] - want).abs() <= 2 * tol).all())
        assert bool((got["logprob"][~there] == 0).all())
    if top:
        index = got["top_index"].long()
        assert bool(((index >= 0) & (index < vocab)).all())
        assert bool(((got["top_logprob"] - logp.gather(1, index)).abs() <= 2 * tol).all())
        best = torch.sort(z, dim=1, descending=True, stable=True)
        if order:
            assert torch.equal(index, best.indices[:, :top])
        else:
            assert bool(((best.values[:, :top] - z.gather(1, index)).abs() <= 2 * zerr * temperature).all())
            assert all(len(set(row)) == top for row in index.tolist())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,d,n,top,temperature,pad,skew", [
    (1, 1, 1, 1, 1, 1.0, 0, 0), (1, 1000, 64, 1, 8, 1.0, 0, 0), (16, 1003, 72, 3, 20, 0.7, 0, 0), (3, 257, 129, 2, 64, 2.0, 0, 0),
    (130, 777, 200, 1, 5, 1.0, 8, 0), (129, 640, 77, 16, 33, 1.3, 3, 1), (300, 9001, 64, 1, 32, 1.0, 0, 0), (2, 64, 40, 64, 64, 1.0, 0, 0),
    (300, 3001, 2056, 1, 10, 1.0, 0, 0), (40, 3001, 2304, 2, 10, 1.0, 0, 0), (20, 900, 4200, 2, 10, 1.0, 0, 0)])
def test_scores_with_exact_logits(dtype, rows, vocab, d, n, top, temperature, pad, skew):
    """The best words in their order, ties to the lower index: the logits are exact."""
    x, w = grid((rows, d), dtype, 1, 16, 2.0 ** -4), grid((vocab, d), dtype, 2, 20, 2.0 ** -round(math.log2(10 * d ** 0.5)))
    tokens = torch.randint(-1, vocab, (rows, n), generator=gen(3), device="cuda", dtype=torch.int32)
    tokens[0, 0], tokens[-1, -1] = vocab - 1, 0
    score_check(x, w, tokens, top, dtype, temperature, score(x, w, tokens, top, dtype, temperature, pad, skew))
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("rows,vocab,d,n,top", [(5, 3000, 513, 0, 9), (200, 5000, 1000, 200, 0), (17, 131, 4100, 256, 12), (1, 40000, 128, 1, 1)])
def test_scores(rows, vocab, d, n, top):
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, 2 * d ** -0.5)
    tokens = torch.randint(0, vocab, (rows, n), generator=gen(3), device="cuda", dtype=torch.int32)
    score_check(x, w, tokens, top, "bf16", 1.0, score(x, w, tokens, top), order=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,d,n,top,pad,skew", [
    (1, 40001, 77, 1, 8, 0, 0), (32, 25003, 130, 5, 64, 0, 0), (31, 129, 2051, 9, 3, 0, 0), (2, 140001, 64, 4, 10, 3, 1), (20, 900, 4201, 2, 10, 0, 1),
    (7, 1, 9, 1, 1, 0, 0), (5, 33, 1, 200, 33, 0, 0), (17, 20000, 72, 3, 5, 8, 4)])
def test_scores_of_few_rows_anywhere(dtype, rows, vocab, d, n, top, pad, skew):
    """Rows that start at any element, words that fill none or several tiles of a CTA; a row of NaN beside the others."""
    x, w = grid((rows, d), dtype, 1, 16, 2.0 ** -4), grid((vocab, d), dtype, 2, 20, 2.0 ** -round(math.log2(10 * d ** 0.5)))
    tokens = torch.randint(-1, vocab, (rows, n), generator=gen(3), device="cuda", dtype=torch.int32)
    score_check(x, w, tokens, top, dtype, 0.8, score(x, w, tokens, top, dtype, 0.8, pad, skew))
    if rows > 1:
        x[rows - 1] = NAN
        got = score(x, w, tokens, top, dtype, 0.8, pad, skew)
        score_check(x[:-1], w, tokens[:-1], top, dtype, 0.8, {name: v[:-1] for name, v in got.items()})
        assert bool(got["lse"][-1].isnan())
    assert api.ds4moe_ops_status() == 0


def test_scores_of_equal_and_of_sorted_logits():
    """Every logit the same: the first words. Logits that rise or fall with the index: lists that change at every word."""
    rows, vocab, d, top = 40, 2000, 64, 50
    x = torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = 1.0, 1.0
    w = torch.zeros((vocab, d), dtype=torch.bfloat16, device="cuda")
    tokens = torch.arange(rows, device="cuda", dtype=torch.int32)[:, None]
    score_check(x, w, tokens, top, "bf16", 1.0, score(x, w, tokens, top))
    v = torch.arange(vocab, device="cuda")
    w[:, 0], w[:, 1] = (v // 128 * 128 / 256.0).to(w.dtype), (v % 128 / 256.0).to(w.dtype)  # index / 256, in two parts
    score_check(x, w, tokens, top, "bf16", 1.0, score(x, w, tokens, top))
    score_check(-x, w, tokens, top, "bf16", 0.01, score(-x, w, tokens, top, temperature=0.01))


@pytest.mark.parametrize("rows,vocab,d,top", [(2, 140000, 64, 10), (40, 140000, 72, 64), (1030, 140000, 64, 9), (1100, 999, 72, 64),
                                              (1025, 3000, 64, 33), (33, 20000, 4100, 5), (128, 700, 136, 3), (32, 5000, 16392, 7)])
def test_scores_of_long_vocabularies_and_many_rows(rows, vocab, d, top):
    """More partials and chunks than a team's threads hold, more best words than a warp has lanes, sums in several accumulators."""
    x, w = grid((rows, d), "bf16", 1, 16, 2.0 ** -4), grid((vocab, d), "bf16", 2, 20, 2.0 ** -round(math.log2(10 * d ** 0.5)))
    tokens = torch.randint(-1, vocab, (rows, 5), generator=gen(3), device="cuda", dtype=torch.int32)
    score_check(x, w, tokens, top, "bf16", 1.0, score(x, w, tokens, top))
    x[::3] = 0  # rows of equal logits
    got = score(x, w, tokens, top)
    assert torch.equal(got["top_index"][::3].cpu(), torch.arange(top, dtype=torch.int32).expand((rows + 2) // 3, top))
    assert api.ds4moe_ops_status() == 0


def test_scores_in_blocks_of_rows():
    rows, vocab, d, n, top = 700, 1500, 72, 2, 4
    x, w = grid((rows, d), "bf16", 1, 16, 2.0 ** -4), grid((vocab, d), "bf16", 2, 20, 2.0 ** -6)
    tokens = torch.randint(-1, vocab, (rows, n), generator=gen(3), device="cuda", dtype=torch.int32)
    whole_call = score(x, w, tokens, top)
    score_check(x, w, tokens, top, "bf16", 1.0, whole_call)
    for block in (128, 256, 640):
        size = api.ds4moe_logprobs_workspace(block, vocab, n, top) + 32
        got = score(x, w, tokens, top, ws_bytes=size // 16 * 16)
        assert all(torch.equal(got[name], whole_call[name]) for name in got)
    with pytest.raises(api.Ds4MoeError) as ei:
        score(x, w, tokens, top, ws_bytes=api.ds4moe_logprobs_workspace(127, vocab, n, top))
    assert ei.value.code == api.DS4MOE_ERR_CAPACITY
    few = score(x[:5], w, tokens[:5], top)  # fewer rows than a block need only their own
    assert torch.equal(few["top_index"], whole_call["top_index"][:5])


def test_scores_of_closed_words_and_rows_that_are_not_finite():
    rows, vocab, d, top = 20, 700, 64, 30
    x = grid((rows, d), "bf16", 1, 16, 2.0 ** -4).abs() + 0.25
    w = grid((vocab, d), "bf16", 2, 20, 2.0 ** -4)
    w[64:690, 3] = -math.inf  # all but 74 words, whole tiles among them
    tokens = torch.randint(0, vocab, (rows, 3), generator=gen(3), device="cuda", dtype=torch.int32)
    tokens[:, 0] = 100
    got = score(x, w, tokens, top)
    z = x.double() @ torch.where(w.isinf(), 0, w).double().T
    z[:, 64:690] = -math.inf
    logp = z - torch.logsumexp(z, 1, keepdim=True)
    assert bool((got["logprob"][:, 0] == -math.inf).all())
    assert torch.equal(got["top_index"].long(), torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top])
    assert bool(((got["top_logprob"] - logp.gather(1, got["top_index"].long())).abs() <= 2.0 ** -14 * z[:, :60].abs().max()).all())
    entropy = -torch.where(z == -math.inf, 0.0, logp * logp.exp()).sum(1)
    assert bool(((got["entropy"] - entropy).abs() <= 1e-4 * (1 + entropy)).all())
    # fewer open words than asked for: the closed ones follow in their order
    w[:, 3] = -math.inf
    w[[7, 300], 3] = 0.0
    got = score(x, w, tokens, top)
    assert bool((got["top_index"][:, :2].sort(1).values == torch.tensor([7, 300], device="cuda")).all())
    assert got["top_index"][0, 2:].tolist() == [i for i in range(40) if i != 7][:28]
    assert bool((got["top_logprob"][:, 2:] == -math.inf).all()) and bool(got["entropy"].isfinite().all())
    # rows of nothing else, and rows with NaN
    w[:, 3] = -math.inf
    x[4, 5] = NAN
    got = score(x, w, tokens, 3)
    fine = [t for t in range(rows) if t != 4]
    assert bool((got["lse"][fine] == -math.inf).all()) and bool(got["entropy"].isnan().all())
    assert bool(got["lse"][4].isnan()) and bool(got["logprob"][4].isnan().all())
    assert got["top_index"][4].tolist() == [-1, -1, -1] and got["top_index"][5].tolist() == [0, 1, 2]
    w = grid((vocab, d), "bf16", 2, 20, 2.0 ** -6)
    w[333] = NAN  # one word
    got = score(x, w, tokens, 3)
    assert not bool((got["top_index"] == 333).any()) and bool(got["lse"].isnan().all())
    assert api.ds4moe_ops_status() == 0


def test_scores_of_foreign_tokens():
    rows, vocab, d = 10, 300, 40
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    tokens = torch.randint(0, vocab, (rows, 4), generator=gen(3), device="cuda", dtype=torch.int32)
    tokens[2] = torch.tensor([5, 5, -1, 5], device="cuda")  # the same token again
    got = score(x, w, tokens, 0)
    score_check(x, w, tokens, 0, "bf16", 1.0, got)
    assert got["logprob"][2, 0] == got["logprob"][2, 1] == got["logprob"][2, 3]
    assert api.ds4moe_ops_status() == 0
    tokens[3, 1], tokens[4, 0], tokens[5, 2] = vocab, -2, 2 ** 31 - 1
    score_check(x, w, tokens, 0, "bf16", 1.0, score(x, w, tokens, 0))
    assert api.ds4moe_ops_status() == 1 and api.ds4moe_ops_status() == 0


def test_scores_of_large_logits():
    rows, vocab, d = 12, 900, 64
    x, w = grid((rows, d), "bf16", 1, 16, 1.0), grid((vocab, d), "bf16", 2, 20, 1.0)  # logits in the thousands
    tokens = torch.randint(0, vocab, (rows, 2), generator=gen(3), device="cuda", dtype=torch.int32)
    for t in (1.0, 1e-3, 1e3):
        got = score(x, w, tokens, 7, temperature=t)
        z = x.double() @ w.double().T
        logp = torch.log_softmax(z / t, 1)
        assert torch.equal(got["top_index"].long(), torch.sort(z, dim=1, descending=True, stable=True).indices[:, :7])
        want = logp.gather(1, tokens.long())
        assert bool(((got["logprob"] - want).abs() <= 2.0 ** -20 * (1 + want.abs())).all())
        assert bool(got["entropy"].isfinite().all()) and bool((got["entropy"] >= 0).all())


# ----------------------------------------------------------------------------------------- distillation


def distilled(x, w, ids, teacher, dloss, dtype="bf16", temperature=1.0, pad=0, ws_bytes=None, want="xw"):
    (rows, d), vocab, k = x.shape, w.shape[0], ids.shape[1]
    size = api.ds4moe_distill_workspace(rows, vocab, d, k)
    ws = torch.full((size + 16,), 255, dtype=torch.uint8, device="cuda")
    loss, lse, logq = full((rows,)), full((rows,)), full((rows, k))
    xb, wb = strided(x, d + pad)[0], strided(w, d + pad)[0]
    api.ds4moe_distill(xb, wb, ids, teacher, loss, lse, logq, rows, vocab, d, k, dtype, temperature, ws, size, d + pad, d + pad, stream())
    (dxb, dx), (dwb, dw) = strided(full((rows, d), dtype), d + pad, fill=7.0), strided(full((vocab, d), dtype), d + pad, fill=7.0)
    api.ds4moe_distill_grad(xb, wb, ids, teacher, lse, logq, dloss, dxb if "x" in want else None, dwb if "w" in want else None, rows, vocab, d,
                            k, dtype, temperature, ws, ws_bytes or size, d + pad, d + pad, d + pad, d + pad, stream())
    assert bool((ws[size:] == 255).all())
    out = (loss, lse, logq, dx.clone(), dw.clone())
    dx.fill_(7.0), dw.fill_(7.0)
    assert bool((dxb == 7.0).all()) and bool((dwb == 7.0).all())
    return out


def teacher_p(ids, teacher, vocab, temperature):
    there = (ids >= 0) & (ids < vocab) & (teacher > -math.inf)
    t = torch.where(there, teacher.double() / temperature, -math.inf)
    some = there.any(1)
    p = torch.softmax(torch.where(some[:, None], t, 0.0), 1)
    return torch.where(there, p, 0.0), some


def distill_check(x, w, ids, teacher, dloss, dtype, temperature, got):
    loss, lse, logq, dx, dw = got
    d, vocab = x.shape[1], w.shape[0]
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    z = x64 @ w64.T / temperature
    there = (ids >= 0) & (ids < vocab)
    at = torch.where(there, ids, 0).long()
    p, some = teacher_p(ids, teacher, vocab, temperature)
    want_lse = torch.logsumexp(z, 1)
    want_logq = torch.where(there, z.gather(1, at) - want_lse[:, None], 0.0)
    want = (torch.xlogy(p, p) - p * want_logq).sum(1)
    zerr = ((d + 8) * 2.0 ** -23 * (x64.abs() @ w64.abs().T).max(1).values / temperature).detach()
    tol = 2 * zerr + 2.0 ** -21 * (1 + want_lse.abs() + z.abs().max(1).values).detach()
    assert bool(((lse - want_lse).abs() <= tol).all())
    assert bool(((logq - want_logq).abs() <= 2 * tol[:, None]).all())
    # p is off by a few units of 2^-22 and of its logits' distance; log p by as much
    far = torch.where(p > 0, torch.log(p.clamp(min=1e-300)).abs(), 0.0).max(1).values
    assert bool(((loss - want).abs() <= 2 * tol + 2.0 ** -20 * (1 + far) * (1 + far + want_logq.abs().max(1).values.detach())).all())
    assert bool((loss[~some] == 0).all())
    g = torch.where(some, dloss.double(), 0.0)
    gx, gw = torch.autograd.grad((want * g).sum(), (x64, w64))
    q = torch.softmax(z, 1).detach()
    hot = torch.zeros_like(q).scatter_add_(1, at, p)
    g = g / temperature
    dz = ((q - hot) * g[:, None]).abs()
    gmax = g.abs().max()
    off = (ULP[dtype] + 2.0 ** -20) * dz + ((2 * tol[:, None] + 2.0 ** -20) * q + 2.0 ** -20 * (1 + far[:, None]) * hot) * g.abs()[:, None]
    off = off + (2.0 ** -25 * 2.0 ** -13 * gmax if dtype == "fp16" else 0)
    sub = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -130
    if dx is not None:
        lim = _tolerance(gx, dz @ w64.abs().detach(), vocab, dtype) + off @ w64.abs().detach() + sub
        assert bool(((dx.double() - gx).abs() <= lim).all())
        assert not bool(dx[~some].any())
    if dw is not None:
        lim = _tolerance(gw, dz.T @ x64.abs().detach(), x.shape[0], dtype) + off.T @ x64.abs().detach() + sub
        assert bool(((dw.double() - gw).abs() <= lim).all())


def lists(rows, vocab, k, seed=3, missing=0.1):
    ids = torch.rand((rows, vocab), generator=gen(seed), device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    ids[torch.rand((rows, k), generator=gen(seed + 1), device="cuda") < missing] = -1
    return ids, torch.randn((rows, k), generator=gen(seed + 2), device="cuda") * 2 + 5


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,d,k,temperature,pad", [
    (1, 1, 1, 1, 1.0, 0), (1, 1000, 64, 32, 1.0, 0), (16, 1003, 72, 5, 2.0, 0), (3, 257, 129, 256, 0.7, 0), (130, 777, 200, 100, 1.0, 8),
    (129, 640, 77, 33, 4.0, 3), (300, 9001, 64, 8, 1.0, 0)])
def test_distillation(dtype, rows, vocab, d, k, temperature, pad):
    x, w = normal((rows, d), dtype, 1), normal((vocab, d), dtype, 2, 2.0 * d ** -0.5)
    ids, teacher = lists(rows, vocab, k)
    if rows > 2:
        ids[1] = -1                             # no teacher
        ids[2, 0], ids[0, -1] = vocab - 1, 0    # (perhaps twice in their rows)
    dloss = torch.rand(rows, generator=gen(8), device="cuda") / rows
    distill_check(x, w, ids, teacher, dloss, dtype, temperature, distilled(x, w, ids, teacher, dloss, dtype, temperature, pad))
    assert api.ds4moe_ops_status() == 0


def test_distillation_of_words_named_twice():
    rows, vocab, d, k = 40, 500, 64, 12
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    ids, teacher = lists(rows, vocab, k, missing=0)
    ids[:, 3], ids[:, 7], ids[::2, 8] = ids[:, 0], ids[:, 0], ids[::2, 1]
    dloss = torch.ones(rows, device="cuda")
    distill_check(x, w, ids, teacher, dloss, "bf16", 1.5, distilled(x, w, ids, teacher, dloss, temperature=1.5))


def test_distillation_from_one_word_is_the_cross_entropy():
    rows, vocab, d = 60, 2000, 72
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    labels = torch.randint(0, vocab, (rows,), generator=gen(3), device="cuda", dtype=torch.int32)
    labels[::9] = -1
    dloss = torch.rand(rows, generator=gen(4), device="cuda")
    loss, lse, _, dx, dw = distilled(x, w, labels[:, None], torch.randn((rows, 1), generator=gen(5), device="cuda"), dloss)
    from test_gpu_mm16 import _ce
    want = _ce(x, w, labels, dloss, "bf16", ignore=-1)
    # the same logits and sums, joined in another order
    assert bool(((loss - want[0]).abs() <= 2.0 ** -19 * (1 + want[0].abs())).all()) and bool(((lse - want[1]).abs() <= 2.0 ** -19 * want[1].abs()).all())
    for got, ref in ((dx, want[2]), (dw, want[3])):
        # dz's label terms may round the other way: a step of bf16 at a few places
        assert bool(((got.double() - ref.double()).norm() <= 2.0 ** -8 * ref.double().norm()).all())


def test_distillation_of_foreign_ids_and_rows_that_teach_nothing():
    rows, vocab, d, k = 24, 400, 64, 6
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    ids, teacher = lists(rows, vocab, k, missing=0)
    teacher[3] = -math.inf       # no entry above -inf
    teacher[4, 2] = -math.inf    # one of no weight
    ids[5, 0], ids[6, 1], ids[7] = vocab, -5, -1
    dloss = torch.ones(rows, device="cuda")
    got = distilled(x, w, ids, teacher, dloss)
    distill_check(x, w, ids, teacher, dloss, "bf16", 1.0, got)
    assert got[0][3] == 0 and got[0][7] == 0 and got[2][5, 0] == 0
    assert api.ds4moe_ops_status() == 1 and api.ds4moe_ops_status() == 0
    teacher[8, 1], teacher[9, 0], dloss[10] = NAN, math.inf, NAN
    loss, lse, logq, dx, dw = distilled(x, w, ids, teacher, dloss)
    assert loss.isfinite().logical_not().nonzero().flatten().tolist() == [8, 9]
    assert dx.isfinite().all(1).logical_not().nonzero().flatten().tolist() == [8, 9, 10]
    api.ds4moe_ops_status()


def test_distillation_of_closed_words():
    """Words whose logit is -inf: probability 0. A teacher that names one has an infinite loss, and a finite gradient."""
    rows, vocab, d, k = 20, 700, 64, 5
    x, w = normal((rows, d), "bf16", 1).abs() + 0.1, normal((vocab, d), "bf16", 2, d ** -0.5)
    w[64:300, 3] = -math.inf
    ids = torch.randint(300, vocab, (rows, k), generator=gen(3), device="cuda", dtype=torch.int32)
    ids[4, 2] = 100
    teacher = torch.randn((rows, k), generator=gen(4), device="cuda")
    loss, lse, logq, dx, dw = distilled(x, w, ids, teacher, torch.ones(rows, device="cuda"), want="w")
    assert loss.isinf().nonzero().flatten().tolist() == [4] and logq[4, 2] == -math.inf
    assert bool(dw.isfinite().all()) and dw[64:300].any(1).nonzero().flatten().tolist() == [36]


def test_distillation_in_small_pieces_and_blocks():
    rows, vocab, d, k = 300, 2000, 136, 7
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    ids, teacher = lists(rows, vocab, k)
    dloss = torch.rand(rows, generator=gen(8), device="cuda")
    small = 16 + 4 * rows * (d + 1 + k) + 512 * 304 + 48  # the documented smallest size: 256 words a piece
    distill_check(x, w, ids, teacher, dloss, "bf16", 1.0, distilled(x, w, ids, teacher, dloss, ws_bytes=small))
    loss, lse, logq = full((rows,)), full((rows,)), full((rows, k))
    size = api.ds4moe_logprobs_workspace(128, vocab, k, 0)  # the forward's own blocks of rows
    ws = torch.full((size + 16,), 255, dtype=torch.uint8, device="cuda")
    api.ds4moe_distill(x, w, ids, teacher, loss, lse, logq, rows, vocab, d, k, workspace=ws, workspace_bytes=size, stream=stream())
    assert bool((ws[size:] == 255).all())
    want = distilled(x, w, ids, teacher, dloss)
    assert torch.equal(loss, want[0]) and torch.equal(lse, want[1]) and torch.equal(logq, want[2])


def test_distillation_gradient_against_differences():
    rows, vocab, d, k, t = 12, 300, 40, 9, 1.7
    x, w = normal((rows, d), "bf16", 1), normal((vocab, d), "bf16", 2, d ** -0.5)
    ids, teacher = lists(rows, vocab, k)
    ids[:, 4] = ids[:, 2]
    c = torch.rand(rows, generator=gen(4), device="cuda")
    _, _, _, dx, dw = distilled(x, w, ids, teacher, c, temperature=t)
    p, _ = teacher_p(ids, teacher, vocab, t)

    def f(x, w):
        logq = torch.log_softmax(x @ w.T / t, 1).gather(1, ids.clamp(min=0).long())
        return (c.double() * (torch.xlogy(p, p) - p * logq).sum(1)).sum()

    at, h = [x.double(), w.double()], 1e-4
    for i, got in enumerate((dx, dw)):
        v = torch.randn(at[i].shape, generator=gen(9 + i), device="cuda", dtype=torch.float64)
        hi, lo = [s + h * v if j == i else s for j, s in enumerate(at)], [s - h * v if j == i else s for j, s in enumerate(at)]
        want, have = (f(*hi) - f(*lo)) / (2 * h), (got.double() * v).sum()
        # dz and the result are each rounded to bf16 (2^-9 of a term on average); four deviations
        assert abs(have - want) <= 4 * 2 * 2.0 ** -9 * (got.double() * v).norm() + 1e-6


def test_distillation_of_no_rows():
    dw = full((30, 16), "bf16")
    api.ds4moe_distill_grad(None, None, None, None, None, None, None, None, dw, 0, 30, 16, 3, stream=stream())
    assert not bool(dw.any())


# -------------------------------------------------------------------------------------------- together


def test_a_student_block_and_head_learn_from_a_teachers_scores():
    """A teacher's head names its best words; the student's block and head are scored, distilled and differentiated through
    the operators, and compared with 64-bit autograd; then the same on several streams and in a graph, bit for bit."""
    rows, d, f, vocab, k, t = 200, 136, 72, 3000, 16, 1.5
    counts = [0, 3, 150, 47]
    off = offsets(counts)
    x, w, down = normal((rows, d), "bf16", 1), normal((4, 2 * f, d), "bf16", 2, d ** -0.5), normal((4, d, f), "bf16", 3, f ** -0.5)
    head, other = normal((vocab, d), "bf16", 4, 2 * d ** -0.5), normal((vocab, d), "bf16", 5, 2 * d ** -0.5)
    ones = torch.full((rows,), 1.0 / rows, device="cuda")
    size = max(api.ds4moe_logprobs_workspace(rows, vocab, 1, k), api.ds4moe_distill_workspace(rows, vocab, d, k))

    def buffers():
        b = {name: full(s, "bf16", 9.0) for name, s in dict(h=(rows, f), z=(rows, 2 * f), y=(rows, d), dy=(rows, d), dh=(rows, f), dz=(rows, 2 * f), dx=(rows, d),
                                                           dw=(4, 2 * f, d), ddown=(4, d, f), dhead=(vocab, d)).items()}
        b.update({name: full(s, "fp32", 9.0) for name, s in dict(entropy=(rows,), top=(rows, k), loss=(rows,), lse=(rows,), logq=(rows, k)).items()})
        b["ids"] = torch.full((rows, k), 9, dtype=torch.int32, device="cuda")
        b["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        return b

    def calls(b):
        s = stream()
        sizes, ws = dict(rows=rows, vocab=vocab, d=d, stream=s), dict(workspace=b["ws"], workspace_bytes=size)
        api.ds4moe_logprobs(x, other, None, None, None, b["entropy"], b["ids"], b["top"], n_tokens=0, top_k=k, temperature=1.0, **sizes, **ws)
        api.ds4moe_grouped_glu(x, w, off, b["h"], rows, f, d, 4, zout=b["z"], stream=s)
        api.ds4moe_grouped_mm(b["h"], down, off, b["y"], rows, d, f, 4, stream=s)
        api.ds4moe_distill(b["y"], head, b["ids"], b["top"], b["loss"], b["lse"], b["logq"], top_k=k, temperature=t, **sizes, **ws)
        api.ds4moe_distill_grad(b["y"], head, b["ids"], b["top"], b["lse"], b["logq"], ones, b["dy"], b["dhead"], top_k=k, temperature=t, **sizes, **ws)
        api.ds4moe_grouped_mm_dx(b["dy"], down, off, b["dh"], rows, d, f, 4, stream=s)
        api.ds4moe_grouped_mm_dw(b["dy"], b["h"], off, b["ddown"], rows, d, f, 4, stream=s)
        api.ds4moe_grouped_glu_grad(b["dh"], x, w, off, b["z"], b["dz"], b["dx"], b["dw"], rows, f, d, 4, stream=s)

    first = buffers()
    calls(first)
    torch.cuda.synchronize()
    x64, w64, down64, head64 = (v.double().requires_grad_() for v in (x, w, down, head))
    y64 = torch.cat([(lambda a: (torch.nn.functional.silu(a[:, :f]) * a[:, f:]) @ down64[e].T)(x64[lo:hi] @ w64[e].T) for e, lo, hi in groups_of(counts)])
    teacher = torch.log_softmax(x.double() @ other.double().T, 1)
    assert bool(((first["top"] - teacher.gather(1, first["ids"].long())).abs() <= 1e-4).all())
    p = torch.softmax(first["top"].double() / t, 1)
    logq = torch.log_softmax(y64 @ head64.T / t, 1).gather(1, first["ids"].long())
    loss = (torch.xlogy(p, p) - p * logq).sum(1)
    (loss / rows).sum().backward()
    # every tensor handed on is rounded to bf16 (2^-9 of an element on average, at most eight of them on the longest way)
    assert float((first["loss"] - loss.detach()).norm() / loss.detach().norm()) <= 8 * 2.0 ** -9
    for name, leaf in (("dx", x64), ("dw", w64), ("ddown", down64), ("dhead", head64)):
        rel = float((first[name].double() - leaf.grad).norm() / leaf.grad.norm())
        assert rel <= 8 * 2.0 ** -9, (name, rel)
    sets, streams = [buffers() for _ in range(3)], [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        for st, b in zip(streams, sets):
            with torch.cuda.stream(st):
                calls(b)
    torch.cuda.synchronize()
    captured = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(captured)
    for _ in range(2):
        for name, v in captured.items():
            if name != "ws":
                v.fill_(1)
        graph.replay()
    torch.cuda.synchronize()
    for b in sets + [captured]:
        for name, v in first.items():
            if name != "ws":
                assert torch.equal(v, b[name]), name
    assert api.ds4moe_ops_status() == 0


def test_host_memory_is_refused():
    x = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")
    host = torch.zeros((1, 16, 8), dtype=torch.bfloat16).pin_memory()
    with pytest.raises(api.Ds4MoeError) as ei:
        api.ds4moe_grouped_glu(x, host, None, x, 4, 8, 8, stream=stream())
    assert ei.value.code == api.DS4MOE_ERR_INVALID_ARG and "w is not device memory" in str(ei.value)
    f = torch.zeros((4, 1), device="cuda")
    with pytest.raises(api.Ds4MoeError) as ei:
        api.ds4moe_logprobs(x, x, torch.zeros((4, 1), dtype=torch.int32), f, f, f, None, None, 4, 4, 8, workspace=x, workspace_bytes=1 << 12, stream=stream())
    assert "tokens is not device memory" in str(ei.value)
    with pytest.raises(ValueError):  # a list with gaps between its rows
        api.ds4moe_distill(x, x, torch.zeros((4, 6), dtype=torch.int32, device="cuda")[:, :3], f, f, f, f, 4, 4, 8, 3, workspace=x, workspace_bytes=1 << 12)
