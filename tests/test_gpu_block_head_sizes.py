"""GPU: the gated block, the scores and the distillation at the sizes where they change their form: workspaces made for
more rows, pieces of the vocabulary above 16384 words, selections among words that are not numbers, ragged weight gradients
on pairs of CTAs, groups on both sides of a tile. Tolerances as in test_gpu_block_head."""
import math

import pytest
import torch

from quantized_moe_gb300 import ds4moe as api
from test_gpu_block_head import block, distill_check, distilled, grid, lists, score, score_check
from test_gpu_mm16 import NAN, gen, groups_of, normal, offsets, stream, whole

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab,n,top,most,rows", [(129280, 1, 0, 33, 32), (32000, 100, 0, 40, 13), (32000, 1, 8, 33, 32), (5000, 6, 3, 100, 17)])
def test_scores_of_fewer_rows_than_the_workspace_was_made_for(vocab, n, top, most, rows):
    d = 64
    x, w = grid((rows, d), "bf16", 1, 16, 2.0 ** -4), grid((vocab, d), "bf16", 2, 20, 2.0 ** -6)
    tokens = torch.randint(-1, vocab, (rows, n), generator=gen(3), device="cuda", dtype=torch.int32)
    got = score(x, w, tokens, top, ws_bytes=api.ds4moe_logprobs_workspace(most, vocab, n, top))
    score_check(x, w, tokens, top, "bf16", 1.0, got)
    own = score(x, w, tokens, top)
    assert all(torch.equal(got[name], own[name]) for name in own)
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("rows", [1, 7, 40, 200, 1100])
@pytest.mark.parametrize("top", [2, 5, 40])
def test_best_words_among_words_that_are_not_numbers(rows, top):
    """Whole tiles and chunks of NaN come before closed words (-inf) and a few open ones: the open words are listed first and
    then the closed ones in their order, as if the others were not there."""
    vocab, d = 13000, 64
    x, w = grid((rows, d), "bf16", 1, 16, 2.0 ** -4), grid((vocab, d), "bf16", 2, 20, 2.0 ** -6)
    x[:, 0] = 1.0
    w[:, 0] = -math.inf
    w[:11900] = NAN  # 46 tiles of 256, 371 chunks of 32, and part of the next
    open_words = [11950, 12345, vocab - 1]
    w[open_words, 0] = 0.0
    w[12000:12300] = NAN
    tokens = torch.zeros((rows, 1), dtype=torch.int32, device="cuda")
    got = score(x, w, tokens, top)
    z = x.double() @ w.double().T
    z = torch.where(torch.arange(vocab, device="cuda") < 11900, NAN, z)
    number = ~z[0].isnan()
    places = number.nonzero().flatten()
    want = places[torch.sort(z[:, number], dim=1, descending=True, stable=True).indices[:, :top]]
    assert torch.equal(got["top_index"].long(), want)
    assert bool(got["lse"].isnan().all()) and bool(got["top_logprob"].isnan().all())
    # fewer words that are numbers than asked for
    w[:, 0], w[11900:vocab - 1] = NAN, NAN
    w[vocab - 1] = 1.0
    got = score(x, w, tokens, top)
    assert got["top_index"][0].tolist() == [vocab - 1] + [-1] * (top - 1)
    # a word of infinite logit comes first, and the row has no log probabilities
    w = grid((vocab, d), "bf16", 2, 20, 2.0 ** -6)
    w[12345, 0] = math.inf
    got = score(x, w, tokens, top)
    assert bool((got["top_index"][:, 0] == 12345).all())
    z = x.double() @ w.double().T
    assert torch.equal(got["top_index"].long(), torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top])
    assert all(bool(got[name].isnan().all()) for name in ("lse", "entropy", "logprob", "top_logprob"))
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("rows,vocab", [(12, 900), (300, 9001), (20, 140000)])
@pytest.mark.parametrize("t", [1.0, 1e-3, 1e3, 0.3])
def test_entropy_of_exact_logits(rows, vocab, t):
    """The logits are exact (whole numbers below 2^24), so that what is left is the sums' and the exponentials' rounding: at
    most 73 roundings one after the other in each of two sums (chunks of 32 words in four accumulators, the joins), as a
    random walk of sqrt(146) steps of 2^-24, below 2^-20, twice that allowed for; and the factor 1 / T, whose rounding of up
    to 2^-23 moves the entropy by the variance of log p as much."""
    d = 64
    x, w = grid((rows, d), "bf16", 1, 16, 1.0), grid((vocab, d), "bf16", 2, 20, 1.0)
    x[rows // 2:] = (x[rows // 2:].float() * 0.01).round().to(x.dtype)  # rows of small logits, with a large entropy
    tokens = torch.zeros((rows, 1), dtype=torch.int32, device="cuda")
    got = score(x, w, tokens, 0, temperature=t)["entropy"].double()
    logp = torch.log_softmax(x.double() @ w.double().T / t, 1)
    p = logp.exp()
    want = -torch.where(p > 0, p * logp, 0.0).sum(1)
    var = torch.where(p > 0, p * (logp + want[:, None]) ** 2, 0.0).sum(1)
    assert bool(((got - want).abs() <= 2.0 ** -19 * (1 + want) + 2.0 ** -23 * var).all())


@pytest.mark.parametrize("dtype,rows,vocab,d,k,temperature", [
    ("bf16", 1, 40000, 64, 8, 1.0), ("fp16", 16, 40007, 72, 32, 2.0), ("bf16", 128, 40000, 200, 16, 1.0), ("bf16", 512, 33000, 64, 8, 1.0),
    ("bf16", 513, 33000, 64, 8, 1.0), ("fp16", 700, 33001, 72, 5, 1.0), ("bf16", 64, 40000, 1024, 8, 1.0), ("bf16", 512, 140000, 64, 8, 0.8),
    ("bf16", 64, 16000, 1024, 8, 1.0), ("fp16", 512, 16128, 1024, 8, 1.0), ("bf16", 200, 9000, 712, 8, 1.0), ("bf16", 40, 140001, 77, 8, 1.0)])
def test_distillation_over_long_vocabularies(dtype, rows, vocab, d, k, temperature):
    """Pieces above 16384 words, several of them, the step from 512 to 513 rows, sums of dx in several accumulators, and over
    clusters; listed words on both sides of where pieces may end."""
    x, w = normal((rows, d), dtype, 1), normal((vocab, d), dtype, 2, 2.0 * d ** -0.5)
    ids, teacher = lists(rows, vocab, k)
    ends = [e + o for e in (256, 8192, 14592, 16128, 16384, 20224, 32768, 65536) for o in (-1, 0, 1) if e + o < vocab] + [0, vocab - 1]
    for i, word in enumerate(ends):
        ids[i % rows, i // rows % k] = word
    dloss = torch.rand(rows, generator=gen(8), device="cuda") / rows
    got = distilled(x, w, ids, teacher, dloss, dtype, temperature)
    distill_check(x, w, ids, teacher, dloss, dtype, temperature, got)
    # a workspace made for more rows changes nothing
    again = distilled(x, w, ids, teacher, dloss, dtype, temperature)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert api.ds4moe_ops_status() == 0


def ragged(groups, average, spread, seed=5):
    g = torch.Generator().manual_seed(seed)
    return [max(0, average + int(v)) for v in (torch.randn(groups, generator=g) * spread).round().tolist()]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("counts,n,k", [
    (ragged(16, 200, 60), 1040, 1024), ([128] * 40, 600, 1000), ([0, 500, 1, 700, 15, 17, 900, 33] * 4, 520, 1280), ([20005, 17, 0, 300], 1040, 1024),
    ([1, 16384, 16385], 1288, 1024), (ragged(64, 256, 40), 776, 712), (ragged(30, 150, 100), 1024, 2200), ([3000], 4104, 1024)])
def test_ragged_weight_gradients_on_pairs(dtype, counts, n, k):
    """Groups with ends that are no multiple of 16, empty and long ones, next to rows that are not finite."""
    rows, g = sum(counts) + 9, len(counts)
    dy, x = whole((rows, n), dtype, 1), whole((rows, k), dtype, 2)
    dy[sum(counts):], x[sum(counts):] = NAN, NAN
    dw = torch.full((g, n, k), 7.0, dtype=x.dtype, device="cuda")
    api.ds4moe_grouped_mm_dw(dy, x, offsets(counts), dw, rows, n, k, g, dtype, stream=stream())
    for e, lo, hi in groups_of(counts):
        assert torch.equal(dw[e], (dy[lo:hi].double().T @ x[lo:hi].double()).to(dw.dtype)), (e, lo, hi)
    last = max(e for e, c in enumerate(counts) if c)  # a group's rows stay out of its neighbours'
    x[sum(counts[:last]) + counts[last] // 2, 3] = math.inf
    api.ds4moe_grouped_mm_dw(dy, x, offsets(counts), dw, rows, n, k, g, dtype, stream=stream())
    for e, lo, hi in groups_of(counts):
        if e != last:
            assert torch.equal(dw[e], (dy[lo:hi].double().T @ x[lo:hi].double()).to(dw.dtype)), (e, lo, hi)
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("counts", [[20, 400] * 8, [10, 0, 30, 900, 5, 1500, 300, 256], [257] * 8, [256] * 8, [200] * 8, [320, 321, 384, 385, 0, 448, 1, 255],
                                    [2000] + [30] * 9, [448, 449, 512, 447, 500, 433, 434, 441], [700, 1, 1, 1]])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_groups_beside_wide_tiles(dtype, counts):
    """Groups that fit a tile of both accumulators, and that do not, in every mixture: blocks and both products."""
    rows, g, n, k = sum(counts) + 3, len(counts), 2568, 264
    x, w = whole((rows, k), dtype, 1), whole((g, 2 * n, k), dtype, 2)
    x[sum(counts):] = NAN
    off = offsets(counts)
    h, z, clean = block(x, w, off, n, "relu", dtype)
    y, dx = (torch.full((rows, 2 * n), 7.0, dtype=x.dtype, device="cuda") for _ in range(2))
    api.ds4moe_grouped_mm(x, w, off, y, rows, 2 * n, k, g, dtype, stream=stream())
    api.ds4moe_grouped_mm_dx(x, w.transpose(1, 2).contiguous(), off, dx, rows, k, 2 * n, g, dtype, stream=stream())
    assert clean and torch.equal(z, y) and torch.equal(z, dx) and bool((y[sum(counts):] == 7.0).all()) and bool((h[sum(counts):] == 7.0).all())
    for e, lo, hi in groups_of(counts):
        ref = x[lo:hi].double() @ w[e].double().T
        assert torch.equal(z[lo:hi], ref.to(z.dtype)), e
        assert torch.equal(h[lo:hi], (ref[:, :n].clamp(min=0) * ref[:, n:]).to(h.dtype)), e
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("rows,vocab,top", [(1023, 3001, 28), (1024, 3001, 28), (1024, 3001, 29), (1031, 140001, 28), (2050, 999, 31), (1024, 40, 28)])
def test_best_words_of_many_rows(rows, vocab, top):
    """On both sides of where a warp instead of a block searches for a row's best words; equal logits in some rows."""
    x, w = grid((rows, 64), "bf16", 1, 16, 2.0 ** -4), grid((vocab, 64), "bf16", 2, 20, 2.0 ** -6)
    x[::7] = 0
    tokens = torch.randint(-1, vocab, (rows, 2), generator=gen(3), device="cuda", dtype=torch.int32)
    score_check(x, w, tokens, top, "bf16", 1.0, score(x, w, tokens, top))
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("average,spread", [(190, 120), (300, 30), (256, 5), (400, 200)])
def test_a_thousand_groups_beside_wide_tiles(average, spread):
    counts, n, k = ragged(1024, average, spread), 72, 64
    rows, g = sum(counts), len(counts)
    x, w, off = whole((rows, k), "bf16", 1), whole((g, 2 * n, k), "bf16", 2), offsets(counts)
    h, z, clean = block(x, w, off, n, "relu", "bf16")
    y = torch.full((rows, 2 * n), 7.0, dtype=x.dtype, device="cuda")
    api.ds4moe_grouped_mm(x, w, off, y, rows, 2 * n, k, g, "bf16", stream=stream())
    ref = torch.cat([x[lo:hi].double() @ w[e].double().T for e, lo, hi in groups_of(counts)])
    assert clean and torch.equal(z, ref.to(z.dtype)) and torch.equal(y, z)
    assert torch.equal(h, (ref[:, :n].clamp(min=0) * ref[:, n:]).to(h.dtype))
    assert api.ds4moe_ops_status() == 0
