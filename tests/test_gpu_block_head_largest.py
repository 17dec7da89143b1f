"""GPU: the gated block, the scores and the distillation at the ends of their ranges: 2^23 features, 2^24 words, sums of 2^24 terms."""
import pytest
import torch

from quantized_moe_gb300 import ds4moe as api
from test_gpu_block_head import block, grid, score, score_check
from test_gpu_mm16 import gen, stream, whole

pytestmark = pytest.mark.gpu
MOST = 1 << 24


@pytest.mark.parametrize("rows", [1, 3, 300])
def test_a_block_of_as_many_features_as_there_may_be(rows):
    n, k = MOST // 2, 8
    x, w = whole((rows, k), "bf16", 1), whole((1, 2 * n, k), "bf16", 2)
    h, z, clean = block(x, w, None, n, "relu", "bf16")
    assert clean
    for lo in range(0, n, 1 << 20):  # (in pieces: the 64-bit form of all features would take 80 GB)
        a, b = (x.double() @ w[0, o + lo:o + lo + (1 << 20)].double().T for o in (0, n))
        assert torch.equal(h[:, lo:lo + (1 << 20)], (a.clamp(min=0) * b).to(h.dtype))
        assert torch.equal(z[:, lo:lo + (1 << 20)], a.to(z.dtype)) and torch.equal(z[:, n + lo:n + lo + (1 << 20)], b.to(z.dtype))
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("rows,top", [(1, 64), (2, 5), (33, 9)])
def test_scores_of_as_many_words_as_there_may_be(rows, top):
    x, w = grid((rows, 8), "bf16", 1, 16, 2.0 ** -4), grid((MOST, 8), "bf16", 2, 20, 2.0 ** -5)
    tokens = torch.randint(0, MOST, (rows, 6), generator=gen(3), device="cuda", dtype=torch.int32)
    tokens[0, 0], tokens[-1, 1] = MOST - 1, 0
    score_check(x, w, tokens, top, "bf16", 1.0, score(x, w, tokens, top))
    assert api.ds4moe_ops_status() == 0


@pytest.mark.parametrize("rows", [2, 40])
def test_scores_of_as_long_sums_as_there_may_be(rows):
    vocab = 5
    x, w = whole((rows, MOST), "bf16", 1, 1), whole((vocab, MOST), "bf16", 2, 1)
    x[:, MOST // 64:] = 0  # (sums below 2^24 / 64: a step of the logits' fp32 is well below 1)
    x[:, -1], w[:, -1] = 1, 1
    tokens = torch.randint(0, vocab, (rows, 1), generator=gen(3), device="cuda", dtype=torch.int32)
    z = torch.stack([(x[t, :MOST // 64].double() * w[:, :MOST // 64].double()).sum(1) + 1 for t in range(rows)])
    got = score(x, w, tokens, vocab, temperature=100.0)
    logp = torch.log_softmax(z / 100, 1)
    assert torch.equal(got["top_index"].long(), torch.sort(z, dim=1, descending=True, stable=True).indices)
    # exact logits; lse and the quotients are off by a few steps of fp32
    assert bool(((got["logprob"] - logp.gather(1, tokens.long())).abs() <= 2.0 ** -20 * (1 + z.abs().max() / 100)).all())
    assert bool(((got["top_logprob"] - logp.gather(1, got["top_index"].long())).abs() <= 2.0 ** -20 * (1 + z.abs().max() / 100)).all())
    assert api.ds4moe_ops_status() == 0


def test_the_distillation_over_as_many_words_as_there_may_be():
    """Where the student's words have equal logits, q is 1 / vocab: the gradient is -p x at the listed words and x / vocab elsewhere."""
    rows, d, k = 3, 8, 4
    x, w = whole((rows, d), "bf16", 1), torch.zeros((MOST, d), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([[0, 1, MOST - 1, 5], [7, MOST // 2, 9, -1], [MOST - 2, 4, 3, 2]], dtype=torch.int32, device="cuda")
    teacher = torch.randn((rows, k), generator=gen(3), device="cuda")
    loss, lse, logq = (torch.empty(s, device="cuda") for s in ((rows,), (rows,), (rows, k)))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    size = api.ds4moe_distill_workspace(rows, MOST, d, k)
    args = dict(rows=rows, vocab=MOST, d=d, top_k=k, workspace=torch.empty(size, dtype=torch.uint8, device="cuda"), workspace_bytes=size, stream=stream())
    api.ds4moe_distill(x, w, ids, teacher, loss, lse, logq, **args)
    api.ds4moe_distill_grad(x, w, ids, teacher, lse, logq, torch.ones(rows, device="cuda"), dx, dw, **args)
    # sums of 2^24 ones (each thread's, a warp's, a block's): exact but for the logarithm
    assert bool(((lse - 24 * 0.6931471805599453).abs() <= 2.0 ** -18).all())
    p = torch.softmax(torch.where(ids >= 0, teacher, -float("inf")).double(), 1)
    assert not bool(dx.any())  # (W is zero)
    want = torch.zeros((MOST, d), dtype=torch.float64, device="cuda") + x.double().sum(0) / MOST
    for t in range(rows):
        for j in range(k):
            if ids[t, j] >= 0:
                want[ids[t, j]] -= p[t, j] * x[t].double()
    # dz and the result each rounded to bf16; q is off by lse's error, 2^-18, and its exponential's
    size_of = torch.zeros((MOST, d), dtype=torch.float64, device="cuda") + x.double().abs().sum(0) / MOST
    for t in range(rows):
        for j in range(k):
            if ids[t, j] >= 0:
                size_of[ids[t, j]] += p[t, j] * x[t].double().abs()
    assert bool(((dw.double() - want).abs() <= 2 * 2.0 ** -8 * size_of + 2.0 ** -16 * size_of + 2.0 ** -60).all())
    assert api.ds4moe_ops_status() == 0
