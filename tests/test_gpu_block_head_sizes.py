"""GPU: the gated block, the scores and the distillation at the sizes where they change their form: workspaces made for
more rows, pieces of the vocabulary above 16384 words, selections among words that are not numbers, ragged weight gradients
on pairs of CTAs, groups on both sides of a tile. Tolerances as in test_gpu_block_head."""
import pytest
import torch

from quantized_moe_gb300 import ds4moe as api
from test_gpu_block_head import grid, score, score_check
from test_gpu_mm16 import gen

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
