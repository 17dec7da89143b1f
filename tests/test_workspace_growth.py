"""CPU: a workspace for the largest batch serves every smaller one. The queries never fall as the rows grow, and a call of
fewer rows is not refused the bytes that were returned for more."""
import itertools

import pytest

from quantized_moe_gb300 import build as b
from quantized_moe_gb300 import ds4moe as api

b.build()
P = 16  # a pointer that no call follows: without a device it ends there, with one its checks do
VOCABS = (1, 33, 700, 32000, 50257, 129280, 151936)
STEPS = [*range(1, 48), 63, 64, 65, 89, 90, 103, 104, 127, 128, 129, 255, 256, 257, 300, 504, 505, 511, 512, 513, 520, 1000, 2049]


def rising(sizes):
    return all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("vocab", VOCABS)
def test_queries_never_fall(vocab):
    for n, top in itertools.product((0, 1, 4, 5, 100, 256), (0, 1, 8, 64)):
        if top <= vocab:
            assert rising([api.ds4moe_logprobs_workspace(r, vocab, n, top) for r in STEPS]), (n, top)
    for d, k in itertools.product((1, 72, 4096), (1, 32, 256)):
        assert rising([api.ds4moe_distill_workspace(r, vocab, d, k) for r in STEPS]), (d, k)
        assert rising([api.ds4moe_cross_entropy_workspace(r, vocab, d) for r in STEPS]), d
        assert rising([api.ds4moe_linear_grad_workspace(r, vocab, "silu") for r in STEPS])


@pytest.mark.parametrize("vocab,n,top", [(129280, 1, 0), (32000, 100, 0), (32000, 1, 0), (50257, 1, 0), (32000, 1, 8), (700, 200, 3)])
def test_fewer_rows_are_not_refused(vocab, n, top):
    for most in (33, 34, 40, 46, 64, 100, 127, 128, 200):
        size = api.ds4moe_logprobs_workspace(most, vocab, n, top)
        for rows in (1, 5, 11, 13, 24, 31, 32, 33):
            if rows > most:
                continue
            with pytest.raises(api.Ds4MoeError) as ei:
                api.ds4moe_logprobs(P, P, P, P, P, P, P, P, rows, vocab, 64, n, top, workspace=P, workspace_bytes=size)
            assert ei.value.code != api.DS4MOE_ERR_CAPACITY, (most, rows)
            if top == 0:
                size_d = api.ds4moe_distill_workspace(most, vocab, 64, n)
                with pytest.raises(api.Ds4MoeError) as ei:
                    api.ds4moe_distill(P, P, P, P, P, P, P, rows, vocab, 64, n, workspace=P, workspace_bytes=size_d)
                assert ei.value.code != api.DS4MOE_ERR_CAPACITY, (most, rows)


def test_a_gradient_of_fewer_rows_keeps_its_pieces():
    """The distillation's gradient takes up to 512 rows in pieces of up to 64 MB: a workspace for more rows holds them."""
    for vocab in VOCABS:
        for rows in (8, 100, 264, 512):
            wide = max(16384, (1 << 25) // ((rows + 7) // 8 * 8) // 256 * 256)
            piece = 2 * ((rows + 7) // 8 * 8) * min(wide, (vocab + 255) // 256 * 256)
            for most in (rows, 513, 700, 2000):
                assert api.ds4moe_distill_workspace(most, vocab, 72, 9) >= piece + 16 + 4 * rows * (72 + 1 + 9)
