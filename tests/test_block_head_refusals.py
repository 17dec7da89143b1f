"""CPU: what the gated block, the scores and the distillation refuse before touching a device."""
import pytest

from quantized_moe_gb300 import build as b
from quantized_moe_gb300 import ds4moe as api

b.build()
P = 16  # a pointer that no refused call follows
INVALID, FORMAT, CAPACITY = api.DS4MOE_ERR_INVALID_ARG, api.DS4MOE_ERR_UNSUPPORTED_FORMAT, api.DS4MOE_ERR_CAPACITY


def block(**kw):
    api.ds4moe_grouped_glu(**{**dict(x=P, w=P, offsets=P, h=P, rows=4, n=8, k=8, n_groups=2), **kw})


def block_grad(**kw):
    api.ds4moe_grouped_glu_grad(**{**dict(dh=P, x=P, w=P, offsets=P, z=P, dz=P, dx=P, dw=P, rows=4, n=8, k=8, n_groups=2), **kw})


def score(**kw):
    api.ds4moe_logprobs(**{**dict(x=P, w=P, tokens=P, logprob=P, lse=P, entropy=P, top_index=P, top_logprob=P, rows=4, vocab=100,
                                  d=8, n_tokens=1, top_k=3, workspace=P, workspace_bytes=1 << 20), **kw})


def distill(**kw):
    api.ds4moe_distill(**{**dict(x=P, w=P, ids=P, teacher=P, loss=P, lse=P, logq=P, rows=4, vocab=100, d=8, top_k=3, workspace=P,
                                 workspace_bytes=1 << 20), **kw})


def distill_grad(**kw):
    api.ds4moe_distill_grad(**{**dict(x=P, w=P, ids=P, teacher=P, lse=P, logq=P, dloss=P, dx=P, dw=P, rows=4, vocab=100, d=8,
                                      top_k=3, workspace=P, workspace_bytes=1 << 20), **kw})


NAN = float("nan")


@pytest.mark.parametrize("call,kw,code,msg", [
    (block, dict(rows=-1), INVALID, "rows=-1"), (block, dict(n=0), INVALID, "n=0"), (block, dict(n=(1 << 23) + 1), INVALID, "n="),
    (block, dict(k=0), INVALID, "k=0"), (block, dict(act=4), INVALID, "act=4"), (block, dict(dtype="fp32"), FORMAT, "dtype=2"),
    (block, dict(n_groups=0), INVALID, "n_groups=0"), (block, dict(n_groups=1025), INVALID, "n_groups=1025"),
    (block, dict(offsets=None), INVALID, "offsets is NULL"), (block, dict(ldh=7), INVALID, "ldh=7"), (block, dict(ldz=15), INVALID, "ldz=15"),
    (block, dict(ldx=7), INVALID, "ldx=7"), (block, dict(ldw=7), INVALID, "ldw=7"), (block, dict(w_stride=127), INVALID, "w_stride=127"),
    (block_grad, dict(rows=1 << 25), INVALID, "rows="), (block_grad, dict(n=-1), INVALID, "n=-1"), (block_grad, dict(lddh=7), INVALID, "lddh=7"),
    (block_grad, dict(lddz=15), INVALID, "lddz=15"), (block_grad, dict(lddx=7), INVALID, "lddx=7"), (block_grad, dict(lddw=7), INVALID, "lddw=7"),
    (block_grad, dict(dw_stride=127), INVALID, "dw_stride=127"), (block_grad, dict(act=-1), INVALID, "act=-1"),
    (block_grad, dict(offsets=None), INVALID, "offsets is NULL"), (block_grad, dict(rows=0, offsets=None), INVALID, "offsets is NULL"),
    (block_grad, dict(dtype=9), FORMAT, "dtype=9"),
    (score, dict(vocab=0), INVALID, "vocab=0"), (score, dict(d=0), INVALID, "d=0"), (score, dict(n_tokens=-1), INVALID, "n_tokens=-1"),
    (score, dict(n_tokens=257), INVALID, "n_tokens=257"), (score, dict(top_k=65), INVALID, "top_k=65"), (score, dict(top_k=-1), INVALID, "top_k=-1"),
    (score, dict(vocab=5, top_k=6), INVALID, "top_k=6"), (score, dict(temperature=0.0), INVALID, "temperature"),
    (score, dict(temperature=-1.0), INVALID, "temperature"), (score, dict(temperature=NAN), INVALID, "temperature"),
    (score, dict(temperature=1e4), INVALID, "temperature"), (score, dict(dtype="fp32"), FORMAT, "dtype=2"),
    (score, dict(workspace_bytes=4 * 4 * 100), CAPACITY, "workspace_bytes"), (score, dict(workspace_bytes=-1), CAPACITY, "workspace_bytes"),
    (score, dict(workspace_bytes=-2 ** 63), CAPACITY, "workspace_bytes"), (score, dict(ldx=7), INVALID, "ldx=7"), (score, dict(ldw=7), INVALID, "ldw=7"),
    (distill, dict(top_k=0), INVALID, "top_k=0"), (distill, dict(top_k=257), INVALID, "top_k=257"), (distill, dict(rows=-3), INVALID, "rows=-3"),
    (distill, dict(temperature=float("inf")), INVALID, "temperature"), (distill, dict(workspace_bytes=100), CAPACITY, "workspace_bytes"),
    (distill, dict(dtype=5), FORMAT, "dtype=5"), (distill, dict(vocab=(1 << 24) + 1), INVALID, "vocab="),
    (distill_grad, dict(workspace_bytes=2000), CAPACITY, "smallest piece"), (distill_grad, dict(workspace_bytes=-2 ** 63), CAPACITY, "smallest piece"),
    (distill_grad, dict(lddx=7), INVALID, "lddx=7"), (distill_grad, dict(lddw=7), INVALID, "lddw=7"), (distill_grad, dict(temperature=1e-4), INVALID, "temperature"),
    (distill_grad, dict(top_k=300), INVALID, "top_k=300"),
])
def test_refusals(call, kw, code, msg):
    with pytest.raises(api.Ds4MoeError) as ei:
        call(**kw)
    assert ei.value.code == code
    assert msg in api.ds4moe_last_error()


def test_no_rows_is_no_work():
    block(rows=0, x=None, w=None, offsets=None, h=None)
    score(rows=0, x=None, w=None, tokens=None, workspace=None, workspace_bytes=0)
    distill(rows=0, x=None, w=None, ids=None, workspace=None, workspace_bytes=0)
    distill_grad(dx=None, dw=None, workspace=None, workspace_bytes=1 << 20)  # nothing asked for


def test_workspace_sizes():
    # the logits are kept for the best words alone
    assert api.ds4moe_logprobs_workspace(4096, 129280, 4, 8) >= 4 * 4096 * 129280
    assert api.ds4moe_logprobs_workspace(4096, 129280, 4, 0) < 4096 * 129280 // 4
    assert api.ds4moe_logprobs_workspace(0, 10, 1, 1) > 0 and api.ds4moe_distill_workspace(0, 10, 10, 3) > 0
    # one piece of the vocabulary, not the logits
    assert api.ds4moe_distill_workspace(4096, 129280, 4096, 64) < 4096 * 129280 * 2 // 4
    # what the header gives for the smallest gradient
    rows, vocab, d, k = 70, 2000, 136, 5
    least = 16 + 4 * rows * (d + 1 + k) + 512 * 72 + 48
    with pytest.raises(api.Ds4MoeError) as ei:
        distill_grad(rows=rows, vocab=vocab, d=d, top_k=k, workspace_bytes=least - 48 - 16)
    assert ei.value.code == CAPACITY
