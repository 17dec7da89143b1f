"""CPU: what the operators on 16-bit matrices refuse before touching a device."""
import pytest

from quantized_moe_gb300 import build as b
from quantized_moe_gb300 import ds4moe as api

b.build()
P = 16  # a pointer that no refused call follows


def grouped(**kw):
    a = dict(x=P, w=P, offsets=P, y=P, rows=4, n=8, k=8, n_groups=2)
    a.update(kw)
    api.ds4moe_grouped_mm(**a)


def grouped_dw(**kw):
    a = dict(dy=P, x=P, offsets=P, dw=P, rows=4, n=8, k=8, n_groups=2)
    a.update(kw)
    api.ds4moe_grouped_mm_dw(**a)


def linear(**kw):
    a = dict(x=P, w=P, bias=None, residual=None, y=P, rows=4, n=8, k=8)
    a.update(kw)
    api.ds4moe_linear(**a)


def linear_grad(**kw):
    a = dict(dy=P, x=P, w=P, z=P, dx=P, dw=P, db=P, rows=4, n=8, k=8, act="silu", workspace=P, workspace_bytes=1 << 20)
    a.update(kw)
    api.ds4moe_linear_grad(**a)


def loss(**kw):
    a = dict(x=P, w=P, labels=P, loss=P, lse=P, rows=4, vocab=100, d=8, workspace=P, workspace_bytes=1 << 20)
    a.update(kw)
    api.ds4moe_cross_entropy(**a)


def loss_grad(**kw):
    a = dict(x=P, w=P, labels=P, lse=P, dloss=P, dx=P, dw=P, rows=4, vocab=100, d=8, workspace=P, workspace_bytes=1 << 20)
    a.update(kw)
    api.ds4moe_cross_entropy_grad(**a)


INVALID, FORMAT, CAPACITY = api.DS4MOE_ERR_INVALID_ARG, api.DS4MOE_ERR_UNSUPPORTED_FORMAT, api.DS4MOE_ERR_CAPACITY


@pytest.mark.parametrize("call,kw,code,msg", [
    (grouped, dict(rows=-1), INVALID, "rows=-1"), (grouped, dict(n=0), INVALID, "n=0"), (grouped, dict(k=-3), INVALID, "k=-3"),
    (grouped, dict(rows=(1 << 24) + 1), INVALID, "rows="), (grouped, dict(n_groups=0), INVALID, "n_groups=0"),
    (grouped, dict(n_groups=1025), INVALID, "n_groups=1025"), (grouped, dict(dtype="fp32"), FORMAT, "dtype=2"),
    (grouped, dict(dtype=7), FORMAT, "dtype=7"), (grouped, dict(ldx=7), INVALID, "ldx=7"), (grouped, dict(ldw=-8), INVALID, "ldw=-8"),
    (grouped, dict(ldy=1), INVALID, "ldy=1"), (grouped, dict(w_stride=63), INVALID, "w_stride=63"),
    (grouped_dw, dict(dtype="bf16", dw_dtype="fp16"), FORMAT, "dw_dtype"), (grouped_dw, dict(lddw=7), INVALID, "lddw=7"),
    (grouped_dw, dict(dw_stride=8), INVALID, "dw_stride=8"), (grouped_dw, dict(lddy=5), INVALID, "lddy=5"),
    (linear, dict(act=4), INVALID, "act=4"), (linear, dict(act=-1), INVALID, "act=-1"), (linear, dict(ldr=7), INVALID, "ldr=7"),
    (linear, dict(ldz=7), INVALID, "ldz=7"), (linear, dict(k=(1 << 24) + 1), INVALID, "k="),
    (linear_grad, dict(workspace_bytes=15), CAPACITY, "workspace_bytes"), (linear_grad, dict(lddx=7), INVALID, "lddx=7"),
    (linear_grad, dict(act=9), INVALID, "act=9"), (linear_grad, dict(rows=-2), INVALID, "rows=-2"),
    (loss, dict(vocab=0), INVALID, "vocab=0"), (loss, dict(d=0), INVALID, "d=0"), (loss, dict(workspace_bytes=47), CAPACITY, "workspace_bytes"),
    (loss, dict(dtype=2), FORMAT, "dtype=2"), (loss_grad, dict(workspace_bytes=2000), CAPACITY, "smallest piece"),
    (loss_grad, dict(lddw=7), INVALID, "lddw=7"), (loss_grad, dict(workspace_bytes=-1), CAPACITY, "workspace_bytes"),
])
def test_refusals(call, kw, code, msg):
    with pytest.raises(api.Ds4MoeError) as ei:
        call(**kw)
    assert ei.value.code == code
    assert msg in api.ds4moe_last_error()


@pytest.mark.parametrize("call,kw", [(linear, dict(act="tanh")), (grouped, dict(dtype="int8"))])
def test_unknown_names_are_refused(call, kw):
    with pytest.raises(ValueError):
        call(**kw)


def test_no_rows_is_no_work():
    grouped(rows=0, x=None, w=None, offsets=None, y=None)
    linear(rows=0, x=None, w=None, y=None)
    loss(rows=0, x=None, w=None, labels=None, loss=None, lse=None, workspace=None, workspace_bytes=0)


def test_workspace_sizes():
    assert api.ds4moe_linear_grad_workspace(100, 33, "silu") >= 2 * 100 * 33 + 4 * 33
    assert api.ds4moe_linear_grad_workspace(100, 33, "none") < api.ds4moe_linear_grad_workspace(100, 33, "silu")
    # one piece of the vocabulary, not the logits
    assert api.ds4moe_cross_entropy_workspace(4096, 129280, 4096) < 4096 * 129280 * 2 // 4
    assert api.ds4moe_cross_entropy_workspace(0, 10, 10) > 0
