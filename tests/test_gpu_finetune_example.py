"""GPU: the fine-tuning example's gradients against 64-bit autograd, and its loss going down."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("finetune_step", os.path.join(ROOT, "examples", "finetune_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_match_autograd(example):
    rows, d, f, n, k, vocab = 96, 256, 136, 8, 3, 1000
    w = example.make_weights(d, f, n, vocab)
    x = torch.randn((rows, d), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    labels = torch.randint(0, vocab, (rows,), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda", dtype=torch.int32)
    labels[::6] = example.IGNORE
    loss, grads = example.loss_and_gradients(w, x, labels, k)
    ex = example.Experts(x, w["router"], k)
    p = {name: t.double().requires_grad_(name != "router") for name, t in w.items()}
    x64 = x.double()
    m = x64
    for j in range(k):
        e = ex.idx[:, j].long()
        g, u = torch.einsum("td,tfd->tf", x64, p["gate"][e]), torch.einsum("td,tfd->tf", x64, p["up"][e])
        y = torch.einsum("tf,tdf->td", torch.nn.functional.silu(g) * u, p["down"][e])
        m = m + ex.weight[:, j].double()[:, None] * y
    o = torch.nn.functional.gelu(m @ p["dense"].T + p["bias"]) + m
    want = torch.nn.functional.cross_entropy(o @ p["head"].T, labels.long(), ignore_index=example.IGNORE)
    want.backward()
    # every tensor handed from one operator to the next is rounded to bf16 (2^-9 of an element on average, at
    # most ten of them on the longest way); the loss is a mean over independent errors
    assert abs(float(loss) - float(want.detach())) <= 10 * 2.0 ** -9
    for name, grad in grads.items():
        rel = float((grad.double() - p[name].grad).norm() / p[name].grad.norm())
        assert rel <= 10 * 2.0 ** -9, (name, rel)


def test_the_loss_goes_down(example):
    losses = example.train(12)
    assert losses[-1] < losses[0] - 1.0
    assert all(b < a + 0.05 for a, b in zip(losses, losses[1:]))
