"""Training steps of a block whose experts, dense layer and head are kept in bf16.

    x  --router-->  top-k experts            ds4moe_route_noalloc (the quantized layer's router)
       --> h = silu(Wg x) * (Wu x)           ds4moe_grouped_mm, twice
       --> m = x + sum_j w_j Wd h            ds4moe_grouped_mm
       --> o = gelu(W m + b) + m             ds4moe_linear
       --> loss of o against the labels      ds4moe_cross_entropy
and back through the same operators' gradients, followed by a step of gradient descent. The router's
weights stay fixed. Everything runs on the current stream without synchronising.

    python examples/finetune_step.py [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_moe_gb300 import ds4moe as api  # noqa: E402

BF16 = torch.bfloat16
IGNORE = -100


def stream():
    return torch.cuda.current_stream().cuda_stream


def make_weights(d, f, n_experts, vocab, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)

    return {"router": torch.randn((n_experts, d), generator=g, device="cuda") * 0.02,
            "gate": normal(n_experts, f, d, scale=d ** -0.5), "up": normal(n_experts, f, d, scale=d ** -0.5),
            "down": normal(n_experts, d, f, scale=f ** -0.5), "dense": normal(d, d, scale=d ** -0.5),
            "bias": normal(d, scale=0.1), "head": normal(vocab, d, scale=d ** -0.5)}


class Experts:
    """The grouped products of one routed batch: slot s of the rows ordered by expert is token token[s]."""

    def __init__(self, x, router, top_k):
        rows, d = x.shape
        self.n, self.k = router.shape[0], top_k
        self.idx = torch.empty((rows, top_k), dtype=torch.int32, device="cuda")
        self.weight = torch.empty((rows, top_k), dtype=torch.float32, device="cuda")
        api.ds4moe_route_noalloc(router, None, x, rows, d, self.n, top_k, self.idx, self.weight, stream())
        flat = self.idx.flatten().long()
        self.order = torch.sort(flat, stable=True).indices
        self.token = self.order // top_k
        counts = torch.zeros(self.n, dtype=torch.int64, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))
        self.offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)

    def mm(self, x, w):
        y = torch.empty((x.shape[0], w.shape[1]), dtype=BF16, device="cuda")
        api.ds4moe_grouped_mm(x, w, self.offsets, y, x.shape[0], w.shape[1], w.shape[2], self.n, stream=stream())
        return y

    def mm_grad(self, dy, x, w):
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        sizes = dict(rows=x.shape[0], n=w.shape[1], k=w.shape[2], n_groups=self.n, stream=stream())
        api.ds4moe_grouped_mm_dx(dy, w, self.offsets, dx, **sizes)
        api.ds4moe_grouped_mm_dw(dy, x, self.offsets, dw, **sizes)
        return dx, dw

    def gather(self, per_token):
        return per_token[self.token]

    def combine(self, per_slot):
        """sum_j w_j y_j of each token, in its top-k order, in fp32."""
        slots = torch.empty_like(per_slot)
        slots[self.order] = per_slot
        return (slots.view(-1, self.k, per_slot.shape[1]).float() * self.weight[..., None]).sum(1)


def loss_and_gradients(w, x, labels, top_k):
    """The mean loss over the labelled rows, and the gradient of every trained weight."""
    rows, d = x.shape
    vocab = w["head"].shape[0]
    # ---- forward
    ex = Experts(x, w["router"], top_k)
    xe = ex.gather(x)
    gate, up = ex.mm(xe, w["gate"]), ex.mm(xe, w["up"])
    h = (torch.nn.functional.silu(gate.float()) * up.float()).to(BF16)
    ye = ex.mm(h, w["down"])
    m = (x.float() + ex.combine(ye)).to(BF16)
    o, z = torch.empty_like(m), torch.empty_like(m)
    api.ds4moe_linear(m, w["dense"], w["bias"], m, o, rows, d, d, "gelu", zout=z, stream=stream())
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    size = max(api.ds4moe_cross_entropy_workspace(rows, vocab, d), api.ds4moe_linear_grad_workspace(rows, d, "gelu"))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    head = dict(rows=rows, vocab=vocab, d=d, ignore_index=IGNORE, workspace=ws, workspace_bytes=size, stream=stream())
    api.ds4moe_cross_entropy(o, w["head"], labels, loss, lse, **head)
    kept = (labels != IGNORE).sum().clamp(min=1)
    # ---- backward
    grads = {name: torch.empty_like(w[name]) for name in ("dense", "bias", "head")}
    do, dm = torch.empty_like(o), torch.empty_like(m)
    dloss = (1.0 / kept.float()).expand(rows).contiguous()
    api.ds4moe_cross_entropy_grad(o, w["head"], labels, lse, dloss, do, grads["head"], **head)
    api.ds4moe_linear_grad(do, m, w["dense"], z, dm, grads["dense"], grads["bias"], rows, d, d, "gelu", workspace=ws,
                           workspace_bytes=size, stream=stream())
    dm = dm.float() + do.float()  # through the dense layer, and past it
    dye = (ex.gather(dm) * ex.weight.flatten()[ex.order][:, None]).to(BF16)
    dh, grads["down"] = ex.mm_grad(dye, h, w["down"])
    s = torch.sigmoid(gate.float())
    dgate = (dh.float() * up.float() * s * (1 + gate.float() * (1 - s))).to(BF16)
    dup = (dh.float() * gate.float() * s).to(BF16)
    _, grads["gate"] = ex.mm_grad(dgate, xe, w["gate"])
    _, grads["up"] = ex.mm_grad(dup, xe, w["up"])
    return loss.sum() / kept, grads


def train(steps, rows=512, d=512, f=256, n_experts=16, top_k=4, vocab=4000, lr=1.0, seed=0):
    """The losses of `steps` steps on one batch."""
    w = make_weights(d, f, n_experts, vocab, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn((rows, d), generator=g, device="cuda").to(BF16)
    labels = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    labels[::10] = IGNORE
    losses = []
    for _ in range(steps):
        loss, grads = loss_and_gradients(w, x, labels, top_k)
        for name, grad in grads.items():
            w[name] = (w[name].float() - lr * grad.float()).to(BF16)
        losses.append(loss)
    flags = api.ds4moe_ops_status()
    if flags:
        raise RuntimeError(f"the operators raised flags {flags:#x}")
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    for i, v in enumerate(train(ap.parse_args().steps)):
        print(f"step {i:3d}  loss {v:.4f}")
