"""Cases of the 16-bit operators that stand next to the quantized MoE layer: the experts' matrix
products grouped by ragged token counts (with both gradients), the dense product with bias,
activation and residual in its epilogue (with its gradients), and the softmax cross entropy over
a large vocabulary (with its gradients).

`own` selects what `run` does: False computes each operator in elementary torch operations in 32
bits, rounded once at the end; True calls the library's entry points. `exact` is the definition in
64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IGNORE = -100


def listed():
    return [
        # one token's eight routed experts out of 256: the gate product of a decode step, one row
        # per touched expert; reading the touched weights is all there is
        dict(name="experts-token", op="grouped", direction="y", dtype="bf16", rows=8, groups=256, n=2048, k=4096,
             spread="distinct"),
        # 512 tokens with Zipf-skewed routing, eight experts each: the down product of a short
        # prompt (few rows per expert, some experts with hundreds, some with none)
        dict(name="experts-512", op="grouped", direction="y", dtype="bf16", rows=4096, groups=256, n=4096, k=2048,
             spread="zipf"),
        # 4096 tokens, uniform routing: the gate product of a long prompt
        dict(name="experts-4096", op="grouped", direction="y", dtype="fp16", rows=32768, groups=256, n=2048, k=4096,
             spread="uniform"),
        # the gradient of the same product with respect to its tokens
        dict(name="experts-4096-dx", op="grouped", direction="dx", dtype="bf16", rows=32768, groups=256, n=2048,
             k=4096, spread="uniform"),
        # and with respect to the weights of every expert
        dict(name="experts-4096-dw", op="grouped", direction="dw", dtype="bf16", rows=32768, groups=256, n=2048,
             k=4096, spread="uniform", dw_dtype="bf16"),
        # a small fine-tuning batch: odd row counts, experts without rows, widths that no tile
        # divides, gradients accumulated by the optimizer in 32 bits
        dict(name="experts-ragged-dw", op="grouped", direction="dw", dtype="fp16", rows=1537, groups=24, n=1000,
             k=712, spread="zipf", dw_dtype="fp32"),
        # a projection for one token with the residual stream added
        dict(name="dense-token", op="linear", direction="y", dtype="bf16", rows=1, n=4096, k=4096, act="none",
             bias=True, residual=True, packed=False),
        # widths that are no multiple of anything, read out of a wider buffer
        dict(name="dense-odd", op="linear", direction="y", dtype="fp16", rows=333, n=1001, k=517, act="gelu",
             bias=True, residual=False, packed=True),
        # the projection of a long prompt
        dict(name="dense-4096", op="linear", direction="y", dtype="bf16", rows=4096, n=4096, k=4096, act="silu",
             bias=True, residual=True, packed=False),
        # a training step through a dense layer of the shared expert's width
        dict(name="dense-4096-grad", op="linear", direction="grad", dtype="bf16", rows=4096, n=2048, k=4096,
             act="silu", bias=True, residual=True, packed=False),
        # scoring a drafted continuation of 16 tokens: losses only
        dict(name="loss-16", op="loss", direction="y", dtype="bf16", rows=16, vocab=129280, d=4096),
        # a training step of the head: losses and both gradients
        dict(name="loss-2048-grad", op="loss", direction="grad", dtype="bf16", rows=2048, vocab=129280, d=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A matrix width: usually a multiple of 8, as models have them, sometimes any number."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.3 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["grouped", "grouped", "linear", "linear", "loss"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "grouped":
        return dict(op=op, direction=rng.choice(["y", "dx", "dw"]), dtype=dtype, rows=_log(rng, 1, 32768),
                    groups=_log(rng, 1, 256), n=_width(rng, 64, 4096), k=_width(rng, 64, 4096),
                    spread=rng.choice(["uniform", "zipf"]), dw_dtype=rng.choice([dtype, "fp32"]))
    if op == "linear":
        return dict(op=op, direction=rng.choice(["y", "y", "grad"]), dtype=dtype, rows=_log(rng, 1, 8192),
                    n=_width(rng, 64, 4096), k=_width(rng, 64, 4096),
                    act=rng.choice(["none", "relu", "silu", "gelu"]), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, packed=rng.random() < 0.3)
    return dict(op=op, direction=rng.choice(["y", "grad"]), dtype=dtype, rows=_log(rng, 1, 2048),
                vocab=_log(rng, 1000, 129280), d=_width(rng, 64, 4096))


def _shares(case):
    """The share of the rows that each group gets."""
    g = case["groups"]
    if case["spread"] == "zipf":
        w = [(i + 1) ** -1.1 for i in range(g)]
        return [v / sum(w) for v in w]
    return [1.0 / g] * g


def _counts(case, gen):
    """Rows of each group: int32 [groups] on the host."""
    g, rows = case["groups"], case["rows"]
    if case["spread"] == "distinct":
        counts = torch.zeros(g, dtype=torch.int64)
        counts[torch.randperm(g, generator=gen)[:rows]] = 1
        return counts
    p = torch.tensor(_shares(case), dtype=torch.float64)[torch.randperm(g, generator=gen)]
    return torch.bincount(torch.multinomial(p, rows, replacement=True, generator=gen), minlength=g)


def _inputs(case, seed):
    dt = DTYPES[case["dtype"]]
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        t = torch.empty(shape, dtype=dt, device="cuda")
        return t.normal_(0.0, scale, generator=gen)

    s = {"case": case}
    if case["op"] == "grouped":
        rows, n, k, g = case["rows"], case["n"], case["k"], case["groups"]
        counts = _counts(case, host)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
        if case["direction"] == "y":
            s["x"], s["w"] = normal(rows, k), normal(g, n, k, scale=k ** -0.5)
        elif case["direction"] == "dx":
            s["dy"], s["w"] = normal(rows, n), normal(g, n, k, scale=k ** -0.5)
        else:
            s["dy"], s["x"] = normal(rows, n), normal(rows, k)
    elif case["op"] == "linear":
        rows, n, k = case["rows"], case["n"], case["k"]
        # packed: the operand is one half of a projection's output that holds two
        s["x"] = normal(rows, 2 * k)[:, k:] if case["packed"] else normal(rows, k)
        s["w"] = normal(n, k, scale=k ** -0.5)
        if case["direction"] == "y":
            s["bias"] = normal(n) if case["bias"] else None
            s["residual"] = normal(rows, n) if case["residual"] else None
        else:
            s["dy"] = normal(rows, n)
            s["z"] = None if case["act"] == "none" else normal(rows, n)  # what the forward kept
    else:
        rows, vocab, d = case["rows"], case["vocab"], case["d"]
        s["x"], s["w"] = normal(rows, d), normal(vocab, d, scale=1.3 * d ** -0.5)
        labels = torch.randint(0, vocab, (rows,), generator=host)
        skip = torch.rand(rows, generator=host) < 0.1  # padding: no loss and no gradient
        labels[skip] = IGNORE
        s["labels"] = labels.to(torch.int32).cuda()
        s["dloss"] = torch.full((rows,), 1.0 / max(1, int((~skip).sum())), device="cuda")  # of the mean
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    dt = DTYPES[case["dtype"]]
    empty = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device="cuda")
    if case["op"] == "grouped":
        out = {"y": (case["rows"], case["n"]), "dx": (case["rows"], case["k"]),
               "dw": (case["groups"], case["n"], case["k"])}[case["direction"]]
        s["out"] = empty(*out, dtype=DTYPES[case["dw_dtype"]] if case["direction"] == "dw" else dt)
    elif case["op"] == "linear":
        if case["direction"] == "y":
            s["y"] = empty(case["rows"], case["n"])
        else:
            s["dx"], s["dw"], s["db"] = empty(case["rows"], case["k"]), empty(case["n"], case["k"]), empty(case["n"])
            # the scratch that a program keeps: dz, and 32-bit partial sums of db
            s["scratch"] = empty(2 * case["rows"] * (case["n"] + 8) + 1024 * (case["n"] + 64) + (1 << 16),
                                 dtype=torch.uint8)
    else:
        rows, vocab, d = case["rows"], case["vocab"], case["d"]
        s["loss"], s["lse"] = empty(rows, dtype=torch.float32), empty(rows, dtype=torch.float32)
        # the scratch that a program keeps: softmax partials or one piece of the vocabulary (8192 wide)
        s["scratch"] = empty(rows * (2 * 8192 + 4 * d + vocab // 8 + 256) + (1 << 20), dtype=torch.uint8)
        if case["direction"] == "grad":
            s["dx"], s["dw"] = empty(rows, d), empty(vocab, d)
    return s


# ------------------------------------------------------------------------------------- plain form


def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


def _plain_grouped(s):
    case, out = s["case"], s["out"]
    ends = s["offsets"].tolist()
    for g in range(case["groups"]):
        lo, hi = ends[g], ends[g + 1]
        if lo == hi:
            if case["direction"] == "dw":
                out[g] = 0
        elif case["direction"] == "y":
            out[lo:hi] = s["x"][lo:hi].float() @ s["w"][g].float().T
        elif case["direction"] == "dx":
            out[lo:hi] = s["dy"][lo:hi].float() @ s["w"][g].float()
        else:
            out[g] = s["dy"][lo:hi].float().T @ s["x"][lo:hi].float()
    return out


def _plain_linear(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["direction"] == "y":
        z = s["x"].float() @ s["w"].float().T
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(dt)
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), case["act"])
    return {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.T @ s["x"].float()).to(dt), "db": dz.sum(0).to(dt)}


def _plain_loss(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    x, w, labels = s["x"].float(), s["w"].float(), s["labels"].long()
    kept = labels != IGNORE
    at = torch.where(kept, labels, 0).unsqueeze(1)
    z = x @ w.T
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    loss = torch.where(kept, (lse - z.gather(1, at)).squeeze(1), 0.0)
    out = {"loss": loss, "lse": lse.squeeze(1)}
    if case["direction"] == "grad":
        dz = e / total
        dz.scatter_add_(1, at, torch.full_like(total, -1.0))
        dz *= torch.where(kept, s["dloss"], 0.0).unsqueeze(1)
        out["dx"], out["dw"] = (dz @ w).to(dt), (dz.T @ x).to(dt)
    return out


# ------------------------------------------------------------------------- the library's operators


def _own_grouped(s):
    from quantized_moe_gb300 import ds4moe as api

    c, stream = s["case"], torch.cuda.current_stream().cuda_stream
    sizes = dict(rows=c["rows"], n=c["n"], k=c["k"], n_groups=c["groups"], dtype=c["dtype"], stream=stream)
    if c["direction"] == "y":
        api.ds4moe_grouped_mm(s["x"], s["w"], s["offsets"], s["out"], **sizes)
    elif c["direction"] == "dx":
        api.ds4moe_grouped_mm_dx(s["dy"], s["w"], s["offsets"], s["out"], **sizes)
    else:
        api.ds4moe_grouped_mm_dw(s["dy"], s["x"], s["offsets"], s["out"], dw_dtype=c["dw_dtype"], **sizes)
    return s["out"]


def _own_linear(s):
    from quantized_moe_gb300 import ds4moe as api

    c, stream = s["case"], torch.cuda.current_stream().cuda_stream
    sizes = dict(rows=c["rows"], n=c["n"], k=c["k"], act=c["act"], dtype=c["dtype"], ldx=s["x"].stride(0),
                 stream=stream)
    if c["direction"] == "y":
        api.ds4moe_linear(s["x"], s["w"], s["bias"], s["residual"], s["y"], **sizes)
        return s["y"]
    api.ds4moe_linear_grad(s["dy"], s["x"], s["w"], s["z"], s["dx"], s["dw"], s["db"], workspace=s["scratch"],
                           workspace_bytes=s["scratch"].numel(), **sizes)
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def _own_loss(s):
    from quantized_moe_gb300 import ds4moe as api

    c, stream = s["case"], torch.cuda.current_stream().cuda_stream
    sizes = dict(rows=c["rows"], vocab=c["vocab"], d=c["d"], dtype=c["dtype"], ignore_index=IGNORE,
                 workspace=s["scratch"], workspace_bytes=s["scratch"].numel(), stream=stream)
    api.ds4moe_cross_entropy(s["x"], s["w"], s["labels"], s["loss"], s["lse"], **sizes)
    out = {"loss": s["loss"], "lse": s["lse"]}
    if c["direction"] == "grad":
        api.ds4moe_cross_entropy_grad(s["x"], s["w"], s["labels"], s["lse"], s["dloss"], s["dx"], s["dw"], **sizes)
        out["dx"], out["dw"] = s["dx"], s["dw"]
    return out


def run(state):
    forms = {"grouped": (_plain_grouped, _own_grouped), "linear": (_plain_linear, _own_linear),
             "loss": (_plain_loss, _own_loss)}
    return forms[state["case"]["op"]][1 if own else 0](state)


def work(case):
    size = 2
    if case["op"] == "grouped":
        rows, n, k, g = case["rows"], case["n"], case["k"], case["groups"]
        if case["spread"] == "distinct":
            touched = min(rows, g)
        else:
            touched = sum(1 - (1 - p) ** rows for p in _shares(case))  # expected
        if case["direction"] == "dw":
            weights = g * n * k * (4 if case["dw_dtype"] == "fp32" else size)
        else:
            weights = touched * n * k * size
        return {"bytes": int(weights + rows * (n + k) * size + (g + 1) * 4), "flops": 2 * rows * n * k}
    if case["op"] == "linear":
        rows, n, k = case["rows"], case["n"], case["k"]
        if case["direction"] == "y":
            extra = n * case["bias"] + rows * n * case["residual"]
            return {"bytes": size * (rows * k + n * k + rows * n + extra), "flops": 2 * rows * n * k}
        held = rows * n * (1 + (case["act"] != "none"))
        return {"bytes": size * (held + 2 * rows * k + 2 * n * k + n), "flops": 4 * rows * n * k}
    rows, vocab, d = case["rows"], case["vocab"], case["d"]
    if case["direction"] == "y":
        return {"bytes": size * (rows * d + vocab * d) + 12 * rows, "flops": 2 * rows * vocab * d}
    return {"bytes": size * (2 * rows * d + 2 * vocab * d) + 16 * rows, "flops": 6 * rows * vocab * d}


def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits."""
    s = _inputs(case, seed)
    f64 = {name: t.double() if torch.is_tensor(t) and t.is_floating_point() and t.dim() < 3 else t
           for name, t in s.items()}
    if case["op"] == "grouped":
        counts = (s["offsets"][1:] - s["offsets"][:-1]).cpu()
        parts = {name: f64[name].split(counts.tolist()) for name in ("x", "dy") if name in f64}
        if case["direction"] == "dw":
            dw = [torch.einsum("tn,tk->nk", a, b) for a, b in zip(parts["dy"], parts["x"])]
            return torch.stack(dw)
        if case["direction"] == "y":
            return torch.cat([torch.einsum("tk,nk->tn", a, s["w"][e].double()) for e, a in enumerate(parts["x"])])
        return torch.cat([torch.einsum("tn,nk->tk", a, s["w"][e].double()) for e, a in enumerate(parts["dy"])])
    if case["op"] == "linear":
        act = {"none": lambda z: z, "relu": torch.nn.functional.relu, "silu": torch.nn.functional.silu,
               "gelu": torch.nn.functional.gelu}[case["act"]]
        if case["direction"] == "y":
            z = torch.einsum("tk,nk->tn", f64["x"], f64["w"])
            y = act(z if s["bias"] is None else z + f64["bias"])
            return y if s["residual"] is None else y + f64["residual"]
        dz = f64["dy"]
        if s["z"] is not None:
            z = f64["z"].requires_grad_()
            (dz,) = torch.autograd.grad(act(z), z, dz)
        return {"dx": torch.einsum("tn,nk->tk", dz, f64["w"]), "dw": torch.einsum("tn,tk->nk", dz, f64["x"]),
                "db": torch.einsum("tn->n", dz)}
    rows, vocab = case["rows"], case["vocab"]
    labels, kept = s["labels"].long(), s["labels"] != IGNORE
    grad = case["direction"] == "grad"
    chunks = [(v, min(v + 16384, vocab)) for v in range(0, vocab, 16384)]
    lse = torch.full((rows,), -math.inf, dtype=torch.float64, device="cuda")
    own_z = torch.zeros(rows, dtype=torch.float64, device="cuda")
    for lo, hi in chunks:
        z = f64["x"] @ f64["w"][lo:hi].T
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        here = (labels >= lo) & (labels < hi)
        own_z[here] = z[here, labels[here] - lo]
    out = {"loss": torch.where(kept, lse - own_z, 0.0), "lse": lse}
    if grad:
        dx, dw = torch.zeros_like(f64["x"]), []
        for lo, hi in chunks:
            dz = torch.exp(f64["x"] @ f64["w"][lo:hi].T - lse[:, None])
            here = (labels >= lo) & (labels < hi)
            dz[here, labels[here] - lo] -= 1
            dz *= torch.where(kept, f64["dloss"], 0.0)[:, None]
            dx += dz @ f64["w"][lo:hi]
            dw.append(dz.T @ f64["x"])
        out["dx"], out["dw"] = dx, torch.cat(dw)
    return out
