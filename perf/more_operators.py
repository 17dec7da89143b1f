"""Cases of the operators for a 16-bit block and its head: the gated feed-forward product of the experts
(with its gradients), the log probabilities of given tokens with entropy and top alternatives, and the
distillation from a teacher's top logits (with its gradients).

`own` selects what `run` does: False computes each operator in elementary torch operations in 32 bits,
rounded once at the end; True calls the library's entry points. `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one token's eight routed experts out of 256: gate, up and their product in a decode step
        dict(name="block-token", op="block", direction="y", dtype="bf16", rows=8, groups=256, n=2048, k=4096,
             act="silu", spread="distinct", keep=False),
        # 512 tokens with Zipf-skewed routing, eight experts each: a short prompt
        dict(name="block-512", op="block", direction="y", dtype="bf16", rows=4096, groups=256, n=2048, k=4096,
             act="silu", spread="zipf", keep=False),
        # the always-on shared expert of a 4096-token prompt: one dense block
        dict(name="block-shared-4096", op="block", direction="y", dtype="bf16", rows=4096, groups=0, n=2048, k=4096,
             act="silu", spread="uniform", keep=False),
        # a training batch over 64 experts: the forward pass that keeps what its gradient needs
        dict(name="block-train", op="block", direction="y", dtype="bf16", rows=16384, groups=64, n=2048, k=4096,
             act="silu", spread="uniform", keep=True),
        # and its gradients
        dict(name="block-train-grad", op="block", direction="grad", dtype="bf16", rows=16384, groups=64, n=2048,
             k=4096, act="silu", spread="uniform"),
        # a small fine-tuning batch: odd row counts, experts without rows, widths that no tile divides
        dict(name="block-ragged-grad", op="block", direction="grad", dtype="fp16", rows=1537, groups=24, n=1000,
             k=712, act="gelu", spread="zipf"),
        # one generated token: its own log probability and the eight best words
        dict(name="score-1", op="score", dtype="bf16", rows=1, vocab=129280, d=4096, tokens=1, top=8,
             temperature=1.0),
        # a drafted continuation of 16 tokens, three candidates a place, at the sampling temperature
        dict(name="score-16", op="score", dtype="bf16", rows=16, vocab=129280, d=4096, tokens=3, top=8,
             temperature=0.7),
        # a scored prompt with its twenty best alternatives: also the teacher's side of a distillation
        dict(name="score-2048", op="score", dtype="bf16", rows=2048, vocab=129280, d=4096, tokens=1, top=20,
             temperature=1.0),
        # the loss alone on a small held-out batch, odd sizes
        dict(name="distill-held-out", op="distill", direction="y", dtype="fp16", rows=333, vocab=32003, d=1000,
             listed=20, temperature=1.0),
        # a training step of a small head
        dict(name="distill-small-grad", op="distill", direction="grad", dtype="fp16", rows=512, vocab=32000, d=1024,
             listed=100, temperature=2.0),
        # a training step of the large head
        dict(name="distill-2048-grad", op="distill", direction="grad", dtype="bf16", rows=2048, vocab=129280, d=4096,
             listed=32, temperature=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A matrix width: usually a multiple of 8, as models have them, sometimes any number."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.3 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["block", "block", "score", "distill"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "block":
        return dict(op=op, direction=rng.choice(["y", "grad"]), dtype=dtype, rows=_log(rng, 1, 16384),
                    groups=rng.choice([0, _log(rng, 1, 64)]), n=_width(rng, 64, 2048), k=_width(rng, 64, 4096),
                    act=rng.choice(["none", "relu", "silu", "gelu"]), spread=rng.choice(["uniform", "zipf"]),
                    keep=rng.random() < 0.5)
    case = dict(op=op, dtype=dtype, rows=_log(rng, 1, 2048), vocab=_log(rng, 1000, 129280), d=_width(rng, 64, 4096),
                temperature=rng.choice([0.7, 1.0, 1.0, 2.0]))
    if op == "score":
        case.update(tokens=_log(rng, 1, 32), top=rng.choice([0, _log(rng, 1, 32)]))
    else:
        case.update(direction=rng.choice(["y", "grad"]), listed=_log(rng, 1, 128))
    return case


# ----------------------------------------------------------------------------------------- inputs


def _shares(case):
    """The share of the rows that each expert gets."""
    g = max(1, case["groups"])
    if case["spread"] == "zipf":
        w = [(i + 1) ** -1.1 for i in range(g)]
        return [v / sum(w) for v in w]
    return [1.0 / g] * g


def _counts(case, gen):
    """Rows of each expert: int64 [groups] on the host."""
    g, rows = max(1, case["groups"]), case["rows"]
    if case["spread"] == "distinct":
        counts = torch.zeros(g, dtype=torch.int64)
        counts[torch.randperm(g, generator=gen)[:rows]] = 1
        return counts
    p = torch.tensor(_shares(case), dtype=torch.float64)[torch.randperm(g, generator=gen)]
    return torch.bincount(torch.multinomial(p, rows, replacement=True, generator=gen), minlength=g)


def _ids(rows, vocab, n, gen):
    """n distinct words a row, in any order: one out of each of n equal parts of the vocabulary."""
    part = vocab // n
    ids = torch.randint(0, part, (rows, n), generator=gen, device="cuda") + part * torch.arange(n, device="cuda")
    return ids.gather(1, torch.rand((rows, n), generator=gen, device="cuda").argsort(1))


def _inputs(case, seed):
    dt = DTYPES[case["dtype"]]
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        t = torch.empty(shape, dtype=dt, device="cuda")
        return t.normal_(0.0, scale, generator=gen)

    def grid(*shape, scale, step):
        """Normal numbers on a grid of 8-bit whole numbers times a power of two: their products and sums are
        exact in 32 bits, so that the order of the logits, ties among them, does not hang on a rounding."""
        t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, scale, generator=gen)
        return (t.round_().clamp_(-127, 127) * step).to(dt)

    s = {"case": case}
    if case["op"] == "block":
        rows, n, k, g = case["rows"], case["n"], case["k"], max(1, case["groups"])
        s["counts"] = _counts(case, host)
        if case["groups"]:
            s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), s["counts"].cumsum(0)]).to(torch.int32).cuda()
        else:
            s["offsets"] = None  # one dense block
        s["x"], s["w"] = normal(rows, k), normal(g, 2 * n, k, scale=k ** -0.5)
        if case["direction"] == "grad":
            s["dh"], s["z"] = normal(rows, n), normal(rows, 2 * n)
        return s
    rows, vocab, d = case["rows"], case["vocab"], case["d"]
    if case["op"] == "score":
        # logits of standard deviation between 0.9 and 1.9
        s["x"] = grid(rows, d, scale=16.0, step=2.0 ** -4)
        s["w"] = grid(vocab, d, scale=20.0, step=2.0 ** -round(math.log2(20.0 * d ** 0.5 / 1.3)))
        tokens = _ids(rows, vocab, case["tokens"], gen)
        tokens[torch.rand(tokens.shape, generator=gen, device="cuda") < 0.05] = -1  # places without a token
        s["tokens"] = tokens.to(torch.int32)
        return s
    n = case["listed"]
    s["x"], s["w"] = normal(rows, d), normal(vocab, d, scale=1.3 * d ** -0.5)
    ids = _ids(rows, vocab, n, gen)
    # a teacher's best logits fall off like the logarithm of their rank
    teacher = 12.0 - 1.5 * torch.log(torch.arange(1, n + 1, device="cuda").float()) + 0.3 * torch.randn((rows, n), generator=gen, device="cuda")
    ids[torch.rand(ids.shape, generator=gen, device="cuda") < 0.02] = -1  # shorter lists
    padding = torch.rand(rows, generator=gen, device="cuda") < 0.05       # rows without a teacher
    ids[padding] = -1
    s["ids"], s["teacher"] = ids.to(torch.int32), teacher
    s["dloss"] = torch.where(padding, 0.0, 1.0 / max(1, rows - int(padding.sum())))  # of the mean
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    dt = DTYPES[case["dtype"]]
    empty = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    f32, i32 = torch.float32, torch.int32
    rows = case["rows"]
    if case["op"] == "block":
        n, k, g = case["n"], case["k"], max(1, case["groups"])
        if case["direction"] == "y":
            s["h"] = empty(rows, n)
            s["zout"] = empty(rows, 2 * n) if case["keep"] else None
        else:
            s["dz"], s["dx"], s["dw"] = empty(rows, 2 * n), empty(rows, k), empty(g, 2 * n, k)
        return s
    vocab, d = case["vocab"], case["d"]
    if case["op"] == "score":
        s["logprob"], s["lse"], s["entropy"] = empty(rows, case["tokens"], dtype=f32), empty(rows, dtype=f32), empty(rows, dtype=f32)
        top = case["top"]
        s["top_index"], s["top_logprob"] = (empty(rows, top, dtype=i32), empty(rows, top, dtype=f32)) if top else (None, None)
        # the scratch that a program keeps: softmax partials, lists, and logits to pick the best from
        s["scratch"] = empty(4 * rows * vocab * (top > 0) + rows * (vocab // 4 + 32 * case["tokens"] + 256) + (1 << 20),
                             dtype=torch.uint8)
        return s
    s["loss"], s["lse"], s["logq"] = empty(rows, dtype=f32), empty(rows, dtype=f32), empty(rows, case["listed"], dtype=f32)
    # the scratch that a program keeps: softmax partials and lists, or one piece of the vocabulary (16384 wide)
    s["scratch"] = empty((rows + 8) * (2 * min(vocab + 256, 16384) + 4 * d + vocab // 4 + 32 * case["listed"] + 256) + (1 << 20),
                         dtype=torch.uint8)
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
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _plain_block(s):
    case = s["case"]
    n, act = case["n"], case["act"]
    if case["groups"]:
        ends = s["offsets"].tolist()
        groups = list(zip(ends[:-1], ends[1:]))
    else:
        groups = [(0, case["rows"])]
    if case["direction"] == "y":
        h, zout = s["h"], s["zout"]
        for g, (lo, hi) in enumerate(groups):
            if lo == hi:
                continue
            z = s["x"][lo:hi].float() @ s["w"][g].float().T
            h[lo:hi] = _act(z[:, :n], act) * z[:, n:]
            if zout is not None:
                zout[lo:hi] = z
        return h if zout is None else {"h": h, "z": zout}
    dall, dx, dw = s["dz"], s["dx"], s["dw"]
    for g, (lo, hi) in enumerate(groups):
        if lo == hi:
            dw[g] = 0
            continue
        dh, gate, up = s["dh"][lo:hi].float(), s["z"][lo:hi, :n].float(), s["z"][lo:hi, n:].float()
        dz = torch.cat([dh * up * _act_slope(gate, act), dh * _act(gate, act)], 1)
        dall[lo:hi] = dz
        dx[lo:hi] = dz @ s["w"][g].float()
        dw[g] = dz.T @ s["x"][lo:hi].float()
    return {"dz": dall, "dx": dx, "dw": dw}


def _softmax_parts(z):
    """(the row's largest, exp(z - largest), its sum)"""
    most = z.max(1, keepdim=True).values
    e = torch.exp(z - most)
    return most, e, e.sum(1, keepdim=True)


def _plain_score(s):
    case = s["case"]
    z = s["x"].float() @ s["w"].float().T
    t = z * (1 / case["temperature"])
    most, e, total = _softmax_parts(t)
    lse = most + torch.log(total)
    entropy = torch.log(total) - (e * (t - most)).sum(1, keepdim=True) / total
    there = s["tokens"] >= 0
    at = torch.where(there, s["tokens"], 0).long()
    out = {"logprob": torch.where(there, t.gather(1, at) - lse, 0.0), "lse": lse.squeeze(1), "entropy": entropy.squeeze(1)}
    if case["top"]:
        index = torch.empty((case["rows"], case["top"]), dtype=torch.int64, device=z.device)
        for j in range(case["top"]):  # the first of the largest, which the next pass leaves out
            index[:, j] = z.argmax(1)
            z.scatter_(1, index[:, j:j + 1], -math.inf)
        out["top_index"], out["top_logprob"] = index.to(torch.int32), t.gather(1, index) - lse
    return out


def _plain_distill(s):
    case = s["case"]
    dt, scale = DTYPES[case["dtype"]], 1 / case["temperature"]
    x, w = s["x"].float(), s["w"].float()
    there = s["ids"] >= 0
    taught = there.any(1)
    at = torch.where(there, s["ids"], 0).long()
    teacher = torch.where(there, s["teacher"] * scale, -math.inf)
    _, p, total = _softmax_parts(torch.where(taught[:, None], teacher, 0.0))
    p = torch.where(there, p / total, 0.0)
    logp = torch.where(p > 0, torch.log(p), 0.0)
    z = (x @ w.T) * scale
    most, e, total = _softmax_parts(z)
    lse = most + torch.log(total)
    logq = torch.where(there, z.gather(1, at) - lse, 0.0)
    out = {"loss": (p * (logp - logq)).sum(1), "lse": lse.squeeze(1), "logq": logq}
    if case["direction"] == "grad":
        dz = e / total
        dz.scatter_add_(1, at, -p)
        dz *= torch.where(taught, s["dloss"] * scale, 0.0)[:, None]
        out["dx"], out["dw"] = (dz @ w).to(dt), (dz.T @ x).to(dt)
    return out


# ------------------------------------------------------------------------- the library's operators


def _own_block(s):
    from quantized_moe_gb300 import ds4moe as api

    c, stream = s["case"], torch.cuda.current_stream().cuda_stream
    sizes = dict(rows=c["rows"], n=c["n"], k=c["k"], n_groups=max(1, c["groups"]), act=c["act"], dtype=c["dtype"],
                 stream=stream)
    if c["direction"] == "y":
        api.ds4moe_grouped_glu(s["x"], s["w"], s["offsets"], s["h"], zout=s["zout"], **sizes)
        return s["h"] if s["zout"] is None else {"h": s["h"], "z": s["zout"]}
    api.ds4moe_grouped_glu_grad(s["dh"], s["x"], s["w"], s["offsets"], s["z"], s["dz"], s["dx"], s["dw"], **sizes)
    return {"dz": s["dz"], "dx": s["dx"], "dw": s["dw"]}


def _own_score(s):
    from quantized_moe_gb300 import ds4moe as api

    c = s["case"]
    api.ds4moe_logprobs(s["x"], s["w"], s["tokens"], s["logprob"], s["lse"], s["entropy"], s["top_index"],
                        s["top_logprob"], rows=c["rows"], vocab=c["vocab"], d=c["d"], n_tokens=c["tokens"],
                        top_k=c["top"], dtype=c["dtype"], temperature=c["temperature"], workspace=s["scratch"],
                        workspace_bytes=s["scratch"].numel(), stream=torch.cuda.current_stream().cuda_stream)
    out = {"logprob": s["logprob"], "lse": s["lse"], "entropy": s["entropy"]}
    if c["top"]:
        out["top_index"], out["top_logprob"] = s["top_index"], s["top_logprob"]
    return out


def _own_distill(s):
    from quantized_moe_gb300 import ds4moe as api

    c = s["case"]
    sizes = dict(rows=c["rows"], vocab=c["vocab"], d=c["d"], top_k=c["listed"], dtype=c["dtype"],
                 temperature=c["temperature"], workspace=s["scratch"], workspace_bytes=s["scratch"].numel(),
                 stream=torch.cuda.current_stream().cuda_stream)
    api.ds4moe_distill(s["x"], s["w"], s["ids"], s["teacher"], s["loss"], s["lse"], s["logq"], **sizes)
    out = {"loss": s["loss"], "lse": s["lse"], "logq": s["logq"]}
    if c["direction"] == "grad":
        api.ds4moe_distill_grad(s["x"], s["w"], s["ids"], s["teacher"], s["lse"], s["logq"], s["dloss"], s["dx"], s["dw"],
                                **sizes)
        out["dx"], out["dw"] = s["dx"], s["dw"]
    return out


def run(state):
    forms = {"block": (_plain_block, _own_block), "score": (_plain_score, _own_score),
             "distill": (_plain_distill, _own_distill)}
    return forms[state["case"]["op"]][1 if own else 0](state)


def work(case):
    size, rows = 2, case["rows"]
    if case["op"] == "block":
        n, k, g = case["n"], case["k"], max(1, case["groups"])
        if case["spread"] == "distinct":
            touched = min(rows, g)
        else:
            touched = sum(1 - (1 - p) ** rows for p in _shares(case))  # expected
        weights = touched * 2 * n * k * size
        offsets = (g + 1) * 4 if case["groups"] else 0
        if case["direction"] == "y":
            return {"bytes": int(weights + rows * (k + n + 2 * n * case["keep"]) * size + offsets), "flops": 4 * rows * n * k}
        return {"bytes": int(weights + g * 2 * n * k * size + rows * (5 * n + 2 * k) * size + offsets), "flops": 8 * rows * n * k}
    vocab, d = case["vocab"], case["d"]
    if case["op"] == "score":
        return {"bytes": size * (rows * d + vocab * d) + rows * (8 * case["tokens"] + 8 + 8 * case["top"]),
                "flops": 2 * rows * vocab * d}
    lists = rows * (12 * case["listed"] + 8)
    if case["direction"] == "y":
        return {"bytes": size * (rows * d + vocab * d) + lists, "flops": 2 * rows * vocab * d}
    return {"bytes": size * (2 * rows * d + 2 * vocab * d) + lists + 4 * rows, "flops": 6 * rows * vocab * d}


# ---------------------------------------------------------------------------- definition, 64 bits


def _exact_block(case, s):
    act = {"none": lambda z: z, "relu": torch.nn.functional.relu, "silu": torch.nn.functional.silu,
           "gelu": torch.nn.functional.gelu}[case["act"]]
    counts = s["counts"].tolist()
    x = s["x"].double().split(counts)
    if case["direction"] == "y":
        z = [torch.einsum("tk,nk->tn", a, s["w"][e].double()) for e, a in enumerate(x)]
        h = torch.cat([act(g) * u for g, u in (v.chunk(2, 1) for v in z)])
        return {"h": h, "z": torch.cat(z)} if case["keep"] else h
    z = s["z"].double().requires_grad_()
    gate, up = z.chunk(2, 1)
    (dz,) = torch.autograd.grad(act(gate) * up, z, s["dh"].double())
    parts = dz.split(counts)
    return {"dz": dz, "dx": torch.cat([torch.einsum("tn,nk->tk", a, s["w"][e].double()) for e, a in enumerate(parts)]),
            "dw": torch.stack([torch.einsum("tn,tk->nk", a, b) for a, b in zip(parts, x)])}


def _exact_score(case, s):
    w, x = s["w"], s["x"].double()
    z = torch.cat([x @ part.double().T for part in w.split(16384)], 1)
    logp = z / case["temperature"]
    lse = torch.logsumexp(logp, 1, keepdim=True)
    logp = logp - lse
    tokens = s["tokens"].long()
    out = {"logprob": logp.gather(1, tokens.clamp(min=0)).masked_fill(tokens < 0, 0.0), "lse": lse.squeeze(1),
           "entropy": torch.stack([-(row.exp() * row).sum() for row in logp])}
    if case["top"]:
        # (a stable sort keeps equal logits in the order of their indices)
        order = torch.stack([torch.sort(row, descending=True, stable=True).indices[:case["top"]] for row in z])
        out["top_index"], out["top_logprob"] = order.to(torch.int32), logp.gather(1, order)
    return out


def _exact_distill(case, s):
    rows, vocab, n = case["rows"], case["vocab"], case["listed"]
    x, w, t = s["x"].double(), s["w"], case["temperature"]
    ids = s["ids"].long()
    there = ids >= 0
    p = torch.zeros((rows, n), dtype=torch.float64, device="cuda")
    for r in there.any(1).nonzero().flatten().tolist():
        p[r, there[r]] = torch.softmax(s["teacher"][r, there[r]].double() / t, 0)
    chunks = [(v, min(v + 16384, vocab)) for v in range(0, vocab, 16384)]
    lse = torch.full((rows,), -math.inf, dtype=torch.float64, device="cuda")
    own_z = torch.zeros((rows, n), dtype=torch.float64, device="cuda")
    for lo, hi in chunks:
        z = x @ w[lo:hi].double().T / t
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        here = (ids >= lo) & (ids < hi)
        own_z = torch.where(here, z.gather(1, (ids - lo).clamp(0, hi - lo - 1)), own_z)
    logq = (own_z - lse[:, None]).masked_fill(~there, 0.0)
    out = {"loss": (torch.xlogy(p, p) - p * logq).sum(1), "lse": lse, "logq": logq}
    if case["direction"] == "grad":
        g = torch.where(there.any(1), s["dloss"].double(), 0.0) / t
        dx, dw = torch.zeros_like(x), []
        for lo, hi in chunks:
            wd = w[lo:hi].double()
            dz = torch.exp(x @ wd.T / t - lse[:, None])
            here = (ids >= lo) & (ids < hi)
            dz.scatter_add_(1, (ids - lo).clamp(0, hi - lo - 1), torch.where(here, -p, 0.0))
            dz *= g[:, None]
            dx += dz @ wd
            dw.append(dz.T @ x)
        out["dx"], out["dw"] = dx, torch.cat(dw)
    return out


def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits."""
    return {"block": _exact_block, "score": _exact_score, "distill": _exact_distill}[case["op"]](case, _inputs(case, seed))
