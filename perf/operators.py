"""Cases for the operators of a sharded training step: their plain forms in
elementary torch operations, and the library's own calls (``own``).

Three operators over virtual ranks whose buffers live on one GPU:

``xent``     softmax cross entropy of hidden states against an output
             projection whose vocabulary rows are split over the ranks:
             losses and log-sum-exps ("loss"), or the gradients of the hidden
             states and of every rank's rows ("grad");
``balance``  the load-balance loss of a mixture-of-experts router over every
             rank's tokens, with per-expert counts and the gradient of every
             rank's router logits;
``ortho``    one matrix per rank orthogonalised by Newton-Schulz steps.
"""

import math

import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def listed():
    return [
        # scoring a handful of tokens with a small character-level vocabulary: launch latency
        {"name": "xent loss tiny f32", "op": "xent", "grad": False, "ranks": 2, "tokens": 7, "vocab": 259, "dim": 64, "dtype": "f32"},
        # scoring one short prompt against a large vocabulary: the projection's bytes count
        {"name": "xent loss short bf16", "op": "xent", "grad": False, "ranks": 8, "tokens": 48, "vocab": 128003, "dim": 4096, "dtype": "bf16"},
        # evaluation of a batch
        {"name": "xent loss batch f16", "op": "xent", "grad": False, "ranks": 4, "tokens": 4096, "vocab": 50257, "dim": 2048, "dtype": "f16"},
        # gradients of a small model kept in single precision
        {"name": "xent grad small f32", "op": "xent", "grad": True, "ranks": 3, "tokens": 301, "vocab": 8009, "dim": 520, "dtype": "f32"},
        # gradients of a medium model's micro-batch
        {"name": "xent grad batch f16", "op": "xent", "grad": True, "ranks": 2, "tokens": 2048, "vocab": 32003, "dim": 2048, "dtype": "f16"},
        # gradients of a large model's micro-batch, eight vocabulary shards
        {"name": "xent grad large bf16", "op": "xent", "grad": True, "ranks": 8, "tokens": 8192, "vocab": 100277, "dim": 4096, "dtype": "bf16"},
        # a few tokens per rank, few experts: launch latency
        {"name": "balance tiny f32", "op": "balance", "ranks": 4, "tokens": 61, "experts": 8, "topk": 2, "dtype": "f32"},
        # an ordinary micro-batch on eight ranks
        {"name": "balance batch bf16", "op": "balance", "ranks": 8, "tokens": 4096, "experts": 64, "topk": 6, "dtype": "bf16"},
        # many experts, long sequences
        {"name": "balance large f32", "op": "balance", "ranks": 8, "tokens": 16384, "experts": 256, "topk": 8, "dtype": "f32"},
        # attention-head sized matrices, one per rank
        {"name": "ortho small f32", "op": "ortho", "ranks": 8, "rows": 128, "cols": 200, "dtype": "f32"},
        # a projection and its feed-forward shape, eight ranks' gradients at once
        {"name": "ortho batch bf16", "op": "ortho", "ranks": 8, "rows": 1024, "cols": 4096, "dtype": "bf16"},
        # tall single-precision gradients of a large layer
        {"name": "ortho large f32", "op": "ortho", "ranks": 2, "rows": 8190, "cols": 2048, "dtype": "f32"},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    dtype = rng.choice(["f32", "f16", "bf16"])
    ranks = rng.randint(1, 8)
    kind = rng.choice(["loss", "grad", "balance", "ortho"])
    if kind in ("loss", "grad"):
        step = 4 if dtype == "f32" else 8                  # rows of whole 16-byte vectors
        while True:
            dim = step * _log_uniform(rng, 64 // step, 6144 // step)
            vocab = _log_uniform(rng, 256, 131072)
            tokens = _log_uniform(rng, 1, 8192)
            if tokens * vocab * dim <= (8192 * 100277 * 4096) // (4 if dtype == "f32" else 1):
                break
        return {"op": "xent", "grad": kind == "grad", "ranks": ranks, "tokens": tokens, "vocab": vocab, "dim": dim,
                "dtype": dtype}
    if kind == "balance":
        experts = _log_uniform(rng, 4, 384)
        return {"op": "balance", "ranks": ranks, "tokens": _log_uniform(rng, 1, 16384), "experts": experts,
                "topk": rng.randint(1, min(8, experts)), "dtype": dtype}
    while True:
        rows, cols = _log_uniform(rng, 16, 8192), _log_uniform(rng, 16, 8192)
        small, large = min(rows, cols), max(rows, cols)
        if ranks * (3 * small * small * large + small ** 3) <= 2 * (3 * 2048 * 2048 * 8190 + 2048 ** 3):
            break
    return {"op": "ortho", "ranks": ranks, "rows": rows, "cols": cols, "dtype": dtype}


def shards(vocab, ranks):
    """Rows of the vocabulary per rank: equal blocks, the last ones shorter."""
    block = -(-vocab // ranks)
    return [max(0, min(block, vocab - r * block)) for r in range(ranks)]


def _prepare_xent(c, g):
    t, v, d, dt = c["tokens"], c["vocab"], c["dim"], DTYPE[c["dtype"]]
    # normalised hidden states with a few larger channels; logits of a standard deviation near 2
    x = torch.randn(t, d, generator=g, device="cuda") * (1 + 2 * (torch.rand(d, generator=g, device="cuda") < 0.02))
    x = x.to(dt)
    sizes = shards(v, c["ranks"])
    w = [(torch.randn(n, d, generator=g, device="cuda") * (2 / math.sqrt(d))).to(dt) for n in sizes]
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    target[torch.rand(t, generator=g, device="cuda") < 0.06] = -1          # prompt and padding positions: no loss
    s = {"x": x, "w": w, "target": target}
    if c["grad"]:
        # the forward pass has run: its log-sum-exps are at hand, with each token's weight in the mean
        s["lse"] = torch.cat([torch.logsumexp(p.float() @ torch.cat(w).float().t(), 1) for p in x.split(4096)])
        weight = 0.5 + torch.rand(t, generator=g, device="cuda")
        s["dloss"] = weight / weight.sum() * (1024.0 if dt == torch.float16 else 1.0)   # f16 trains with a scaled loss
    return s


def _prepare_balance(c, g):
    t, e, k, dt = c["tokens"], c["experts"], c["topk"], DTYPE[c["dtype"]]
    skew = torch.randn(e, generator=g, device="cuda")                      # some experts are liked more
    logits = [(torch.randn(t, e, generator=g, device="cuda") + skew).to(dt) for _ in range(c["ranks"])]
    experts = [z.float().topk(k, 1).indices.to(torch.int32) for z in logits]
    for z in experts:                                                       # padded positions and dropped choices
        z[torch.rand(t, generator=g, device="cuda") < 0.04] = -1
        z[torch.rand(t, k, generator=g, device="cuda") < 0.02] = -1
    return {"logits": logits, "experts": experts, "coef": 0.01 * (1024.0 if dt == torch.float16 else 1.0)}


def _prepare_ortho(c, g):
    m, n, dt = c["rows"], c["cols"], DTYPE[c["dtype"]]
    r = max(2, min(m, n) // 16)
    # gradients: a few strong directions over the noise of a micro-batch
    fade = torch.logspace(0, -2, r, device="cuda")
    return {"grad": [((torch.randn(m, r, generator=g, device="cuda") * fade) @ torch.randn(r, n, generator=g, device="cuda")
                      * 0.02 + 0.004 * torch.randn(m, n, generator=g, device="cuda")).to(dt) for _ in range(c["ranks"])]}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"xent": _prepare_xent, "balance": _prepare_balance, "ortho": _prepare_ortho}[case["op"]](case, g)
    s["case"] = dict(case)
    return s


# --- plain forms -------------------------------------------------------------

def _plain_xent(s):
    x, target = s["x"].float(), s["target"]
    w = torch.cat(s["w"]).float()
    v = w.shape[0]
    logits = x @ w.t()
    counted = (target >= 0) & (target < v)
    at = target.clamp(0, v - 1)[:, None]
    if not s["case"]["grad"]:
        top = logits.amax(1, keepdim=True)
        lse = (logits - top).exp().sum(1).log() + top[:, 0]
        return {"loss": torch.where(counted, lse - logits.gather(1, at)[:, 0], 0.0), "lse": lse}
    p = (logits - s["lse"][:, None]).exp()
    p.scatter_add_(1, at, torch.full_like(at, -1, dtype=p.dtype))
    p *= (s["dloss"] * counted)[:, None]
    dt = s["x"].dtype
    dw = (p.t() @ x).to(dt)
    return {"dx": (p @ w).to(dt), "dw": list(dw.split([q.shape[0] for q in s["w"]]))}


def _plain_balance(s):
    ranks, e, k = s["case"]["ranks"], s["case"]["experts"], s["case"]["topk"]
    z, idx = torch.stack(s["logits"]).float(), torch.stack(s["experts"]).long()
    chosen = (idx >= 0) & (idx < e)
    valid = chosen.any(2)
    p = (z - z.amax(2, keepdim=True)).exp()
    p = p / p.sum(2, keepdim=True) * valid[..., None]
    rank = torch.arange(ranks, device=z.device)[:, None, None]
    counts = torch.zeros(ranks * e, dtype=torch.int64, device=z.device)
    counts.scatter_add_(0, (rank * e + idx.clamp(0, e - 1)).reshape(-1), chosen.reshape(-1).long())
    counts = counts.view(ranks, e)
    total = counts.sum(0)
    n = valid.sum().clamp(min=1).double()
    f = total / (n * k)
    scale = s["coef"] * e / n
    loss = scale * (f * p.double().sum((0, 1))).sum()
    f = f.float()
    dz = scale.float() * p * (f - (p * f).sum(2, keepdim=True))
    return {"counts": torch.cat([counts, total[None]]), "loss": loss.float().view(1),
            "dlogits": list(dz.to(s["logits"][0].dtype).unbind(0))}


def _plain_ortho(s):
    x = torch.stack(s["grad"]).float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / (x.double().square().sum((1, 2), keepdim=True).sqrt() + 1e-7).float()
    a, b, c = NEWTON_SCHULZ
    for _ in range(5):
        gram = x @ x.transpose(1, 2).contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if tall:
        x = x.transpose(1, 2)
    return {"update": list(x.to(s["grad"][0].dtype).unbind(0))}


# --- the library's calls -----------------------------------------------------

def _own_xent(s):
    from double_binary_tree_amd import emucomm as E
    c = s["case"]
    if "workspace" not in s:                      # a training program keeps these from step to step
        s["workspace"] = E.cross_entropy_workspace(s["x"], s["w"], grad=c["grad"])
        if c["grad"]:
            s["dx"], s["dw"] = torch.empty_like(s["x"]), [torch.empty_like(w) for w in s["w"]]
        else:
            s["out"] = [torch.empty(c["tokens"], device="cuda") for _ in range(2)]
    if not c["grad"]:
        loss, lse = s["out"]
        E.cross_entropy_tensors(s["x"], s["w"], s["target"], loss, lse, workspace=s["workspace"])
        return {"loss": loss, "lse": lse}
    E.cross_entropy_grad_tensors(s["x"], s["w"], s["target"], s["lse"], s["dloss"], s["dx"], s["dw"],
                                 workspace=s["workspace"])
    return {"dx": s["dx"], "dw": s["dw"]}


def _own_balance(s):
    from double_binary_tree_amd import emucomm as E
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = E.balance_loss_workspace(s["logits"])
        s["counts"] = torch.empty(c["ranks"] + 1, c["experts"], dtype=torch.int64, device="cuda")
        s["loss"] = torch.empty(1, device="cuda")
        s["dlogits"] = [torch.empty_like(z) for z in s["logits"]]
    E.balance_loss_tensors(s["logits"], s["experts"], s["coef"], s["counts"], s["loss"], s["dlogits"],
                           workspace=s["workspace"])
    return {"counts": s["counts"], "loss": s["loss"], "dlogits": s["dlogits"]}


def _own_ortho(s):
    from double_binary_tree_amd import emucomm as E
    if "workspace" not in s:
        s["workspace"] = E.orthogonalize_workspace(s["grad"])
        s["update"] = [torch.empty_like(x) for x in s["grad"]]
    E.orthogonalize_tensors(s["grad"], s["update"], steps=5, workspace=s["workspace"])
    return {"update": s["update"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"xent": _own_xent, "balance": _own_balance, "ortho": _own_ortho}[op](state)
    return {"xent": _plain_xent, "balance": _plain_balance, "ortho": _plain_ortho}[op](state)


# --- the work that a pass cannot do without ----------------------------------

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    r = case["ranks"]
    if case["op"] == "xent":
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        if not case["grad"]:
            return {"bytes": (t + v) * d * size + 16 * t, "flops": 2 * t * v * d}
        # the logits are not kept, so their product is part of the gradient
        return {"bytes": 2 * (t + v) * d * size + 16 * t, "flops": 6 * t * v * d}
    if case["op"] == "balance":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        return {"bytes": r * t * (2 * e * size + 4 * k) + 8 * e * (r + 1) + 4, "flops": 12 * r * t * e}
    m, n = sorted((case["rows"], case["cols"]))
    # both squares are symmetric: half their products are needed
    return {"bytes": 2 * r * m * n * size, "flops": 5 * r * (m * m * n + m * m * m + 2 * m * m * n)}


# --- the definitions in 64 bits ----------------------------------------------

def _exact_xent(c, s):
    x, w = s["x"].double(), [q.double() for q in s["w"]]
    first, out = 0, []
    scores = [torch.mm(x, q.t().contiguous()) for q in w]
    label = torch.full((c["tokens"],), float("nan"), dtype=torch.float64, device="cuda")
    rows = torch.arange(c["tokens"], device="cuda")
    kept = (s["target"] >= 0) & (s["target"] < c["vocab"])
    if not c["grad"]:
        lse = torch.logsumexp(torch.stack([torch.logsumexp(z, 1) for z in scores if z.shape[1]]), 0)
        for z in scores:
            here = (s["target"] >= first) & (s["target"] < first + z.shape[1])
            label[here] = z[rows[here], s["target"][here] - first]
            first += z.shape[1]
        return {"loss": torch.where(kept, lse - label, torch.zeros_like(lse)), "lse": lse}
    dx = torch.zeros_like(x)
    scale = torch.where(kept, s["dloss"].double(), torch.zeros_like(s["dloss"], dtype=torch.float64))
    for z, q in zip(scores, w):
        z.sub_(s["lse"].double()[:, None]).exp_()
        here = (s["target"] >= first) & (s["target"] < first + z.shape[1])
        z[rows[here], s["target"][here] - first] -= 1.0
        z.mul_(scale[:, None])
        dx += torch.mm(z, q)
        out.append(torch.mm(z.t().contiguous(), x))
        first += z.shape[1]
    return {"dx": dx, "dw": out}


def _exact_balance(c, s):
    e, counts, soft, live = c["experts"], [], [], []
    for z, idx in zip(s["logits"], s["experts"]):
        idx = idx.long()
        ok = (idx >= 0) & (idx < e)
        counts.append(torch.bincount(idx[ok], minlength=e))
        live.append(ok.sum(1) > 0)
        soft.append(torch.softmax(z.double(), 1))
    total = sum(counts)
    n = max(1, int(sum(v.sum() for v in live)))
    share = total.double() / (n * c["topk"])
    mean = sum((p * v[:, None]).sum(0) for p, v in zip(soft, live)) / n
    loss = s["coef"] * e * torch.dot(share, mean)
    grads = [s["coef"] * e / n * v[:, None] * p * (share - (p @ share)[:, None]) for p, v in zip(soft, live)]
    return {"counts": torch.stack(counts + [total]), "loss": loss.view(1), "dlogits": grads}


def _exact_ortho(c, s):
    a, b, d = NEWTON_SCHULZ
    out = []
    for g in s["grad"]:
        y = g.double()
        y = y / (torch.linalg.vector_norm(y) + 1e-7)
        for _ in range(5):
            if y.shape[0] <= y.shape[1]:
                k = torch.mm(y, y.t().contiguous())
                y = a * y + torch.mm(b * k + d * torch.mm(k, k), y)
            else:
                k = torch.mm(y.t().contiguous(), y)
                y = a * y + torch.mm(y, b * k + d * torch.mm(k, k))
        out.append(y)
    return {"update": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"xent": _exact_xent, "balance": _exact_balance, "ortho": _exact_ortho}[case["op"]](case, s)
