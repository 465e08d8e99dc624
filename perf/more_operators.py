"""Cases of the operators at a language model's two ends and of its experts'
router: the token embedding with its gradient, the linear softmax cross entropy
over the vocabulary with its gradients, and the router (probabilities, choices,
counts, balance and z losses) with its gradient; each with its plain form, its
exact values and its work.

``run(state)`` makes one pass: in plain torch operations in 32 bits where
``own`` is false, through the package's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# the cases


def listed():
    return [
        # eight sequences look one token up each: latency
        dict(name="embedding_decode", op="embedding", tokens=8, hidden=4096, vocab=32000,
             table="bf16", out="bf16", scale=1.0, padded=0.0),
        # BERT-base rows (64 sequences of 512, a tenth padding), fp16, and the
        # gradient of its table
        dict(name="embedding_train_bert", op="embedding_train", tokens=32768, hidden=768,
             vocab=30522, table="fp16", out="fp16", grad="fp16", scale=1.0, padded=0.1),
        # a training batch of a 7B-shaped model, onto an fp32 residual stream,
        # scaled
        dict(name="embedding_train_7b", op="embedding_train", tokens=16384, hidden=4096,
             vocab=32000, table="bf16", out="fp32", grad="bf16", scale=64.0, padded=0.0),
        # odd sizes, 32-bit rows
        dict(name="embedding_train_odd", op="embedding_train", tokens=2999, hidden=1001,
             vocab=5003, table="fp32", out="fp32", grad="fp32", scale=0.7, padded=0.05),
        # the log-probabilities of eight tokens, as a scorer takes them: one
        # read of the head's weights
        dict(name="loss_score", op="loss", tokens=8, hidden=4096, vocab=32000, dtype="bf16",
             scale=1.0, left_out=0.0),
        # masked-language-model training of a BERT-base batch: 15% of the
        # positions have a target
        dict(name="loss_train_bert", op="loss_train", tokens=8192, hidden=768, vocab=30522,
             dtype="fp16", grad="fp16", reduction="mean", scale=1.0, left_out=0.85),
        # a training batch of a 7B-shaped model (four sequences of 2048)
        dict(name="loss_train_7b", op="loss_train", tokens=8192, hidden=4096, vocab=32000,
             dtype="bf16", grad="bf16", reduction="mean", scale=1.0, left_out=0.0),
        # a wide vocabulary over a narrow model, gradients kept in 32 bits
        dict(name="loss_train_wide", op="loss_train", tokens=4096, hidden=1024, vocab=131072,
             dtype="bf16", grad="fp32", reduction="sum", scale=1.0, left_out=0.1),
        # odd sizes, a gradient for every token's own loss, a temperature
        dict(name="loss_train_odd", op="loss_train", tokens=1021, hidden=1001, vocab=5003,
             dtype="fp16", grad="fp16", reduction="none", scale=0.7, left_out=0.3),
        # eight sequences decode one token each, two of eight experts a token
        dict(name="route_decode", op="route", tokens=8, experts=8, topk=2, dtype="fp32",
             normalize=True, barred=0.0, padded=0.0),
        # a training batch of a model with 256 experts, eight a token
        dict(name="route_train", op="route_train", tokens=65536, experts=256, topk=8,
             dtype="fp32", normalize=True, barred=0.0, padded=0.0),
        # odd sizes, 16-bit scores (ties), some experts barred, some tokens
        # with none left
        dict(name="route_train_odd", op="route_train", tokens=3001, experts=17, topk=3,
             dtype="bf16", normalize=False, barred=0.2, padded=0.1),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _hidden(rng):
    hidden = _spread(rng, 64, 8192)
    return max(64, hidden // 8 * 8) if rng.random() < 0.7 else hidden


def draw(rng):
    op = rng.choice(["embedding", "embedding_train", "loss", "loss_train", "loss_train", "route",
                     "route_train"])
    if op in ("embedding", "embedding_train"):
        hidden = _hidden(rng)
        table = rng.choice(["fp16", "bf16", "fp32"])
        return dict(op=op, hidden=hidden, table=table, out=rng.choice([table, "fp32"]),
                    grad=rng.choice([table, "fp32"]),
                    tokens=_spread(rng, 1, min(65536, 16384 * 4096 // 2 // hidden)),
                    vocab=_spread(rng, 500, min(131072, 32000 * 4096 // 2 // hidden)),
                    scale=rng.choice([1.0, round(math.sqrt(hidden), 3)]),
                    padded=rng.choice([0.0, 0.1, 0.6]))
    if op in ("loss", "loss_train"):
        hidden = _hidden(rng)
        vocab = _spread(rng, 500, 131072)
        most = min(16384, 8192 * 4096 * 32000 // (hidden * vocab), 4096 * 131072 // vocab)
        dtype = rng.choice(["fp16", "bf16"])
        return dict(op=op, tokens=_spread(rng, 1, most), hidden=hidden, vocab=vocab, dtype=dtype,
                    grad=rng.choice([dtype, "fp32"]),
                    reduction=rng.choice(["mean", "sum", "none"]),
                    scale=rng.choice([1.0, round(rng.uniform(0.3, 2.0), 3)]),
                    left_out=rng.choice([0.0, 0.1, 0.85]))
    experts = _spread(rng, 2, 512)
    return dict(op=op, tokens=_spread(rng, 1, min(65536, 65536 * 256 // experts)), experts=experts,
                topk=min(experts, rng.choice([1, 2, 3, 4, 6, 8])),
                dtype=rng.choice(["fp16", "bf16", "fp32"]), normalize=rng.choice([True, False]),
                barred=rng.choice([0.0, 0.0, 0.2]), padded=rng.choice([0.0, 0.1]))


# ---------------------------------------------------------------------------
# inputs


def _tokens(case, gen, share):
    """Token ids as texts have them (the k-th most frequent about 1/k as often
    as the first), a share of them -1."""
    u = torch.rand(case["tokens"], device="cuda", generator=gen, dtype=torch.float64)
    ids = (torch.exp(u * math.log(case["vocab"] + 1.0)) - 1.0).long().clamp_(0, case["vocab"] - 1)
    if share:
        gone = torch.rand(case["tokens"], device="cuda", generator=gen) < share
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype, scale=1.0):
        return torch.randn(*shape, device="cuda", generator=gen).mul_(scale).to(dtype)

    s = {"case": case}
    T = case["tokens"]
    if case["op"] in ("embedding", "embedding_train"):
        s["ids"] = _tokens(case, gen, case["padded"])
        s["table"] = normal(case["vocab"], case["hidden"], dtype=DTYPES[case["table"]], scale=0.02)
        if case["op"] == "embedding_train":
            s["dy"] = normal(T, case["hidden"], dtype=DTYPES[case["out"]], scale=1e-2)
        return s
    if case["op"] in ("loss", "loss_train"):
        dt, H = DTYPES[case["dtype"]], case["hidden"]
        s["targets"] = _tokens(case, gen, case["left_out"])
        w = torch.randn(case["vocab"], H, device="cuda", generator=gen).mul_(1.5 / math.sqrt(H))
        # a model part of the way through its training: the target's score
        # stands above the others', which lie around 1.5
        toward = 2.0 * torch.rand(T, 1, device="cuda", generator=gen)
        x = torch.randn(T, H, device="cuda", generator=gen)
        x += toward * w[s["targets"].clamp(min=0)]
        s["w"], s["x"] = w.to(dt), x.to(dt)
        if case["op"] == "loss_train":
            # the gradient of the loss: a loss scale (mean), a share of the
            # batch (sum), weights of the tokens (none)
            if case["reduction"] == "none":
                s["d"] = torch.rand(T, device="cuda", generator=gen)
            else:
                s["d"] = torch.full((), 4096.0 if case["reduction"] == "mean" else 0.5,
                                    device="cuda")
        return s
    T, E = case["tokens"], case["experts"]
    want = torch.linspace(0.0, 2.0, E, device="cuda")
    z = torch.randn(T, E, device="cuda", generator=gen) + want
    if case["barred"]:
        z[torch.rand(T, E, device="cuda", generator=gen) < case["barred"]] = -math.inf
    if case["padded"]:
        z[torch.rand(T, device="cuda", generator=gen) < case["padded"]] = -math.inf
    s["logits"] = z.to(DTYPES[case["dtype"]])
    if case["op"] == "route_train":
        s["d_weights"] = normal(T, case["topk"], dtype=torch.float32, scale=1e-2)
        s["d_losses"] = torch.tensor([1e-2, 1e-3], device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass


def run(state):
    op = state["case"]["op"]
    if op in ("embedding", "embedding_train"):
        return _embedding_own(state) if own else _embedding_plain(state)
    if op in ("loss", "loss_train"):
        return _loss_own(state) if own else _loss_plain(state)
    return _route_own(state) if own else _route_plain(state)


def _embedding_own(s):
    import zero_sharded_optimizer_flatten_gb300 as Z
    c = s["case"]
    out = {"y": Z.zero_embedding(s["ids"], s["table"], scale=c["scale"], dtype=DTYPES[c["out"]])}
    if c["op"] == "embedding_train":
        out["dtable"] = Z.zero_embedding_backward(s["dy"], s["ids"], c["vocab"], scale=c["scale"],
                                                  dtype=DTYPES[c["grad"]])
    return out


def _embedding_plain(s):
    c = s["case"]
    kept = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
    at = torch.where(kept, s["ids"], torch.zeros_like(s["ids"]))
    y = s["table"][at].float() * c["scale"] * kept[:, None]
    out = {"y": y.to(DTYPES[c["out"]])}
    if c["op"] == "embedding_train":
        d = torch.zeros(c["vocab"], c["hidden"], device="cuda")
        d.index_add_(0, at, s["dy"].float() * kept[:, None])
        out["dtable"] = (d * c["scale"]).to(DTYPES[c["grad"]])
    return out


def _loss_own(s):
    import zero_sharded_optimizer_flatten_gb300 as Z
    c = s["case"]
    ce = Z.zero_linear_cross_entropy(s["x"], s["w"], s["targets"], scale=c["scale"])
    out = {"losses": ce.losses, "lse": ce.lse, "total": ce.total}
    if c["op"] == "loss_train":
        out["dx"], out["dw"] = Z.zero_linear_cross_entropy_backward(
            s["x"], s["w"], s["targets"], ce, s["d"], reduction=c["reduction"], scale=c["scale"],
            dw_dtype=DTYPES[c["grad"]])
    return out


def _loss_plain(s):
    c = s["case"]
    x, w = s["x"].float(), s["w"].float()
    kept = (s["targets"] >= 0) & (s["targets"] < c["vocab"])
    at = torch.where(kept, s["targets"], torch.zeros_like(s["targets"]))[:, None]
    z = (x @ w.t()) * c["scale"]
    top = z.max(dim=1, keepdim=True).values
    lse = (z - top).exp().sum(dim=1, keepdim=True).log() + top
    losses = torch.where(kept, (lse - z.gather(1, at))[:, 0], torch.zeros_like(lse[:, 0]))
    count = kept.sum().float()
    total = losses.sum()
    out = {"losses": losses, "lse": torch.where(kept, lse[:, 0], torch.zeros_like(losses)),
           "total": torch.stack([total / count.clamp(min=1.0), total, count])}
    if c["op"] == "loss_train":
        g = s["d"] / count.clamp(min=1.0) if c["reduction"] == "mean" else s["d"]
        g = (g * kept * c["scale"])[:, None]
        dz = (z - lse).exp()
        dz.scatter_add_(1, at, torch.full_like(lse, -1.0))
        dz *= g
        out["dx"] = (dz @ w).to(s["x"].dtype)
        out["dw"] = (dz.t() @ x).to(DTYPES[c["grad"]])
    return out


def _route_own(s):
    import zero_sharded_optimizer_flatten_gb300 as Z
    c = s["case"]
    r = Z.zero_expert_route(s["logits"], c["topk"], normalize=c["normalize"])
    out = {"ids": r.ids, "weights": r.weights, "counts": r.counts, "losses": r.losses}
    if c["op"] == "route_train":
        out["dlogits"] = Z.zero_expert_route_backward(s["logits"], r, s["d_weights"],
                                                      s["d_losses"])
    return out


def _route_plain(s):
    c = s["case"]
    z = s["logits"].float()
    T, E = z.shape
    K = c["topk"]
    top = z.max(dim=1, keepdim=True).values
    there = top > -math.inf
    top = torch.where(there, top, torch.zeros_like(top))
    e = (z - top).exp()
    total = e.sum(dim=1, keepdim=True)
    p = torch.where(there, e / total, torch.zeros_like(e))
    lse = torch.where(there, total.log() + top, torch.zeros_like(top))
    value, order = torch.sort(z, dim=1, descending=True, stable=True)
    chosen, kept = order[:, :K], value[:, :K] > -math.inf
    ids = torch.where(kept, chosen, torch.full_like(chosen, -1))
    weights = p.gather(1, chosen) * kept
    share = weights.sum(dim=1, keepdim=True)
    if c["normalize"]:
        weights = torch.where(there, weights / share, torch.zeros_like(weights))
    counts = torch.zeros(E, dtype=torch.int64, device="cuda")
    counts.scatter_add_(0, chosen.reshape(-1), kept.reshape(-1).long())
    n = there.sum().float().clamp(min=1.0)
    load = counts.float() * (E / (K * n))
    balance = (load * (p.sum(dim=0) / n)).sum()
    out = {"ids": ids.to(torch.int32), "weights": weights, "counts": counts.to(torch.int32),
           "losses": torch.stack([balance, lse.square().sum() / n])}
    if c["op"] == "route_train":
        d = s["d_weights"] * kept
        a = (s["d_losses"][0] / n * load).expand(T, E)
        if c["normalize"]:
            direct = weights * (d - (d * weights).sum(dim=1, keepdim=True))
        else:
            a = a.scatter_add(1, chosen, d)
        dz = p * (a - (a * p).sum(dim=1, keepdim=True))
        dz = dz + s["d_losses"][1] * 2.0 / n * lse * p
        if c["normalize"]:
            dz = dz.scatter_add(1, chosen, direct)
        out["dlogits"] = dz.to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------------------
# the work of one pass


def _distinct(case, share):
    """Expected different ids of a case's tokens."""
    V = case["vocab"]
    k = np.arange(V, dtype=np.float64)
    q = (np.log(k + 2.0) - np.log(k + 1.0)) / math.log(V + 1.0)
    kept = case["tokens"] * (1.0 - share)
    return float(np.sum(-np.expm1(kept * np.log1p(-np.minimum(q, 1.0 - 1e-12)))))


def work(case):
    T = case["tokens"]
    if case["op"] in ("embedding", "embedding_train"):
        H, V = case["hidden"], case["vocab"]
        rows = T * (1.0 - case["padded"])
        total = 8 * T + _distinct(case, case["padded"]) * H * BYTES[case["table"]]
        total += T * H * BYTES[case["out"]]
        flops = rows * H
        if case["op"] == "embedding_train":
            total += rows * H * BYTES[case["out"]] + V * H * BYTES[case["grad"]]
            flops += 2 * rows * H
        return {"bytes": int(total), "flops": int(flops)}
    if case["op"] in ("loss", "loss_train"):
        H, V, e = case["hidden"], case["vocab"], BYTES[case["dtype"]]
        rows = T * (1.0 - case["left_out"])
        total = 8 * T + (rows + V) * H * e + 8 * T + 12
        flops = rows * V * (2.0 * H + 4)
        if case["op"] == "loss_train":
            total += T * H * e + V * H * BYTES[case["grad"]]
            flops += rows * V * (4.0 * H + 4)
        return {"bytes": int(total), "flops": int(flops)}
    E, K, e = case["experts"], case["topk"], BYTES[case["dtype"]]
    total = T * E * e + T * K * 8 + 4 * E + 8
    flops = T * E * (K + 6)
    if case["op"] == "route_train":
        total += T * E * e + T * K * 4 + 8
        flops += 8 * T * E
    return {"bytes": int(total), "flops": int(flops)}


# ---------------------------------------------------------------------------
# the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("embedding", "embedding_train"):
        return _embedding_exact(s)
    if case["op"] in ("loss", "loss_train"):
        return _loss_exact(s)
    return _route_exact(s)


def _embedding_exact(s):
    c = s["case"]
    kept = ((s["ids"] >= 0) & (s["ids"] < c["vocab"])).nonzero()[:, 0]
    ids = s["ids"][kept]
    y = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device="cuda")
    y[kept] = s["table"].double()[ids] * c["scale"]
    out = {"y": y}
    if c["op"] == "embedding_train":
        d = torch.zeros(c["vocab"], c["hidden"], dtype=torch.float64, device="cuda")
        out["dtable"] = d.index_add_(0, ids, s["dy"].double()[kept]) * c["scale"]
    return out


def _loss_exact(s):
    """By autograd over the tokens that have a target, some at a time."""
    c = s["case"]
    train = c["op"] == "loss_train"
    T = c["tokens"]
    kept = ((s["targets"] >= 0) & (s["targets"] < c["vocab"])).nonzero()[:, 0]
    n = max(1, kept.numel())
    w = s["w"].double().requires_grad_(train)
    losses = torch.zeros(T, dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(losses)
    dx = torch.zeros(T, c["hidden"], dtype=torch.float64, device="cuda")
    if train:
        w.grad = torch.zeros_like(w)
    for rows in kept.split(max(1, (1 << 26) // c["vocab"])):
        x = s["x"][rows].double().requires_grad_(train)
        z = (x @ w.t()) * c["scale"]
        norm = torch.logsumexp(z, dim=1)
        loss = norm - z.gather(1, s["targets"][rows][:, None])[:, 0]
        losses[rows], lse[rows] = loss.detach(), norm.detach()
        if train:
            d = s["d"].double()
            d = d[rows] if c["reduction"] == "none" else d / n if c["reduction"] == "mean" else d
            (loss * d).sum().backward()
            dx[rows] = x.grad
    count = torch.tensor(float(kept.numel()), dtype=torch.float64, device="cuda")
    out = {"losses": losses, "lse": lse, "total": torch.stack([losses.sum() / n, losses.sum(), count])}
    if train:
        out["dx"], out["dw"] = dx, w.grad
    return out


def _route_exact(s):
    c = s["case"]
    train = c["op"] == "route_train"
    E, K = c["experts"], c["topk"]
    T = c["tokens"]
    rows = (s["logits"] > -math.inf).any(dim=1).nonzero()[:, 0]
    z = s["logits"][rows].double().requires_grad_(train)
    n = max(1, rows.numel())
    lse = torch.logsumexp(z, dim=1)
    p = torch.exp(z - lse[:, None])
    left = s["logits"][rows].double()
    chosen = torch.zeros(rows.numel(), K, dtype=torch.int64, device="cuda")
    kept = torch.zeros(rows.numel(), K, dtype=torch.bool, device="cuda")
    place = torch.arange(E, device="cuda").expand_as(left)
    for k in range(K):  # the largest left, the first of equal ones
        most = left.max(dim=1, keepdim=True).values
        first = torch.where(left == most, place, torch.full_like(place, E)).min(dim=1).values
        chosen[:, k], kept[:, k] = first, most[:, 0] > -math.inf
        left.scatter_(1, first[:, None], -math.inf)
    weights = torch.where(kept, p.gather(1, chosen), torch.zeros((), dtype=torch.float64, device="cuda"))
    if c["normalize"]:
        weights = weights / weights.sum(dim=1, keepdim=True)
    counts = (chosen[kept][:, None] == torch.arange(E, device="cuda")).sum(dim=0) \
        if chosen.numel() * E <= 1 << 28 else torch.bincount(chosen[kept], minlength=E)
    balance = (counts.double() * p.sum(dim=0)).sum() * E / (K * n * n)
    zloss = lse.square().sum() / n
    whole = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    whole[rows] = weights.detach()
    out = {"ids": None, "weights": whole, "counts": None,
           "losses": torch.stack([balance, zloss]).detach()}
    if train:
        d = s["d_losses"].double()
        loss = (weights * s["d_weights"].double()[rows]).sum() + d[0] * balance + d[1] * zloss
        loss.backward()
        dz = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        dz[rows] = torch.nan_to_num(z.grad)
        out["dlogits"] = dz
    return out
