"""Cases of the training-step operators: gradient norm and clipping over many
tensors, the block join (norms before and after a block with its gate and
residual scale), and the expert permutation (tokens sorted by expert, brought
back with weights), each with its plain form, its exact values and its work.

``run(state)`` makes one pass: in plain torch operations in 32 bits where
``own`` is false, through the package's entry points where it is true.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# the cases


def listed():
    return [
        # the gradients of the two-block MLP group (1.05M parameters, 10
        # tensors), clipped into its flat 16-bit replica: launches count
        dict(name="clip_mlp", op="clip", layout="mlp", dtype="fp16", out="fp16", max_norm=1.0),
        # the gradients of the 101M-parameter ToyModel (50 tensors)
        dict(name="clip_toy", op="clip", layout="toy", dtype="bf16", out="bf16", max_norm=1.0),
        # 1500 small tensors of odd sizes (norm gains, biases, adapters), fp32
        # and 16-bit mixed, clipped into one 16-bit replica at odd offsets
        dict(name="clip_many", op="clip", layout="ragged", tensors=1500, total=12_000_000,
             dtype="mixed", out="bf16", max_norm=0.5),
        # the norm alone, as a logger or an overflow check takes it, of the
        # fp32 gradients of one LLaMA-13B MLP layer (212M elements)
        dict(name="norm_layer_13b", op="norm", layout="layer", hidden=5120, ffn=13824,
             dtype="fp32"),
        # one token through a join, as a serving step makes it: latency
        dict(name="join_one_token", op="join", rows=1, hidden=4096, kind="rms", gate="channel",
             post=True, pre=True, dtype="bf16", res="bf16", param="bf16", scale=0.5),
        # a prompt of a 13B-shaped model on an fp32 residual stream
        dict(name="join_prompt", op="join", rows=8191, hidden=5120, kind="rms", gate="none",
             post=False, pre=True, dtype="bf16", res="fp32", param="bf16", scale=1.0),
        # training rows of a 7B-shaped model, norms on both sides, gated
        dict(name="join_train_7b", op="join_train", rows=16384, hidden=4096, kind="rms",
             gate="channel", post=True, pre=True, dtype="bf16", res="bf16", param="bf16",
             scale=0.25),
        # BERT-base rows: LayerNorm of the sum, its biases, fp16
        dict(name="join_train_bert", op="join_train", rows=32768, hidden=768, kind="layer",
             gate="none", post=False, pre=True, dtype="fp16", res="fp16", param="fp32",
             scale=1.0),
        # an odd hidden size, a gate for every element, LayerNorm on both sides
        dict(name="join_train_odd", op="join_train", rows=3001, hidden=1021, kind="layer",
             gate="full", post=True, pre=True, dtype="fp32", res="fp32", param="fp32",
             scale=0.7),
        # eight sequences decode one token each, two of eight experts a token
        dict(name="experts_decode", op="experts", tokens=8, topk=2, experts=8, hidden=4096,
             dtype="bf16", weights="fp32", drop=0.0),
        # a training batch of a 7B-shaped model with 64 experts
        dict(name="experts_train", op="experts_train", tokens=16384, topk=2, experts=64,
             hidden=4096, dtype="bf16", weights="fp32", drop=0.0),
        # ragged: odd sizes, 32-bit rows, a tenth of the choices dropped
        dict(name="experts_train_odd", op="experts_train", tokens=2999, topk=3, experts=17,
             hidden=1001, dtype="fp32", weights="fp32", drop=0.1),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["clip", "norm", "join", "join_train", "experts", "experts_train"])
    if op in ("clip", "norm"):
        tensors = _spread(rng, 1, 1500)
        total = max(tensors, _spread(rng, 50_000, 100_000_000))
        c = dict(op=op, layout="ragged", tensors=tensors, total=total,
                 dtype=rng.choice(["fp16", "bf16", "fp32", "mixed"]))
        if op == "clip":
            c["out"] = "bf16" if c["dtype"] == "mixed" else c["dtype"]
            c["max_norm"] = round(math.exp(rng.uniform(math.log(0.05), math.log(20.0))), 3)
        return c
    if op in ("join", "join_train"):
        hidden = _spread(rng, 64, 8192)
        if rng.random() < 0.7:
            hidden = max(64, hidden // 8 * 8)
        most = 16384 * 4096 // 2 // hidden
        act = rng.choice(["fp16", "bf16", "fp32"])
        post, pre = rng.choice([(True, True), (True, False), (False, True)])
        return dict(op=op, rows=_spread(rng, 1, min(most, 65536)), hidden=hidden,
                    kind=rng.choice(["rms", "layer"]),
                    gate=rng.choice(["none", "channel", "row", "full"]), post=post, pre=pre,
                    dtype=act, res=rng.choice([act, "fp32"]), param=rng.choice([act, "fp32"]),
                    scale=round(rng.uniform(0.1, 1.0), 3))
    topk = rng.choice([1, 2, 3, 4, 6, 8])
    hidden = _spread(rng, 64, 8192)
    if rng.random() < 0.7:
        hidden = max(64, hidden // 8 * 8)
    most = 16384 * 4096 // (hidden * topk)
    dtype = rng.choice(["fp16", "bf16", "fp32"])
    return dict(op=op, tokens=_spread(rng, 1, max(1, min(most, 65536))), topk=topk,
                experts=max(topk, _spread(rng, 2, 512)), hidden=hidden, dtype=dtype,
                weights=rng.choice([dtype, "fp32"]), drop=rng.choice([0.0, 0.0, 0.1, 0.5]))


# ---------------------------------------------------------------------------
# inputs


def _sizes(case):
    """Element counts of a group's tensors, in parameter order."""
    if case["layout"] == "mlp":
        return [256 * 1024, 1024, 1024 * 256, 256] * 2 + [256 * 10, 10]
    if case["layout"] == "toy":
        return [1024 * 4096, 4096, 4096 * 1024, 1024] * 12 + [1024 * 10, 10]
    if case["layout"] == "layer":
        return [case["hidden"] * case["ffn"]] * 3
    rng = random.Random(case["tensors"] * 1_000_003 + case["total"])
    share = [math.exp(rng.gauss(0.0, 1.0)) for _ in range(case["tensors"])]
    unit = case["total"] / sum(share)
    return [max(1, int(s * unit)) for s in share]


def _kinds(case, n):
    if case["dtype"] != "mixed":
        return [DTYPES[case["dtype"]]] * n
    return [torch.float32 if k % 3 == 0 else torch.bfloat16 for k in range(n)]


def _gradients(case, gen):
    """One tensor each, values ~N(0, 1e-2) with 1% of the entries times 100."""
    sizes = _sizes(case)
    flat = torch.randn(sum(sizes), device="cuda", generator=gen).mul_(1e-2)
    far = torch.randint(0, flat.numel(), (flat.numel() // 100,), device="cuda", generator=gen)
    flat[far] *= 100.0
    at, grads = 0, []
    for n, dt in zip(sizes, _kinds(case, len(sizes))):
        grads.append(flat[at:at + n].to(dt, copy=True))
        at += n
    return grads


def _experts(case, gen):
    """Each token's choices without repeats, some experts more wanted than
    others; dropped ones are -1."""
    T, K, E = case["tokens"], case["topk"], case["experts"]
    want = torch.linspace(0.0, 2.0, E, device="cuda")
    score = torch.randn(T, E, device="cuda", generator=gen) + want
    value, ids = score.topk(K, dim=1)
    weights = torch.softmax(value, dim=1).to(DTYPES[case["weights"]])
    if case["drop"]:
        gone = torch.rand(T, K, device="cuda", generator=gen) < case["drop"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32), weights


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype, scale=1.0, shift=0.0):
        x = torch.randn(*shape, device="cuda", generator=gen)
        return x.mul_(scale).add_(shift).to(dtype)

    s = {"case": case}
    if case["op"] in ("clip", "norm"):
        s["grads"] = grads = _gradients(case, gen)
        if case["op"] == "clip":
            total = sum(g.numel() for g in grads)
            s["flat"] = torch.zeros(total, dtype=DTYPES[case["out"]], device="cuda")
            at, views = 0, []
            for g in grads:
                views.append(s["flat"][at:at + g.numel()])
                at += g.numel()
        if own:  # the prepared call that a training loop keeps for its buffers
            import zero_sharded_optimizer_flatten_gb300 as Z
            if case["op"] == "clip":
                s["call"] = Z.ClipGradNorm(grads, case["max_norm"], out=views)
            else:
                s["call"] = Z.GradNorm(grads)
        return s
    if case["op"] in ("join", "join_train"):
        R, H = case["rows"], case["hidden"]
        act, res, par = DTYPES[case["dtype"]], DTYPES[case["res"]], DTYPES[case["param"]]
        s["x"] = normal(R, H, dtype=res, scale=2.0)
        s["b"] = normal(R, H, dtype=act, scale=0.5, shift=0.1)
        s["w_post"] = normal(H, dtype=par, scale=0.1, shift=1.0) if case["post"] else None
        s["w_pre"] = normal(H, dtype=par, scale=0.1, shift=1.0) if case["pre"] else None
        layer = case["kind"] == "layer"
        s["bias_post"] = normal(H, dtype=par, scale=0.1) if layer and case["post"] else None
        s["bias_pre"] = normal(H, dtype=par, scale=0.1) if layer and case["pre"] else None
        shape = {"none": None, "channel": (H,), "row": (R, 1), "full": (R, H)}[case["gate"]]
        s["gate"] = None if shape is None else normal(*shape, dtype=act, scale=0.3, shift=0.5)
        if case["op"] == "join_train":
            s["d_o"] = normal(R, H, dtype=res, scale=1e-2)
            s["d_n"] = normal(R, H, dtype=act, scale=1e-2) if case["pre"] else None
        return s
    T, K, H, dt = case["tokens"], case["topk"], case["hidden"], DTYPES[case["dtype"]]
    s["ids"], s["weights"] = _experts(case, gen)
    s["x"] = normal(T, H, dtype=dt)
    s["ys"] = normal(T * K, H, dtype=dt)
    if case["op"] == "experts_train":
        s["dy"] = normal(T, H, dtype=dt, scale=1e-2)
        s["dxs"] = normal(T * K, H, dtype=dt, scale=1e-2)
    return s


# ---------------------------------------------------------------------------
# one pass


def run(state):
    op = state["case"]["op"]
    if op == "clip":
        return _clip_own(state) if own else _clip_plain(state)
    if op == "norm":
        return [state["call"]()] if own else [_norm_plain(state["grads"])]
    if op == "join":
        return _join_own(state) if own else _join_plain(state)
    if op == "join_train":
        return _join_train_own(state) if own else _join_train_plain(state)
    return _experts_own(state) if own else _experts_plain(state)


def _clip_own(s):
    norm = s["call"]()
    return {"norm": norm, "flat": s["flat"]}


def _norm_plain(grads):
    return torch.cat([g.float() for g in grads]).square().sum().sqrt()


def _clip_plain(s):
    flat = torch.cat([g.float() for g in s["grads"]])
    norm = flat.square().sum().sqrt()
    coef = torch.clamp(s["case"]["max_norm"] / (norm + 1e-6), max=1.0)
    s["flat"].copy_(flat * coef)
    return {"norm": norm, "flat": s["flat"]}


EPS = 1e-6


def _own_params(s):
    c = s["case"]
    return dict(w_post=s["w_post"], bias_post=s["bias_post"], w_pre=s["w_pre"],
                bias_pre=s["bias_pre"], gate=s["gate"], kind=c["kind"], scale=c["scale"], eps=EPS)


def _join_own(s):
    import zero_sharded_optimizer_flatten_gb300 as Z
    o, n, _ = Z.zero_block_join(s["x"], s["b"], **_own_params(s))
    return {"o": o, "n": n}


def _join_train_own(s):
    import zero_sharded_optimizer_flatten_gb300 as Z
    params = _own_params(s)
    o, n, stats = Z.zero_block_join(s["x"], s["b"], want_stats=True, **params)
    grads = Z.zero_block_join_backward(s["x"], s["b"], s["d_o"], s["d_n"], stats, **params)
    return {"o": o, "n": n, **grads}


def _normed(v, kind):
    """(v - mean) / deviation and 1 / deviation of every row; no mean for rms."""
    if kind == "layer":
        v = v - v.mean(dim=-1, keepdim=True)
    r = torch.rsqrt(v.square().mean(dim=-1, keepdim=True) + EPS)
    return v * r, r


def _affine(v, w, bias):
    v = v * w.float()
    return v if bias is None else v + bias.float()


def _join_parts(s):
    c = s["case"]
    x, b = s["x"].float(), s["b"].float()
    bh = rb = oh = ro = n = None
    u = b
    if c["post"]:
        bh, rb = _normed(b, c["kind"])
        u = _affine(bh, s["w_post"], s["bias_post"])
    g = c["scale"] if s["gate"] is None else c["scale"] * s["gate"].float()
    o = x + g * u
    if c["pre"]:
        oh, ro = _normed(o, c["kind"])
        n = _affine(oh, s["w_pre"], s["bias_pre"])
    return g, u, bh, rb, o, oh, ro, n


def _join_plain(s):
    g, u, bh, rb, o, oh, ro, n = _join_parts(s)
    return {"o": o.to(s["x"].dtype), "n": None if n is None else n.to(s["b"].dtype)}


def _normed_backward(t, vh, r, kind):
    """Gradient of _normed's input from that of its output."""
    d = t - vh * (t * vh).mean(dim=-1, keepdim=True)
    if kind == "layer":
        d = d - t.mean(dim=-1, keepdim=True)
    return d * r


def _join_train_plain(s):
    c = s["case"]
    g, u, bh, rb, o, oh, ro, n = _join_parts(s)
    out = {"o": o.to(s["x"].dtype), "n": None if n is None else n.to(s["b"].dtype)}
    for k in ("dgate", "dw_post", "dbias_post", "dw_pre", "dbias_pre"):
        out[k] = None
    do = s["d_o"].float()
    if c["pre"]:
        dn = s["d_n"].float()
        out["dw_pre"] = (dn * oh).sum(dim=0).to(s["w_pre"].dtype)
        if s["bias_pre"] is not None:
            out["dbias_pre"] = dn.sum(dim=0).to(s["bias_pre"].dtype)
        do = do + _normed_backward(dn * s["w_pre"].float(), oh, ro, c["kind"])
    out["dx"] = do.to(s["x"].dtype)
    if s["gate"] is not None:
        dg = c["scale"] * do * u
        if c["gate"] == "channel":
            dg = dg.sum(dim=0)
        elif c["gate"] == "row":
            dg = dg.sum(dim=1, keepdim=True)
        out["dgate"] = dg.to(s["gate"].dtype)
    du = g * do
    if c["post"]:
        out["dw_post"] = (du * bh).sum(dim=0).to(s["w_post"].dtype)
        if s["bias_post"] is not None:
            out["dbias_post"] = du.sum(dim=0).to(s["bias_post"].dtype)
        du = _normed_backward(du * s["w_post"].float(), bh, rb, c["kind"])
    out["db"] = du.to(s["b"].dtype)
    return out


def _experts_own(s):
    import zero_sharded_optimizer_flatten_gb300 as Z
    c = s["case"]
    order = Z.zero_expert_sort(s["ids"], c["experts"])
    out = {"offsets": order.offsets, "rows": order.rows, "pairs": order.pairs,
           "xs": Z.zero_expert_dispatch(s["x"], order),
           "y": Z.zero_expert_combine(s["ys"], s["weights"], order)}
    if c["op"] == "experts_train":
        out["dys"], out["dweights"] = Z.zero_expert_combine_backward(s["dy"], s["ys"],
                                                                     s["weights"], order)
        out["dx"] = Z.zero_expert_dispatch_backward(s["dxs"], order)
    return out


def _experts_plain(s):
    c = s["case"]
    T, K = s["ids"].shape
    E, H = c["experts"], c["hidden"]
    ids = s["ids"].reshape(-1)
    kept = (ids >= 0) & (ids < E)
    key = torch.where(kept, ids, torch.full_like(ids, E))
    pairs = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    counts.scatter_add_(0, key.long(), torch.ones_like(key, dtype=torch.int64))
    offsets = (counts.cumsum(0) - counts).to(torch.int32)
    place = torch.empty_like(pairs)
    place[pairs] = torch.arange(T * K, device="cuda")
    sorted_kept = kept[pairs]
    xs = s["x"][pairs // K] * sorted_kept[:, None]
    w = (s["weights"].float().reshape(-1) * kept).reshape(T, K, 1)
    ys = s["ys"][place].float().reshape(T, K, H)
    y = (w * torch.where(kept.reshape(T, K, 1), ys, torch.zeros_like(ys))).sum(dim=1)
    out = {"offsets": offsets,
           "rows": torch.where(kept, place, torch.full_like(place, -1)).to(torch.int32).reshape(T, K),
           "pairs": torch.where(sorted_kept, pairs, torch.full_like(pairs, -1)).to(torch.int32),
           "xs": xs, "y": y.to(s["ys"].dtype)}
    if c["op"] == "experts_train":
        dy = s["dy"].float()
        dys = (dy[pairs // K] * w.reshape(-1)[pairs][:, None]).to(s["ys"].dtype)
        dw = (dy[:, None, :] * ys).sum(dim=2) * kept.reshape(T, K)
        dxs = s["dxs"][place].float().reshape(T, K, H)
        out["dys"], out["dweights"] = dys, dw.to(s["weights"].dtype)
        out["dx"] = (dxs * kept.reshape(T, K, 1)).sum(dim=1).to(s["dxs"].dtype)
    return out


# ---------------------------------------------------------------------------
# the work of one pass


def work(case):
    if case["op"] in ("clip", "norm"):
        sizes = _sizes(case)
        read = sum(n * k.itemsize for n, k in zip(sizes, _kinds(case, len(sizes))))
        write = sum(sizes) * BYTES[case["out"]] if case["op"] == "clip" else 0
        return {"bytes": read + write + 4, "flops": (3 if write else 2) * sum(sizes)}
    if case["op"] in ("join", "join_train"):
        R, H = case["rows"], case["hidden"]
        act, res, par = (BYTES[case[k]] for k in ("dtype", "res", "param"))
        gate = {"none": 0, "channel": H, "row": R, "full": R * H}[case["gate"]] * act
        vectors = (int(case["post"]) + int(case["pre"])) * (2 if case["kind"] == "layer" else 1)
        row = 2 * res + act + (act if case["pre"] else 0)
        total = R * H * row + gate + vectors * H * par
        flops = R * H * (4 + 5 * int(case["post"]) + 5 * int(case["pre"]))
        if case["op"] == "join_train":
            row = 3 * res + 2 * act + (act if case["pre"] else 0)
            total += R * H * row + 2 * gate + 2 * vectors * H * par
            flops += R * H * (8 + 12 * int(case["post"]) + 12 * int(case["pre"]))
        return {"bytes": total, "flops": flops}
    T, K, H = case["tokens"], case["topk"], case["hidden"]
    e, w = BYTES[case["dtype"]], BYTES[case["weights"]]
    keep = 1.0 - case["drop"]
    total = 4 * T * K * 3 + 4 * (case["experts"] + 1) + T * K * w
    total += T * H * e * 2 + T * K * H * e * (1 + keep)
    flops = 2 * T * K * H
    if case["op"] == "experts_train":
        total += T * H * e * 2 + T * K * H * e * (1 + 2 * keep) + 2 * T * K * w
        flops += 4 * T * K * H
    return {"bytes": total, "flops": flops}


# ---------------------------------------------------------------------------
# the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("clip", "norm"):
        sq = 0.0
        for g in s["grads"]:
            sq += float(g.double().pow(2).sum())
        norm = torch.tensor(math.sqrt(sq), dtype=torch.float64)
        if case["op"] == "norm":
            return [norm]
        factor = min(1.0, case["max_norm"] / (float(norm) + 1e-6))
        return {"norm": norm, "flat": torch.cat([g.double() * factor for g in s["grads"]])}
    if case["op"] in ("join", "join_train"):
        return _join_exact(s)
    return _experts_exact(s)


def _join_exact(s):
    c = s["case"]
    train = c["op"] == "join_train"
    names = ("x", "b", "gate", "w_post", "bias_post", "w_pre", "bias_pre")
    v = {k: None if s[k] is None else s[k].double().requires_grad_(train) for k in names}

    def norm(t, w, bias):
        H = t.shape[-1]
        if c["kind"] == "layer":
            t = t - t.sum(-1, keepdim=True) / H
        t = t / (t.pow(2).sum(-1, keepdim=True) / H + EPS).sqrt() * w
        return t if bias is None else t + bias

    u = norm(v["b"], v["w_post"], v["bias_post"]) if c["post"] else v["b"]
    if v["gate"] is not None:
        u = u * v["gate"]
    o = v["x"] + c["scale"] * u
    n = norm(o, v["w_pre"], v["bias_pre"]) if c["pre"] else None
    out = {"o": o.detach(), "n": None if n is None else n.detach()}
    if train:
        loss = (o * s["d_o"].double()).sum()
        if n is not None:
            loss = loss + (n * s["d_n"].double()).sum()
        loss.backward()
        for k in names:
            out["dx" if k == "x" else "db" if k == "b" else "d" + k] = \
                None if v[k] is None else v[k].grad
    return out


def _experts_exact(s):
    c = s["case"]
    K, E = c["topk"], c["experts"]
    ids = s["ids"].reshape(-1).cpu().tolist()
    lists = [[] for _ in range(E)]
    for p, e in enumerate(ids):
        if 0 <= e < E:
            lists[e].append(p)
    order = [p for members in lists for p in members]
    M = len(order)
    at = torch.tensor(order, dtype=torch.int64, device="cuda")
    token = at // K
    w = s["weights"].double().reshape(-1)[at][:, None]
    ys = s["ys"][:M].double()
    xs = torch.zeros(s["ys"].shape, dtype=torch.float64, device="cuda")
    xs[:M] = s["x"][token].double()
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    y.index_add_(0, token, w * ys)
    out = {"offsets": None, "rows": None, "pairs": None, "xs": xs, "y": y}
    if c["op"] == "experts_train":
        dy = s["dy"].double()[token]
        dys = torch.zeros_like(xs)
        dys[:M] = w * dy
        dw = torch.zeros(s["weights"].numel(), dtype=torch.float64, device="cuda")
        dw[at] = (dy * ys).sum(1)
        dx = torch.zeros_like(y)
        dx.index_add_(0, token, s["dxs"][:M].double())
        out["dys"], out["dweights"], out["dx"] = dys, dw.reshape(s["weights"].shape), dx
    return out
