"""The operators on rows of scores, as cases that are timed and checked: routing tokens to experts
(``route``, and ``route_train`` with its gradient), grouping the routed choices by expert (``group``),
and log probabilities of given tokens with entropy and top alternatives (``logprobs``, and
``logprobs_train`` with its gradient).

``run`` computes a case in plain torch operations, or, where ``own`` is true, with this library's
calls; ``exact`` computes it again from the definitions in 64 bits.

Definitions.  Routing: p = softmax or sigmoid of a row's scores; experts are chosen by s = p + bias
(without a bias by the scores themselves), the best ``top_k`` inside the best ``top_groups`` groups, a
group's score being the sum of its best ``group_best`` s; ties go to the lowest index; the weights are
scale * p, or scale * p / (sum of the chosen p).  Grouping: the choices (flat indices of a [rows, top_k]
id array) ordered by expert, stably, each expert's segment padded to a multiple of ``align`` with -1;
ids of -1 are dropped.  Log probabilities: of scale * logits, a row with target -1 has log probability 0
and rank -1; the rank counts the logits above the target's, and equal ones at lower indices.
"""
import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one decoded token's router, the smallest call: its time is launch and host latency
        _route("route", "route_step", rows=1, experts=128, top_k=8, dtype="bf16"),
        # a long prompt through a router with sigmoid scores, a balance bias and expert groups
        _route("route", "route_prompt_groups", rows=16384, experts=256, top_k=8, dtype="f32",
               score="sigmoid", bias=True, groups=8, top_groups=4, group_best=2, scale=2.5),
        # a training step's router whose weights stay plain probabilities: the gradient reaches every expert
        _route("route_train", "route_train_softmax", rows=8192, experts=64, top_k=6, dtype="f16",
               renormalize=False),
        # a training step's router over many experts, with the balance bias and renormalised weights
        _route("route_train", "route_train_sigmoid", rows=32768, experts=512, top_k=8, dtype="f32",
               score="sigmoid", bias=True, scale=1.5),
        # the choices of a small decode batch, segments padded to a matrix tile of 16 rows
        _group("group_step", rows=32, top_k=8, experts=128, align=16),
        # the choices of a long prompt, segments padded to tiles of 128 rows, some padding tokens dropped
        _group("group_prompt", rows=16384, top_k=8, experts=256, align=128, dropped=0.03),
        # a training step's choices over many crowded and empty experts, no padding, an odd count
        _group("group_train", rows=262147, top_k=5, experts=1000, align=1, skew=1.0),
        # four sequences' next-token logits with the 20 best alternatives: few rows, a long axis
        _logits("logprobs", "logprobs_step", rows=4, vocab=131072, dtype="bf16", top_k=20),
        # every prompt position scored, with 8 alternatives
        _logits("logprobs", "logprobs_prompt", rows=2048, vocab=131072, dtype="bf16", top_k=8),
        # constrained decoding at a temperature: most of the vocabulary masked, an odd vocabulary in padded rows
        _logits("logprobs", "logprobs_masked", rows=257, vocab=50021, dtype="f32", top_k=5, pad=27,
                scale=1.4, masked=0.9, ignored=0.1),
        # a policy-gradient step: log probabilities and entropies of the sampled tokens, and the logits' gradient
        _logits("logprobs_train", "logprobs_train_long", rows=2048, vocab=131072, dtype="bf16", ignored=0.2),
        # the same on a small odd batch in full precision
        _logits("logprobs_train", "logprobs_train_odd", rows=501, vocab=32003, dtype="f32", ignored=0.05),
    ]


def _route(op, name, rows, experts, top_k, dtype, score="softmax", bias=False, groups=1, top_groups=1,
           group_best=1, renormalize=True, scale=1.0, pad=0):
    return {"name": name, "op": op, "rows": rows, "experts": experts, "top_k": top_k, "dtype": dtype,
            "score": score, "bias": bias, "groups": groups, "top_groups": top_groups,
            "group_best": group_best, "renormalize": renormalize, "scale": scale, "pad": pad}


def _group(name, rows, top_k, experts, align, dropped=0.0, skew=0.0):
    return {"name": name, "op": "group", "rows": rows, "top_k": top_k, "experts": experts,
            "align": align, "dropped": dropped, "skew": skew}


def _logits(op, name, rows, vocab, dtype, top_k=0, scale=1.0, masked=0.0, ignored=0.0, pad=0):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "top_k": top_k,
            "scale": scale, "masked": masked, "ignored": ignored, "pad": pad}


def draw(rng):
    def spread(lo, hi):   # uniform over the logarithm
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["route", "route_train", "group", "logprobs", "logprobs_train"])
    if op == "group":
        top_k = rng.choice([1, 2, 4, 5, 6, 8])
        c = _group("", rows=spread(1, 262144), top_k=top_k, experts=spread(1, 1024),
                   align=rng.choice([1, 1, 8, 16, 64, 100, 128]),
                   dropped=rng.choice([0.0, 0.02, 0.3]), skew=rng.choice([0.0, 0.7, 1.3]))
    elif op.startswith("route"):
        groups = rng.choice([1, 1, 2, 4, 8])
        size = spread(max(1, 8 // groups), 1024 // groups)
        experts = groups * size
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(12, top_groups * size))
        c = _route(op, "", rows=spread(1, min(32768, 16000000 // experts)), experts=experts,
                   top_k=top_k, dtype=rng.choice(["f32", "f16", "bf16"]),
                   score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                   top_groups=top_groups, group_best=rng.choice([1, min(2, size)]),
                   renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 2.5]),
                   pad=rng.choice([0, 0, 3, 8]))
    else:
        vocab = spread(100, 262144)
        c = _logits(op, "", rows=spread(1, min(4096, 130000000 // vocab)), vocab=vocab,
                    dtype=rng.choice(["f32", "f16", "bf16"]),
                    top_k=0 if op == "logprobs_train" else rng.choice([0, 1, 5, 20, 64]),
                    scale=rng.choice([1.0, 1.0, 0.8, 1.4]), masked=rng.choice([0.0, 0.0, 0.5, 0.95]),
                    ignored=rng.choice([0.0, 0.1]), pad=rng.choice([0, 0, 1, 8, 64]))
    del c["name"]
    return c


def _matrix(g, rows, cols, pad, spread, dtype):
    """A [rows, cols] view of rows that are cols + pad apart, as a padded projection leaves it."""
    return (torch.randn(rows, cols + pad, generator=g, device="cuda") * spread).to(dtype)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    rows = case["rows"]
    if case["op"] == "group":
        # experts by a power law of their number (skew 0: evenly), as a router leaves them; -1 for padding tokens
        law = torch.arange(1, case["experts"] + 1, device="cuda", dtype=torch.float64) ** -case["skew"]
        law = law[torch.randperm(case["experts"], generator=g, device="cuda")]
        at = torch.rand(rows * case["top_k"], generator=g, device="cuda", dtype=torch.float64)
        ids = torch.searchsorted(torch.cumsum(law, 0) / law.sum(), at).clamp_(max=case["experts"] - 1)
        gone = torch.rand(rows, 1, generator=g, device="cuda") < case["dropped"]
        s["ids"] = ids.to(torch.int32).view(rows, case["top_k"]).masked_fill_(gone, -1)
    elif case["op"].startswith("route"):
        s["x"] = _matrix(g, rows, case["experts"], case["pad"], 1.5, _DTYPES[case["dtype"]])
        s["b"] = torch.randn(case["experts"], generator=g, device="cuda") * 0.05 if case["bias"] else None
        s["dw"] = torch.randn(rows, case["top_k"], generator=g, device="cuda")
    else:
        # logits of a trained model: a wide spread, and a target that is most often a likely token
        x = _matrix(g, rows, case["vocab"], case["pad"], 3.0, _DTYPES[case["dtype"]])
        t = torch.randint(0, case["vocab"], (rows,), generator=g, device="cuda")
        lift = torch.rand(rows, generator=g, device="cuda") * 20
        x[torch.arange(rows, device="cuda"), t] += lift.to(x.dtype)
        if case["masked"]:
            gone = torch.rand(rows, case["vocab"], generator=g, device="cuda") < case["masked"]
            gone[torch.arange(rows, device="cuda"), t] = False
            x.masked_fill_(gone, float("-inf"))
        off = torch.rand(rows, generator=g, device="cuda") < case["ignored"]
        s["x"], s["t"] = x, t.masked_fill_(off, -1).to(torch.int32)
        s["dlp"] = torch.randn(rows, generator=g, device="cuda")
        s["dh"] = torch.randn(rows, generator=g, device="cuda") * 0.1
    return s


# --- plain forms ---------------------------------------------------------------------------------

def _plain_route(x, bias, c):
    x32 = x.float()
    wide = x32.double()   # the choice is made in 64 bits: scores next to each other decide it
    if c["score"] == "softmax":
        p64 = torch.exp(wide - wide.amax(1, keepdim=True))
        p64 = p64 / p64.sum(1, keepdim=True)
        p = torch.exp(x32 - x32.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p64, p = 1 / (1 + torch.exp(-wide)), 1 / (1 + torch.exp(-x32))
    s = wide if bias is None else p64 + bias.double()
    size = c["experts"] // c["groups"]
    by_group = (p64 if bias is None and c["group_best"] == 2 else s).view(-1, c["groups"], size)
    of_group = torch.topk(by_group, c["group_best"], dim=2).values.sum(2)
    kept = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
    keep = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, kept, True)
    s = s.view(-1, c["groups"], size).masked_fill(~keep[:, :, None], float("-inf")).view(x.shape)
    ids = torch.sort(s, dim=1, descending=True, stable=True).indices[:, : c["top_k"]]
    w = p.gather(1, ids)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return ids, w * c["scale"], p


def _plain_route_grad(ids, w, p, dw, c):
    g = p.gather(1, ids)
    if c["renormalize"]:
        share = g / g.sum(1, keepdim=True)
        dg = (dw - (dw * share).sum(1, keepdim=True)) * (c["scale"] / g.sum(1, keepdim=True))
    else:
        dg = dw * c["scale"]
    dp = torch.zeros_like(p).scatter_(1, ids, dg)
    if c["score"] == "softmax":
        return p * (dp - (dp * p).sum(1, keepdim=True))
    return dp * p * (1 - p)


def _plain_group(ids, c):
    flat = ids.reshape(-1).long()
    n, experts, align = flat.numel(), c["experts"], c["align"]
    key = torch.where(flat >= 0, flat, experts)
    ranked, order = torch.sort(key, stable=True)
    edge = torch.searchsorted(ranked, torch.arange(experts + 1, device=ids.device))
    counts = edge[1:] - edge[:-1]
    ends = torch.cumsum((counts + align - 1) // align * align, 0)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    room = n + experts * (align - 1)
    to = torch.where(ranked < experts, starts[ranked] + torch.arange(n, device=ids.device) - edge[ranked], room)
    out = torch.full((room + 1,), -1, dtype=torch.int32, device=ids.device)
    out[to] = order.to(torch.int32)
    place = torch.empty(n, dtype=torch.int32, device=ids.device)
    place[order] = torch.where(to < room, to, -1).to(torch.int32)
    return {"order": out[:room], "place": place.view(ids.shape), "starts": starts.to(torch.int32),
            "counts": counts.to(torch.int32)}


def _plain_logprobs(x, t, c):
    x32 = x.float()
    at = torch.arange(x.shape[1], device=x.device)
    given = t >= 0
    target = t.long().clamp(min=0)[:, None]
    m = x32.amax(1, keepdim=True)
    d = (x32 - m) * c["scale"]
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    xt = x32.gather(1, target)
    out = {"lse": (m * c["scale"] + torch.log(s))[:, 0], "stats": torch.cat([m, s], 1),
           "logprob": torch.where(given, ((xt - m) * c["scale"] - torch.log(s))[:, 0], 0.0),
           "entropy": (torch.log(s) - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / s)[:, 0]}
    ahead = ((x32 > xt) | ((x32 == xt) & (at < target))).sum(1)
    out["rank"] = torch.where(given, ahead, -1).to(torch.int32)
    if c["top_k"]:
        # one whole number for each logit, larger for what comes first: the value's order, then the lower index
        bits = (x32 + 0.0).view(torch.int32).long()
        first = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 32) - at
        ids = torch.topk(first, c["top_k"], dim=1).indices
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = (x32.gather(1, ids) - m) * c["scale"] - torch.log(s)
    return out, d, e


def _plain_logprobs_grad(x, t, dlp, dh, c, out, d, e):
    s = out["stats"][:, 1:]
    p, logp = e / s, d - torch.log(s)
    a = torch.where(t >= 0, dlp, 0.0)[:, None]
    dz = -a * p - dh[:, None] * torch.where(p > 0, p * (logp + out["entropy"][:, None]), 0.0)
    dz.scatter_add_(1, t.long().clamp(min=0)[:, None], a)
    return (dz * c["scale"]).to(x.dtype)


def run(state):
    s = state
    if s["op"] == "group":
        if own:
            import sorting_lsd_radix_amd as rs
            order, place, starts, counts = rs.group_choices(s["ids"], s["experts"], align=s["align"])
            return {"order": order, "place": place, "starts": starts, "counts": counts}
        return _plain_group(s["ids"], s)
    if s["op"].startswith("route"):
        if own:
            import sorting_lsd_radix_amd as rs
            how = {"score": s["score"], "renormalize": s["renormalize"], "scale": s["scale"]}
            ids, w = rs.route_topk(s["x"], s["top_k"], bias=s["b"], groups=s["groups"],
                                   top_groups=s["top_groups"], group_best=s["group_best"], **how)
            out = {"ids": ids, "weights": w}
            if s["op"] == "route_train":
                out["dscores"] = rs.route_topk_grad(s["x"], ids, w, s["dw"], **how)
            return out
        ids, w, p = _plain_route(s["x"], s["b"], s)
        out = {"ids": ids.to(torch.int32), "weights": w}
        if s["op"] == "route_train":
            out["dscores"] = _plain_route_grad(ids, w, p, s["dw"], s).to(s["x"].dtype)
        return out
    if own:
        import sorting_lsd_radix_amd as rs
        r = rs.token_logprobs(s["x"], s["t"], top_k=s["top_k"], scale=s["scale"])
        out = {"lse": r.lse, "stats": r.stats, "logprob": r.logprob, "entropy": r.entropy, "rank": r.rank}
        if s["top_k"]:
            out["top_ids"], out["top_logprobs"] = r.top_ids, r.top_logprobs
        if s["op"] == "logprobs_train":
            out["dlogits"] = rs.token_logprobs_grad(s["x"], r.stats, s["t"], dlogprob=s["dlp"],
                                                    entropy=r.entropy, dentropy=s["dh"], scale=s["scale"])
        return out
    out, d, e = _plain_logprobs(s["x"], s["t"], s)
    if s["op"] == "logprobs_train":
        out["dlogits"] = _plain_logprobs_grad(s["x"], s["t"], s["dlp"], s["dh"], s, out, d, e)
    return out


def work(case):
    rows = case["rows"]
    if case["op"] == "group":
        n = rows * case["top_k"]
        room = n + case["experts"] * (case["align"] - 1)
        return {"bytes": 4 * (2 * n + room + 2 * case["experts"] + 1), "flops": 0}
    size = _SIZES[case["dtype"]]
    if case["op"].startswith("route"):
        e = rows * case["experts"]
        b = e * size + rows * case["top_k"] * 8 + (4 * case["experts"] if case["bias"] else 0)
        if case["op"] == "route_train":
            b += e * size + rows * case["top_k"] * 4
        return {"bytes": b, "flops": e * (8 if case["op"] == "route_train" else 4)}
    v = rows * case["vocab"]
    b = v * size + rows * (4 + 24 + 8 * case["top_k"])
    if case["op"] == "logprobs_train":
        b += v * size + 8 * rows
    return {"bytes": b, "flops": v * (14 if case["op"] == "logprobs_train" else 6)}


# --- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "group":
        return None   # whole numbers only
    s = prepare(case, seed)
    parts = []
    step = max(1, 40_000_000 // s["x"].shape[1])   # rows at a time
    for r in range(0, case["rows"], step):
        rows = slice(r, r + step)
        x = s["x"][rows].to(torch.float64)
        parts.append(_exact_route(x, s, rows) if case["op"].startswith("route") else _exact_logprobs(x, s, rows))
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_route(x, s, rows):
    n = torch.arange(x.shape[0], device=x.device)
    p = torch.softmax(x, 1) if s["score"] == "softmax" else torch.sigmoid(x)
    key = x.clone() if s["b"] is None else p + s["b"].double()
    if s["groups"] > 1:
        score = (p if s["b"] is None and s["group_best"] == 2 else key).reshape(len(n), s["groups"], -1)
        score = score.sort(dim=2, descending=True).values[:, :, : s["group_best"]].sum(2)
        lose = score.argsort(dim=1, descending=True, stable=True)[:, s["top_groups"]:]
        out = key.reshape(len(n), s["groups"], -1)
        out[n[:, None], lose] = -torch.inf
        key = out.reshape(x.shape)
    ids = key.argsort(dim=1, descending=True, stable=True)[:, : s["top_k"]]
    chosen = p[n[:, None], ids]
    total = chosen.sum(1, keepdim=True) if s["renormalize"] else torch.ones_like(chosen[:, :1])
    w = s["scale"] * chosen / total
    out = {"ids": ids, "weights": w}
    if s["op"] == "route_train":
        # the Jacobian's product, written out: d w_j / d p_l = scale ([j = l] / total - p_j / total^2 if renormalised)
        dw = s["dw"][rows].double()
        dp = s["scale"] * dw / total
        if s["renormalize"]:
            dp = dp - (w * dw).sum(1, keepdim=True) / total
        dx = torch.zeros_like(x)
        if s["score"] == "softmax":
            dx -= p * (dp * chosen).sum(1, keepdim=True)
            dx[n[:, None], ids] += dp * chosen
        else:
            dx[n[:, None], ids] = dp * chosen * torch.sigmoid(-x[n[:, None], ids])
        out["dscores"] = dx
    return out


def _exact_logprobs(x, s, rows):
    n = torch.arange(x.shape[0], device=x.device)
    t = s["t"][rows].long()
    given = t >= 0
    t = torch.where(given, t, torch.zeros_like(t))
    lp = torch.log_softmax(x * s["scale"], 1)
    p = lp.exp()
    m = x.max(1).values
    lse = torch.logsumexp(x * s["scale"], 1)
    entropy = -torch.special.xlogy(p, p).sum(1)
    zero = torch.zeros_like(lse)
    out = {"lse": lse, "stats": torch.stack([m, (lse - m * s["scale"]).exp()], 1), "entropy": entropy,
           "logprob": torch.where(given, lp[n, t], zero)}
    xt = x[n, t][:, None]
    before = torch.arange(x.shape[1], device=x.device) < t[:, None]
    out["rank"] = torch.where(given, torch.where(before, x >= xt, x > xt).sum(1), -torch.ones_like(t))
    if s["top_k"]:
        ids = x.sort(dim=1, descending=True, stable=True).indices[:, : s["top_k"]]
        out["top_ids"], out["top_logprobs"] = ids, lp.gather(1, ids)
    if s["op"] == "logprobs_train":
        a = torch.where(given, s["dlp"][rows].double(), zero)
        dz = -p * a[:, None] - s["dh"][rows].double()[:, None] * (torch.special.xlogy(p, p) + p * entropy[:, None])
        dz[n, t] += a
        out["dlogits"] = dz * s["scale"]
    return out
