"""The operators that move rows of a model's matrices by index, and what they feed, as cases that are
timed and checked: tokens brought into the order of their experts (``gather``, and ``gather_train`` with
its gradient) and back with their weights (``combine``, ``combine_train``), rows of an embedding table
(``embed``) and the table's gradient (``embed_grad``), and penalties, biases and masks on logits
(``adjust``).

``run`` computes a case in plain torch operations, or, where ``own`` is true, with this library's
calls; ``exact`` computes it again from the definitions in 64 bits.

Definitions.  order [room] holds a choice (an index into the flattened [rows, top_k]) or -1 at every
position of the experts' segments, place [rows, top_k] the position of a choice or -1.  Gathering:
y_i = w_c x_t for the choice c = order_i of row t = c div top_k, 0 where there is none.  Combining:
out_t = sum over j of w_tj y_(place_tj), without the choices that have no place.  Gradients of both for
rows and weights.  Embedding: out_i = scale * table[id_i], 0 for an id outside the table; the table's
gradient is scale times the sum of the gradients of the rows that took it.  Adjusting: a token of the
history has its logit l divided (l > 0) or multiplied by the row's repetition penalty; one that occurs
behind the prompt, c times, loses frequency * c + presence; then the row's bias of the token is added (the
last of several for one token), and a token whose mask bit is 0 gets -inf.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # the tokens of a small decode batch to their experts: latency, and the zeros of the padding
        _rows("gather", "gather_step", rows=32, top_k=8, experts=128, align=16, width=4096, dtype="bf16"),
        # a long prompt's tokens to their experts, segments padded to tiles of 128 rows, some padding tokens dropped
        _rows("gather", "gather_prompt", rows=16384, top_k=8, experts=256, align=128, width=4096,
              dtype="bf16", dropped=0.03),
        # a training step that weights the tokens before the experts, with both gradients; odd sizes, full precision
        _rows("gather_train", "gather_train_odd", rows=3001, top_k=5, experts=100, align=1, width=1001,
              dtype="f32", weighted=True, skew=0.7),
        # the experts' rows of a small decode batch summed by their weights
        _rows("combine", "combine_step", rows=32, top_k=8, experts=128, align=16, width=4096,
              dtype="bf16", weighted=True),
        # the same for a long prompt
        _rows("combine", "combine_prompt", rows=16384, top_k=8, experts=256, align=128, width=4096,
              dtype="bf16", weighted=True, dropped=0.03),
        # a training step's sum by weights, and the gradients of the experts' rows and of the weights
        _rows("combine_train", "combine_train", rows=8192, top_k=6, experts=64, align=64, width=2048,
              dtype="f16", weighted=True),
        # the embeddings of four sequences' next tokens, the smallest call
        _embed("embed", "embed_step", tokens=4, vocab=131072, width=4096, dtype="bf16"),
        # the embeddings of a batch of prompts, scaled by the root of their width, with padding tokens
        _embed("embed", "embed_prompt", tokens=32768, vocab=131072, width=5120, dtype="f16",
               scale=math.sqrt(5120), dropped=0.05),
        # a training step's gradient of a large table: most rows have no token, a few have a thousand
        _embed("embed_grad", "embed_grad_large", tokens=16384, vocab=131072, width=2048, dtype="bf16"),
        # the same with more tokens than rows, odd sizes and full precision
        _embed("embed_grad", "embed_grad_odd", tokens=50021, vocab=32003, width=1001, dtype="f32",
               scale=math.sqrt(1001), dropped=0.05),
        # sampling a small batch with every rule, an odd vocabulary in padded rows
        _adjust("adjust_step", rows=8, vocab=50021, dtype="f32", history=1000, biases=30, masked=0.9, pad=27),
        # a large decode batch with long histories
        _adjust("adjust_batch", rows=256, vocab=131072, dtype="bf16", history=8192, biases=300, masked=0.5),
    ]


def _rows(op, name, rows, top_k, experts, align, width, dtype, weighted=False, dropped=0.0, skew=0.0, pad=0):
    return {"name": name, "op": op, "rows": rows, "top_k": top_k, "experts": experts, "align": align,
            "width": width, "dtype": dtype, "weighted": weighted, "dropped": dropped, "skew": skew, "pad": pad}


def _embed(op, name, tokens, vocab, width, dtype, scale=1.0, dropped=0.0, skew=1.0, pad=0):
    return {"name": name, "op": op, "tokens": tokens, "vocab": vocab, "width": width, "dtype": dtype,
            "scale": scale, "dropped": dropped, "skew": skew, "pad": pad}


def _adjust(name, rows, vocab, dtype, history, penalties=True, biases=0, masked=0.0, pad=0, to="same"):
    return {"name": name, "op": "adjust", "rows": rows, "vocab": vocab, "dtype": dtype, "history": history,
            "penalties": penalties, "biases": biases, "masked": masked, "pad": pad, "to": to}


def draw(rng):
    def spread(lo, hi):   # uniform over the logarithm
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(["gather", "gather_train", "combine", "combine_train", "embed", "embed_grad", "adjust"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    size = _SIZES[dtype]
    pad = rng.choice([0, 0, 3, 8])
    if op == "adjust":
        vocab = spread(100, 262144)
        c = _adjust("", rows=spread(1, min(1024, 30000000 // vocab)), vocab=vocab, dtype=dtype,
                    history=spread(1, 20000), penalties=rng.random() < 0.8, biases=rng.choice([0, 0, 5, 300]),
                    masked=rng.choice([0.0, 0.5, 0.99]), pad=pad, to=rng.choice(["same", "f32"]))
    elif op.startswith("embed"):
        width = spread(16, 8192)
        # the table, and the rows taken of it, in bytes no more than the large listed ones
        vocab = spread(100, min(262144, 400000000 // (width * size)))
        c = _embed(op, "", tokens=spread(1, min(131072, 300000000 // (width * size))), vocab=vocab,
                   width=width, dtype=dtype, scale=rng.choice([1.0, math.sqrt(width)]),
                   dropped=rng.choice([0.0, 0.1]), skew=rng.choice([0.0, 0.7, 1.0, 1.3]), pad=pad)
    else:
        top_k = rng.choice([1, 2, 4, 5, 6, 8, 12])
        experts = spread(top_k, 512)
        align = rng.choice([1, 1, 8, 16, 64, 100, 128])
        width = spread(16, 8192)
        room = max(1, 250000000 // (width * size) - experts * (align - 1)) // top_k
        c = _rows(op, "", rows=spread(1, max(1, min(32768, room))), top_k=top_k, experts=experts,
                  align=align, width=width, dtype=dtype,
                  weighted=op.endswith("train") or rng.random() < 0.5,
                  dropped=rng.choice([0.0, 0.02, 0.3]), skew=rng.choice([0.0, 0.7, 1.3]), pad=pad)
    del c["name"]
    return c


def _room(case):
    return case["rows"] * case["top_k"] + case["experts"] * (case["align"] - 1)


def _law(g, n, skew):
    """n numbers' probabilities, by a power law (skew 0: even) in a random order, summed up."""
    law = torch.arange(1, n + 1, device="cuda", dtype=torch.float64) ** -skew
    law = law[torch.randperm(n, generator=g, device="cuda")]
    return torch.cumsum(law, 0) / law.sum()


def _take(g, law, shape):
    at = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
    return torch.searchsorted(law, at).clamp_(max=law.numel() - 1)


def _matrix(g, rows, cols, dtype, pad=0, spread=1.0):
    """A [rows, cols] view of rows that are cols + pad apart, as a fused projection leaves it."""
    out = torch.empty(rows, cols + pad, device="cuda", dtype=_DTYPES[dtype])
    step = max(1, (1 << 28) // (cols + pad))
    for r in range(0, rows, step):
        part = out[r:r + step]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * spread)
    return out[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "adjust":
        rows, vocab = case["rows"], case["vocab"]
        s["x"] = _matrix(g, rows, vocab, case["dtype"], case["pad"], 3.0)
        law = _law(g, vocab, 1.0)
        s["history"] = _take(g, law, (rows, case["history"])).to(torch.int32)
        s["lengths"] = torch.randint(0, case["history"] + 1, (rows,), generator=g, device="cuda").to(torch.int32)
        part = torch.rand(rows, generator=g, device="cuda")
        s["prompts"] = (s["lengths"] * part).to(torch.int32)
        s["repetition"] = 1 + torch.rand(rows, generator=g, device="cuda") * 0.5
        s["presence"] = torch.rand(rows, generator=g, device="cuda")
        s["frequency"] = torch.rand(rows, generator=g, device="cuda") * 0.3
        s["bias_ids"] = s["bias"] = s["mask"] = None
        if case["biases"]:
            ids = torch.randint(0, vocab, (rows, case["biases"]), generator=g, device="cuda")
            few = torch.rand(rows, case["biases"], generator=g, device="cuda") < 0.3
            s["bias_ids"] = ids.masked_fill_(few, -1).to(torch.int32)
            s["bias"] = torch.randn(rows, case["biases"], generator=g, device="cuda") * 5
        if case["masked"]:
            # 32 tokens to a word, lowest bit first; what a grammar allows
            words = (vocab + 31) // 32
            allowed = torch.rand(rows, words, 32, generator=g, device="cuda") >= case["masked"]
            bit = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
            word = (allowed * bit).sum(2)
            s["mask"] = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
    elif case["op"].startswith("embed"):
        n, vocab = case["tokens"], case["vocab"]
        ids = _take(g, _law(g, vocab, case["skew"]), (n,))
        gone = torch.rand(n, generator=g, device="cuda") < case["dropped"]
        s["ids"] = ids.masked_fill_(gone, -1).to(torch.int32)
        if case["op"] == "embed":
            s["table"] = _matrix(g, vocab, case["width"], case["dtype"], case["pad"], 0.02)
        else:
            s["dout"] = _matrix(g, n, case["width"], case["dtype"], case["pad"])
    else:
        rows, k, experts, align = case["rows"], case["top_k"], case["experts"], case["align"]
        ids = _take(g, _law(g, experts, case["skew"]), (rows, k))
        gone = torch.rand(rows, 1, generator=g, device="cuda") < case["dropped"]
        s["order"], s["place"] = _grouped(ids.masked_fill_(gone, -1).reshape(-1), experts, align, _room(case))
        s["place"] = s["place"].view(rows, k)
        w = torch.rand(rows, k, generator=g, device="cuda") + 0.01
        s["w"] = w / w.sum(1, keepdim=True) if case["weighted"] else None
        wide, dtype, pad = case["width"], case["dtype"], case["pad"]
        if case["op"].startswith("gather"):
            s["x"] = _matrix(g, rows, wide, dtype, pad)
        else:
            s["y"] = _matrix(g, _room(case), wide, dtype, pad)
        if case["op"] == "gather_train":
            s["dy"] = _matrix(g, _room(case), wide, dtype, pad)
        if case["op"] == "combine_train":
            s["dout"] = _matrix(g, rows, wide, dtype, pad)
    return s


def _grouped(flat, experts, align, room):
    """order and place of the choices: by expert, stably, segments padded to multiples of align."""
    n = flat.numel()
    key = torch.where(flat >= 0, flat, experts)
    ranked, by = torch.sort(key, stable=True)
    edge = torch.searchsorted(ranked, torch.arange(experts + 1, device="cuda"))
    ends = torch.cumsum((edge[1:] - edge[:-1] + align - 1) // align * align, 0)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    to = torch.where(ranked < experts, starts[ranked] + torch.arange(n, device="cuda") - edge[ranked], room)
    order = torch.full((room + 1,), -1, dtype=torch.int32, device="cuda")
    order[to] = by.to(torch.int32)
    place = torch.empty(n, dtype=torch.int32, device="cuda")
    place[by] = torch.where(to < room, to, -1).to(torch.int32)
    return order[:room].clone(), place


# --- plain forms ---------------------------------------------------------------------------------

def _plain_gather(x, s):
    """Rows of x, by their weights if there are any, in the order of the experts' segments."""
    c = s["order"].long()
    real = c >= 0
    c = c.clamp(min=0)
    y = x[c // s["top_k"]].float()
    if s["w"] is not None:
        y = y * s["w"].reshape(-1)[c][:, None]
    return torch.where(real[:, None], y, 0.0).to(x.dtype)


def _plain_combine(y, s):
    """The sum of each row's choices in y, by their weights if there are any."""
    out = None
    for j in range(s["top_k"]):
        p = s["place"][:, j].long()
        part = torch.where((p >= 0)[:, None], y[p.clamp(min=0)].float(), 0.0)
        if s["w"] is not None:
            part = part * s["w"][:, j:j + 1]
        out = part if out is None else out + part
    return out.to(y.dtype)


def _plain_dots(x, y, s):
    """The products of each row of x with the rows of y at its choices."""
    dots = []
    for j in range(s["top_k"]):
        p = s["place"][:, j].long()
        part = (x.float() * y[p.clamp(min=0)].float()).sum(1)
        dots.append(torch.where(p >= 0, part, 0.0))
    return torch.stack(dots, 1)


def _plain_embed(table, ids, scale):
    at = ids.long()
    real = (at >= 0) & (at < table.shape[0])
    out = table[torch.where(real, at, 0)].float() * scale
    return torch.where(real[:, None], out, 0.0).to(table.dtype)


def _plain_embed_grad(dout, ids, vocab, scale):
    at = ids.long()
    at = torch.where((at >= 0) & (at < vocab), at, vocab)
    total = torch.zeros(vocab + 1, dout.shape[1], device=dout.device)
    total.index_add_(0, at, dout.float())
    return (total[:vocab] * scale).to(dout.dtype)


def _plain_adjust(x, s):
    rows, vocab = x.shape
    l = x.float()
    if s["penalties"]:
        step = torch.arange(s["history"].shape[1], device=x.device)
        valid = step < s["lengths"][:, None]
        late = valid & (step >= s["prompts"][:, None])
        token = s["history"].long()
        seen = torch.zeros(rows, vocab, device=x.device).scatter_add_(1, token, valid.float())
        count = torch.zeros(rows, vocab, device=x.device).scatter_add_(1, token, late.float())
        by = s["repetition"][:, None]
        l = torch.where(seen > 0, torch.where(l > 0, l / by, l * by), l)
        l = l - torch.where(count > 0, s["frequency"][:, None] * count + s["presence"][:, None], 0.0)
    if s["bias_ids"] is not None:
        # the last entry of a token counts
        ids, n = s["bias_ids"].long(), s["bias_ids"].shape[1]
        entry = torch.where(ids >= 0, torch.arange(n, device=x.device), -1)
        last = torch.full((rows, vocab), -1, dtype=torch.int64, device=x.device)
        last.scatter_reduce_(1, ids.clamp(min=0), entry, "amax")
        l = l + torch.where(last >= 0, s["bias"].gather(1, last.clamp(min=0)), 0.0)
    if s["mask"] is not None:
        at = torch.arange(vocab, device=x.device)
        l = torch.where((s["mask"][:, at // 32] >> (at % 32)) & 1 == 1, l, float("-inf"))
    return l.to(x.dtype) if s["to"] == "same" else l


def run(state):
    s = state
    if s["op"] == "adjust":
        if not own:
            return _plain_adjust(s["x"], s)
        import sorting_lsd_radix_amd as rs
        how = {}
        if s["penalties"]:
            how = {"history": s["history"], "lengths": s["lengths"], "prompt_lengths": s["prompts"],
                   "repetition": s["repetition"], "presence": s["presence"], "frequency": s["frequency"]}
        return rs.adjust_logits(s["x"], bias_ids=s["bias_ids"], bias=s["bias"], mask=s["mask"],
                                dtype=None if s["to"] == "same" else torch.float32, **how)
    if s["op"] == "embed":
        if not own:
            return _plain_embed(s["table"], s["ids"], s["scale"])
        import sorting_lsd_radix_amd as rs
        return rs.embed_tokens(s["table"], s["ids"], scale=s["scale"])
    if s["op"] == "embed_grad":
        if not own:
            return _plain_embed_grad(s["dout"], s["ids"], s["vocab"], s["scale"])
        import sorting_lsd_radix_amd as rs
        return rs.embed_tokens_grad(s["dout"], s["ids"], s["vocab"], scale=s["scale"])
    if s["op"].startswith("gather"):
        if own:
            import sorting_lsd_radix_amd as rs
            out = {"y": rs.gather_choices(s["x"], s["order"], s["place"], weights=s["w"])}
            if s["op"] == "gather_train":
                out["dx"], out["dw"] = rs.gather_choices_grad(s["dy"], s["x"], s["place"], s["w"])
            return out
        out = {"y": _plain_gather(s["x"], s)}
        if s["op"] == "gather_train":
            out["dx"], out["dw"] = _plain_combine(s["dy"], s), _plain_dots(s["x"], s["dy"], s)
        return out
    if own:
        import sorting_lsd_radix_amd as rs
        out = {"out": rs.combine_choices(s["y"], s["place"], weights=s["w"])}
        if s["op"] == "combine_train":
            out["dy"], out["dw"] = rs.combine_choices_grad(s["dout"], s["y"], s["order"], s["place"], s["w"])
        return out
    out = {"out": _plain_combine(s["y"], s)}
    if s["op"] == "combine_train":
        out["dy"], out["dw"] = _plain_gather(s["dout"], s), _plain_dots(s["dout"], s["y"], s)
    return out


def _kinds(n, vocab, skew):
    """How many of `vocab` tokens n draws by the power law meet."""
    law = torch.arange(1, vocab + 1, dtype=torch.float64) ** -skew
    return float((1 - (1 - law / law.sum()) ** n).sum())


def work(case):
    if case["op"] == "adjust":
        v = case["rows"] * case["vocab"]
        size = _SIZES[case["dtype"]]
        b = v * (size + (size if case["to"] == "same" else 4))
        if case["penalties"]:
            b += case["rows"] * (4 * case["history"] // 2 + 20)   # histories are half full
        b += case["rows"] * (8 * case["biases"] + (case["vocab"] + 31) // 32 * 4 * (case["masked"] > 0))
        return {"bytes": b, "flops": 4 * v}
    size = _SIZES[case["dtype"]] * case["width"]
    if case["op"].startswith("embed"):
        n = case["tokens"]
        kept = int(n * (1 - case["dropped"]))
        if case["op"] == "embed":
            taken = _kinds(kept, case["vocab"], case["skew"])
            return {"bytes": int(size * (n + taken)) + 4 * n, "flops": n * case["width"]}
        return {"bytes": size * (kept + case["vocab"]) + 4 * n, "flops": kept * case["width"]}
    rows, n, room = case["rows"], case["rows"] * case["top_k"], _room(case)
    kept = int(n * (1 - case["dropped"]))
    weights = 4 * n if case["weighted"] else 0
    if case["op"].startswith("gather"):
        b, f = size * (rows + room) + 4 * room + weights, kept * case["width"]
        if case["op"] == "gather_train":   # reads the rows' gradients and the rows again, writes theirs and the weights'
            b += size * (kept + 2 * rows) + 12 * n
            f *= 5
    else:
        b, f = size * (kept + rows) + 4 * n + weights, 2 * kept * case["width"]
        if case["op"] == "combine_train":   # reads the gradient and the experts' rows again, writes the rows' gradients
            b += size * (rows + kept + room) + 4 * room + 12 * n
            f = 5 * kept * case["width"]
    return {"bytes": b, "flops": f}


# --- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adjust":
        return _exact_adjust(s)
    if case["op"] == "embed":
        out = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(s["ids"] >= 0)[:, 0]
        out[at] = s["table"].index_select(0, s["ids"][at].long()).double() * case["scale"]
        return out
    if case["op"] == "embed_grad":
        out = torch.zeros(case["vocab"], case["width"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(s["ids"] >= 0)[:, 0]
        out.index_put_((s["ids"][at].long(),), s["dout"][at].double(), accumulate=True)
        return out.mul_(case["scale"])
    rows, k, room, wide = case["rows"], case["top_k"], _room(case), case["width"]
    one = torch.ones(rows, k, dtype=torch.float64, device="cuda")
    w = one if s["w"] is None else s["w"].double()
    place = s["place"].long()
    out = {}
    if case["op"].startswith("gather"):
        x = s["x"].double()
        y = torch.zeros(room, wide, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(place[:, j] >= 0)[:, 0]
            y[place[t, j]] = x[t] * w[t, j, None]
        out["y"] = y
        if case["op"] == "gather_train":
            out["dx"], out["dw"] = _exact_back(x, s["dy"], s["order"].long(), w)
        return out
    out["out"], dots = _exact_back(s["dout"].double() if "dout" in s else None, s["y"], s["order"].long(), w)
    if case["op"] == "combine_train":
        dy = torch.zeros(room, wide, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(place[:, j] >= 0)[:, 0]
            dy[place[t, j]] = s["dout"][t].double() * w[t, j, None]
        out["dy"], out["dw"] = dy, dots
    return out


def _exact_back(x, y, order, w):
    """The rows of y summed by their weights, and their products with the rows of x, by position."""
    rows, k = w.shape
    at = torch.nonzero(order >= 0)[:, 0]
    out = torch.zeros(rows, y.shape[1], dtype=torch.float64, device="cuda")
    dots = torch.zeros(rows * k, dtype=torch.float64, device="cuda")
    step = max(1, 100_000_000 // y.shape[1])   # positions at a time
    for i in range(0, at.numel(), step):
        c = order[at[i:i + step]]
        part = y[at[i:i + step]].double()
        if x is not None:
            dots[c] = (x[c // k] * part).sum(1)
        out.index_put_((c // k,), part * w.reshape(-1)[c, None], accumulate=True)
    return out, dots.view(rows, k)


def _exact_adjust(s):
    x = s["x"]
    rows, vocab = x.shape
    out = x.double()
    for r in range(rows):
        l = out[r]
        if s["penalties"]:
            n, prompt = int(s["lengths"][r]), int(s["prompts"][r])
            seen = torch.unique(s["history"][r, :n].long())
            by = s["repetition"][r].double()
            l[seen] = torch.where(l[seen] > 0, l[seen] / by, l[seen] * by)
            late, count = torch.unique(s["history"][r, prompt:n].long(), return_counts=True)
            l[late] -= s["frequency"][r].double() * count + s["presence"][r].double()
        if s["bias_ids"] is not None:
            entries = dict(zip(s["bias_ids"][r].tolist(), s["bias"][r].tolist()))
            entries.pop(-1, None)
            if entries:
                at = torch.tensor(list(entries), device=x.device)
                l[at] += torch.tensor(list(entries.values()), dtype=torch.float64, device=x.device)
        if s["mask"] is not None:
            bits = s["mask"][r].view(torch.uint8)[:, None] >> torch.arange(8, dtype=torch.uint8, device=x.device) & 1
            l[bits.reshape(-1)[:vocab] == 0] = -torch.inf
    return out
