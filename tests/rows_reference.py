"""The calls on rows of scores from their definitions, in numpy and 64 bits, with bounds on what
32-bit arithmetic may be off.  Shares no code with the library."""
import numpy as np

U = 2.0 ** -24                                        # half a step of f32, relative
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SMALLEST = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def row_order(x):
    """Indices of each row in its order: larger first, equal ones by index, NaN last."""
    x = np.where(x == 0, 0.0, x)
    key = np.where(np.isnan(x), -np.inf, x)
    last = np.isnan(x)
    out = np.empty(x.shape, np.int64)
    for r in range(x.shape[0]):
        out[r] = np.lexsort((np.arange(x.shape[1]), -key[r], last[r]))
    return out


# --- routing --------------------------------------------------------------------------------------

def probabilities(x, score):
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        m = x.max(1, keepdims=True)                   # NaN if the row has one
        e = np.exp(x - m)
        p = e / e.sum(1, keepdims=True)
        p[np.all(x == -np.inf, axis=1)] = 0.0
        return p


def route(x, k, bias=None, score="softmax", groups=1, top_groups=1, group_best=1,
          renormalize=True, scale=1.0):
    """(ids, weights, p) of f64 scores."""
    rows, experts = x.shape
    p = probabilities(x, score)
    masked = ~(x > -np.inf)
    with np.errstate(all="ignore"):
        s = x if bias is None else np.where(masked, -np.inf, p + bias.astype(np.float64))
    s = np.where(s > -np.inf, s, -np.inf)             # NaN is masked
    size = experts // groups
    ids = np.empty((rows, k), np.int64)
    for r in range(rows):
        by = p[r] if bias is None and group_best == 2 else s[r]
        by = np.where((s[r] > -np.inf) & (by > -np.inf), by, -np.inf)
        scores = []
        for g in range(groups):
            best = sorted((v for v in by[g * size:(g + 1) * size] if v > -np.inf), reverse=True)
            scores.append(sum(best[:group_best]) if best else -np.inf)
        kept = sorted(range(groups), key=lambda g: (-scores[g], g))[:top_groups]
        can = [e for e in range(experts) if e // size in kept]
        ids[r] = sorted(can, key=lambda e: (-s[r, e], e))[:k]
    chosen = np.take_along_axis(p, ids, 1)
    with np.errstate(all="ignore"):
        w = scale * chosen
        if renormalize:
            total = chosen.sum(1, keepdims=True)
            w = np.where(total == 0, 0.0, w / total)
    return ids, w, p


def route_grad(x, ids, dw, score="softmax", renormalize=True, scale=1.0):
    """dscores in f64 and a bound on what f32 arithmetic may be off."""
    p = probabilities(x, score)
    rows, k = ids.shape
    n = np.arange(rows)[:, None]
    chosen = p[n, ids]
    total = chosen.sum(1, keepdims=True)
    w = scale * (chosen / np.where(total == 0, 1.0, total) if renormalize else chosen)
    d = (dw * w).sum(1, keepdims=True)
    part = w * (dw - d / scale if renormalize else dw)
    # f32: every operation is off by U relative.  D sums k products of inputs that are off by U
    # themselves: at most (k + 2) U sum |dw w|.  The term is then a difference, a division and two
    # products (5 more), and 1 - p is 1 / (1 + exp x): 4 U, and exp's argument is exact.
    spread = np.abs(dw * w).sum(1, keepdims=True) / (scale if renormalize else 1.0)
    off = U * (k + 12) * np.abs(w) * (np.abs(dw) + (spread if renormalize else 0.0))
    dx = np.zeros_like(x)
    bound = np.zeros_like(x)
    if score == "sigmoid":
        q = 1.0 / (1.0 + np.exp(np.where(np.isnan(x), 0, x)))[n, ids]
        np.add.at(dx, (n, ids), part * q)
        # 1 - p below f32's smallest normal number is a multiple of 2^-149, off by half of that
        np.add.at(bound, (n, ids), off * q + 2.0 ** -149 * np.abs(part))
    else:
        if not renormalize:
            # p: x - m is rounded once (|x - m| U in the exponent), exp 2 U, the sum of the row
            # at most (experts / 64 + 8) U and its terms' own errors, one division
            far = np.where(p > 0, np.abs(x - x.max(1, keepdims=True)), 0.0)
            far = far + (p * far).sum(1, keepdims=True)
            dx -= p * d
            bound += p * (np.abs(d) * U * (far + x.shape[1] / 64 + 20) +
                          U * (k + 2) * np.abs(dw * w).sum(1, keepdims=True))
        np.add.at(dx, (n, ids), part)
        np.add.at(bound, (n, ids), off)
    return dx, bound


# --- grouping -------------------------------------------------------------------------------------

def group(ids, experts, align):
    """order, place, starts, counts; ids as unsigned numbers."""
    ids = ids.reshape(-1).astype(np.uint32)
    n = ids.size
    order = np.full(n + experts * (align - 1), -1, np.int64)
    place = np.full(n, -1, np.int64)
    counts = np.bincount(ids[ids < experts], minlength=experts)
    starts = np.concatenate([[0], np.cumsum((counts + align - 1) // align * align)])
    by = np.argsort(ids, kind="stable")
    by = by[ids[by] < experts]
    rank = np.arange(by.size) - (np.cumsum(counts) - counts)[ids[by]]
    place[by] = starts[ids[by]] + rank
    order[place[by]] = by
    return order, place, starts, counts


# --- log probabilities -----------------------------------------------------------------------------

def logprobs(x, targets, k, scale):
    """Everything token_logprobs gives, of f64 logits, and bounds on what f32 may be off."""
    rows, vocab = x.shape
    with np.errstate(all="ignore"):
        nan = np.isnan(x).any(1) | (x == np.inf).any(1)
        m = np.where(np.isnan(x), -np.inf, x).max(1)
        empty = np.all(x == -np.inf, axis=1)
        c = float(scale)
        d = (x - np.where(m == -np.inf, 0, m)[:, None]) * c
        e = np.exp(d)
        s = e.sum(1)
        t = np.where(e > 0, e * d, 0.0).sum(1)
        ln_s = np.where(empty, 0.0, np.log(s))
        lse = np.where(empty, -np.inf, m * c + ln_s)
        entropy = np.where(empty, 0.0, ln_s - t / s)
        s = np.where(nan, np.nan, s)
        lse = np.where(nan, np.nan, lse)
        entropy = np.where(nan, np.nan, entropy)
        ln_p = np.where(empty[:, None], -np.inf, d - np.log(s)[:, None])
    out = {"stats": np.stack([m, s], 1), "lse": lse, "entropy": entropy}
    order = row_order(x)
    if targets is not None:
        given = targets < vocab
        at = np.where(given, targets, 0)
        n = np.arange(rows)
        out["logprob"] = np.where(given, ln_p[n, at], 0.0)
        rank = np.empty((rows, vocab), np.int64)
        np.put_along_axis(rank, order, np.arange(vocab)[None].repeat(rows, 0), 1)
        out["rank"] = np.where(given & ~np.isnan(x[n, at]), rank[n, at], -1)
    if k:
        out["top_ids"] = order[:, :k]
        out["top_logprobs"] = np.take_along_axis(ln_p, out["top_ids"], 1)
    # Bounds.  d in powers of two comes from x - r (1), times a = scale * log2 e (1, and 2 in a):
    # 4 U |d| in the exponent, ln2 of that relative in e, and 2 for exp2.  Against a thread's
    # reference |d| is at most |x - m| in those units and 16 + 16 more, weighted by e: W is the mean
    # of |x - m|.  A thread adds vocab / 256 / parts terms (at most vocab / 256 + 8), then 30 joins of 3.
    w = np.where(np.isfinite(entropy), np.abs(t) / np.where(s > 0, s, 1), 0) / np.log(2)
    es = U * (vocab / 256 + 8 + 100 + 3 * (w + 34))
    far = np.where(np.isfinite(ln_p), np.abs(ln_p), 0.0)
    off = {"stats": np.stack([0 * es, es * np.where(np.isfinite(s), s, 0)], 1),
           "lse": es + 4 * U * (np.abs(np.where(np.isfinite(m), m, 0)) * c + np.abs(ln_s)),
           "entropy": es * (2 + 2 * w) + 8 * U * (np.abs(ln_s) + w)}
    if targets is not None:
        out_far = np.where(targets < vocab, far[np.arange(rows), np.where(targets < vocab, targets, 0)], 0)
        off["logprob"] = es + 4 * U * (out_far + 2 * np.abs(ln_s))
    if k:
        off["top_logprobs"] = es[:, None] + 4 * U * (np.take_along_axis(far, out["top_ids"], 1) +
                                                     2 * np.abs(ln_s)[:, None])
    return out, off


def logprobs_grad(x, targets, scale, g=None, h=None, q=None):
    """dlogits in f64 and a bound on what f32 may be off (the stats are the library's own, f32)."""
    rows, vocab = x.shape
    c = float(scale)
    out, off = logprobs(x, targets, 0, scale)
    empty = np.all(x == -np.inf, axis=1)
    zero = np.zeros(rows)
    given = targets < vocab if targets is not None else np.zeros(rows, bool)
    g = zero if g is None else np.where(given, g, 0.0)
    h = zero if h is None else h
    q = zero if q is None else q
    m, s = out["stats"].T
    with np.errstate(all="ignore"):
        d = (x - np.where(empty, 0, m)[:, None]) * c
        p = np.where(empty[:, None], 0.0, np.exp(d) / np.where(empty, 1, s)[:, None])
        ln_p = d - np.log(np.where(empty, 1, s))[:, None]
        plnp = np.where(p > 0, p * (ln_p + out["entropy"][:, None]), 0.0)
        dx = c * ((q - g)[:, None] * p - h[:, None] * plnp)
        far = np.where(p > 0, np.abs(d), 0.0)
        ln_s = np.abs(np.log(np.where(empty, 1, s)))
        # e: 4 U |d| / ln2 * ln2 in the exponent and 2 for exp2; the coefficients 12 operations on
        # terms q, g, h H, h ln s, h d; s and H are off by their own bounds.  The chip's exp2 gives 0
        # below f32's smallest normal number, 2^-126: e is off by up to that beside its relative error
        size = (np.abs(q) + np.abs(g))[:, None] + np.abs(h)[:, None] * (out["entropy"][:, None] + ln_s[:, None] + far)
        bound = c * p * (size * (U * (4 * far + 24) + (off["stats"][:, 1] / np.where(s > 0, s, 1))[:, None]) +
                         np.abs(h)[:, None] * off["entropy"][:, None]) + \
            c * size * 2.0 ** -126 / np.where(s > 0, s, 1)[:, None]
    n = np.arange(rows)[given & ~empty]
    dx[n, targets[n] if targets is not None else 0] += c * g[n]
    if targets is not None:
        bound[n, targets[n]] += 4 * U * c * np.abs(g[n])
    return dx, bound
