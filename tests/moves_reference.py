"""The calls that move rows by index, and the adjusting of logits, from their definitions, in numpy
and 64 bits, with bounds on what 32-bit arithmetic may be off.  Shares no code with the library."""
import numpy as np

U = 2.0 ** -24                                        # half a step of f32, relative


def gather(x, order, k, w=None):
    """(y, bound): a product of two f32 numbers is rounded once."""
    y = np.zeros((len(order), x.shape[1]))
    bound = np.zeros_like(y)
    for i, c in enumerate(order):
        if 0 <= c < x.shape[0] * k:
            y[i] = x[c // k] * (1.0 if w is None else w.reshape(-1)[c])
            bound[i] = 0.0 if w is None else U * np.abs(y[i])
    return y, bound


def combine(y, place, w=None):
    """(out, bound): k products and k sums, each rounded relative to at most the sum of what is added up."""
    rows, k = place.shape
    out = np.zeros((rows, y.shape[1]))
    size = np.zeros_like(out)
    for t in range(rows):
        for j in range(k):
            p = place[t, j]
            if 0 <= p < y.shape[0]:
                part = y[p] * (1.0 if w is None else w[t, j])
                out[t] += part
                size[t] += np.abs(part)
    return out, 2 * k * U * size * (1 + 2.0 ** -10)


def dots(x, y, place):
    """(products of the rows of x with the rows of y at their choices, bound).  A wave or more shares a
    row of more than 32 vectors of at most 8 elements, whose lanes add width / 64 + 8 products each at
    most; 4 to 32 lanes share a shorter one, a vector each: 8 products.  The lanes and waves add up in at
    most 16 steps more."""
    rows, k = place.shape
    out = np.zeros((rows, k))
    size = np.zeros_like(out)
    for t in range(rows):
        for j in range(k):
            p = place[t, j]
            if 0 <= p < y.shape[0]:
                out[t, j] = np.sum(x[t] * y[p])
                size[t, j] = np.sum(np.abs(x[t] * y[p]))
    return out, (x.shape[1] / 64 + 40) * U * size


def embed(table, ids, scale):
    out = np.zeros((len(ids), table.shape[1]))
    real = (ids >= 0) & (ids < table.shape[0])
    out[real] = table[ids[real]] * scale
    return out, (0.0 if scale == 1 else U) * np.abs(out)


def embed_grad(dout, ids, vocab, scale, old=None):
    """(dtable, bound): n rows are n - 1 sums, whatever their order, then a product and a sum."""
    out = np.zeros((vocab, dout.shape[1]))
    size = np.zeros_like(out)
    count = np.zeros((vocab, 1))
    for i, v in enumerate(ids):
        if 0 <= v < vocab:
            out[v] += dout[i]
            size[v] += np.abs(dout[i])
            count[v] += 1
    out *= scale
    size *= abs(scale)
    if old is not None:
        out = out + old
        size = size + np.abs(old)
    return out, (count + 2) * U * size * (count > 0) * (1 + 2.0 ** -10)


def adjust(x, history=None, lengths=None, prompts=None, repetition=None, presence=None, frequency=None,
           bias_ids=None, bias=None, allowed=None):
    """(logits, bound): a division or product, frequency * count + presence and its subtraction, a
    sum, each rounded relative to at most the terms' sizes."""
    rows, vocab = x.shape
    out = x.copy()
    size = np.abs(x)
    with np.errstate(all="ignore"):
        for r in range(rows):
            if history is not None:
                n = history.shape[1]
                length = n if lengths is None else min(max(int(lengths[r]), 0), n)
                prompt = 0 if prompts is None else min(max(int(prompts[r]), 0), length)
                tokens = history[r, :length].astype(np.int64)
                inside = (tokens >= 0) & (tokens < vocab)
                late = tokens[prompt:][inside[prompt:]]
                count = np.bincount(late, minlength=vocab).astype(np.float64)
                seen = np.bincount(tokens[inside], minlength=vocab) > 0
                by = 1.0 if repetition is None else repetition[r]
                out[r, seen] = np.where(out[r, seen] > 0, out[r, seen] / by, out[r, seen] * by)
                size[r] = np.maximum(size[r], np.abs(out[r]))
                f = 0.0 if frequency is None else frequency[r]
                p = 0.0 if presence is None else presence[r]
                some = count > 0
                out[r, some] -= (f * count + p)[some]
                size[r, some] += (abs(f) * count + abs(p))[some]
            if bias_ids is not None:
                entries = {int(v): bias[r, i] for i, v in enumerate(bias_ids[r]) if 0 <= v < vocab}
                for v, b in entries.items():
                    out[r, v] += b
                    size[r, v] += abs(b)
        if allowed is not None:
            out[~allowed] = -np.inf
    return out, 5 * U * np.where(np.isfinite(size), size, 0.0)


def mask_words(allowed):
    """[rows, ceil(vocab / 32)] int32 words of [rows, vocab] truth values, the lowest bit first."""
    rows, vocab = allowed.shape
    words = (vocab + 31) // 32
    bits = np.zeros((rows, words * 32), bool)
    bits[:, :vocab] = allowed
    bits[:, vocab:] = np.random.default_rng(rows * vocab).random((rows, words * 32 - vocab)) < 0.5   # behind the row
    return np.packbits(bits, axis=1, bitorder="little").view("<i4").copy()
