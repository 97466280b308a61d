"""Calls that move rows by index and the adjusting of logits, on the CPU: what they refuse before
anything is launched, their size queries, and the reference's gradients against differences."""
import numpy as np
import pytest

import moves_reference as ref
import sorting_lsd_radix_amd as rs

# never-dereferenced addresses: every case fails a host check first
A, B, C, D, E, F, G, H, I, J = (0x100000000 * i for i in range(1, 11))


def refused(status, call, *args, **kw):
    with pytest.raises(rs.RsError) as ei:
        call(*args, **kw)
    assert ei.value.status == status, (args, kw, ei.value)


BAD, SIZE, LAP, OFF, TEMP = (rs.RS_ERR_INVALID_VALUE, rs.RS_ERR_UNSUPPORTED_SIZE, rs.RS_ERR_OVERLAP,
                             rs.RS_ERR_MISALIGNED, rs.RS_ERR_TEMP_TOO_SMALL)

COMMON = [
    (dict(et=3), BAD), (dict(et=-1), BAD), (dict(k=0), BAD), (dict(k=65), SIZE), (dict(width=0), BAD),
    (dict(width=1 << 30), SIZE), (dict(rows=1 << 30), SIZE), (dict(room=1 << 30), SIZE),
    (dict(rows=1 << 25, k=32), SIZE), (dict(k=(1 << 32) + 8), SIZE), (dict(width=(1 << 32) + 64), SIZE),
    (dict(rows=1 << 24, width=1 << 20), SIZE), (dict(x=None), BAD), (dict(y=None), BAD), (dict(place=None), BAD),
    (dict(x=A + 1), OFF), (dict(et=0, x=A + 2, xs=64), OFF), (dict(y=B + 1), OFF), (dict(place=D + 2), OFF),
    (dict(weights=E + 1), OFF), (dict(xs=1 << 60), BAD),
]


def gather(et=2, x=A, xs=64, order=C, room=200, place=D, weights=E, rows=16, k=8, width=64, y=B, ys=64):
    rs.rs_gather_choices(et, x, xs, order, room, place, weights, rows, k, width, y, ys, stream=0)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(order=None), BAD), (dict(ys=63), BAD), (dict(order=C + 1), OFF),
    (dict(y=A + 64), LAP), (dict(y=C - 128), LAP), (dict(y=D + 16), LAP), (dict(y=E), LAP),
])
def test_gather_refusals(kw, status):
    refused(status, gather, **kw)


def gather_grad(et=2, y=B, ys=64, room=200, x=A, xs=64, place=D, weights=E, rows=16, k=8, width=64, dx=F, dxs=64,
                dw=G):
    rs.rs_gather_choices_grad(et, y, ys, room, x, xs, place, weights, rows, k, width, dx, dxs, dw, stream=0)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dx=None), BAD), (dict(dw=None), BAD), (dict(weights=None), BAD), (dict(dxs=63), BAD), (dict(dw=G + 2), OFF),
    (dict(dx=F + 1), OFF), (dict(dx=A), LAP), (dict(dx=B), LAP), (dict(dx=D), LAP), (dict(dw=E), LAP), (dict(dw=F), LAP),
])
def test_gather_grad_refusals(kw, status):
    refused(status, gather_grad, **kw)


def combine(et=2, y=B, ys=64, room=200, place=D, weights=E, rows=16, k=8, width=64, x=A, xs=64):
    rs.rs_combine_choices(et, y, ys, room, place, weights, rows, k, width, x, xs, stream=0)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(xs=63), BAD), (dict(x=B + 128), LAP), (dict(x=D), LAP), (dict(x=E), LAP),
])
def test_combine_refusals(kw, status):
    refused(status, combine, **kw)


def combine_grad(et=2, x=A, xs=64, y=B, ys=64, order=C, room=200, place=D, weights=E, rows=16, k=8, width=64, dy=F,
                 dys=64, dw=G):
    rs.rs_combine_choices_grad(et, x, xs, y, ys, order, room, place, weights, rows, k, width, dy, dys, dw, stream=0)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(order=None), BAD), (dict(weights=None), BAD), (dict(dy=None), BAD), (dict(dw=None), BAD), (dict(dys=63), BAD),
    (dict(order=C + 2), OFF), (dict(dw=G + 2), OFF), (dict(dy=A), LAP), (dict(dy=B), LAP), (dict(dy=C), LAP),
    (dict(dw=D), LAP), (dict(dw=E), LAP), (dict(dw=F + 8), LAP),
])
def test_combine_grad_refusals(kw, status):
    refused(status, combine_grad, **kw)


def embed(et=2, table=A, ts=64, ids=B, n=100, vocab=1000, width=64, scale=1.0, out=C, os=64):
    rs.rs_embed_tokens(et, table, ts, ids, n, vocab, width, scale, out, os, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(et=3), BAD), (dict(vocab=0), BAD), (dict(width=0), BAD), (dict(vocab=1 << 30), SIZE), (dict(n=1 << 30), SIZE),
    (dict(width=1 << 30), SIZE), (dict(vocab=(1 << 32) + 5), SIZE), (dict(vocab=1 << 29, width=1 << 12), SIZE),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(table=None), BAD), (dict(ids=None), BAD),
    (dict(out=None), BAD), (dict(os=63), BAD), (dict(ts=1 << 60), BAD), (dict(table=A + 1), OFF), (dict(ids=B + 2), OFF),
    (dict(out=C + 1), OFF), (dict(out=A + 64), LAP), (dict(out=B), LAP),
])
def test_embed_refusals(kw, status):
    refused(status, embed, **kw)


def test_embed_of_no_tokens_launches_nothing():
    embed(n=0, table=None, ids=None, out=None)


def embed_grad(et=2, dout=A, ds=64, ids=B, n=100, vocab=1000, width=64, scale=1.0, acc=0, tt=2, table=C, ts=64, temp=D,
               size=1 << 24):
    return rs.rs_embed_tokens_grad(et, dout, ds, ids, n, vocab, width, scale, acc, tt, table, ts, temp, size, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(et=3), BAD), (dict(tt=1), BAD), (dict(et=0, tt=2), BAD), (dict(vocab=0), BAD), (dict(width=0), BAD),
    (dict(vocab=1 << 30), SIZE), (dict(n=1 << 30), SIZE), (dict(width=1 << 30), SIZE), (dict(width=(1 << 32) + 5), SIZE),
    (dict(n=1 << 29, width=1 << 12), SIZE), (dict(scale=float("nan")), BAD), (dict(dout=None), BAD),
    (dict(ids=None), BAD), (dict(table=None), BAD), (dict(ts=63), BAD), (dict(dout=A + 1), OFF), (dict(ids=B + 2), OFF),
    (dict(table=C + 1), OFF), (dict(temp=D + 8), OFF), (dict(size=3), TEMP), (dict(table=A), LAP), (dict(table=B), LAP),
    (dict(table=D), LAP), (dict(temp=A), LAP), (dict(temp=B + 16), LAP),
])
def test_embed_grad_refusals(kw, status):
    refused(status, embed_grad, **kw)


def test_embed_grad_size_query():
    def query(n, vocab=131072, width=4096):
        return rs.rs_embed_tokens_grad(2, None, 0, None, n, vocab, width, 1.0, 0, 2, None, 0, None, 0)
    assert 0 < query(0) <= query(1) <= query(1000) <= query(1 << 20)
    assert query(1 << 20) < (1 << 20) * 4096 * 2   # less than the gradients themselves
    refused(SIZE, query, 1 << 30)


def adjust(et=2, logits=A, ls=1000, rows=8, vocab=1000, history=B, hs=100, hlen=100, lengths=C, prompts=C, rep=D, pres=D,
           freq=D, ids=E, istr=10, bias=F, bs=10, blen=10, mask=G, ms=32, ot=2, out=H, os=1000):
    rs.rs_adjust_logits(et, logits, ls, rows, vocab, history, hs, hlen, lengths, prompts, rep, pres, freq, ids, istr, bias,
                        bs, blen, mask, ms, ot, out, os, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(et=3), BAD), (dict(ot=1), BAD), (dict(et=0, ot=2), BAD), (dict(vocab=0), BAD), (dict(vocab=1 << 30), SIZE),
    (dict(rows=1 << 30), SIZE), (dict(hlen=1 << 30), SIZE), (dict(blen=1 << 30), SIZE), (dict(vocab=(1 << 32) + 9), SIZE),
    (dict(rows=1 << 29, vocab=1 << 12), SIZE),
    (dict(logits=None), BAD), (dict(out=None), BAD), (dict(history=None), BAD), (dict(ids=None), BAD),
    (dict(bias=None), BAD), (dict(ids=None, bias=None), BAD), (dict(os=999), BAD), (dict(ls=1 << 60), BAD),
    (dict(hs=1 << 61), BAD), (dict(ms=1 << 61), BAD), (dict(logits=A + 1), OFF), (dict(out=H + 1), OFF),
    (dict(history=B + 2), OFF), (dict(lengths=C + 2), OFF), (dict(prompts=C + 1), OFF), (dict(rep=D + 2), OFF),
    (dict(pres=D + 2), OFF), (dict(freq=D + 2), OFF), (dict(ids=E + 2), OFF), (dict(bias=F + 2), OFF),
    (dict(mask=G + 2), OFF), (dict(out=A + 2), LAP), (dict(out=A, os=1001), LAP), (dict(out=A, ot=0), LAP),
    (dict(out=B), LAP), (dict(out=C), LAP), (dict(out=D), LAP), (dict(out=E), LAP), (dict(out=F), LAP),
    (dict(out=G), LAP),
])
def test_adjust_refusals(kw, status):
    refused(status, adjust, **kw)


def test_adjust_of_no_rows_launches_nothing():
    adjust(rows=0, logits=None, out=None)


# --- the reference's gradients against differences -------------------------------------------------

def differences(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + h
        up = f()
        x[i] = old - h
        g[i] = (up - f()) / (2 * h)
        x[i] = old
    return g


def test_gradients_of_choices():
    rng = np.random.default_rng(1)
    order = np.array([3, -1, 0, 5, 2, -1, 1])
    place = np.array([[2, 6], [4, 0], [-1, 3]])
    x, w = rng.standard_normal((3, 4)), rng.standard_normal((3, 2))
    dy = rng.standard_normal((7, 4))

    def loss():
        return (ref.gather(x, order, 2, w)[0] * dy).sum()
    # every function here is linear in each argument: differences are exact but for rounding
    assert np.allclose(differences(loss, x), ref.combine(dy, place, w)[0], atol=1e-9)
    assert np.allclose(differences(loss, w), ref.dots(x, dy, place)[0], atol=1e-9)
    y, dout = rng.standard_normal((7, 4)), rng.standard_normal((3, 4))

    def loss():
        return (ref.combine(y, place, w)[0] * dout).sum()
    assert np.allclose(differences(loss, y), ref.gather(dout, order, 2, w)[0], atol=1e-9)
    assert np.allclose(differences(loss, w), ref.dots(dout, y, place)[0], atol=1e-9)


def test_gradient_of_embedding():
    rng = np.random.default_rng(2)
    ids = np.array([3, 0, 3, -1, 7, 3])
    table, dout = rng.standard_normal((5, 4)), rng.standard_normal((6, 4))

    def loss():
        return (ref.embed(table, ids, -1.5)[0] * dout).sum()
    assert np.allclose(differences(loss, table), ref.embed_grad(dout, ids, 5, -1.5)[0], atol=1e-9)


def test_mask_words():
    allowed = np.zeros((1, 40), bool)
    allowed[0, [0, 33]] = True
    words = ref.mask_words(allowed)
    assert words.shape == (1, 2) and words[0, 0] == 1 and words[0, 1] & 0xFF == 2


def test_wrappers_refuse_host_memory():
    torch = pytest.importorskip("torch")
    x, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    p, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for call in (lambda: rs.gather_choices(x, i, p), lambda: rs.gather_choices_grad(x, x, p, w),
                 lambda: rs.combine_choices(x, p), lambda: rs.combine_choices_grad(x, x, i, p, w),
                 lambda: rs.embed_tokens(x, i), lambda: rs.embed_tokens_grad(x, i, 9), lambda: rs.adjust_logits(x)):
        with pytest.raises(TypeError):
            call()
