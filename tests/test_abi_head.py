"""Refusals of the language-model head on the host (no GPU needed)."""
import ctypes

import pytest
import torch

import bit_quantized_lora_quant_amd as q

P = ctypes.c_void_p
FAKE = 0x100000
BIG = 1 << 50


def _h(rows=8, dim=128, vocab=100, ldh=None, ldw=None, hidden=FAKE, weight=FAKE, labels=FAKE):
    return q.HeadDescriptor(hidden, rows, dim, dim if ldh is None else ldh, weight, vocab,
                            dim if ldw is None else ldw, labels)


def _ptr(v):
    return P(v) if v else None


def _score(h, logp=FAKE, stats=FAKE, ws=FAKE, ws_bytes=BIG):
    return q.lib().qlora_head_logprobs(ctypes.byref(h), _ptr(logp), _ptr(stats), _ptr(ws),
                                       ws_bytes, None)


def _back(h, stats=FAKE, w=FAKE, g=None, dh=FAKE, ldd=None, dw=None, ldo=None, ws=FAKE,
          ws_bytes=BIG):
    return q.lib().qlora_head_logprobs_bwd(
        ctypes.byref(h), _ptr(stats), _ptr(w), _ptr(g), _ptr(dh), h.dim if ldd is None else ldd,
        _ptr(dw), h.dim if ldo is None else ldo, _ptr(ws), ws_bytes, None)


def _ce(h, red=0, loss=FAKE, logp=FAKE, dh=None, ldd=None, dw=None, ldo=None, ws=FAKE,
        ws_bytes=BIG):
    return q.lib().qlora_head_cross_entropy(
        ctypes.byref(h), red, _ptr(loss), _ptr(logp), _ptr(dh), h.dim if ldd is None else ldd,
        _ptr(dw), h.dim if ldo is None else ldo, _ptr(ws), ws_bytes, None)


def _bytes(h, grads=0):
    return q.lib().qlora_head_workspace_bytes(ctypes.byref(h), grads)


@pytest.mark.parametrize("h,want", [
    (_h(rows=-1), "INVALID_ARG"), (_h(dim=0), "INVALID_ARG"), (_h(vocab=0), "INVALID_ARG"),
    (_h(ldh=127), "INVALID_ARG"), (_h(ldw=120), "INVALID_ARG"), (_h(hidden=0), "INVALID_ARG"),
    (_h(hidden=FAKE + 8), "INVALID_ARG"), (_h(weight=0), "INVALID_ARG"),
    (_h(weight=FAKE + 2), "INVALID_ARG"), (_h(labels=0), "INVALID_ARG"),
    (_h(labels=FAKE + 4), "INVALID_ARG"), (_h(dim=96, ldh=128, ldw=128), "UNSUPPORTED"),
    (_h(dim=1 << 17), "UNSUPPORTED"), (_h(ldh=132), "UNSUPPORTED"), (_h(ldw=129), "UNSUPPORTED"),
    (_h(ldh=1 << 22), "UNSUPPORTED"), (_h(ldw=1 << 22), "UNSUPPORTED"),
    (_h(rows=1 << 24), "UNSUPPORTED"), (_h(vocab=(1 << 22) + 1), "UNSUPPORTED")])
def test_bad_heads(h, want):
    code = getattr(q, "QLORA_ERR_" + want)
    assert _score(h) == code and _back(h) == code and _ce(h) == code
    if want == "UNSUPPORTED":
        assert all(_bytes(h, g) == 0 for g in range(4))


def test_refusals():
    bad, h = q.QLORA_ERR_INVALID_ARG, _h()
    assert _score(h, logp=None) == bad and _score(h, stats=FAKE + 2) == bad
    for kw in (dict(stats=None), dict(w=None), dict(g=FAKE + 1), dict(dh=None),
               dict(dh=FAKE + 8), dict(ldd=127), dict(ldd=132), dict(ldd=1 << 22),
               dict(dw=FAKE + 2), dict(dw=FAKE, ldo=64)):
        assert _back(h, **kw) == bad, kw
    for kw in (dict(red=2), dict(red=-1), dict(loss=None), dict(loss=FAKE + 2),
               dict(logp=FAKE + 1), dict(dh=FAKE + 4), dict(dh=FAKE, ldd=129),
               dict(dw=FAKE, ldo=1 << 22)):
        assert _ce(h, **kw) == bad, kw
    # in place needs the same stride
    assert _back(_h(ldh=136), dh=FAKE, ldd=128) == bad
    assert _ce(_h(ldh=136), dh=FAKE, ldd=144) == bad
    none = _h(rows=0, hidden=0, labels=0)
    assert _score(none, logp=None, ws=None) == q.QLORA_OK
    assert _back(none, stats=None, w=None, dh=None, ws=None) == q.QLORA_OK


def test_workspaces():
    h = _h(rows=700, dim=256, vocab=5000)
    sizes = [_bytes(h, g) for g in range(4)]
    assert 0 < sizes[0] < sizes[1] <= sizes[3] and sizes[2] <= sizes[3]
    assert _bytes(h, 4) == 0 and _bytes(h, -1) == 0
    short = q.QLORA_ERR_WORKSPACE
    assert _score(h, ws=None) == short and _score(h, ws_bytes=sizes[0] - 1) == short
    assert _score(h, ws=FAKE + 64) == short
    assert _back(h, ws_bytes=sizes[1] - 1) == short
    assert _back(h, dw=FAKE, ws_bytes=sizes[3] - 1) == short
    assert _ce(h, ws_bytes=sizes[0] - 1) == short
    assert _ce(h, dh=FAKE, ws_bytes=sizes[1] - 1) == short
    # what a call keeps does not grow with its rows: hidden, and a panel of 2^29
    many, few = _bytes(_h(rows=1 << 17, dim=4096, vocab=128256), 1), \
        _bytes(_h(rows=4096, dim=4096, vocab=128256), 1)
    assert many - few < (1 << 17) * (4096 * 2 + 100) and few < 3 << 29


def _raises(fn, *args, **kw):
    with pytest.raises(q.QloraError) as e:
        fn(*args, **kw)
    assert e.value.status == q.QLORA_ERR_INVALID_ARG


def test_binding_refusals():
    bf = torch.bfloat16
    h, W, y = torch.zeros((4, 64), dtype=bf), torch.zeros((50, 64), dtype=bf), \
        torch.zeros(4, dtype=torch.int64)
    for f in (q.qlora_head_logprobs, q.qlora_head_cross_entropy):
        _raises(f, h, W, y)                                     # on the host
        _raises(f, h.float(), W, y)
        _raises(f, h, W.float(), y)
        _raises(f, h, W[:, :32], y)
        _raises(f, torch.zeros((64, 4), dtype=bf).t(), W, y)
        _raises(f, h, torch.zeros((64, 50), dtype=bf).t(), y)
        _raises(f, h[0], W, y[:1])
        _raises(f, h, W, y.int())
        _raises(f, h, W, y[:3])
    _raises(q.qlora_head_logprobs, h, W, y, logp=torch.zeros(3))
    _raises(q.qlora_head_logprobs, h, W, y, stats=torch.zeros(4))
    _raises(q.qlora_head_cross_entropy, h, W, y, "none")
    _raises(q.qlora_head_cross_entropy, h, W, y, dhidden=torch.zeros((4, 64)))
    _raises(q.qlora_head_cross_entropy, h, W, y, dweight=torch.zeros((4, 64), dtype=bf))
    s, w = torch.zeros((4, 2)), torch.zeros(4)
    _raises(q.qlora_head_logprobs_bwd, h, W, y, s, w)
    _raises(q.qlora_head_logprobs_bwd, h, W, y, s[:3], w)
    _raises(q.qlora_head_logprobs_bwd, h, W, y, s, w.double())
    _raises(q.qlora_head_logprobs_bwd, h, W, y, s, w, grad_scale=w)
