"""Refusals of the losses on packed logits on the host (no GPU needed)."""
import ctypes

import pytest
import torch

import bit_quantized_lora_quant_amd as q

P = ctypes.c_void_p
FAKE = 0x100000
BIG = 1 << 40


def _z(rows=8, vocab=100, ld=None, dtype=1, data=FAKE, labels=FAKE, reserved=0):
    return q.LogitsDescriptor(data, dtype, reserved, rows, vocab, vocab if ld is None else ld,
                              labels)


def _ptr(v):
    return P(v) if v else None


def _score(z, logp=FAKE, stats=FAKE, ws=FAKE, ws_bytes=BIG):
    return q.lib().qlora_token_logprobs(ctypes.byref(z), _ptr(logp), _ptr(stats), _ptr(ws),
                                        ws_bytes, None)


def _back(z, stats=FAKE, w=FAKE, g=None, dz=2 * FAKE, ldd=None):
    return q.lib().qlora_token_logprobs_bwd(ctypes.byref(z), _ptr(stats), _ptr(w), _ptr(g),
                                            _ptr(dz), z.vocab if ldd is None else ldd, None)


def _pref(z, pairs=2, cu=FAKE, beta=0.1, smooth=0.0, kind=0, mean=0, loss=FAKE, dz=None, ldd=0,
          ws_bytes=BIG, ref=FAKE, h=True):
    p = q.PreferenceParams(beta, smooth, kind, mean)
    return q.lib().qlora_preference_loss(ctypes.byref(z), pairs, _ptr(cu), _ptr(ref),
                                         ctypes.byref(p) if h else None, _ptr(loss), None, None,
                                         None, None, None, _ptr(dz), ldd, P(FAKE), ws_bytes, None)


def _pol(z, n=2, cu=FAKE, adv=FAKE, old=None, ref=None, lo=0.2, hi=0.2, kl=0.0, red=0, tok=0,
         out=FAKE, ws_bytes=BIG):
    p = q.PolicyParams(lo, hi, kl, red, tok)
    return q.lib().qlora_policy_loss(ctypes.byref(z), n, _ptr(cu), _ptr(adv), _ptr(old), _ptr(ref),
                                     ctypes.byref(p), _ptr(out), None, None, None, None, 0,
                                     P(FAKE), ws_bytes, None)


@pytest.mark.parametrize("z,want", [
    (_z(rows=-1), "INVALID_ARG"), (_z(vocab=0), "INVALID_ARG"), (_z(ld=99), "INVALID_ARG"),
    (_z(dtype=2), "INVALID_ARG"), (_z(reserved=1), "INVALID_ARG"), (_z(data=0), "INVALID_ARG"),
    (_z(data=FAKE + 1), "INVALID_ARG"), (_z(data=FAKE + 2, dtype=0), "INVALID_ARG"),
    (_z(labels=0), "INVALID_ARG"), (_z(labels=FAKE + 4), "INVALID_ARG"),
    (_z(rows=1 << 24), "UNSUPPORTED"), (_z(vocab=1 << 30), "UNSUPPORTED"),
    (_z(ld=1 << 30), "UNSUPPORTED")])
def test_bad_logits(z, want):
    want = getattr(q, "QLORA_ERR_" + want)
    assert _score(z) == want and _back(z) == want and _pref(z) == want and _pol(z) == want
    if z.data and z.data % 4 == 0 and z.labels and z.labels % 8 == 0:
        assert q.lib().qlora_loss_workspace_bytes(ctypes.byref(z), 2) == 0


def test_token_logprobs_refusals():
    bad = q.QLORA_ERR_INVALID_ARG
    assert _score(_z(), logp=None) == bad and _score(_z(), stats=FAKE + 2) == bad
    assert _score(_z(), ws=None) == q.QLORA_ERR_WORKSPACE
    assert _score(_z(), ws_bytes=0) == q.QLORA_ERR_WORKSPACE
    assert _score(_z(rows=0, data=0, labels=0), logp=None) == q.QLORA_OK
    for kw in (dict(stats=None), dict(w=None), dict(dz=None), dict(ldd=99), dict(w=FAKE + 2),
               dict(dz=FAKE + 1), dict(g=FAKE + 2)):
        assert _back(_z(), **kw) == bad, kw
    assert _back(_z(ld=128), dz=FAKE, ldd=100) == bad       # in place needs the same stride
    assert _back(_z(rows=0, data=0, labels=0), dz=None, stats=None, w=None) == q.QLORA_OK


def test_preference_refusals():
    bad = q.QLORA_ERR_INVALID_ARG
    nan, inf = float("nan"), float("inf")
    for kw in (dict(pairs=0), dict(pairs=-1), dict(cu=None), dict(h=False), dict(loss=None),
               dict(beta=0.0), dict(beta=-1.0), dict(beta=nan), dict(beta=inf), dict(smooth=-0.1),
               dict(smooth=0.6), dict(smooth=nan), dict(kind=3), dict(kind=-1),
               dict(kind=1, smooth=0.1), dict(mean=2), dict(dz=FAKE, ldd=99), dict(ref=FAKE + 1)):
        assert _pref(_z(), **kw) == bad, kw
    for pairs in (1 << 21, 1 << 23):
        assert _pref(_z(), pairs=pairs) == q.QLORA_ERR_UNSUPPORTED
    z = _z()
    need = q.lib().qlora_loss_workspace_bytes(ctypes.byref(z), 4)
    assert need > 0 and _pref(z, ws_bytes=need - 1) == q.QLORA_ERR_WORKSPACE


def test_policy_refusals():
    bad = q.QLORA_ERR_INVALID_ARG
    nan, inf = float("nan"), float("inf")
    for kw in (dict(n=0), dict(cu=None), dict(adv=None), dict(out=None), dict(lo=-0.1),
               dict(lo=1.5), dict(hi=-0.1), dict(hi=inf), dict(kl=-1.0, ref=FAKE),
               dict(kl=nan, ref=FAKE), dict(kl=0.1), dict(red=2), dict(tok=2), dict(old=FAKE + 2)):
        assert _pol(_z(), **kw) == bad, kw
    for n in (1 << 22, 1 << 24):
        assert _pol(_z(), n=n) == q.QLORA_ERR_UNSUPPORTED
    z = _z()
    need = q.lib().qlora_loss_workspace_bytes(ctypes.byref(z), 2)
    assert _pol(z, ws_bytes=need - 1) == q.QLORA_ERR_WORKSPACE


def _raises(fn, *args, **kw):
    with pytest.raises(q.QloraError) as e:
        fn(*args, **kw)
    assert e.value.status == q.QLORA_ERR_INVALID_ARG


def test_binding_refusals():
    z, y = torch.zeros(4, 50), torch.zeros(4, dtype=torch.int64)
    cu = torch.tensor([0, 2, 4], dtype=torch.int32)
    _raises(q.qlora_token_logprobs, z, y)                           # on the host
    _raises(q.qlora_preference_loss, z, y, cu)
    _raises(q.qlora_policy_loss, z, y, cu, torch.zeros(2))
    _raises(q.qlora_token_logprobs, z.half(), y)
    _raises(q.qlora_token_logprobs, z.t(), torch.zeros(50, dtype=torch.int64))
    _raises(q.qlora_token_logprobs, z, y.int())
    _raises(q.qlora_token_logprobs, z, y[:3])
    _raises(q.qlora_token_logprobs, z, y, logp=torch.zeros(3))
    _raises(q.qlora_token_logprobs_bwd, z, y, torch.zeros(4, 2), torch.zeros(3))
    _raises(q.qlora_token_logprobs_bwd, z, y, torch.zeros(4, 1), torch.zeros(4))
    _raises(q.qlora_token_logprobs_bwd, z, y, torch.zeros(4, 2), torch.zeros(4),
            dlogits=torch.zeros(4, 49))
    _raises(q.qlora_preference_loss, z, y, cu.long())
    _raises(q.qlora_preference_loss, z, y, cu[:2])                  # one sequence is no pair
    _raises(q.qlora_preference_loss, z, y, cu, torch.zeros(3))
    _raises(q.qlora_preference_loss, z, y, cu, loss_type="other")
    _raises(q.qlora_policy_loss, z, y, cu, torch.zeros(4))          # per token only when asked
    _raises(q.qlora_policy_loss, z, y, cu, torch.zeros(2), token_advantages=True)
    _raises(q.qlora_policy_loss, z, y, cu, torch.zeros(2), reduction="mean")


def test_rows_and_sequences_share_a_grid():
    z = _z(rows=(1 << 24) - 2)
    want = q.QLORA_ERR_UNSUPPORTED
    assert _pref(z, pairs=1) == want and _pol(z, n=2) == want
    assert q.lib().qlora_loss_workspace_bytes(ctypes.byref(z), 2) == 0
    assert q.lib().qlora_loss_workspace_bytes(ctypes.byref(z), 1) > 0
