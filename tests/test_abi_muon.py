"""Refusals of the orthogonalised update on the host (no GPU needed)."""
import ctypes

import pytest
import torch

import bit_quantized_lora_quant_amd as q

P = ctypes.c_void_p
FAKE = 0x100000
BIG = 1 << 50
NAN, INF = float("nan"), float("inf")


def _ns(a=3.4, b=-4.7, c=2.0, eps=1e-7, steps=5, reserved=0):
    return q.NewtonSchulz(a, b, c, eps, steps, reserved)


def _ortho(rows=8, cols=100, ldi=None, ldo=None, x=FAKE, out=2 * FAKE, dtype=0, reserved=0,
           count=1, ns=None, ws=FAKE, ws_bytes=BIG):
    m = (q.OrthoMatrix * 1)(q.OrthoMatrix(x, out, rows, cols, cols if ldi is None else ldi,
                                          cols if ldo is None else ldo, dtype, reserved))
    n = _ns() if ns is None else ns
    return q.lib().qlora_orthogonalize(ctypes.byref(n), m, count, P(ws) if ws else None, ws_bytes,
                                       None)


def _step(rows=8, cols=100, p=FAKE, g=FAKE, m=FAKE, pb=FAKE, ldp=None, ldg=None, ldm=None,
          ldb=None, dtype=0, reserved=0, count=1, lr=0.1, mu=0.9, wd=0.0, ns=None, nesterov=1,
          adjust=1, ws=FAKE, ws_bytes=BIG):
    ld = lambda v: cols if v is None else v  # noqa: E731
    t = (q.MuonTensor * 1)(q.MuonTensor(p, g, m, pb, rows, cols, ld(ldp), ld(ldg), ld(ldm), ld(ldb),
                                        dtype, reserved))
    h = q.MuonHparams(lr, mu, wd, _ns() if ns is None else ns, nesterov, adjust)
    return q.lib().qlora_muon_step(ctypes.byref(h), t, count, P(ws) if ws else None, ws_bytes, None)


def _bytes(*shapes):
    return q.qlora_muon_workspace_bytes(shapes)


BAD_NS = [_ns(a=NAN), _ns(b=INF), _ns(c=-INF), _ns(eps=0), _ns(eps=-1), _ns(eps=NAN), _ns(eps=INF),
          _ns(steps=0), _ns(steps=33), _ns(reserved=1)]


@pytest.mark.parametrize("ns", BAD_NS)
def test_bad_coefficients(ns):
    assert _ortho(ns=ns) == q.QLORA_ERR_INVALID_ARG and _step(ns=ns) == q.QLORA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), "INVALID_ARG"), (dict(cols=-1), "INVALID_ARG"),
    (dict(rows=129, cols=129), "UNSUPPORTED"), (dict(rows=1 << 30), "UNSUPPORTED"),
    (dict(cols=1 << 30), "UNSUPPORTED"), (dict(dtype=2), "INVALID_ARG"),
    (dict(reserved=1), "INVALID_ARG"), (dict(count=-1), "INVALID_ARG"),
    (dict(ws=None), "WORKSPACE"), (dict(ws_bytes=100), "WORKSPACE"), (dict(ws=FAKE + 8), "WORKSPACE")])
def test_bad_shapes(kw, want):
    code = getattr(q, "QLORA_ERR_" + want)
    assert _ortho(**kw) == code and _step(**kw) == code


def test_orthogonalize_refusals():
    bad = q.QLORA_ERR_INVALID_ARG
    for kw in (dict(x=None), dict(out=None), dict(x=FAKE + 2), dict(out=FAKE + 1),
               dict(x=FAKE + 1, dtype=1), dict(ldi=99), dict(ldo=99), dict(ldi=1 << 30),
               dict(out=FAKE, ldo=128)):
        assert _ortho(**kw) == bad, kw
    assert _ortho(rows=0, x=None, out=None, ws=None) == q.QLORA_OK
    assert _ortho(cols=0, x=None, out=None, ws=None) == q.QLORA_OK
    assert _ortho(count=0, ws=None) == q.QLORA_OK
    n = _ns()
    assert q.lib().qlora_orthogonalize(None, None, 0, None, 0, None) == bad
    assert q.lib().qlora_orthogonalize(ctypes.byref(n), None, 1, P(FAKE), BIG, None) == bad


def test_step_refusals():
    bad = q.QLORA_ERR_INVALID_ARG
    for kw in (dict(p=None), dict(g=None), dict(m=None), dict(p=FAKE + 2), dict(g=FAKE + 2),
               dict(g=FAKE + 1, dtype=1), dict(m=FAKE + 1), dict(pb=FAKE + 1), dict(ldp=99),
               dict(ldg=99), dict(ldm=99), dict(ldb=99), dict(ldm=1 << 30), dict(lr=-1),
               dict(lr=NAN), dict(lr=INF), dict(mu=1.0), dict(mu=-0.1), dict(mu=NAN), dict(wd=-1),
               dict(wd=INF), dict(nesterov=2), dict(adjust=3), dict(adjust=-1)):
        assert _step(**kw) == bad, kw
    assert _step(rows=0, p=None, g=None, m=None, ws=None) == q.QLORA_OK
    assert _step(count=0, ws=None) == q.QLORA_OK
    assert q.lib().qlora_muon_step(None, None, 0, None, 0, None) == bad


def test_workspace_bytes():
    assert 0 < _bytes((8, 1024)) < _bytes((8, 1024), (1024, 8)) < _bytes((128, 1024), (1024, 8))
    assert _bytes((129, 129)) == 0 and _bytes((-1, 4)) == 0 and _bytes((4, 1 << 30)) == 0
    assert _bytes(*[(1, (1 << 30) - 1)] * 5) == 0       # more than 2^24 chunks
    assert _bytes() == 0 and _bytes((0, 5)) == 0
    for s in ((8, 1024), (64, 22016), (4096, 128)):
        need = _bytes(s)
        assert _ortho(*s, ws_bytes=need - 1) == q.QLORA_ERR_WORKSPACE
        assert _step(*s, ws_bytes=need - 1) == q.QLORA_ERR_WORKSPACE


def _raises(fn, *args, status=q.QLORA_ERR_INVALID_ARG, **kw):
    with pytest.raises(q.QloraError) as e:
        fn(*args, **kw)
    assert e.value.status == status


def test_binding_refusals():
    x = torch.zeros(4, 50)
    _raises(q.qlora_orthogonalize, [x])                              # on the host
    _raises(q.qlora_orthogonalize, [x.double()])
    _raises(q.qlora_orthogonalize, [x.t()])
    _raises(q.qlora_orthogonalize, [x[0]])
    _raises(q.qlora_orthogonalize, [x], out=[])
    _raises(q.qlora_orthogonalize, [x], out=[x.bfloat16()])
    _raises(q.qlora_orthogonalize, [x], out=[torch.zeros(50, 4)])
    _raises(q.qlora_orthogonalize, [x], coefficients=(1.0, 2.0))
    good = (x, x.clone(), x.clone(), x.bfloat16())
    _raises(q.MuonPlan, [good])                                      # on the host
    _raises(q.MuonPlan, [good[:3]])
    _raises(q.MuonPlan, [(x.bfloat16(),) + good[1:]])
    _raises(q.MuonPlan, [(x, x.half()) + good[2:]])
    _raises(q.MuonPlan, [(x, x, x[:, :40], None)])
    _raises(q.MuonPlan, [(x, x, x, x)])
    _raises(q.MuonPlan, [(x.t(), x.t(), x.t(), None)])
    _raises(q.qlora_muon_step, [], 0.1, adjust="other")
    assert q.qlora_muon_step([], 0.1) is None
    assert q.qlora_orthogonalize([]) == []


def test_nothing_is_written_twice():
    """Two tensors of a call that begin at one place would be written by workgroups of
    both; a gradient, which is only read, may serve two."""
    x, y, z, w = (torch.zeros(4, 50) for _ in range(4))
    b = x.bfloat16()
    for bad in ([(x, y, z, None), (x, y, w, None)],                  # a parameter
                [(x, y, z, None), (w, y, z, None)],                  # a momentum
                [(x, y, x, None)],
                [(x, y, z, b), (w, y, y.clone(), b)]):
        with pytest.raises(q.QloraError, match="twice"):
            q.MuonPlan(bad)
    with pytest.raises(q.QloraError, match="twice"):
        q.qlora_orthogonalize([x, y], out=[z, z])
    e = torch.zeros(0, 5)
    for fine in ([(x, y, z, None), (w, y, y.clone(), None)],         # refused for the host only
                 [(x, y, z, None), (e, e, e, None), (e, e, e, None)]):
        with pytest.raises(q.QloraError, match="GPU"):
            q.MuonPlan(fine)
