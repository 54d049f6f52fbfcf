"""Zero matrices under any eps and any coefficients: zeros, at every padded rank, alone,
among others and in a step."""
import math

import pytest
import torch

from gpu_common import DEV, say
from test_gpu_muon import BF, F32, _check, _matrix, _np
from oracle import muon as omuon

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu
SHAPES = [(8, 1024), (1024, 16), (20, 700), (5000, 32), (33, 400), (3000, 64), (65, 200), (400, 128)]


@pytest.mark.parametrize("kw", [dict(eps=1e-100), dict(eps=1e-160), dict(eps=1e-310),
                                dict(eps=5e-324), dict(coefficients=(1e300, -1e300, 1e300)),
                                dict(eps=1e-300, coefficients=(1e300, 0.0, 0.0), steps=32)])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_zero_matrices(rows, cols, dtype, kw):
    say("zeros %d x %d %s %s" % (rows, cols, dtype, kw))
    z = torch.zeros((rows, cols), dtype=dtype, device=DEV)
    z[0] = -0.0
    out, = q.qlora_orthogonalize([z], **kw)
    assert not out.any()
    p = torch.ones((rows, cols), device=DEV)
    pb = p.to(BF)
    q.qlora_muon_step([(p, z, torch.zeros_like(p), pb)], 0.1, weight_decay=0.5, **kw)
    assert (p == 0.95).all() and torch.equal(pb, p.to(BF))


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_smallest_values_under_a_smaller_eps(rows, cols):
    say("float32's smallest values, %d x %d" % (rows, cols))
    m = torch.zeros((rows, cols), device=DEV)
    m[0, 0] = 2.0 ** -149
    out, = q.qlora_orthogonalize([m], eps=5e-324)
    _check(out, omuon.orthogonalize(_np(m), eps=5e-324), F32)
    assert float(out[0, 0]) != 0 and int((out != 0).sum()) == 1


def test_zeros_among_others():
    say("zeros among others")
    ms = [torch.zeros(s, device=DEV) if i % 2 else _matrix(i, *s) for i, s in enumerate(SHAPES)]
    for m, o in zip(ms, q.qlora_orthogonalize(ms, eps=1e-300)):
        assert o.any() == m.any()
        _check(o, omuon.orthogonalize(_np(m), eps=1e-300), F32)
    bad = torch.zeros((64, 300), device=DEV)
    bad[3, 3] = math.inf
    assert torch.isnan(q.qlora_orthogonalize([bad], eps=1e-300)[0]).all()
