"""The largest sizes of the head and the update that their checks let through."""
import pytest
import torch

from gpu_common import DEV, say
from oracle import muon as omuon
from test_gpu_head import BF, _exact, _logp_tol
from test_gpu_muon import _check, _np

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu


def _random(seed, rows, cols, scale):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn((rows, cols), generator=g, device=DEV) * scale).to(BF)


@pytest.mark.parametrize("T,D,V,step", [(70, 65536, 300, 70), (130, 64, 1 << 22, 16),
                                        ((1 << 21) + 300, 64, 5, 1 << 18),
                                        (300, 1024, 1 << 20, 32)])
def test_largest(T, D, V, step):
    say("largest head T=%d D=%d V=%d" % (T, D, V))
    h, W = _random(1, T, D, 1.5), _random(2, V, D, D ** -0.5)
    y = torch.randint(0, V, (T,), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    y[torch.rand(T, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV) < 0.2] = -100
    y[0], y[-1] = V - 1, 0
    n = int((y >= 0).sum())
    o = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=True)
    only = q.qlora_head_cross_entropy(h, W, y, return_grad=True)
    logp, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    dh, dw = q.qlora_head_logprobs_bwd(h, W, y, stats, torch.full((T,), -1.0 / n, device=DEV),
                                       need_dweight=True)
    assert torch.equal(o.logp, logp) and torch.equal(only.logp, logp)
    total = torch.zeros((), dtype=torch.float64, device=DEV)
    dw_ref = torch.zeros((V, D), dtype=torch.float64, device=DEV)
    err = {k: 0.0 for k in ("o", "only", "bwd")}
    size = 0.0
    for i in range(0, T, step):
        s = slice(i, i + step)
        w = torch.full((len(y[s]),), -1.0 / n, dtype=torch.float64, device=DEV)
        ref, d, dh_ref, part = _exact(h[s], W, y[s], w)
        assert float((logp[s].double() - ref).abs().max()) <= _logp_tol(D, V)
        total += ref.sum()
        dw_ref += part
        size += float(dh_ref.norm() ** 2)
        for k, got in (("o", o.dhidden), ("only", only.dhidden), ("bwd", dh)):
            err[k] += float((got[s].double() - dh_ref).norm() ** 2)
            assert not got[s][y[s] < 0].any()
        del d, part, dh_ref
    assert abs(float(o.loss) + float(total) / n) <= _logp_tol(D, V)
    # (dz and the output rounded once each, without bias)
    assert all((e / size) ** 0.5 < 4e-3 for e in err.values()), err
    for got in (o.dweight, dw):
        assert float((got.double() - dw_ref).norm() / dw_ref.norm()) < 4e-3


@pytest.mark.parametrize("rows,cols", [(1, 1 << 24), ((1 << 22) + 3, 3), (128, 1 << 17), ((1 << 20) + 1, 33)])
def test_longest_matrices(rows, cols):
    say("longest %d x %d" % (rows, cols))
    x = _random(5, rows, cols, 1e-3).float()
    out, = q.qlora_orthogonalize([x])
    # (the polynomial of the short side's product matrix, in float64)
    u = x.double() if rows <= cols else x.double().T
    g = u @ u.T
    n = g.diagonal().sum().sqrt()
    a, b, c = omuon.COEFFICIENTS
    G, P = g / n ** 2, torch.eye(len(g), dtype=torch.float64, device=DEV)
    for _ in range(5):
        p = a * torch.eye(len(g), dtype=torch.float64, device=DEV) + b * G + c * G @ G
        P, G = p @ P, p @ G @ p
    ref = (P / n) @ u
    _check(out, _np(ref if rows <= cols else ref.T), torch.float32)


def test_many_matrices():
    say("3000 matrices")
    g = torch.Generator().manual_seed(6)
    shapes = [tuple(int(v) for v in torch.randint(1, 40, (2,), generator=g)) for _ in range(3000)]
    flat = torch.randn(sum(r * c for r, c in shapes), generator=g).to(DEV)
    xs = [t.view(s) for t, s in zip(flat.split([r * c for r, c in shapes]), shapes)]
    for x, o in list(zip(xs, q.qlora_orthogonalize(xs)))[::7]:
        _check(o, omuon.orthogonalize(_np(x)), torch.float32)
