"""GPU parity of the language-model head without logits against the float64
oracle: log-probabilities, weighted gradients and cross entropy over one row to
several panels, ragged vocabularies and row counts, strides, masks that leave
nothing, special values, in place, on other streams, replayed from graphs and
through autograd."""
import math

import numpy as np
import pytest
import torch

from gpu_common import DEV, host, say
from oracle import head as ohead

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _inputs(seed, T, D, V, ignored=0.3, pad=0, sharp=1.0):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn((V, D + pad), generator=g) / math.sqrt(D)).to(BF)[:, :D]
    y = torch.randint(0, V, (T,), generator=g)
    toward = sharp * 1.3 * math.log(V + 1) * torch.rand((T, 1), generator=g)
    h = torch.zeros((T, D + pad))
    h[:, :D] = 1.5 * torch.randn((T, D), generator=g) + toward * W[y].float()
    h = h.to(BF)[:, :D]
    y[torch.rand(T, generator=g) < ignored] = -100
    return _to(h), _to(W), y.to(DEV)


def _to(x):
    """On the GPU with the strides it has here."""
    full = torch.empty((x.shape[0], x.stride(0)), dtype=x.dtype, device=DEV)
    full[:, :x.shape[1]] = x.to(DEV)
    return full[:, :x.shape[1]]


def _np(t):
    return host(t).double().numpy()


def _exact(h, W, y, w=None):
    """The oracle in float64 on the GPU's inputs (torch on the GPU where it is
    large: the same formulas, row by row of the definition)."""
    hd, Wd, has = h.double(), W.double(), y >= 0
    hd = torch.where(has[:, None], hd, 0.0)
    z = hd @ Wd.T
    lse = torch.logsumexp(z, 1)
    at = y.clamp(min=0)[:, None]
    logp = torch.where(has, z.gather(1, at)[:, 0] - lse, 0.0)
    if w is None:
        return logp, lse
    w = torch.where(has, w.double(), 0.0)
    p = torch.exp(z - lse[:, None])
    d = -w[:, None] * p
    rest = p.scatter(1, at, 0.0).sum(1)
    d.scatter_(1, at, (w * rest)[:, None])
    return logp, d, d @ Wd, d.T @ hd


def _logp_tol(D, V, z=30.0):
    """A logit is a float32 sum of D exact products (each partial sum rounded:
    2^-24 of at most |z| sqrt(D) / 4 on the way, D / 4 adds of four products
    random in sign), then exponentials and float32 sums of a slice: 2^-22 of
    their own, as in the losses on given logits."""
    return z * 2.0 ** -24 * (4 + math.sqrt(D) / 8) + (math.log(V + 1) + 5) * 2.0 ** -22 + 2.0 ** -18


def _check_grad(got, d, other, ref, axis_len):
    """Each dz is rounded to bf16 once (half a step, 2^-8 relative to the value's
    power of two at most) from a value itself 2^-11 off (the fp16 exponential) and
    2^-17 (statistics): a sum of products errs by at most the sum of
    |dz| |other| (2^-8 / 2 ... taken whole), then half a step of the output."""
    bound = torch.matmul(d.abs(), other.abs()) * (2.0 ** -8 + 2.0 ** -11)
    # fp16's smallest steps: exponentials below 2^-14 of their slice's largest lose
    # 2^-25 of it at most
    bound = bound + d.abs().amax(1, keepdim=True) * 2.0 ** -24 * other.abs().sum(0)
    bound = bound + ref.abs() * 2.0 ** -8 + 1e-30
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    # and on the whole: rounding dz and the output, no bias
    if ref.norm() > 0 and ref.numel() > 1000:
        assert float(err.norm() / ref.norm()) < 4e-3


SHAPES = [  # T, D, V, row padding
    (1, 64, 1, 0), (1, 64, 2, 0), (1, 128, 5, 8), (3, 64, 63, 0), (5, 192, 64, 0), (64, 64, 127, 0),
    (65, 256, 129, 16), (17, 320, 255, 0), (128, 64, 257, 0), (129, 448, 300, 0),
    (33, 1024, 1000, 0), (200, 512, 4099, 8), (256, 256, 256, 0), (257, 320, 513, 0),
    (700, 576, 2000, 0), (1, 4096, 32000, 0), (16, 1024, 32003, 0), (331, 1024, 5003, 0),
    (1500, 128, 777, 0), (2, 8192, 1003, 0), (40, 64, 128256, 0),
    # few tiles: the inner index is cut
    (38, 6848, 1652, 0), (71, 2880, 2662, 0), (2481, 1024, 700, 0), (9, 384, 12004, 0),
    (300, 4096, 600, 8), (3000, 128, 300, 0), (1000, 2048, 130, 0), (130, 1024, 1, 0),
]


@pytest.mark.parametrize("T,D,V,pad", SHAPES)
def test_logprobs_and_backward(T, D, V, pad):
    say("head logprobs T=%d D=%d V=%d pad=%d" % (T, D, V, pad))
    h, W, y = _inputs(T + V, T, D, V, pad=pad, ignored=0.3 if T > 1 else 0)
    w = torch.randn(T, generator=torch.Generator().manual_seed(1)).to(DEV)
    logp, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    g = torch.tensor([0.75], device=DEV)
    ref, d, dh_ref, dw_ref = _exact(h, W, y, 0.75 * w)
    assert float((logp.double() - ref).abs().max()) <= _logp_tol(D, V)
    assert torch.equal(logp, q.qlora_head_logprobs(h, W, y))
    p = torch.exp(ref)
    has = y >= 0
    assert float((stats[:, 1].double() - (1 - p))[has].abs().max() if has.any() else 0) <= \
        4 * _logp_tol(D, V)
    assert not stats[~has].any() and not logp[~has].any()
    dh, dw = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dweight=True, grad_scale=g)
    _check_grad(dh, d, W.double(), dh_ref, V)
    _check_grad(dw, d.T.contiguous(), torch.where(has[:, None], h.double(), 0.0), dw_ref, T)
    assert not dh[~has].any()
    again = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dweight=True, grad_scale=g)
    assert torch.equal(dh, again[0]) and torch.equal(dw, again[1])
    only, none = q.qlora_head_logprobs_bwd(h, W, y, stats, w, grad_scale=g)
    assert none is None and torch.equal(only, dh)
    none, only = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dhidden=False,
                                           need_dweight=True, grad_scale=g)
    assert none is None and torch.equal(only, dw)


@pytest.mark.parametrize("T,D,V,pad", SHAPES)
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_cross_entropy(T, D, V, pad, reduction):
    say("head cross entropy T=%d D=%d V=%d pad=%d %s" % (T, D, V, pad, reduction))
    h, W, y = _inputs(T + V + 1, T, D, V, pad=pad, ignored=0.3 if T > 1 else 0)
    n = int((y >= 0).sum())
    k = -1.0 / max(n, 1) if reduction == "mean" else -1.0
    w = torch.full((T,), k, device=DEV)
    ref, d, dh_ref, dw_ref = _exact(h, W, y, w.double())
    o = q.qlora_head_cross_entropy(h, W, y, reduction, return_grad=True, need_dweight=True)
    assert float((o.logp.double() - ref).abs().max()) <= _logp_tol(D, V)
    assert abs(float(o.loss) - k * float(ref.sum())) <= _logp_tol(D, V) * -k * n + \
        2.0 ** -23 * abs(float(o.loss))
    _check_grad(o.dhidden, d, W.double(), dh_ref, V)
    _check_grad(o.dweight, d.T.contiguous(), torch.where((y >= 0)[:, None], h.double(), 0.0),
                dw_ref, T)
    plain = q.qlora_head_cross_entropy(h, W, y, reduction)
    assert torch.equal(plain.loss, o.loss) and torch.equal(plain.logp, o.logp)
    assert plain.dhidden is None and plain.dweight is None
    # dh alone is formed from powers of two rounded to bf16 instead of from dz: one
    # rounding as well, of other values, so within the same bounds but not the same bits
    only = q.qlora_head_cross_entropy(h, W, y, reduction, return_grad=True)
    assert torch.equal(only.logp, o.logp) and torch.equal(only.loss, o.loss)
    assert only.dweight is None and not only.dhidden[y < 0].any()
    _check_grad(only.dhidden, d, W.double(), dh_ref, V)
    again = q.qlora_head_cross_entropy(h, W, y, reduction, return_grad=True)
    assert torch.equal(again.dhidden, only.dhidden)


@pytest.mark.parametrize("T,D,V", [(9, 64, 20), (70, 128, 300), (140, 64, 513)])
def test_against_the_oracle(T, D, V):
    say("head oracle T=%d D=%d V=%d" % (T, D, V))
    h, W, y = _inputs(T, T, D, V)
    loss, logp, dh, dw = ohead.cross_entropy(_np(h), _np(W), _np(y).astype(int))
    o = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=True)
    assert abs(float(o.loss) - loss) <= _logp_tol(D, V)
    assert np.max(np.abs(_np(o.logp) - logp)) <= _logp_tol(D, V)
    for got, ref in ((o.dhidden, dh), (o.dweight, dw)):
        assert np.linalg.norm(_np(got) - ref) <= 4e-3 * np.linalg.norm(ref)
