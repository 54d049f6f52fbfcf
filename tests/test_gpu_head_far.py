"""Logits far beyond what float32 holds to a nat: where one entry is likelier than all the
others by more than that, the probabilities are 0 and 1 and the gradients exact."""
import pytest
import torch

from gpu_common import DEV, say
from test_gpu_head import BF, _check_grad, _exact, _inputs, _logp_tol

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu


def _decided(h, W, margin):
    """Rows whose two largest logits differ by more than `margin` of the largest."""
    top = torch.topk(h.double() @ W.double().T, 2, dim=1).values
    return (top[:, 0] - top[:, 1]) > margin * top.abs().amax(1) + 120


@pytest.mark.parametrize("T,D,V", [(50, 64, 500), (70, 1024, 300), (600, 128, 3000)])
@pytest.mark.parametrize("scale", [1e4, 1e7, 1e9, 1e15, 1e30, 2e37])
def test_one_entry_far_above_the_others(T, D, V, scale):
    say("logits of %g, T=%d D=%d V=%d" % (scale, T, D, V))
    h, W, y = _inputs(T, T, D, V, sharp=0)
    h = (h.float() * scale).to(BF)
    # (a float32 sum of D products: 2^-24 sqrt(D) / 4 of the largest, taken four times)
    on = _decided(h, W, 2.0 ** -20 * D ** 0.5)
    assert int(on.sum()) > T // 3
    y[on] = torch.where(torch.arange(T, device=DEV)[on] % 3 == 0,
                        (h[on].double() @ W.double().T).argmax(1), y[on])
    w = torch.linspace(-1, 1, T, device=DEV)
    ref, d, dh_ref, _ = _exact(h, W, y, w)
    logp, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    assert bool(torch.isfinite(logp).all()) and bool(torch.isfinite(stats).all())
    far = float((h.double() @ W.double().T).abs().max())
    assert float((logp.double() - ref).abs().max()) <= _logp_tol(D, V, 3 * far + 30)
    dh, dw = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dweight=True)
    assert bool(torch.isfinite(dh).all())
    _check_grad(dh[on], d[on], W.double(), dh_ref[on], V)
    for need in (False, True):
        o = q.qlora_head_cross_entropy(h, W, y, "sum", return_grad=True, need_dweight=need)
        _, d1, ref1, _ = _exact(h, W, y, torch.full((T,), -1.0, device=DEV))
        assert bool(torch.isfinite(o.dhidden).all()) and torch.equal(o.logp, logp)
        _check_grad(o.dhidden[on], d1[on], W.double(), ref1[on], V)
