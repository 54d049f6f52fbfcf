"""Losses whose log-probabilities are infinite, in a term that the call leaves
out (a coefficient, smoothing or advantage of zero), and other products with
zero: what is left out adds nothing."""
import math

import pytest
import torch

from gpu_common import DEV, say

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _rows(T, V, dtype):
    g = torch.Generator().manual_seed(T + V)
    z = (2 * torch.randn((T, V), generator=g)).to(dtype).to(DEV)
    return z, torch.randint(0, V, (T,), generator=g).to(DEV)


# two launches, and one pass over the rows
FORMS = [(40, 500, F32), (40, 501, BF), (300, 16500, BF), (270, 9001, F32)]


@pytest.mark.parametrize("T,V,dtype", FORMS)
@pytest.mark.parametrize("low", [-math.inf, None])
def test_policy_with_a_masked_target_and_a_reference_that_is_only_watched(T, V, dtype, low):
    say("policy, masked target, kl_coef 0, T=%d V=%d %s" % (T, V, dtype))
    z, y = _rows(T, V, dtype)
    cu = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    adv = torch.tensor([1.0, -0.5], device=DEV)
    old = q.qlora_token_logprobs(z, y)
    for t in (3, T - 2):
        z[t, y[t]] = torch.finfo(dtype).min if low is None else low
    w, alone = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    want = q.qlora_policy_loss(z, y, cu, adv, old, return_grad=True, w=alone)
    assert math.isfinite(float(want.loss))
    o = q.qlora_policy_loss(z, y, cu, adv, old, old, kl_coef=0.0, return_grad=True, w=w)
    assert torch.equal(o.loss, want.loss) and torch.equal(w, alone)
    assert torch.equal(o.dlogits, want.dlogits) and bool(torch.isfinite(o.dlogits).all())
    assert float(o.kl) == math.inf
    # and where the term counts it is infinite, not undefined
    assert float(q.qlora_policy_loss(z, y, cu, adv, old, old, kl_coef=0.1).loss) == math.inf


@pytest.mark.parametrize("T,V,dtype", FORMS)
def test_policy_without_advantage_of_a_token_its_sampler_ruled_out(T, V, dtype):
    say("policy, advantage 0, infinite ratio, T=%d V=%d %s" % (T, V, dtype))
    z, y = _rows(T, V, dtype)
    cu = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    old = q.qlora_token_logprobs(z, y)
    old[5] = -math.inf
    o = q.qlora_policy_loss(z, y, cu, torch.tensor([0.0, 0.0], device=DEV), old, return_grad=True)
    assert float(o.loss) == 0 and not o.dlogits.any()
    # a positive advantage meets the upper clip
    o = q.qlora_policy_loss(z, y, cu, torch.tensor([1.0, 0.0], device=DEV), old, return_grad=True)
    assert math.isfinite(float(o.loss)) and not o.dlogits[5].any() and o.dlogits[4].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["sigmoid", "hinge"])
def test_preference_without_smoothing_of_an_answer_ruled_out(dtype, kind):
    """The other answer of pair 0 holds a masked token: its log ratio is -inf, the
    pair is won, its loss and gradient 0."""
    say("preference, infinite log ratio, %s %s" % (kind, dtype))
    z, y = _rows(24, 700, dtype)
    cu = torch.tensor([0, 6, 12, 18, 24], dtype=torch.int32, device=DEV)
    ref = q.qlora_token_logprobs(z, y)
    half = q.qlora_preference_loss(z[12:], y[12:], cu[:3], ref[12:], 0.2, kind, return_grad=True)
    z[8, y[8]] = -math.inf
    o = q.qlora_preference_loss(z, y, cu, ref, 0.2, kind, return_grad=True)
    assert float(o.loss) == pytest.approx(float(half.loss) / 2, rel=2.0 ** -22)
    assert not o.dlogits[:12].any() and o.dlogits[12:].any()
    assert bool(torch.isfinite(o.dlogits).all()) and float(o.rewards[1]) == -math.inf
    # the pair lost, and the pair won with smoothing: infinite, not undefined
    swap = torch.cat((torch.arange(6, 12), torch.arange(6), torch.arange(12, 24))).to(DEV)
    lost = q.qlora_preference_loss(z[swap], y[swap], cu, ref[swap], 0.2, kind)
    assert float(lost.loss) == math.inf
    if kind == "sigmoid":
        assert float(q.qlora_preference_loss(z, y, cu, ref, 0.2, kind, 0.1).loss) == math.inf


@pytest.mark.parametrize("scale", [math.inf, math.nan])
def test_rows_of_weight_zero_under_an_overflowed_upstream_gradient(scale):
    say("weight 0, upstream gradient %s" % scale)
    for V, dtype in ((700, BF), (701, F32)):
        z, y = _rows(20, V, dtype)
        z[3] = math.nan                                # not read
        y[5], y[6] = -100, -1
        _, stats = q.qlora_token_logprobs(z, y, return_stats=True)
        w = torch.linspace(0.5, 1.0, 20, device=DEV)
        w[[0, 3, 19]] = 0
        d = q.qlora_token_logprobs_bwd(z, y, stats, w, grad_scale=torch.tensor([scale], device=DEV))
        assert not d[[0, 3, 5, 6, 19]].any()
        assert bool((~torch.isfinite(d[1])).any())
        # padding rows of a loss, whose weights are zero
        cu = torch.tensor([2, 9, 16], dtype=torch.int32, device=DEV)
        leaf = torch.where(torch.isnan(z), 0, z).requires_grad_()
        loss, _, _ = q.PreferenceLossFn.apply(leaf, y, cu)
        (loss * scale).backward()
        assert not leaf.grad[:2].any() and not leaf.grad[16:].any()
