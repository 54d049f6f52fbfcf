"""The autograd functions have first derivatives only: differentiating a
gradient again raises, where it would come out as if the backward were constant."""
import pytest
import torch

from gpu_common import DEV, say

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu


def _loss(name, leaf):
    if name == "linear" or name == "linear act8":
        g = torch.Generator().manual_seed(1)
        t = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
        W, _ = q.qlora_quantize_nf4(torch.randn((64, 128), generator=g).to(DEV))
        Y = q.QLoRALinearFn.apply(leaf.to(torch.bfloat16), t(4, 128), t(64, 4), W, 8.0, None,
                                  name != "linear")
        return (Y.float() ** 2).sum()
    y = torch.arange(8, device=DEV)
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    if name == "logprobs":
        return (q.TokenLogprobsFn.apply(leaf, y) ** 2).sum()
    if name == "preference":
        return q.PreferenceLossFn.apply(leaf, y, cu)[0]
    return q.PolicyLossFn.apply(leaf, y, cu, torch.ones(2, device=DEV))[0]


NAMES = ["logprobs", "preference", "policy", "linear", "linear act8"]


def _leaf():
    return torch.randn((8, 128), generator=torch.Generator().manual_seed(2)).to(DEV).requires_grad_()


@pytest.mark.parametrize("name", NAMES)
def test_second_derivatives_are_refused(name):
    say("twice: %s" % name)
    leaf = _leaf()
    d, = torch.autograd.grad(_loss(name, leaf), leaf)
    loss = _loss(name, leaf)
    twice, = torch.autograd.grad(loss, leaf, create_graph=True)
    assert torch.equal(d, twice.detach())            # the first one as without a graph
    with pytest.raises(RuntimeError):
        torch.autograd.grad((twice ** 2).sum(), leaf, retain_graph=True)
    # a penalty on the gradient beside the loss itself, which would go unseen
    with pytest.raises(RuntimeError):
        (loss + (twice ** 2).sum()).backward()


@pytest.mark.parametrize("name", NAMES)
def test_a_graph_of_the_gradient_that_is_not_used(name):
    say("graph kept: %s" % name)
    leaf, other = _leaf(), _leaf()
    _loss(name, leaf).backward()
    _loss(name, other).backward(create_graph=True)
    assert torch.equal(leaf.grad, other.grad.detach())
    # and one of another factor of the loss
    s = torch.tensor(2.0, device=DEV, requires_grad=True)
    third = _leaf()
    (s * _loss(name, third)).backward(create_graph=True)
    assert torch.allclose(third.grad.detach(), 2 * leaf.grad, rtol=2.0 ** -6, atol=1e-6)
    third.grad = other.grad = None
