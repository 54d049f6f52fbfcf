"""The autograd functions inside a region whose saved tensors are recomputed in the
backward, or kept on the host: hooks that give each saved tensor out once."""
import pytest
import torch
from torch.utils.checkpoint import checkpoint

from gpu_common import DEV, say

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu


def _functions():
    g = torch.Generator().manual_seed(1)
    t = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    W, _ = q.qlora_quantize_nf4(torch.randn((192, 128), generator=g).to(DEV))
    A, B, y = t(4, 128), t(192, 4), torch.arange(8, device=DEV)
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    adv = torch.tensor([1.0, -0.5], device=DEV)

    def linear(act8, dropout=None):
        return lambda x: q.QLoRALinearFn.apply(x.to(torch.bfloat16), A.requires_grad_(), B, W, 8.0,
                                               dropout, act8).float().square().sum()

    return {"logprobs": lambda x: q.TokenLogprobsFn.apply(x * 2, y).square().sum(),
            "preference": lambda x: q.PreferenceLossFn.apply(x * 2, y, cu)[0],
            "policy": lambda x: q.PolicyLossFn.apply(x * 2, y, cu, adv)[0],
            "linear": linear(None), "linear act8": linear(True),
            "linear act8 dropout": linear(True, (0.1, 5))}


@pytest.mark.parametrize("name", ["logprobs", "preference", "policy", "linear", "linear act8",
                                  "linear act8 dropout"])
def test_recomputed_and_offloaded(name):
    say("recomputed: %s" % name)
    f = _functions()[name]
    x = torch.randn((8, 128), generator=torch.Generator().manual_seed(2)).to(DEV)

    def grad(run):
        leaf = x.clone().requires_grad_()
        loss = run(leaf)
        loss.backward()
        return loss.detach(), leaf.grad

    want = grad(f)
    for run in (lambda v: checkpoint(f, v, use_reentrant=False),
                lambda v: checkpoint(f, v, use_reentrant=True)):
        got = grad(run)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    leaf = x.clone().requires_grad_()
    with torch.autograd.graph.save_on_cpu():
        loss = f(leaf)
    loss.backward()
    assert torch.equal(want[1], leaf.grad)
