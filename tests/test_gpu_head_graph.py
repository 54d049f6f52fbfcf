"""The head's autograd functions, forward and backward, captured into a graph and replayed
on other inputs."""
import pytest
import torch

from gpu_common import DEV, say
from test_gpu_head import _inputs

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu
SIZE = dict(T=300, D=128, V=2000)


def _grads(name, h, W, y):
    h, W = h.detach().requires_grad_(), W.detach().requires_grad_()
    if name == "logprobs":
        out = q.HeadLogprobsFn.apply(h, W, y)
        loss = (out * out).mean()
    else:
        loss, out = q.HeadCrossEntropyFn.apply(h, W, y, name)
        loss = 3 * loss
    return (out.detach(), loss.detach()) + torch.autograd.grad(loss, (h, W))


@pytest.mark.parametrize("name", ["logprobs", "mean", "sum"])
def test_forward_and_backward_replayed(name):
    say("graph of a head's forward and backward, %s" % name)
    h, W, y = (t.clone() for t in _inputs(60, **SIZE))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _grads(name, h, W, y)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _grads(name, h, W, y)
    for i, ignored in enumerate((0.0, 0.5, 0.9, 1.0, 0.3)):
        new = _inputs(61 + i, ignored=ignored, **SIZE)
        for t, x in zip((h, W, y), new):
            t.copy_(x)
        want = _grads(name, *new)
        for t in got:
            t.view(torch.uint8).fill_(0xA5) if t.dim() else t.fill_(7.0)
        torch.randn(1 << 20, device=DEV).sum().item()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
