"""Logits that are a narrow view of a wide buffer (one position of every sequence,
the answer's part of a padded vocabulary): the gradient that a call allocates is
as large as the view, its rows at the view's alignment."""
import pytest
import torch

from gpu_common import DEV, say

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,width,dtype", [(12, 1000, 64000, torch.bfloat16), (12, 1003, 60001, torch.bfloat16),
                                             (9, 777, 50003, torch.float32), (300, 16403, 40004, torch.bfloat16)])
def test_gradient_of_a_narrow_view(T, V, width, dtype):
    say("narrow view T=%d V=%d of %d %s" % (T, V, width, dtype))
    g = torch.Generator(device=DEV).manual_seed(V)
    buf = torch.randn((T, width), generator=g, device=DEV).to(dtype)
    z, y = buf[:, :V], torch.randint(0, V, (T,), generator=g, device=DEV)
    cu = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    adv = torch.tensor([1.0, -0.5], device=DEV)
    size, phase = buf.element_size(), 16 // buf.element_size()
    _, stats = q.qlora_token_logprobs(z, y, return_stats=True)
    w = torch.linspace(0.5, 1, T, device=DEV)
    for call in (lambda t, **k: q.qlora_token_logprobs_bwd(t, y, stats, w, **k),
                 lambda t, **k: q.qlora_preference_loss(t, y, cu, return_grad=True, **k).dlogits,
                 lambda t, **k: q.qlora_policy_loss(t, y, cu, adv, return_grad=True, **k).dlogits):
        d = call(z)
        held = d.untyped_storage().nbytes()      # (apart: a failing line would print the storage)
        assert held <= T * (V + 16) * size
        assert (d.stride(0) - z.stride(0)) % phase == 0 and d.stride(0) >= V
        wide = torch.empty_like(buf)
        assert torch.equal(d, call(z, dlogits=wide[:, :V]))
    leaf = buf.clone().requires_grad_()
    q.PreferenceLossFn.apply(leaf[:, :V], y, cu)[0].backward()
    assert torch.equal(leaf.grad[:, :V], q.qlora_preference_loss(z, y, cu, return_grad=True).dlogits)
    assert not leaf.grad[:, V:].any()
