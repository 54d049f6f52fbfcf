"""The gradient at a target that is nearly certain: w (1 - p) is what is left of
two numbers of the size of w, and comes out to a step of its own."""
import math

import pytest
import torch

from gpu_common import DEV, say

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _rows(T, V, dtype, pad, seed):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((T, V + pad), generator=g).to(dtype).to(DEV)[:, :V]
    y = torch.randint(0, V, (T,), generator=g)
    y[:8] = torch.tensor([0, 1, V // 2, V - 1, 0, 1, V // 2, V - 1])     # edges of a row among them
    w = (0.2 + torch.rand(T, generator=g)) / 3100 * torch.where(torch.rand(T, generator=g) < 0.5, -1, 1)
    return g, z, y.to(DEV), w.to(DEV)


@pytest.mark.parametrize("V,dtype,pad", [(777, BF, 0), (1000, BF, 3), (5003, BF, 1), (32000, BF, 0),
                                         (1001, F32, 0), (8200, F32, 2)])
def test_gradient_of_a_certain_target(V, dtype, pad):
    """From given statistics (m = z_y, sum = 1 + d) the value is w d / (1 + d):
    the difference is exact, quotient and product round once each, and the
    output's type adds half a step."""
    say("certain targets V=%d %s" % (V, dtype))
    T = 64
    g, z, y, w = _rows(T, V, dtype, pad, V)
    z[torch.arange(T), y] = 30.0
    rest = 10.0 ** -(2 + 4.5 * torch.rand(T, generator=g).double())      # 1e-2 to 3e-7
    rest[:4] = 0.0                                                        # certain: exactly zero
    stats = torch.stack((torch.full((T,), 30.0), (1 + rest).float()), 1).to(DEV)
    d = q.qlora_token_logprobs_bwd(z, y, stats, w)
    got = torch.gather(d, 1, y[:, None])[:, 0].double()
    s = stats[:, 1].double()
    want = w.double() * (s - 1) / s
    half = torch.finfo(dtype).eps / 2 if dtype == BF else 0.0
    err = (got - want).abs()
    assert bool((err <= (half + 2.0 ** -22) * want.abs()).all()), \
        float((err / want.abs().clamp(min=1e-30)).max())
    assert not got[:4].any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_of_a_target_below_the_maximum(dtype):
    """p = exp(z_y - m) / sum for a z_y that is not the largest: exp is off by
    2^-22 of itself."""
    say("targets below the maximum %s" % dtype)
    T, V = 64, 900
    g, z, y, w = _rows(T, V, dtype, 0, 5)
    z[torch.arange(T), y] = (torch.rand(T, generator=g) * 4 + 20).to(dtype).to(DEV)
    stats = torch.stack((torch.full((T,), 24.0), 1 + torch.rand(T, generator=g)), 1).to(DEV)
    d = q.qlora_token_logprobs_bwd(z, y, stats, w)
    got = torch.gather(d, 1, y[:, None])[:, 0].double()
    zy = torch.gather(z, 1, y[:, None])[:, 0].double()
    p = torch.exp(zy - 24) / stats[:, 1].double()
    want = w.double() * (1 - p)
    half = torch.finfo(dtype).eps / 2 if dtype == BF else 0.0
    assert bool(((got - want).abs() <= (half + 2.0 ** -22) * want.abs()
                 + 2.0 ** -22 * w.double().abs()).all())


@pytest.mark.parametrize("V,dtype", [(777, BF), (1001, F32), (40000, BF)])
def test_the_only_token_left_has_no_gradient(V, dtype):
    say("one token left V=%d %s" % (V, dtype))
    g, z, y, w = _rows(16, V, dtype, 0, 3)
    keep = torch.gather(z, 1, y[:, None])
    z.fill_(-math.inf)
    z.scatter_(1, y[:, None], keep)
    logp, stats = q.qlora_token_logprobs(z, y, return_stats=True)
    assert not logp.any()
    assert not q.qlora_token_logprobs_bwd(z, y, stats, w).any()


@pytest.mark.parametrize("T,V,dtype", [(300, 16500, BF), (270, 70001, BF), (290, 9001, F32)])
def test_certain_targets_in_one_pass(T, V, dtype):
    """The policy loss that reads each row once has the same values, bit for bit."""
    say("certain targets, one pass T=%d V=%d %s" % (T, V, dtype))
    g, z, y, _ = _rows(T, V, dtype, 1, 9)
    z[torch.arange(T), y] += (12 + 14 * torch.rand(T, generator=g)).to(dtype).to(DEV)
    cu = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    stats, w = torch.empty((T, 2), device=DEV), torch.empty(T, device=DEV)
    lp = q.qlora_token_logprobs(z, y)
    o = q.qlora_policy_loss(z, y, cu, torch.tensor([0.7, -1.3], device=DEV), lp - 0.05, lp + 0.02,
                            kl_coef=0.1, return_grad=True, stats=stats, w=w)
    assert torch.equal(o.dlogits, q.qlora_token_logprobs_bwd(z, y, stats, w))
    s, zy = stats[:, 1].double(), torch.gather(z, 1, y[:, None])[:, 0].double()
    e = torch.exp(zy - stats[:, 0].double())
    want = w.double() * (s - e) / s
    got = torch.gather(o.dlogits, 1, y[:, None])[:, 0].double()
    half = torch.finfo(dtype).eps / 2 if dtype == BF else 0.0
    # (z_y is the maximum in nearly every row: exp exact there, 2^-22 elsewhere)
    tol = (half + 2.0 ** -22) * want.abs() + torch.where(e < 1, 2.0 ** -22, 0.0) * w.double().abs()
    assert bool(((got - want).abs() <= tol).all())
