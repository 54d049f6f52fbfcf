"""Every row of the head's weight gradient for itself, where a slice of the vocabulary has
one entry that is far likelier than its neighbours in every row: their gradients are
small, and as exact as any other."""
import pytest
import torch

from gpu_common import DEV, say
from test_gpu_head import BF, _exact, _inputs, _logp_tol

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu


def _dominated(seed, T, D, V, margin, every=128):
    """One entry of each `every` about `margin` nats above the others; never a target."""
    h, W, y = _inputs(seed, T, D, V, ignored=0.2, sharp=0.2)
    g = torch.Generator().manual_seed(seed + 1)
    u = torch.randn(D, generator=g).to(DEV)
    u = u / u.norm()
    likely = torch.arange(every // 3, V, every, device=DEV)
    Wf, hf = W.float(), h.float()
    Wf[likely] += margin / 4 * u
    Wf -= (Wf @ u)[:, None] * u * (~torch.isin(torch.arange(V, device=DEV), likely))[:, None]
    hf += (4 - hf @ u)[:, None] * u
    y = torch.where(torch.isin(y, likely), y + 1, y)
    return hf.to(BF), Wf.to(BF), y


def _check_rows(got, d, h, ref, slack):
    """A value of dz is off by 2^-11 (the value in 16 bits), 2^-8 (bf16) and what its float32
    logit leaves, all relative to itself however small it is; products with h are exact in
    float32 and their sum off by 2^-24 a term; then the output's rounding."""
    T = d.shape[0]
    bound = (d.abs().T @ h.abs()) * (2.0 ** -8 + 2.0 ** -11 + slack + T * 2.0 ** -24)
    bound = bound + ref.abs() * 2.0 ** -8 + 2.0 ** -126
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), (float((err / bound).max()),
                                        int((err > bound).any(1).sum()), "rows")


@pytest.mark.parametrize("T,D,V", [(300, 128, 1000), (256, 1024, 1000), (40, 64, 9000),
                                   (2300, 128, 20001)])
@pytest.mark.parametrize("margin", [12.0, 18.0, 24.0, 40.0])
def test_neighbours_of_a_likely_entry(T, D, V, margin):
    say("one likely entry a slice, T=%d D=%d V=%d margin=%g" % (T, D, V, margin))
    h, W, y = _dominated(T + V, T, D, V, margin)
    n = int((y >= 0).sum())
    w = torch.full((T,), -1.0 / n, device=DEV)
    _, d, dh_ref, dw_ref = _exact(h, W, y, w)
    masked = torch.where((y >= 0)[:, None], h.double(), 0.0)
    slack = _logp_tol(D, V, 2 * margin + 30)
    o = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=True)
    _check_rows(o.dweight, d, masked, dw_ref, slack)
    only = q.qlora_head_cross_entropy(h, W, y, need_dweight=True)
    assert torch.equal(only.dweight, o.dweight)
    _, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    dh, dw = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dweight=True)
    _check_rows(dw, d, masked, dw_ref, slack)
    for x in (o.dhidden, dh):
        assert float((x.double() - dh_ref).norm() / dh_ref.norm()) < 4e-3


def _row_of_dw(h, W, y, w, v):
    """Row v of dW in 64 bits, and the parts of its sum: |dz h| over its targets' rows and
    over the others."""
    ref, own, other = 0, 0, 0
    for i in range(0, len(y), 512):
        s = slice(i, i + 512)
        _, d, _, _ = _exact(h[s], W, y[s], w[s])
        hd = torch.where((y[s] >= 0)[:, None], h[s].double(), 0.0)
        ref = ref + d[:, v] @ hd
        mine = (y[s] == v).double()
        own = own + (mine * d[:, v].abs()) @ hd.abs()
        other = other + ((1 - mine) * d[:, v].abs()) @ hd.abs()
        del d
    return ref, own, other


@pytest.mark.parametrize("times", [1, 256, 257, 511, 512, 513, 769, 1020])
@pytest.mark.parametrize("V", [700, 9000])
def test_targets_that_round_alike(times, V):
    """The mean over 1020 targets: 1 / 1020 lies halfway between two bf16 values, and with
    p near 0 every target's dz is off to the same side by 2^-8.  What the roundings
    leave is added however many they are, so that the row is off by its own rounding."""
    say("%d targets that round alike, V=%d" % (times, V))
    T, D = 1020, 192
    h, W, y = _inputs(times, T, D, V, ignored=0.0, sharp=0.0)
    h = (h.float() + torch.linspace(-3, 3, D, device=DEV)).to(BF)
    W[7] = 0
    y = torch.where(y == 7, 8, y)
    y[torch.randperm(T, generator=torch.Generator().manual_seed(1))[:times].to(DEV)] = 7
    w = torch.full((T,), -1.0 / T, device=DEV)
    ref, own, other = _row_of_dw(h, W, y, w, 7)
    # (own: float32 sums of exact products and of what is left of each; statistics)
    bound = ref.abs() * 2.0 ** -8 + own * (T * 2.0 ** -23 + _logp_tol(D, V)) + \
        other * (2.0 ** -8 + 2.0 ** -11 + T * 2.0 ** -24 + _logp_tol(D, V))
    o = q.qlora_head_cross_entropy(h, W, y, need_dweight=True)
    _, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    dw = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dhidden=False, need_dweight=True)[1]
    for name, got in (("cross entropy", o.dweight), ("backward", dw)):
        err = (got[7].double() - ref).abs()
        assert bool((err <= bound).all()), (name, float((err / bound).max()))


def test_targets_that_round_alike_over_panels():
    say("3000 targets that round alike in two panels")
    T, D, V = 4080, 64, 262144
    h, W, y = _inputs(5, T, D, V, ignored=0.0, sharp=0.0)
    h = (h.float() + torch.linspace(-3, 3, D, device=DEV)).to(BF)
    W[7] = 0
    y = torch.where(y == 7, 8, y)
    y[torch.randperm(T, generator=torch.Generator().manual_seed(1))[:3000].to(DEV)] = 7
    ref, own, other = _row_of_dw(h, W, y, torch.full((T,), -1.0 / T, device=DEV), 7)
    bound = ref.abs() * 2.0 ** -8 + own * (T * 2.0 ** -23 + _logp_tol(D, V)) + \
        other * (2.0 ** -8 + 2.0 ** -11 + T * 2.0 ** -24 + _logp_tol(D, V))
    o = q.qlora_head_cross_entropy(h, W, y, need_dweight=True)
    err = (o.dweight[7].double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("T,D,V", [(130, 64, 2), (1020, 192, 12), (1500, 576, 16), (1020, 1088, 40),
                                   (5000, 128, 3), (4200, 2112, 2)])
@pytest.mark.parametrize("ignored", [0.0, 0.6])
def test_few_entries_of_many_rows(T, D, V, ignored):
    """A target's rows by the thousand, of which every one's rounding is made up for."""
    say("few entries T=%d D=%d V=%d ignored=%g" % (T, D, V, ignored))
    h, W, y = _inputs(T + V, T, D, V, ignored=ignored, sharp=0.2)
    h = torch.where((y >= 0)[:, None], h, float("nan"))
    n = int((y >= 0).sum())
    w = torch.full((T,), -1.0 / n, device=DEV)
    o = q.qlora_head_cross_entropy(h, W, y, need_dweight=True)
    _, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    dw = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dhidden=False, need_dweight=True)[1]
    for v in range(0, V, max(1, V // 5)):
        ref, own, other = _row_of_dw(h, W, y, w, v)
        bound = ref.abs() * 2.0 ** -8 + own * (T * 2.0 ** -23 + _logp_tol(D, V)) + \
            other * (2.0 ** -8 + 2.0 ** -11 + T * 2.0 ** -24 + _logp_tol(D, V))
        for got in (o.dweight, dw):
            err = (got[v].double() - ref).abs()
            assert bool((err <= bound).all()), (v, float((err / bound).max()))
    again = q.qlora_head_cross_entropy(h, W, y, need_dweight=True)
    assert torch.equal(again.dweight, o.dweight)
