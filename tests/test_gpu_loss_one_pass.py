"""The policy loss where one launch reads each row of logits once: 256 rows or
more, 32 KB to 256 KB of logits each.  Its gradient against the one that the
general backward forms from the statistics and weights of the same call, which
have to give the same bits, and the weights against the float64 oracle: log
ratios past float32's exponentials, KL terms next to zero, ratios next to a clip
border."""
import math

import numpy as np
import pytest
import torch

from gpu_common import DEV, host, say
from oracle import loss as oloss

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FORMS = [(300, 16400, BF, 0), (300, 17003, BF, 3), (280, 40001, BF, 0), (260, 128256, BF, 0),
         (290, 9001, F32, 1), (270, 20003, F32, 0)]


def _case(T, V, dtype, pad=0, seed=0):
    """Packed rows, a third of them without a target, and the log-probabilities
    that the sequences' statistics give."""
    g = torch.Generator().manual_seed(seed + T + V)
    z = (torch.randn((T, V + pad), generator=g) * 2.5)
    y = torch.randint(0, V, (T,), generator=g)
    z[torch.arange(T), y] += 10 * torch.rand(T, generator=g)
    y[torch.rand(T, generator=g) < 0.3] = -100
    z, y = z.to(dtype).to(DEV)[:, :V], y.to(DEV)
    cu = torch.tensor([1, T // 3, T // 3, T - 2], dtype=torch.int32, device=DEV)
    return g, z, y, cu, q.qlora_token_logprobs(z, y)


def _np(t):
    return host(t).double().numpy()


def _run(z, y, cu, *args, **kw):
    """One call with everything it can return; its gradient has to be the one
    that its statistics and weights stand for."""
    T = len(y)
    stats, w = torch.empty((T, 2), device=DEV), torch.empty(T, device=DEV)
    o = q.qlora_policy_loss(z, y, cu, *args, return_grad=True, stats=stats, w=w, **kw)
    inside = torch.zeros(T, dtype=torch.bool, device=DEV)
    inside[int(cu[0]):int(cu[-1])] = True
    d = q.qlora_token_logprobs_bwd(z, torch.where(inside, y, -1), stats, w)
    assert torch.equal(o.dlogits, d)
    return o, stats, w, inside & (y >= 0)


@pytest.mark.parametrize("T,V,dtype,pad", FORMS)
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_gradient_is_that_of_the_weights(T, V, dtype, pad, reduction):
    say("one pass T=%d V=%d %s %s" % (T, V, dtype, reduction))
    g, z, y, cu, lp = _case(T, V, dtype, pad)
    old = lp - 0.3 * torch.randn(T, generator=g).to(DEV)
    ref = lp + 0.2 * torch.randn(T, generator=g).to(DEV)
    adv = torch.randn(3, generator=g).to(DEV)
    _run(z, y, cu, adv, old, ref, kl_coef=0.05, reduction=reduction)
    _run(z, y, cu, adv, old, reduction=reduction)
    _run(z, y, cu, adv, reduction=reduction)


@pytest.mark.parametrize("T,V,dtype,pad", FORMS)
def test_kl_next_to_the_reference(T, V, dtype, pad):
    """Advantage 0: all of a weight is -kl_coef (exp(d) - 1), for d down to 1e-4.
    logp is off by what the row's sum is, w by share kl_coef exp(d) times that."""
    say("one pass, KL only T=%d V=%d %s" % (T, V, dtype))
    g, z, y, cu, lp = _case(T, V, dtype, pad)
    size = 10.0 ** -torch.randint(2, 5, (T,), generator=g).double()
    ref = (lp.double() + (size * torch.randn(T, generator=g).sign()).to(DEV)).float()
    o, stats, w, use = _run(z, y, cu, torch.zeros(3, device=DEV), lp, ref, kl_coef=0.5)
    # from the statistics of the call itself, what is left is one rounding
    zy = torch.gather(z, 1, y.clamp(min=0)[:, None])[:, 0].double()
    l = zy - stats[:, 0].double() - stats[:, 1].double().log()
    want = torch.where(use, -0.5 * torch.expm1(ref.double() - l) / int(use.sum()), 0.0)
    err, tol = (w.double() - want).abs(), 2.0 ** -24 * want.abs() + 1e-15
    assert bool((err <= tol).all()), float((err / want.abs().clamp(min=1e-30)).max())
    # and the gradient's bits are the weights' (above), to half a step in each row
    p = torch.exp(z[use].double() - stats[use, :1].double()) / stats[use, 1:].double()
    d = -want[use][:, None] * p
    d.scatter_add_(1, y[use][:, None], want[use][:, None])
    half = torch.finfo(dtype).eps / 2
    assert bool(((o.dlogits[use].double() - d).abs() <= (half + 2.0 ** -20) * d.abs()
                 + 2.0 ** -20 * want[use].abs()[:, None]).all())


@pytest.mark.parametrize("T,V,dtype,pad", FORMS)
def test_log_ratios_past_float32(T, V, dtype, pad):
    say("one pass, far ratios T=%d V=%d %s" % (T, V, dtype))
    g, z, y, cu, lp = _case(T, V, dtype, pad)
    far = torch.randint(100, 300, (T,), generator=g).float().to(DEV)
    adv = torch.tensor([0.0, 1.0, 0.7], device=DEV)
    # advantage 0 and a ratio of exp(100) and more; a reference watched, not pulled to
    for old, ref, a in ((lp - far, None, adv * 0), (lp, lp + far, adv), (lp - far, lp + far, adv * 0)):
        o, _, w, use = _run(z, y, cu, a, old, ref, kl_coef=0.0)
        assert bool(torch.isfinite(o.dlogits).all()) and bool(torch.isfinite(w).all())
        assert math.isfinite(float(o.loss))
        if not a.any():
            assert float(o.loss) == 0 and not o.dlogits.any()


@pytest.mark.parametrize("T,V,dtype,pad", FORMS)
def test_clipped_rows_are_those_counted(T, V, dtype, pad):
    say("one pass, clip border T=%d V=%d %s" % (T, V, dtype))
    g, z, y, cu, lp = _case(T, V, dtype, pad)
    off = (torch.randint(-8, 9, (T,), generator=g).double() * 2.0 ** -23).to(DEV)
    old = (lp.double() - math.log(1.2) + off).float()
    o, _, w, use = _run(z, y, cu, torch.tensor([1.0, 1.0, 0.5], device=DEV), old)
    cut = use & (w == 0)
    assert 0 < int(cut.sum()) < int(use.sum())
    assert float(o.clip_frac) == pytest.approx(float(cut.sum()) / float(use.sum()), rel=2.0 ** -23)
    assert torch.equal(use & ~o.dlogits.any(1), cut)


@pytest.mark.parametrize("T,V,dtype,pad", [(300, 16400, BF, 0), (290, 9001, F32, 1),
                                           (120, 16400, BF, 0), (120, 1001, F32, 0)])
@pytest.mark.parametrize("kl", [0.0, 0.05])
def test_weights_against_the_oracle(T, V, dtype, pad, kl):
    """Each weight to its own scale: logp off by e moves w by at most
    share (|A| r + kl_coef exp(d)) e.  e: a row's float32 sum, as each
    exponential is off by 2^-22 and a thread adds V / 256 + 64 terms at most."""
    say("policy weights T=%d V=%d %s kl=%g" % (T, V, dtype, kl))
    g, z, y, cu, lp = _case(T, V, dtype, pad)
    d = 0.3 * torch.randn(T, generator=g)
    for edge in (math.log(0.8), math.log(1.2)):
        d = torch.where((d - edge).abs() < 1e-3, d + 4e-3, d)
    old, ref = lp - d.to(DEV), lp + 0.2 * torch.randn(T, generator=g).to(DEV)
    adv = torch.randn(T, generator=g).to(DEV)
    o, _, w, _ = _run(z, y, cu, adv, old, ref if kl else None, kl_coef=kl, token_advantages=True)
    yn, cun = _np(y).astype(int), _np(cu).astype(int)
    r = oloss.policy(_np(z), yn, cun, _np(adv), _np(old), _np(ref) if kl else None, kl_coef=kl,
                     token_adv=True)
    use = oloss.rows_in(cun, yn, T)
    e = 2.0 ** -22 + (V / 256 + 64) * 2.0 ** -24
    unit = np.abs(_np(adv)) * np.exp(r["logp"] - _np(old)) + kl * np.exp(_np(ref) - r["logp"])
    tol = np.where(use, unit / use.sum() * e, 0) + 2.0 ** -23 * np.abs(r["w"])
    assert np.all(np.abs(_np(w) - r["w"]) <= tol)
    # an element moves by its own weight's error, p's and half a step of its type
    half = torch.finfo(dtype).eps / 2
    bound = (half * np.abs(r["dlogits"]) + (tol + np.abs(r["w"]) * (e + 2.0 ** -20))[:, None])
    assert np.all(np.abs(_np(o.dlogits) - r["dlogits"]) <= bound)


# more rows with a target than the launch has workgroups, so that each takes a
# second row and a third
LOOPS = [(2700, 16411, BF, 2, 1024), (1500, 33003, BF, 5, 512), (900, 70001, BF, 0, 256),
         (820, 66003, BF, 4, 256), (1700, 8203, F32, 0, 1024), (1600, 17001, F32, 1, 512),
         (760, 40001, F32, 2, 256)]


@pytest.mark.parametrize("T,V,dtype,pad,groups", LOOPS)
def test_workgroups_that_take_row_after_row(T, V, dtype, pad, groups):
    """Rows of changing alignment: a workgroup's next row has a head, an edge and
    chunks of its own.  logp within a row's float32 sum of float64 (each
    exponential off by 2^-22, a thread adding V / 256 + 64 terms at most), the
    weights one rounding from the statistics', the gradient theirs."""
    say("one pass, many rows T=%d V=%d %s pad=%d" % (T, V, dtype, pad))
    g, z, y, cu, lp = _case(T, V, dtype, pad)
    y[7], y[T // 2 + 1] = V, V + 5                    # labels out of the vocabulary between
    old = lp - 0.3 * torch.randn(T, generator=g).to(DEV)
    ref = lp + 0.2 * torch.randn(T, generator=g).to(DEV)
    adv = torch.randn(T, generator=g).to(DEV)
    kw = dict(kl_coef=0.05, token_advantages=True)
    o, stats, w = _nan_run(z, y, cu, adv, old, ref, **kw)
    inside = torch.zeros(T, dtype=torch.bool, device=DEV)
    inside[int(cu[0]):int(cu[-1])] = True
    use, bad = inside & (y >= 0) & (y < V), inside & (y >= V)
    assert int(use.sum()) > groups
    zd = z.double()
    zy = torch.gather(zd, 1, y.clamp(0, V - 1)[:, None])[:, 0]
    want = torch.where(use, zy - torch.logsumexp(zd, 1), 0.0)
    e = 2.0 ** -22 + (V / 256 + 64) * 2.0 ** -24
    assert bool(((o.logp.double() - want).abs() <= e + 2.0 ** -24 * want.abs())[~bad].all())
    assert bool(torch.isnan(o.logp[bad]).all()) and bool(torch.isnan(o.dlogits[bad]).all())
    l = zy - stats[:, 0].double() - stats[:, 1].double().log()
    r, k = torch.exp(l - old.double()), torch.exp(ref.double() - l)
    u, c = -adv.double() * r, -adv.double() * r.clamp(0.8, 1.2)
    share = 1 / int((inside & (y >= 0)).sum())
    want = share * (torch.where(c > u, 0.0, u) - 0.05 * (k - 1))
    err, tol = (w.double() - want).abs(), 2.0 ** -23 * want.abs() + 1e-13 * share
    border = ((l - old.double()).exp() - 0.8).abs().minimum((r - 1.2).abs()) < 1e-12
    assert bool((err <= tol)[use & ~border].all())
    # in place, where a row's stores follow the next row's loads
    t = z.clone() if z.is_contiguous() else torch.empty((T, V + pad), dtype=dtype, device=DEV)[:, :V]
    t.copy_(z)
    b = q.qlora_policy_loss(t, y, cu, adv, old, ref, dlogits=t, **kw)
    assert b.dlogits is t and torch.equal(torch.nan_to_num(t, 7.0), torch.nan_to_num(o.dlogits, 7.0))
    assert torch.equal(torch.nan_to_num(b.logp, 7.0), torch.nan_to_num(o.logp, 7.0))


def _nan_run(z, y, cu, *args, **kw):
    """_run for batches with labels out of the vocabulary, whose rows are NaN."""
    T = len(y)
    stats, w = torch.empty((T, 2), device=DEV), torch.empty(T, device=DEV)
    o = q.qlora_policy_loss(z, y, cu, *args, return_grad=True, stats=stats, w=w, **kw)
    inside = torch.zeros(T, dtype=torch.bool, device=DEV)
    inside[int(cu[0]):int(cu[-1])] = True
    d = q.qlora_token_logprobs_bwd(z, torch.where(inside, y, -1), stats, w)
    assert torch.equal(torch.nan_to_num(o.dlogits, 7.0), torch.nan_to_num(d, 7.0))
    return o, stats, w


@pytest.mark.parametrize("T,V,dtype", [(512, 32000, BF), (512, 128256, BF), (600, 32000, BF),
                                       (512, 32003, F32)])
def test_sums_have_no_bias(T, V, dtype):
    """Over many rows the sums' relative errors average out: rounded once they are
    within 2^-24 with mean 0 (1.5e-9 over 512 rows), and what the exponentials add
    is under 2^-25 in the mean.  A bias adds up over a sequence's log ratio."""
    say("bias of the sums T=%d V=%d %s" % (T, V, dtype))
    g = torch.Generator(device=DEV).manual_seed(V)
    z = (torch.randn((T, V), generator=g, device=DEV) * 2.5).to(dtype)
    y = torch.randint(0, V, (T,), generator=g, device=DEV)
    cu = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    stats = torch.empty((3, T, 2), device=DEV)
    q.qlora_token_logprobs(z, y, stats=stats[0])
    q.qlora_preference_loss(z, y, cu, stats=stats[1])
    q.qlora_policy_loss(z, y, cu, torch.ones(2, device=DEV), return_grad=True, stats=stats[2])
    for s in stats:
        exact = torch.exp(z.double() - s[:, :1].double()).sum(1)
        rel = s[:, 1].double() / exact - 1
        assert abs(float(rel.mean())) <= 2.0 ** -25, float(rel.mean())
        assert float(rel.square().mean().sqrt()) <= 2.0 ** -23
