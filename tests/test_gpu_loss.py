"""GPU parity of the losses on packed logits against the float64 oracle: token
log-probabilities, the preference loss and the clipped policy loss, forward
and backward, over ragged vocabularies, strides, masks that leave rows or
sequences empty, infinities, and packings with rows outside; in place, on
other streams, replayed from graphs and through autograd."""
import math

import numpy as np
import pytest
import torch

from gpu_common import DEV, host, say
from oracle import loss as oloss

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _logits(seed, T, V, dtype, pad=0, ignored=0.3):
    g = torch.Generator().manual_seed(seed)
    buf = torch.randn((T, V + pad), generator=g) * 2.5
    labels = torch.randint(0, V, (T,), generator=g)
    buf[torch.arange(T), labels] += 4
    labels[torch.rand(T, generator=g) < ignored] = -100
    z = buf.to(dtype).to(DEV)[:, :V]
    return z, labels.to(DEV)


def _np(t):
    return host(t).double().numpy()


def _tol(V):
    """Relative error of a row's float32 sum, and so absolute of its logp: each
    exponential is off by its argument's rounding (the dominating ones are at
    most log V + 3 below the maximum) and 2 ulp, and a thread adds at most
    V / 256 + 64 terms in a row before the tree."""
    return (math.log(V) + 5) * 2.0 ** -22 + (V / 256 + 64) * 2.0 ** -24


def _check_logp(got, ref, V):
    got = _np(got)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = np.isfinite(ref)
    assert np.array_equal(got[~ok & ~np.isnan(ref)], ref[~ok & ~np.isnan(ref)])
    assert np.all(np.abs(got - ref)[ok] <= _tol(V) + 2.0 ** -24 * np.abs(ref[ok]))


def _check_grad(got, ref, w, V, werr=0.0):
    """d = w (1[y] - p): w to werr (relative), p to _tol(V) + rounding, then
    half a step of the output's type."""
    half = torch.finfo(got.dtype).eps / 2
    got, w = _np(got), np.abs(np.asarray(w, dtype=np.float64))[:, None]
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    tol = half * np.abs(ref) + w * (_tol(V) + 2.0 ** -22 + werr)
    ok = ~np.isnan(ref)
    assert np.all(np.abs(got - ref)[ok] <= tol[ok]), float(np.max((np.abs(got - ref) - tol)[ok]))


SHAPES = [  # T, V, dtype, row padding
    (1, 1, BF, 0), (3, 2, F32, 0), (5, 7, BF, 0), (4, 7, F32, 2), (9, 63, BF, 1), (17, 64, BF, 0),
    (33, 1000, BF, 0), (8, 1001, BF, 0), (8, 1003, F32, 0), (6, 4099, BF, 3), (64, 5003, F32, 1),
    (300, 777, BF, 0), (2, 32000, BF, 0), (16, 32003, BF, 0), (3, 50001, F32, 0),
    (1, 128256, BF, 0), (5, 128256, BF, 7), (2, 131073, BF, 0), (2, 200003, F32, 0),
    (3, 262144, BF, 0),
]


@pytest.mark.parametrize("T,V,dtype,pad", SHAPES)
def test_token_logprobs_and_backward(T, V, dtype, pad):
    say("token logprobs T=%d V=%d %s pad=%d" % (T, V, dtype, pad))
    z, y = _logits(T + V, T, V, dtype, pad)
    logp, stats = q.qlora_token_logprobs(z, y, return_stats=True)
    ref, p = oloss.token_logprobs(_np(z), _np(y).astype(int))
    _check_logp(logp, ref, V)
    assert torch.equal(logp, q.qlora_token_logprobs(z, y))
    w = torch.randn(T, generator=torch.Generator().manual_seed(1)).to(DEV)
    w[0] = 0
    g = torch.tensor([0.75], device=DEV)
    d = q.qlora_token_logprobs_bwd(z, y, stats, w, grad_scale=g)
    assert d.stride(0) == (z.stride(0) if T > 1 else V)
    wn = 0.75 * _np(w)
    _check_grad(d, oloss.token_logprobs_bwd(p, _np(y).astype(int), wn), wn, V)
    assert torch.equal(d, q.qlora_token_logprobs_bwd(z, y, stats, w, grad_scale=g))


@pytest.mark.parametrize("T,V,dtype,pad", [
    (128, 16385, BF, 0), (200, 16391, BF, 1), (127, 16384, BF, 0), (512, 17000, BF, 0),
    (513, 16384, BF, 0), (129, 8193, F32, 0), (256, 32003, F32, 5), (140, 131073, BF, 2)])
def test_rows_given_whole_to_a_workgroup(T, V, dtype, pad):
    say("whole rows T=%d V=%d %s pad=%d" % (T, V, dtype, pad))
    z, y = _logits(T + V, T, V, dtype, pad)
    z[3, : V // 2] = -math.inf
    z[5] = -math.inf
    z[7, V - 1] = math.nan
    y[3], y[5], y[7], y[9] = V - 1, 1, 2, V
    logp, stats = q.qlora_token_logprobs(z, y, return_stats=True)
    ref, _ = oloss.token_logprobs(_np(z), _np(y).astype(int))
    _check_logp(logp, ref, V)
    assert torch.isnan(logp[[5, 7, 9]]).all()
    # the launch that a loss makes of the same rows
    cu = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    o = q.qlora_preference_loss(z, y, cu, stats=torch.empty_like(stats))
    _check_logp(o.logp, ref, V)


@pytest.mark.parametrize("dtype,V", [(BF, 1000), (BF, 1003), (F32, 999)])
def test_gradient_in_place_and_with_another_stride(dtype, V):
    say("dlogits in place, V=%d %s" % (V, dtype))
    z, y = _logits(4, 13, V, dtype, 5)
    _, stats = q.qlora_token_logprobs(z, y, return_stats=True)
    w = torch.linspace(-1, 1, 13, device=DEV)
    ref = q.qlora_token_logprobs_bwd(z, y, stats, w).clone()
    other = torch.full((13, V + 2), 7.0, dtype=dtype, device=DEV)
    q.qlora_token_logprobs_bwd(z, y, stats, w, dlogits=other[:, 1:V + 1])
    assert torch.equal(other[:, 1:V + 1], ref)
    assert (other[:, 0] == 7).all() and (other[:, V + 1] == 7).all()
    behind = torch.as_strided(z, (13, 5), (z.stride(0), 1), V)[:-1].clone()
    assert q.qlora_token_logprobs_bwd(z, y, stats, w, dlogits=z) is z
    assert torch.equal(z, ref)
    assert torch.equal(torch.as_strided(z, (13, 5), (z.stride(0), 1), V)[:-1], behind)


def test_masked_logits_and_rows_that_are_not_read():
    say("masks")
    V = 515
    for dtype in (BF, F32):
        z, y = _logits(8, 10, V, dtype, ignored=0.0)
        z[0, 5:] = float("-inf")
        y[0] = 3
        z[1, ::2] = torch.finfo(dtype).min
        y[1] = 1
        z[2] = float("-inf")                      # a row without anything
        z[3] = torch.finfo(dtype).min             # every logit the lowest: uniform
        z[4, 7] = float("inf")
        z[5, 9] = float("nan")
        z[6] = float("nan")                       # no target: not read
        y[6] = -1
        y[7] = V                                  # out of the vocabulary
        z[8] = float("-inf")
        z[8, 77] = 1.0                            # one value left, and it is the target
        y[8] = 77
        z[9, 12] = float("-inf")                  # the target itself masked
        y[9] = 12
        logp, stats = q.qlora_token_logprobs(z, y, return_stats=True)
        ref, p = oloss.token_logprobs(_np(z), _np(y).astype(int))
        assert np.isnan(ref[[2, 4, 5, 7]]).all() and ref[9] == -np.inf and ref[8] == 0
        assert ref[3] == pytest.approx(-math.log(V))
        _check_logp(logp, ref, V)
        w = torch.ones(10, device=DEV)
        d = q.qlora_token_logprobs_bwd(z, y, stats, w)
        for t in (0, 1, 3, 6, 8, 9):
            r = oloss.token_logprobs_bwd(p, _np(y).astype(int), np.ones(10))[t:t + 1]
            _check_grad(d[t:t + 1], r, [1.0], V)
        assert torch.isnan(d[[2, 4, 5, 7]]).any(1).all()
        w[[2, 4, 5, 7]] = 0                       # weight 0: zeros, whatever the row holds
        assert torch.isfinite(q.qlora_token_logprobs_bwd(z, y, stats, w)).all()


def test_no_rows():
    say("no rows")
    z, y = torch.zeros((0, 50), device=DEV), torch.zeros(0, dtype=torch.int64, device=DEV)
    assert q.qlora_token_logprobs(z, y).shape == (0,)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    o = q.qlora_preference_loss(z, y, cu, return_grad=True)
    assert o.loss.item() == pytest.approx(math.log(2)) and o.dlogits.shape == (0, 50)
    o = q.qlora_policy_loss(z, y, cu, torch.ones(2, device=DEV), return_grad=True)
    assert o.loss.item() == 0 and o.clip_frac.item() == 0


# -------------------------------------------------------------- whole losses
PACKS = [  # lengths, rows before, rows behind, V, dtype
    ([1, 1], 0, 0, 50, BF), ([5, 3], 0, 2, 1000, BF), ([7, 0, 1, 9], 3, 4, 333, F32),
    ([40, 25, 60, 31], 0, 0, 2003, BF), ([300, 280], 0, 10, 515, BF), ([4] * 64, 1, 0, 129, F32),
    ([90, 61, 0, 0, 75, 80], 2, 5, 4100, BF), ([6, 5], 0, 0, 128256, BF), ([3, 4], 1, 1, 140000, F32),
    ([70, 66, 51, 80], 0, 3, 33001, BF), ([150, 128], 1, 2, 70001, BF), ([140, 0, 3, 160], 0, 2, 20011, BF),
    ([131, 130], 0, 4, 20003, F32), ([129, 128], 2, 0, 40001, F32),
]


def _packed(seed, lens, lead, tail, V, dtype, ignored=0.3):
    cu = np.cumsum([lead] + lens).astype(np.int32)
    z, y = _logits(seed, int(cu[-1]) + tail, V, dtype, ignored=ignored)
    return z, y, torch.from_numpy(cu).to(DEV)


def _near(got, ref, rel, ab):
    assert abs(float(got) - ref) <= rel * abs(ref) + ab, (float(got), ref)


@pytest.mark.parametrize("lens,lead,tail,V,dtype", PACKS)
@pytest.mark.parametrize("kind,smooth,mean,ref", [("sigmoid", 0.0, False, True),
                                                  ("sigmoid", 0.2, True, True),
                                                  ("hinge", 0.0, True, False),
                                                  ("ipo", 0.0, True, True)])
def test_preference(lens, lead, tail, V, dtype, kind, smooth, mean, ref):
    say("preference %s V=%d %s %s" % (lens[:6], V, kind, mean))
    z, y, cu = _packed(len(lens) + V, lens, lead, tail, V, dtype)
    beta = 0.1
    rl = None
    if ref:
        rl = q.qlora_token_logprobs(z, y) + 0.2 * torch.randn(
            len(y), generator=torch.Generator().manual_seed(2)).to(DEV)
    stats = torch.empty((len(y), 2), device=DEV)
    w = torch.empty(len(y), device=DEV)
    o = q.qlora_preference_loss(z, y, cu, rl, beta, kind, smooth, mean, return_grad=True,
                                stats=stats, w=w)
    cun, yn = _np(cu).astype(int), _np(y).astype(int)
    r = oloss.preference(_np(z), yn, cun, None if rl is None else _np(rl), beta, kind, smooth, mean)
    _check_logp(o.logp, r["logp"], V)
    # a sequence's sums are off by at most its targets times a row's error
    n = max([1] + [int((yn[a:b] >= 0).sum()) for a, b in zip(cun, cun[1:])])
    err = _tol(V) * (1 if mean else n)
    for got, want, unit in ((o.seq_logp, r["seq_logp"], 1.0), (o.rewards, r["rewards"], beta)):
        assert np.all(np.abs(_np(got) - want) <= unit * err + 2.0 ** -23 * np.abs(want))
    # |dloss / dh| <= beta (sigmoid, hinge) or 2 |h - 1 / 2 beta| (ipo); h is off by 2 err
    hmax = 2 * np.abs(r["rewards"]).max() / beta + 1 / beta
    slope = beta if kind != "ipo" else 2 * hmax
    _near(o.loss, r["loss"], 2.0 ** -22, 2 * slope * err + 4 * err * err)
    # the slope itself moves by beta^2 / 4 (sigmoid) or 2 (ipo) of that
    curve = {"sigmoid": beta * beta / 4, "hinge": 0.0, "ipo": 2.0}[kind]
    werr = 2 * err * curve * 2 + 1e-30
    assert np.all(np.abs(_np(w) - r["w"]) <= werr + 2.0 ** -22 * np.abs(r["w"]))
    wmax = np.abs(r["w"]).max()
    rel = werr / wmax if wmax else 0.0
    _check_grad(o.dlogits, r["dlogits"], np.full(len(yn), wmax), V, rel + 2.0 ** -22)
    # the same gradient through the general backward, and without one
    assert torch.equal(o.dlogits, q.qlora_token_logprobs_bwd(z, y, stats, w))
    bare = q.qlora_preference_loss(z, y, cu, rl, beta, kind, smooth, mean)
    assert torch.equal(bare.loss, o.loss) and bare.dlogits is None


@pytest.mark.parametrize("lens,lead,tail,V,dtype", PACKS)
@pytest.mark.parametrize("reduction,kl,token_adv,old", [("token", 0.0, False, True),
                                                        ("token", 0.05, True, True),
                                                        ("sequence", 0.05, False, True),
                                                        ("sequence", 0.0, False, False)])
def test_policy(lens, lead, tail, V, dtype, reduction, kl, token_adv, old):
    say("policy %s V=%d %s kl=%g" % (lens[:6], V, reduction, kl))
    z, y, cu = _packed(len(lens) + V + 1, lens, lead, tail, V, dtype)
    g = torch.Generator().manual_seed(3)
    T = len(y)
    lp = q.qlora_token_logprobs(z, y)
    ol = rl = None
    if old:
        d = 0.3 * torch.randn(T, generator=g)
        for edge in (math.log(0.8), math.log(1.3)):     # away from the clip borders
            d = torch.where((d - edge).abs() < 1e-3, d + 4e-3, d)
        ol = lp - d.to(DEV)
    if kl:
        rl = lp + 0.2 * torch.randn(T, generator=g).to(DEV)
    adv = torch.randn(T if token_adv else len(lens), generator=g).to(DEV)
    o = q.qlora_policy_loss(z, y, cu, adv, ol, rl, 0.2, 0.3, kl, reduction, token_adv,
                            return_grad=True)
    yn = _np(y).astype(int)
    r = oloss.policy(_np(z), yn, _np(cu).astype(int), _np(adv), None if ol is None else _np(ol),
                     None if rl is None else _np(rl), 0.2, 0.3, kl, reduction, token_adv)
    _check_logp(o.logp, r["logp"], V)
    e = _tol(V)
    # one term moves by |A| r (and kl_coef |exp(d) - 1|) for each unit of logp
    amax = float(adv.abs().max()) * 4 + kl * 4
    _near(o.loss, r["loss"], 2.0 ** -22, amax * e)
    _near(o.kl, r["kl"], 2.0 ** -22, 4 * e)
    _near(o.clip_frac, r["clip_frac"], 2.0 ** -23, 0)
    wmax = np.abs(r["w"]).max()
    share = max(1e-30, wmax)
    _check_grad(o.dlogits, r["dlogits"], np.full(T, share), V, 8 * e * (1 + amax / share / max(1, T))
                + 2.0 ** -22)
    stats, w = torch.empty((T, 2), device=DEV), torch.empty(T, device=DEV)
    b = q.qlora_policy_loss(z, y, cu, adv, ol, rl, 0.2, 0.3, kl, reduction, token_adv, stats=stats,
                            w=w)
    assert b.dlogits is None
    _near(b.loss, r["loss"], 2.0 ** -22, amax * e)
    werr = 8 * e * amax / max(1, 1) * (share if T else 0) + 2.0 ** -22 * np.abs(r["w"]) + 1e-30
    assert np.all(np.abs(_np(w) - r["w"]) <= werr + e * amax)
    d2 = q.qlora_token_logprobs_bwd(z, y, stats, w)
    _check_grad(d2, r["dlogits"], np.full(T, share), V, 8 * e * (1 + amax / share / max(1, T))
                + 2.0 ** -22)


def test_no_target_anywhere():
    say("no target")
    z, y, cu = _packed(1, [4, 5], 0, 1, 300, BF)
    z.fill_(float("nan"))
    y.fill_(-100)
    o = q.qlora_preference_loss(z, y, cu, return_grad=True)
    assert o.loss.item() == pytest.approx(math.log(2)) and not o.dlogits.any()
    for red in ("token", "sequence"):
        o = q.qlora_policy_loss(z, y, cu, torch.ones(2, device=DEV), reduction=red,
                                return_grad=True)
        assert o.loss.item() == 0 and o.clip_frac.item() == 0 and not o.dlogits.any()


def test_cu_seqlens_past_the_rows_are_clamped():
    say("cu clamped")
    z, y, _ = _packed(2, [4, 5], 0, 0, 300, BF)
    good = torch.tensor([0, 4, 9], dtype=torch.int32, device=DEV)
    far = torch.tensor([-3, 4, 1 << 30], dtype=torch.int32, device=DEV)
    adv = torch.ones(2, device=DEV)
    a, b = (q.qlora_preference_loss(z, y, c, return_grad=True) for c in (good, far))
    assert torch.equal(a.loss, b.loss) and torch.equal(a.dlogits, b.dlogits)
    a, b = (q.qlora_policy_loss(z, y, c, adv, return_grad=True) for c in (good, far))
    assert torch.equal(a.loss, b.loss) and torch.equal(a.dlogits, b.dlogits)


def test_saturated_pairs_stay_finite():
    say("saturated")
    z, y, cu = _packed(3, [6, 6, 6, 6], 0, 0, 100, F32, ignored=0.0)
    ref = torch.zeros(24, device=DEV)
    ref[:6], ref[6:12], ref[12:18], ref[18:] = -1e5, 1e5, 1e5, -1e5
    for kind in ("sigmoid", "hinge"):
        o = q.qlora_preference_loss(z, y, cu, ref, 0.1, kind, return_grad=True)
        r = oloss.preference(_np(z), _np(y).astype(int), _np(cu).astype(int), _np(ref), 0.1, kind)
        _near(o.loss, r["loss"], 1e-6, 0)
        assert torch.isfinite(o.dlogits).all() and not o.dlogits[:12].any()


def test_in_place_matches_out_of_place():
    say("whole losses in place")
    for T, V in ((40, 1000), (300, 777)):
        z, y, cu = _packed(4, [T // 2, T - T // 2], 0, 0, V, BF)
        adv = torch.tensor([0.5, -1.5], device=DEV)
        old = q.qlora_token_logprobs(z, y) + 0.1
        for f in (lambda t, **k: q.qlora_preference_loss(t, y, cu, **k),
                  lambda t, **k: q.qlora_policy_loss(t, y, cu, adv, old, **k)):
            a = f(z, return_grad=True)
            t = z.clone()
            b = f(t, dlogits=t)
            assert torch.equal(a.loss, b.loss) and torch.equal(a.dlogits, t)


def test_streams_and_graph_replays():
    say("losses: stream and graph")
    for T, V in ((24, 3001), (400, 1000)):
        z, y, cu = _packed(5, [T // 2, T // 2], 0, 0, V, BF)
        adv = torch.tensor([0.5, -1.5], device=DEV)
        lp = q.qlora_token_logprobs(z, y)
        old, ref = lp + 0.1, lp - 0.2

        def step():
            a = q.qlora_preference_loss(z, y, cu, ref, return_grad=True)
            b = q.qlora_policy_loss(z, y, cu, adv, old, ref, kl_coef=0.1, return_grad=True)
            logp, stats = q.qlora_token_logprobs(z, y, return_stats=True)
            return [a.loss, a.seq_logp, a.rewards, a.dlogits, b.loss, b.kl, b.clip_frac, b.logp,
                    b.dlogits, logp, q.qlora_token_logprobs_bwd(z, y, stats, lp)]

        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            got = step()
        side.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want, got))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        for _ in range(3):
            for t in out:
                t.fill_(7)
            torch.randn(1 << 18, device=DEV).sum().item()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(want, out))


def test_autograd_wrappers():
    say("losses: autograd")
    z, y, cu = _packed(6, [20, 15, 11, 18], 0, 3, 1003, BF)
    lp = q.qlora_token_logprobs(z, y)
    old, ref, adv = lp + 0.05, lp - 0.1, torch.tensor([1.0, -1.0, 0.5, 0.0], device=DEV)
    w = torch.linspace(-1, 1, len(y), device=DEV)

    leaf = z.clone().requires_grad_()
    out = q.TokenLogprobsFn.apply(leaf, y)
    assert torch.equal(out, lp)
    (out * w).sum().backward()
    _, stats = q.qlora_token_logprobs(z, y, return_stats=True)
    assert torch.equal(leaf.grad, q.qlora_token_logprobs_bwd(z, y, stats, w))

    for scale in (1.0, -0.5):
        leaf = z.clone().requires_grad_()
        loss, seq, rew = q.PreferenceLossFn.apply(leaf, y, cu, ref, 0.2, "sigmoid", 0.1)
        o = q.qlora_preference_loss(z, y, cu, ref, 0.2, "sigmoid", 0.1, return_grad=True)
        assert torch.equal(loss, o.loss) and torch.equal(seq, o.seq_logp)
        assert not seq.requires_grad and not rew.requires_grad
        (scale * loss).backward(retain_graph=True)
        assert torch.allclose(leaf.grad.float(), scale * o.dlogits.float(), rtol=2.0 ** -7, atol=1e-9)
        once = leaf.grad.clone()
        leaf.grad = None
        (scale * loss).backward()
        assert torch.equal(once, leaf.grad)

        leaf = z.clone().requires_grad_()
        loss, kl, frac = q.PolicyLossFn.apply(leaf, y, cu, adv, old, ref, 0.2, 0.2, 0.1, "sequence")
        o = q.qlora_policy_loss(z, y, cu, adv, old, ref, kl_coef=0.1, reduction="sequence",
                                return_grad=True)
        assert not kl.requires_grad and not frac.requires_grad
        (scale * loss).backward()
        assert torch.allclose(leaf.grad.float(), scale * o.dlogits.float(), rtol=2.0 ** -6, atol=1e-6)


def test_offsets_past_32_bits():
    # 17,000 rows of 128,256 logits: 2.18e9 values, 4.4 GB
    T, V = 17000, 128256
    say("offsets past 32 bits")
    z = torch.zeros((T, V), dtype=BF, device=DEV)
    y = torch.full((T,), -100, dtype=torch.int64, device=DEV)
    z[T - 1, 5], z[0, 9], z[T - 3, V - 1] = 3.0, 2.0, 4.0
    y[T - 1], y[0], y[T - 3], y[T // 2] = 5, 9, V - 1, 1
    rows = [0, T // 2, T - 3, T - 1]
    ref, p = oloss.token_logprobs(_np(z[rows]), _np(y[rows]).astype(int))
    logp, stats = q.qlora_token_logprobs(z, y, return_stats=True)
    _check_logp(logp[rows], ref, V)
    cu = torch.tensor([0, T // 2, T], dtype=torch.int32, device=DEV)
    want = oloss.token_logprobs_bwd(p, _np(y[rows]).astype(int), -np.full(4, 0.25))
    o = q.qlora_policy_loss(z, y, cu, torch.ones(2, device=DEV), dlogits=z)
    assert o.dlogits is z
    _check_grad(z[rows], want, np.full(4, 0.25), V, 1e-6)
    assert not z[1:T // 2].any() and not z[T - 2].any()


def test_a_training_step_end_to_end():
    """A head whose input is an adapted linear with an 8-bit checkpoint: the
    reference policy's log-probabilities with the adapters at zero, the
    preference loss, its backward through the head into the adapters and one
    optimiser step; the adapters' gradients against differences of the loss."""
    say("training step")
    g = torch.Generator().manual_seed(9)
    M, K, N, V, r = 48, 128, 192, 500, 8
    W, _ = q.qlora_quantize_nf4((torch.randn((N, K), generator=g) * 0.1).to(DEV))
    X = torch.randn((M, K), generator=g).to(BF).to(DEV)
    A = (torch.randn((r, K), generator=g) * 0.1).to(BF).to(DEV)
    B = (torch.randn((N, r), generator=g) * 0.1).to(BF).to(DEV)
    H = (torch.randn((V, N), generator=g) * 0.2).to(DEV)
    y = torch.randint(0, V, (M,), generator=g).to(DEV)
    y[::5] = -100
    cu = torch.tensor([0, 11, 24, 36, 48], dtype=torch.int32, device=DEV)
    base = q.QLoRALinearFn.apply(X, A, torch.zeros_like(B), W, 16.0).float() @ H.T
    ref = q.qlora_token_logprobs(base, y)

    def loss_of(a, b):
        h = q.QLoRALinearFn.apply(X, a, b, W, 16.0, None, True)
        return q.PreferenceLossFn.apply(h.float() @ H.T, y, cu, ref, 0.3)[0]

    a, b = A.clone().requires_grad_(), B.clone().requires_grad_()
    loss_of(a, b).backward()
    # float64 differences of the whole step along the gradient itself
    f = lambda t: host(t).double()  # noqa: E731
    Wd = f(q.qlora_dequantize_nf4(W, torch.float32))

    def loss64(a64, b64):
        h = f(X) @ Wd.T + 16.0 / r * (f(X) @ a64.T) @ b64.T
        o = oloss.preference((h @ f(H).T).numpy(), _np(y).astype(int), _np(cu).astype(int), _np(ref),
                             0.3)
        return o["loss"]

    for i, leaf in enumerate((a, b)):
        d = f(leaf.grad)
        d = d / d.norm()
        pt = [f(A), f(B)]
        up, dn = list(pt), list(pt)
        up[i], dn[i] = pt[i] + 1e-5 * d, pt[i] - 1e-5 * d
        slope = (loss64(*up) - loss64(*dn)) / 2e-5
        # bf16 activations, logits' inputs and gradients: a few steps of 2^-8
        assert float(f(leaf.grad).norm()) == pytest.approx(slope, rel=0.05)
    masters = []
    for leaf in (a, b):
        p = leaf.detach().float()
        masters.append((p, leaf.grad.float(), torch.zeros_like(p), torch.zeros_like(p),
                        leaf.detach()))
    before = [leaf.detach().clone() for leaf in (a, b)]
    q.qlora_adamw_step(masters, 1, 1e-2)
    assert all(not torch.equal(u, v.detach()) for u, v in zip(before, (a, b)))
    assert all(torch.isfinite(v).all() for v in (a, b))


@pytest.mark.parametrize("lens,lead,tail,V,dtype", [
    ([131, 0, 127], 0, 3, 12003, F32), ([150, 107], 1, 0, 16384, BF), ([150, 107], 0, 0, 16376, BF)])
@pytest.mark.parametrize("reduction,kl,token_adv,old", [("token", 0.05, True, True),
                                                        ("sequence", 0.0, False, False)])
def test_policy_where_one_pass_begins(lens, lead, tail, V, dtype, reduction, kl, token_adv, old):
    test_policy(lens, lead, tail, V, dtype, reduction, kl, token_adv, old)


def test_policy_in_one_pass_replayed():
    say("policy loss in one pass: graph")
    T, V = 300, 17000
    z, y, cu = _packed(9, [T // 2, 0, T // 2], 0, 0, V, BF)
    adv = torch.tensor([0.5, 1.0, -1.5], device=DEV)
    lp = q.qlora_token_logprobs(z, y)

    def step():
        b = q.qlora_policy_loss(z, y, cu, adv, lp + 0.1, lp - 0.2, kl_coef=0.1, return_grad=True)
        return [b.loss, b.kl, b.clip_frac, b.logp, b.dlogits]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        for t in out:
            t.fill_(7)
        torch.randn(1 << 18, device=DEV).sum().item()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want, out))
        assert all(torch.equal(u, v) for u, v in zip(want, step()))
