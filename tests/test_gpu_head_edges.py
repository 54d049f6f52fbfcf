"""The language-model head without logits where it can go wrong: special values in
rows that take no part, labels past the vocabulary, nearly certain targets, extreme
logits, several panels, offsets past 32 bits, gradients in place and in wider
buffers, no rows, other streams, graphs, autograd, and a training step from
the adapters through the head to their update."""
import math

import numpy as np
import pytest
import torch
from torch.utils.checkpoint import checkpoint

from gpu_common import DEV, host, say
from oracle import head as ohead
from test_gpu_head import BF, F32, _check_grad, _exact, _inputs, _logp_tol, _np

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V", [(40, 300), (300, 1000)])
def test_rows_without_target_may_hold_anything(T, V):
    say("masked rows with NaN and infinities T=%d V=%d" % (T, V))
    h, W, y = _inputs(1, T, 128, V, ignored=0.4)
    clean = h.clone()
    off = y < 0
    h[off] = torch.tensor([math.nan, math.inf, -math.inf, 3e38], device=DEV,
                          dtype=BF).repeat(32)
    clean[off] = 0
    for f in (lambda x: q.qlora_head_cross_entropy(x, W, y, return_grad=True),
              lambda x: q.qlora_head_cross_entropy(x, W, y, return_grad=True, need_dweight=True)):
        a, b = f(h), f(clean)
        assert torch.isfinite(a.loss) and torch.equal(a.loss, b.loss)
        assert torch.equal(a.logp, b.logp) and torch.equal(a.dhidden, b.dhidden)
        assert a.dweight is None or torch.equal(a.dweight, b.dweight)
        assert not a.dhidden[off].any()
    # a weight of 0 leaves a row out as well, whatever it and the upstream gradient hold
    logp, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    w = torch.ones(T, device=DEV)
    zero = (~off).nonzero()[::3, 0]
    w[zero] = 0
    dh, dw = q.qlora_head_logprobs_bwd(clean, W, y, stats, w, need_dweight=True)
    h[zero] = math.nan
    stats[zero] = math.nan
    dh2, dw2 = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dweight=True)
    assert torch.equal(dh, dh2) and torch.equal(dw, dw2) and not dh[zero].any()
    g = torch.tensor([math.inf], device=DEV)
    dh3, _ = q.qlora_head_logprobs_bwd(h, W, y, stats, w, grad_scale=g)
    assert not dh3[zero].any() and not dh3[off].any()


def test_nothing_to_predict():
    say("no targets, no rows")
    h, W, y = _inputs(2, 70, 64, 300)
    y[:] = -100
    h[:] = math.nan
    o = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=True)
    assert float(o.loss) == 0 and not o.logp.any() and not o.dhidden.any() and not o.dweight.any()
    o = q.qlora_head_cross_entropy(h, W, y, "sum", return_grad=True)
    assert float(o.loss) == 0 and not o.dhidden.any()
    logp, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    assert not logp.any() and not stats.any()
    none = h[:0], W, y[:0]
    o = q.qlora_head_cross_entropy(*none, return_grad=True, need_dweight=True)
    assert float(o.loss) == 0 and o.dhidden.shape == (0, 64) and not o.dweight.any()
    assert q.qlora_head_logprobs(*none).shape == (0,)
    dh, dw = q.qlora_head_logprobs_bwd(*none, torch.zeros((0, 2), device=DEV),
                                       torch.zeros(0, device=DEV), need_dweight=True)
    assert dh.shape == (0, 64) and not dw.any()


@pytest.mark.parametrize("V", [1, 64, 255, 256, 257, 1000])
def test_labels_at_and_past_the_end(V):
    say("labels past the vocabulary V=%d" % V)
    h, W, y = _inputs(3, 90, 64, V, ignored=0)
    y[0], y[1], y[2], y[3], y[4] = V - 1, 0, V, V + 255, 1 << 40
    bad = slice(2, 5)
    ok = torch.ones(90, dtype=torch.bool)
    ok[bad] = False
    logp, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    ref, _ = ohead.logprobs(_np(h), _np(W), _np(y).astype(int))
    assert torch.isnan(logp[bad]).all() and np.isnan(ref[bad]).all()
    assert np.max(np.abs(_np(logp) - ref)[ok.numpy()]) <= _logp_tol(64, V)
    good = q.qlora_head_cross_entropy(h[ok.to(DEV)], W, y[ok.to(DEV)], "sum", return_grad=True)
    for dw in (False, True):
        o = q.qlora_head_cross_entropy(h, W, y, "sum", return_grad=True, need_dweight=dw)
        assert torch.isnan(o.loss) and torch.isnan(o.dhidden[bad]).all()
        assert torch.isfinite(o.dhidden[ok.to(DEV)]).all()
        if not dw:
            assert torch.equal(o.dhidden[ok.to(DEV)], good.dhidden)
        else:
            assert torch.isnan(o.dweight).all()
    w = torch.ones(90, device=DEV)
    dh, dw = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dweight=True)
    assert torch.isnan(dh[bad]).all() and torch.isfinite(dh[ok.to(DEV)]).all()
    assert torch.isnan(dw).all()
    w[bad] = 0
    dh, dw = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dweight=True)
    assert not dh[bad].any() and torch.isfinite(dw).all()


def test_special_hidden_and_weight():
    say("NaN and infinities in rows with a target")
    h, W, y = _inputs(4, 20, 64, 300, ignored=0)
    h[3, 7], h[5, 0] = math.nan, math.inf
    for dw in (False, True):
        o = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=dw)
        rest = torch.ones(20, dtype=torch.bool, device=DEV)
        rest[3] = rest[5] = False
        assert torch.isnan(o.logp[[3, 5]]).all() and torch.isfinite(o.logp[rest]).all()
        assert torch.isnan(o.dhidden[[3, 5]]).all() and torch.isfinite(o.dhidden[rest]).all()
        assert torch.isnan(o.loss)
    W[17, 3] = math.nan
    logp = q.qlora_head_logprobs(h, W, y)
    assert torch.isnan(logp).all()


@pytest.mark.parametrize("dw", [False, True])
@pytest.mark.parametrize("margin", [12.0, 25.0, 60.0, 300.0])
def test_nearly_certain_targets(margin, dw):
    """1 - p far below float32's step of p: the gradient keeps its relative size."""
    say("margin %g dweight=%s" % (margin, dw))
    h, W, y = _inputs(5, 33, 128, 700, ignored=0, sharp=0)
    Wf = W.float()
    h = (h.float() * 0.3 + margin * Wf[y] / Wf[y].pow(2).sum(1, keepdim=True)).to(BF)
    w = torch.full((33,), -1.0, device=DEV, dtype=torch.float64)
    ref, d, dh_ref, dw_ref = _exact(h, W, y, w)
    o = q.qlora_head_cross_entropy(h, W, y, "sum", return_grad=True, need_dweight=dw)
    # (logits as large as the margin: their float32 sums decide what is left beside 1)
    slack = _logp_tol(128, 700, 2 * margin + 30)
    assert float((o.logp.double() - ref).abs().max()) <= slack
    norm, err = dh_ref.norm(dim=1), (o.dhidden.double() - dh_ref).norm(dim=1)
    tiny = norm < 1e-30    # below bf16's range for the outputs' elements
    assert bool((err[~tiny] <= (6e-3 + 2 * slack) * norm[~tiny]).all())
    assert bool((o.dhidden.double().norm(dim=1)[tiny] <= 2e-30).all())


@pytest.mark.parametrize("scale", [1e-3, 30.0, 1e4, 1e15])
def test_extreme_logits(scale):
    say("logits of %g" % scale)
    h, W, y = _inputs(6, 50, 64, 500, sharp=0)
    h = (h.float() * scale).to(BF)
    for dw in (False, True):
        o = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=dw)
        ref, _ = _exact(h, W, y)
        z = float(ref.abs().max())
        assert torch.isfinite(o.loss) and torch.isfinite(o.dhidden).all()
        assert float((o.logp.double() - ref).abs().max()) <= _logp_tol(64, 500, 3 * z + 30)
        assert not dw or torch.isfinite(o.dweight).all()


def test_all_logits_equal():
    say("equal logits")
    h, W, y = _inputs(7, 30, 64, 1000, ignored=0)
    h[:] = 0
    o = q.qlora_head_cross_entropy(h, W, y, return_grad=True)
    assert float((o.logp + math.log(1000)).abs().max()) < 1e-5
    _, d, dh, _ = _exact(h, W, y, torch.full((30,), -1 / 30, device=DEV))
    _check_grad(o.dhidden, d, W.double(), dh, 1000)


@pytest.mark.parametrize("T,D,V", [(5000, 64, 262144), (2300, 128, 262000)])
def test_several_panels(T, D, V):
    """2048 rows of 262144 are a panel: rows, loss and both gradients go over panels
    that their targets do not fill."""
    say("panels T=%d D=%d V=%d" % (T, D, V))
    h, W, y = _inputs(8, T, D, V, ignored=0.35)
    n = int((y >= 0).sum())
    assert n > 2048 or T < 3000
    ref = torch.zeros(T, dtype=torch.float64, device=DEV)
    dh_ref = torch.zeros((T, D), dtype=torch.float64, device=DEV)
    dw_ref = torch.zeros((V, D), dtype=torch.float64, device=DEV)
    for i in range(0, T, 512):
        s = slice(i, i + 512)
        w = torch.full((len(y[s]),), -1.0 / n, device=DEV, dtype=torch.float64)
        ref[s], _, dh_ref[s], part = _exact(h[s], W, y[s], w)
        dw_ref += part
    o = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=True)
    alone = q.qlora_head_cross_entropy(h, W, y, return_grad=True)
    logp, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    assert torch.equal(logp, o.logp) and torch.equal(logp, alone.logp)
    assert float((logp.double() - ref).abs().max()) <= _logp_tol(D, V)
    assert abs(float(o.loss) + float(ref.sum()) / n) <= _logp_tol(D, V)
    dh, dw = q.qlora_head_logprobs_bwd(h, W, y, stats, torch.full((T,), -1.0 / n, device=DEV),
                                       need_dweight=True)
    for got, want in ((o.dhidden, dh_ref), (alone.dhidden, dh_ref), (dh, dh_ref),
                      (o.dweight, dw_ref), (dw, dw_ref)):
        assert float((got.double() - want).norm() / want.norm()) < 4e-3
        assert not (got is not o.dweight and got is not dw) or not got[y < 0].any()


def test_offsets_past_32_bits():
    say("row strides of 2^22 - 8 values")
    h, W, y = _inputs(9, 600, 64, 700)
    ld = (1 << 22) - 8
    o = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=True)
    wide = torch.empty((700, ld), dtype=BF, device=DEV)
    hw, ww = wide[:600, 8:72], wide[:, 128:192]
    hw.copy_(h), ww.copy_(W)
    dh, dw = wide[:600, 256:320], wide[:, 512:576]
    wide[:, 504:512] = 7
    wide[:, 576:584] = 7
    p = q.qlora_head_cross_entropy(hw, ww, y, return_grad=True, need_dweight=True, dhidden=dh,
                                   dweight=dw)
    assert torch.equal(o.loss, p.loss) and torch.equal(o.logp, p.logp)
    assert torch.equal(o.dhidden, dh) and torch.equal(o.dweight, dw)
    assert (wide[:, 504:512] == 7).all() and (wide[:, 576:584] == 7).all()


def test_gradient_in_place_of_hidden():
    say("dhidden over hidden")
    h, W, y = _inputs(10, 150, 128, 900, pad=16)
    want = q.qlora_head_cross_entropy(h, W, y, return_grad=True)
    both = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=True)
    logp, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    w = torch.linspace(-1, 1, 150, device=DEV)
    bwd, _ = q.qlora_head_logprobs_bwd(h, W, y, stats, w)
    for f, ref in ((lambda x: q.qlora_head_cross_entropy(x, W, y, dhidden=x).dhidden, want.dhidden),
                   (lambda x: q.qlora_head_cross_entropy(x, W, y, dhidden=x,
                                                         need_dweight=True).dhidden, both.dhidden),
                   (lambda x: q.qlora_head_logprobs_bwd(x, W, y, stats, w, dhidden=x)[0], bwd)):
        full = torch.full((150, 144), 3.0, dtype=BF, device=DEV)
        x = full[:, :128]
        x.copy_(h)
        assert f(x) is x and torch.equal(x, ref) and (full[:, 128:] == 3).all()


def test_two_streams_at_once():
    say("two calls on two streams")
    a, b = _inputs(11, 500, 256, 3000), _inputs(12, 90, 128, 5000)
    ref = [q.qlora_head_cross_entropy(*x, return_grad=True, need_dweight=True) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    out = []
    for _ in range(3):
        for s, x in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                out.append(q.qlora_head_cross_entropy(*x, return_grad=True, need_dweight=True))
    torch.cuda.synchronize()
    for i, o in enumerate(out):
        for got, want in zip(o, ref[i % 2]):
            assert torch.equal(got, want)


def test_graph_replays_follow_their_inputs():
    """Replays with other masks: how many rows there are is known on the GPU alone."""
    say("graph of cross entropy and weighted backward")
    h, W, y = _inputs(13, 400, 128, 2000)
    w = torch.linspace(-1, 1, 400, device=DEV)
    ws = q.workspace(q.qlora_head_workspace_bytes(h, W, y, True, True), DEV)
    dh, dw = torch.empty_like(h), torch.empty_like(W)
    dh2 = torch.empty_like(h)
    logp = torch.empty(400, device=DEV)
    stats = torch.empty((400, 2), device=DEV)
    keep = {}

    def run():
        keep["o"] = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=True,
                                               dhidden=dh, dweight=dw, ws=ws)
        q.qlora_head_logprobs(h, W, y, logp=logp, stats=stats, ws=ws)
        q.qlora_head_logprobs_bwd(h, W, y, stats, w, dhidden=dh2, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for i, ignored in enumerate((0.0, 0.5, 0.9, 1.0)):
        h2, W2, y2 = _inputs(20 + i, 400, 128, 2000, ignored=ignored)
        h.copy_(h2), W.copy_(W2), y.copy_(y2)
        for t in (dh, dw, dh2, logp, stats):
            t.view(torch.uint8).fill_(0xA5)
        torch.randn(1 << 20, device=DEV).sum().item()
        g.replay()
        torch.cuda.synchronize()
        o = q.qlora_head_cross_entropy(h2, W2, y2, return_grad=True, need_dweight=True)
        lp, st = q.qlora_head_logprobs(h2, W2, y2, return_stats=True)
        d2, _ = q.qlora_head_logprobs_bwd(h2, W2, y2, st, w)
        assert torch.equal(keep["o"].loss, o.loss) and torch.equal(dh, o.dhidden)
        assert torch.equal(dw, o.dweight) and torch.equal(logp, lp) and torch.equal(stats, st)
        assert torch.equal(dh2, d2)


# ------------------------------------------------------------------ autograd
def _leaves(seed, T=60, D=64, V=300):
    h, W, y = _inputs(seed, T, D, V)
    return h.requires_grad_(), W.requires_grad_(), y


@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_cross_entropy_function(reduction):
    say("HeadCrossEntropyFn %s" % reduction)
    h, W, y = _leaves(30)
    ref = q.qlora_head_cross_entropy(h.detach(), W.detach(), y, reduction, return_grad=True,
                                     need_dweight=True)
    loss, logp = q.HeadCrossEntropyFn.apply(h, W, y, reduction)
    assert torch.equal(loss, ref.loss) and torch.equal(logp, ref.logp) and not logp.requires_grad
    loss.backward(retain_graph=True)
    assert torch.equal(h.grad, ref.dhidden) and torch.equal(W.grad, ref.dweight)
    h.grad = W.grad = None
    (loss / 3).backward()               # the saved gradients are as they were
    third = torch.tensor(1 / 3, device=DEV)
    assert torch.equal(h.grad, (ref.dhidden.float() * third).to(BF))
    assert torch.equal(W.grad, (ref.dweight.float() * third).to(BF))
    frozen, _ = q.HeadCrossEntropyFn.apply(h, W.detach(), y, reduction)
    h.grad = None
    frozen.backward()
    alone = q.qlora_head_cross_entropy(h.detach(), W.detach(), y, reduction, return_grad=True)
    assert torch.equal(h.grad, alone.dhidden)
    with torch.no_grad():
        loss, _ = q.HeadCrossEntropyFn.apply(h, W, y, reduction)
    assert not loss.requires_grad and torch.equal(loss, ref.loss)


def test_logprobs_function():
    say("HeadLogprobsFn")
    h, W, y = _leaves(31)
    w = torch.linspace(-2, 2, 60, device=DEV)
    logp = q.HeadLogprobsFn.apply(h, W, y)
    (logp * w).sum().backward()
    _, stats = q.qlora_head_logprobs(h.detach(), W.detach(), y, return_stats=True)
    dh, dw = q.qlora_head_logprobs_bwd(h.detach(), W.detach(), y, stats, w, need_dweight=True)
    assert torch.equal(h.grad, dh) and torch.equal(W.grad, dw)


def _loss(name, h, W, y):
    if name == "logprobs":
        return (q.HeadLogprobsFn.apply(h, W, y) ** 2).sum()
    return q.HeadCrossEntropyFn.apply(h, W, y)[0]


@pytest.mark.parametrize("name", ["logprobs", "cross entropy"])
def test_second_derivatives_are_refused(name):
    say("twice: head %s" % name)
    h, W, y = _leaves(32)
    first = torch.autograd.grad(_loss(name, h, W, y), (h, W))
    twice = torch.autograd.grad(_loss(name, h, W, y), (h, W), create_graph=True)
    for a, b in zip(first, twice):
        assert torch.equal(a, b.detach())
    for b in twice:
        with pytest.raises(RuntimeError):
            torch.autograd.grad((b.float() ** 2).sum(), (h, W), retain_graph=True)


@pytest.mark.parametrize("name", ["logprobs", "cross entropy"])
def test_recomputed_and_offloaded(name):
    say("recomputed: head %s" % name)
    h, W, y = _leaves(33)

    def grads(run):
        h.grad = W.grad = None
        loss = run(h, W)
        loss.backward()
        return loss.detach(), h.grad, W.grad

    f = lambda a, b: _loss(name, a, b, y)  # noqa: E731
    want = grads(f)
    for reentrant in (False, True):
        got = grads(lambda a, b: checkpoint(f, a, b, use_reentrant=reentrant))
        assert all(torch.equal(u, v) for u, v in zip(want, got))
    with torch.autograd.graph.save_on_cpu():
        h.grad = W.grad = None
        loss = f(h, W)
    loss.backward()
    assert torch.equal(h.grad, want[1]) and torch.equal(W.grad, want[2])


def test_a_supervised_step_from_end_to_end():
    """An adapted linear under the head's cross entropy, its backward into the
    adapters and their orthogonalised update; the adapters' gradients against
    differences of the loss in float64, the update against the oracle."""
    from oracle import muon as omuon
    say("supervised step")
    g = torch.Generator().manual_seed(9)
    M, K, N, V, r = 70, 128, 192, 500, 8
    W, _ = q.qlora_quantize_nf4((torch.randn((N, K), generator=g) * 0.1).to(DEV))
    X = torch.randn((M, K), generator=g).to(BF).to(DEV)
    A = (torch.randn((r, K), generator=g) * 0.1).to(BF).to(DEV)
    B = (torch.randn((N, r), generator=g) * 0.1).to(BF).to(DEV)
    H = (torch.randn((V, N), generator=g) * 0.2).to(BF).to(DEV)
    y = torch.randint(0, V, (M,), generator=g).to(DEV)
    y[::5] = -100
    a, b = A.clone().requires_grad_(), B.clone().requires_grad_()
    h = q.QLoRALinearFn.apply(X, a, b, W, 16.0, None, True)
    loss, _ = q.HeadCrossEntropyFn.apply(h, H, y)
    loss.backward()
    f = lambda t: host(t).double()  # noqa: E731
    Wd = f(q.qlora_dequantize_nf4(W, torch.float32))

    def loss64(a64, b64):
        h = f(X) @ Wd.T + 16.0 / r * (f(X) @ a64.T) @ b64.T
        return ohead.cross_entropy(h.numpy(), f(H).numpy(), _np(y).astype(int))[0]

    for i, leaf in enumerate((a, b)):
        d = f(leaf.grad)
        d = d / d.norm()
        up, dn = [f(A), f(B)], [f(A), f(B)]
        up[i], dn[i] = up[i] + 1e-5 * d, dn[i] - 1e-5 * d
        slope = (loss64(*up) - loss64(*dn)) / 2e-5
        # bf16 activations, gradients and products' inputs: a few steps of 2^-8
        assert float(f(leaf.grad).norm()) == pytest.approx(slope, rel=0.05)
    masters = [p.detach().float() for p in (a, b)]
    moments = [torch.zeros_like(p) for p in masters]
    plan = q.MuonPlan([(p, leaf.grad, m, leaf.detach()) for p, leaf, m in
                       zip(masters, (a, b), moments)])
    want = []
    for p, leaf in zip(masters, (a, b)):
        u = np.float32(1 - 0.95) * host(leaf.grad).float().numpy()
        u = np.float32(0.95) * u + np.float32(1 - 0.95) * host(leaf.grad).float().numpy()
        o = omuon.orthogonalize(u)
        want.append(_np(p) - 0.02 * omuon.factor("shape", *p.shape) * o)
    q.qlora_muon_step(plan, 0.02)
    for p, leaf, ref in zip(masters, (a, b), want):
        assert np.max(np.abs(_np(p) - ref)) <= 1e-6 * np.max(np.abs(ref))
        assert torch.equal(leaf.detach(), p.to(BF))


@pytest.mark.parametrize("T,D,V", [(1500, 64, 9000), (2300, 128, 20001), (900, 192, 16128),
                                   (3000, 256, 5000)])
def test_tall_tiles_of_few_steps(T, D, V):
    """Tiles of 256 rows whose inner index is one to four steps long."""
    say("tall tiles T=%d D=%d V=%d" % (T, D, V))
    h, W, y = _inputs(T, T, D, V, ignored=0.05)
    w = torch.linspace(-1, 1, T, device=DEV)
    ref, d, dh_ref, dw_ref = _exact(h, W, y, w)
    masked = torch.where((y >= 0)[:, None], h.double(), 0.0)
    logp, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    assert float((logp.double() - ref).abs().max()) <= _logp_tol(D, V)
    dh, dw = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dweight=True)
    _check_grad(dh, d, W.double(), dh_ref, V)
    _check_grad(dw, d.T.contiguous(), masked, dw_ref, T)
    n = int((y >= 0).sum())
    _, d, dh_ref, dw_ref = _exact(h, W, y, torch.full((T,), -1.0 / n, device=DEV))
    o = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=True)
    assert torch.equal(o.logp, logp)
    _check_grad(o.dhidden, d, W.double(), dh_ref, V)
    _check_grad(o.dweight, d.T.contiguous(), masked, dw_ref, T)
    only = q.qlora_head_cross_entropy(h, W, y, return_grad=True)
    assert torch.equal(only.logp, logp)
    _check_grad(only.dhidden, d, W.double(), dh_ref, V)


@pytest.mark.parametrize("times", [1, 2, 255, 256, 257, 700])
@pytest.mark.parametrize("V", [90, 700, 9000])
def test_one_label_many_times(times, V):
    """The same target in many rows, up to where their roundings are left to average."""
    say("one label %d times, V=%d" % (times, V))
    h, W, y = _inputs(41, 720, 128, V, ignored=0.1, sharp=0.3)
    y[torch.randperm(720, generator=torch.Generator().manual_seed(times))[:times].to(DEV)] = 7
    n = int((y >= 0).sum())
    _, d, _, dw_ref = _exact(h, W, y, torch.full((720,), -1.0 / n, device=DEV))
    masked = torch.where((y >= 0)[:, None], h.double(), 0.0)
    o = q.qlora_head_cross_entropy(h, W, y, need_dweight=True)
    _check_grad(o.dweight, d.T.contiguous(), masked, dw_ref, 720)
    _, stats = q.qlora_head_logprobs(h, W, y, return_stats=True)
    w = torch.full((720,), -1.0 / n, device=DEV)
    dw = q.qlora_head_logprobs_bwd(h, W, y, stats, w, need_dhidden=False, need_dweight=True)[1]
    _check_grad(dw, d.T.contiguous(), masked, dw_ref, 720)


def test_labels_and_weights_of_one_call_in_another():
    """A workspace that held another call's rows, slices and labels leaves nothing in
    the next one's results."""
    say("one workspace for calls of several sizes")
    cases = [_inputs(50, 900, 256, 9000), _inputs(51, 3, 64, 300), _inputs(52, 300, 128, 2000)]
    ws = torch.full((max(q.qlora_head_workspace_bytes(*x, True, True) for x in cases),), 255,
                    dtype=torch.uint8, device=DEV)
    for h, W, y in cases + cases[::-1]:
        a = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=True)
        b = q.qlora_head_cross_entropy(h, W, y, return_grad=True, need_dweight=True, ws=ws)
        c = q.qlora_head_cross_entropy(h, W, y, return_grad=True)
        d = q.qlora_head_cross_entropy(h, W, y, return_grad=True, ws=ws)
        for x, z in ((a, b), (c, d)):
            assert torch.equal(x.loss, z.loss) and torch.equal(x.logp, z.logp)
            assert torch.equal(x.dhidden, z.dhidden)
        assert torch.equal(a.dweight, b.dweight)
