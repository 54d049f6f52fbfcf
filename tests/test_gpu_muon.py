"""GPU parity of the orthogonalised update against the float64 oracle: ranks from 1
to 128 on either side, odd sizes and strides, both types, ill-conditioned and
special values, batches over several launches, in place, streams and graphs."""
import math

import numpy as np
import pytest
import torch

from gpu_common import DEV, host, say
from oracle import muon as omuon

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _np(t):
    return host(t).double().numpy()


def _matrix(seed, rows, cols, dtype=F32, pad=0, decay=2.0, offset=0):
    """Singular values over `decay` decades, in rows of cols + pad values."""
    g = torch.Generator().manual_seed(seed)
    k, n = min(rows, cols), max(rows, cols)
    mix = torch.randn((k, k), generator=g) * torch.logspace(0, -decay, k)
    x = mix @ torch.randn((k, n), generator=g) * 1e-3
    x = x if rows <= cols else x.T
    flat = torch.full((offset + rows * (cols + pad),), 7.0, dtype=dtype, device=DEV)
    m = flat[offset:].view(rows, cols + pad)[:, :cols]
    m.copy_(x.to(dtype))
    return m


def _check(got, ref, dtype):
    """The steps run in float64: products of two float32 values are exact in it, a sum
    of n of them is off by n 2^-53 of the largest eigenvalue, and the polynomial's
    slope is below 2 a^14 < 7e7 there: 22016 2^-53 7e7 < 2e-4 of 2^-20 ... so what
    shows is the one rounding of the result, and 2^-30 of it all."""
    half = torch.finfo(dtype).eps / 2
    err = np.abs(_np(got) - ref)
    assert np.all(err <= half * np.abs(ref) + 2.0 ** -27 * np.max(np.abs(ref), initial=0)), \
        float(np.max(err - half * np.abs(ref)))


SHAPES = [(1, 1), (1, 7), (7, 1), (2, 3), (8, 1024), (1024, 8), (16, 16), (16, 4097), (4097, 16),
          (5, 333), (333, 5), (17, 500), (500, 17), (32, 32), (32, 1000), (1001, 31), (33, 64),
          (48, 700), (700, 50), (64, 2048), (2049, 64), (65, 130), (100, 999), (1003, 127),
          (128, 128), (128, 5000), (4096, 128)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_orthogonalize(rows, cols, dtype):
    say("orthogonalize %d x %d %s" % (rows, cols, dtype))
    m = _matrix(rows + cols, rows, cols, dtype)
    ref = omuon.orthogonalize(_np(m))
    out, = q.qlora_orthogonalize([m])
    assert out.dtype == dtype and out.shape == m.shape
    _check(out, ref, dtype)
    assert torch.equal(out, q.qlora_orthogonalize([m])[0])


@pytest.mark.parametrize("rows,cols,pad,offset", [(16, 1000, 24, 0), (1000, 16, 16, 0),
                                                  (16, 1001, 3, 1), (999, 12, 5, 3),
                                                  (64, 515, 1, 2), (520, 40, 24, 4)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides_and_in_place(rows, cols, pad, offset, dtype):
    say("orthogonalize strided %d x %d + %d at %d %s" % (rows, cols, pad, offset, dtype))
    m = _matrix(1, rows, cols, dtype, pad, offset=offset)
    ref = omuon.orthogonalize(_np(m))
    plain, = q.qlora_orthogonalize([m.contiguous()])
    wide = torch.full((rows, cols + 9), 5.0, dtype=dtype, device=DEV)
    q.qlora_orthogonalize([m], out=[wide[:, 2:2 + cols]])
    _check(wide[:, 2:2 + cols], ref, dtype)
    assert torch.equal(wide[:, 2:2 + cols], plain)
    assert (wide[:, :2] == 5).all() and (wide[:, 2 + cols:] == 5).all()
    q.qlora_orthogonalize([m], out=[m])
    assert torch.equal(m, plain)
    assert (torch.as_strided(m, (rows - 1, pad), (m.stride(0), 1),
                             m.storage_offset() + cols) == 7).all()


@pytest.mark.parametrize("decay", [0.0, 4.0, 8.0])
@pytest.mark.parametrize("rows,cols", [(8, 700), (600, 64), (128, 900)])
def test_condition(rows, cols, decay):
    say("condition 1e%g of %d x %d" % (decay, rows, cols))
    m = _matrix(2, rows, cols, decay=decay)
    _check(q.qlora_orthogonalize([m])[0], omuon.orthogonalize(_np(m)), F32)


def test_steps_coefficients_and_eps():
    m = _matrix(3, 12, 300)
    for kw in (dict(steps=1), dict(steps=2), dict(steps=32, coefficients=(1.5, -0.5, 0.0)),
               dict(eps=10.0), dict(steps=8, coefficients=(2.0, -1.5, 0.5))):
        say("orthogonalize %s" % kw)
        _check(q.qlora_orthogonalize([m], **kw)[0], omuon.orthogonalize(_np(m), **kw), F32)


def test_special_values():
    ms = [torch.zeros((8, 100), device=DEV), _matrix(4, 8, 100), _matrix(5, 8, 100),
          _matrix(6, 100, 8), torch.full((4, 50), 1e-30, device=DEV),
          torch.full((50, 4), 3e38, device=DEV), torch.ones((3, 0), device=DEV),
          torch.ones((0, 3), device=DEV), _matrix(7, 300, 9)]
    ms[1][3, 17] = math.nan
    ms[2][0, 99] = math.inf
    ms[3][99, 7] = -math.inf
    say("special values")
    out = q.qlora_orthogonalize(ms)
    assert not out[0].any()
    assert all(torch.isnan(out[i]).all() for i in (1, 2, 3))
    for i in (4, 5, 8):
        _check(out[i], omuon.orthogonalize(_np(ms[i])), F32)
    assert out[6].shape == (3, 0) and out[7].shape == (0, 3)
    assert q.qlora_orthogonalize([]) == []


def test_block_diagonal_stays_so():
    """The zeros off a grouped B's blocks are exact."""
    m = torch.zeros((96, 24), device=DEV)
    m[:40, :8], m[40:64, 8:16], m[64:, 16:] = (_matrix(8, 40, 8), _matrix(9, 24, 8),
                                               _matrix(10, 32, 8))
    say("block diagonal")
    o, = q.qlora_orthogonalize([m])
    assert torch.equal(o == 0, m == 0)
    _check(o, omuon.orthogonalize(_np(m)), F32)


def _tensors(shapes, seed=0, grad=F32, pads=None, half=True):
    out = []
    for i, (rows, cols) in enumerate(shapes):
        pad = (pads or [0])[i % len(pads or [0])]
        p = _matrix(seed + 4 * i, rows, cols, pad=pad)
        p.mul_(20)
        g = _matrix(seed + 4 * i + 1, rows, cols, grad, pad=pad)
        m = _matrix(seed + 4 * i + 2, rows, cols, pad=0)
        pb = _matrix(seed + 4 * i + 3, rows, cols, BF, pad=pad) if half else None
        out.append((p, g, m, pb))
    return out


def _expect(p, g, m, lr, mu, nesterov, wd, adjust):
    """p in float64 from the momentum and update as float32 makes them."""
    f = np.float32
    p, g, m = (host(t).float().numpy() for t in (p, g, m))
    a, b = f(mu), f(1 - mu)
    m = a * m + b * g
    u = a * m + b * g if nesterov else m
    o = omuon.orthogonalize(u)
    scale = lr * omuon.factor(adjust, *p.shape)
    ref = p.astype(np.float64) * (1 - lr * wd) - scale * o
    # roundings of decay, scale, O, two products and the difference
    tol = 2.0 ** -24 * (3 * np.abs(p) + 4 * scale * np.abs(o) + np.abs(ref)) + scale * 2.0 ** -27
    return m, ref, tol


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("adjust", ["shape", "rms", None])
@pytest.mark.parametrize("grad", [F32, BF])
def test_step(nesterov, adjust, grad):
    shapes = [(8, 1024), (1024, 8), (64, 300), (1, 50), (50, 1), (333, 30), (130, 128), (16, 4100)]
    say("step nesterov=%s adjust=%s grad=%s" % (nesterov, adjust, grad))
    ts = _tensors(shapes, grad=grad, pads=[0, 8, 3])
    ts[3] = ts[3][:3] + (None,)
    ref = [_expect(p, g, m, 0.02, 0.95, nesterov, 0.1, adjust) for p, g, m, _ in ts]
    q.qlora_muon_step(ts, 0.02, nesterov=nesterov, weight_decay=0.1, adjust=adjust)
    for (p, _, m, pb), (m_ref, p_ref, tol) in zip(ts, ref):
        assert np.array_equal(host(m).numpy(), m_ref)
        assert np.all(np.abs(_np(p) - p_ref) <= tol)
        assert pb is None or torch.equal(pb, p.to(BF))


def test_many_tensors_over_launches_and_steps():
    """113 tensors of all ranks in three launches, three steps of one plan, against
    one tensor at a time; new gradients each step; what lies between rows stays."""
    rng = np.random.default_rng(5)
    shapes = []
    for i in range(113):
        r, n = int(rng.integers(1, 129)), int(rng.integers(1, 900))
        shapes.append((r, n) if i % 2 else (n, r))
    say("113 tensors")
    one, all_ = _tensors(shapes, pads=[0, 5]), _tensors(shapes, pads=[0, 5])
    plan = q.MuonPlan(all_)
    for k in range(3):
        grads = [_matrix(1000 * k + i, *s, pad=[0, 5][i % 2]) for i, s in enumerate(shapes)]
        q.qlora_muon_step(plan, 0.01 + k, weight_decay=0.01, grads=grads)
        for t, g in zip(one, grads):
            q.qlora_muon_step([(t[0], g, t[2], t[3])], 0.01 + k, weight_decay=0.01)
    for a, b, (rows, cols) in zip(one, all_, shapes):
        for x, y in ((a[0], b[0]), (a[2], b[2]), (a[3], b[3])):
            # (the slices, and so the order of sums, hang on the call's size)
            assert torch.allclose(x.float(), y.float(), rtol=2.0 ** -7, atol=1e-6)
        pad = b[0].stride(0) - cols
        if rows > 1 and pad > 0:
            between = torch.as_strided(b[0], (rows - 1, pad), (b[0].stride(0), 1), cols)
            assert (between == 140).all() or (between == 7).all()


def test_plan_follows_its_tensors():
    say("plan with moved memory")
    t, = _tensors([(8, 100)])
    same = [x.clone() for x in t]
    plan = q.MuonPlan([t])
    q.qlora_muon_step(plan, 0.1)
    q.qlora_muon_step([tuple(same)], 0.1)
    g = _matrix(77, 8, 100)
    t[1].data = g
    q.qlora_muon_step(plan, 0.1)
    q.qlora_muon_step([(same[0], g, same[2], same[3])], 0.1)
    assert torch.equal(t[0], same[0]) and torch.equal(t[2], same[2])
    for bad in (g.to(BF), g[:, :50], g.T.contiguous().T, g.cpu()):
        with pytest.raises(q.QloraError):
            q.qlora_muon_step(plan, 0.1, grads=[bad])
    with pytest.raises(q.QloraError):
        q.qlora_muon_step(plan, 0.1, grads=[])
    q.qlora_muon_step(plan, 0.1, grads=[g])


def test_other_stream_and_graph():
    say("muon on another stream and from a graph")
    base = _tensors([(16, 700), (900, 16), (64, 200)])
    ref = [tuple(x.clone() for x in t) for t in base]
    for _ in range(4):
        q.qlora_muon_step(ref, 0.05)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan = q.MuonPlan(base)
    with torch.cuda.stream(side):
        q.qlora_muon_step(plan, 0.05)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qlora_muon_step(plan, 0.05)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        torch.ones(1000, device=DEV).sum()
    for a, b in zip(base, ref):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])


def test_plan_dropped_while_another_stream_runs():
    """The workspace of a plan is not handed out again while a step of it on another
    stream than the one it was made on still runs."""
    say("muon plan dropped behind a step on another stream")
    base = _tensors([(64, 4000)] * 3)
    ref = [tuple(x.clone() for x in t) for t in base]
    q.qlora_muon_step(ref, 0.05)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    plan = q.MuonPlan(base)
    n = plan.ws.numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        x = torch.ones((4096, 4096), device=DEV)
        for _ in range(40):                      # the step waits its turn behind these
            x = x @ x * 2.0 ** -12
        q.qlora_muon_step(plan, 0.05)
    del plan
    junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    for a, b in zip(base, ref):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    del junk


# up to four chunks of 4096 padded elements, where a workgroup takes a matrix whole, and
# one more long index, where none does
SMALL = [(16, 1024), (1024, 16), (32, 512), (511, 32), (3, 257), (769, 5), (1, 1), (20, 129)]


@pytest.mark.parametrize("count", [1, 8, 45, 46])
@pytest.mark.parametrize("more", [0, 1])
def test_small_matrices(count, more):
    say("%d small matrices, %d more" % (count, more))
    shapes = [SMALL[i % 8] for i in range(count)]
    if more:
        shapes[0] = (16, 1025)
    ts = _tensors(shapes, pads=[0, 4, 1])
    us = [_matrix(7 + i, *s, pad=i % 3, dtype=BF if i % 2 else F32) for i, s in enumerate(shapes)]
    ref = [_expect(p, g, m, 0.3, 0.9, True, 0.1, "rms") for p, g, m, _ in ts]
    for u, o in zip(us, q.qlora_orthogonalize(us)):
        _check(o, omuon.orthogonalize(_np(u)), u.dtype)
    q.qlora_muon_step(ts, 0.3, 0.9, weight_decay=0.1, adjust="rms")
    for (p, _, m, pb), (m_ref, p_ref, tol) in zip(ts, ref):
        assert np.array_equal(host(m).numpy(), m_ref)
        assert np.all(np.abs(_np(p) - p_ref) <= tol)
        assert torch.equal(pb, p.to(BF))
    for (p, _, _, _), (rows, cols) in zip(ts, shapes):
        pad = p.stride(0) - cols
        if rows > 1 and pad > 0:     # (the values were drawn as 7 and multiplied by 20)
            between = torch.as_strided(p, (rows - 1, pad), (p.stride(0), 1), cols)
            assert (between == 7).all()
    again = q.qlora_orthogonalize(us)
    q.qlora_orthogonalize(us, out=us)
    assert all(torch.equal(a, b) for a, b in zip(us, again))


def test_new_gradients_where_the_last_ones_lay():
    """Gradients of another type or shape are refused also at the last ones' addresses,
    and a refusal leaves the plan as it was."""
    say("muon gradients at one address")
    ts = _tensors([(8, 100), (60, 16)])
    ref = [tuple(x.clone() for x in t) for t in ts]
    plan = q.MuonPlan(ts)
    flat = [torch.zeros(4000, device=DEV) for _ in ts]
    good = [f[:t[1].numel()].view(t[1].shape) for f, t in zip(flat, ts)]
    for k in range(3):
        new = [_matrix(90 + 2 * k + i, *t[1].shape) for i, t in enumerate(ts)]
        for f, g in zip(good, new):
            f.copy_(g)
        # (new tensor objects at one place each step)
        q.qlora_muon_step(plan, 0.1, grads=[x.view(x.shape) for x in good])
        q.qlora_muon_step([(t[0], g, t[2], t[3]) for t, g in zip(ref, new)], 0.1)
        for bad in (flat[0].view(BF)[:800].view(8, 100), flat[0][:1600].view(8, 200)[:, :100]):
            with pytest.raises(q.QloraError):
                q.qlora_muon_step(plan, 0.1, grads=[bad, good[1]])
        for a, b in zip(ts, ref):
            assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    assert [g.data_ptr() for _, g, _, _ in plan.tensors] == [g.data_ptr() for g in good]
