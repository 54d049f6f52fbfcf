"""GPU parity of the 8-bit activation checkpoints and of the linear backward
that reads them: codes, scales and values bit for bit against the oracle;
dA and dB within a float32 accumulation bound of the float64 gradients for
the given checkpoint; dX as the plain backward's; dropout, grouping, ragged
shapes, other streams, graph replays and the autograd wrapper."""
import numpy as np
import pytest
import torch

from gpu_common import DEV, assert_close, bf16_np, host, oracle, say, to_dev
from oracle import act8 as oact
from oracle import dropout as odrop

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu
U = 2.0 ** -24      # half a step of float32
BF = torch.bfloat16


def _acts(seed, M, K, scale=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp(rng.standard_normal((1, K))) * scale
    return torch.from_numpy(x.astype(np.float32)).to(BF)


def _same(a, b):
    a, b = (np.asarray(v, dtype=np.float32) for v in (a, b))
    nan = np.isnan(a)
    assert np.array_equal(nan, np.isnan(b))
    assert np.array_equal(a.view(np.uint32)[~nan], b.view(np.uint32)[~nan])


def _round_trip(x):
    a = q.qlora_act8_quantize(x.to(DEV))
    codes, scale = oact.quantize(bf16_np(x))
    assert np.array_equal(host(a.codes).numpy(), codes)
    _same(host(a.scale).numpy(), scale)
    with np.errstate(invalid="ignore"):
        ref = oact.dequantize(codes, scale)
    _same(host(q.qlora_act8_dequantize(a, torch.float32)).numpy(), ref)
    _same(host(q.qlora_act8_dequantize(a)).float().numpy(),
          torch.from_numpy(ref).to(BF).float().numpy())


@pytest.mark.parametrize("M,K", [(1, 64), (3, 192), (31, 64), (32, 128), (33, 4160), (100, 320),
                                 (257, 1024), (2, 22016), (4096, 64), (1000, 704)])
def test_round_trip_bit_exact(M, K):
    say("act8 round trip %dx%d" % (M, K))
    _round_trip(_acts(M * 7 + K, M, K))


@pytest.mark.parametrize("scale", [2.0 ** -130, 2.0 ** -126, 2.0 ** -70, 2.0 ** 60, 2.0 ** 123])
def test_round_trip_far_magnitudes(scale):
    say("act8 magnitudes %g" % scale)
    x = torch.from_numpy(np.random.default_rng(5).uniform(-1, 1, (37, 128)).astype(np.float32))
    _round_trip((x.double() * scale).float().to(BF))


def test_every_quotient_next_to_a_half():
    # all 128 mantissas against all 128 maxima of one binade, and the binades below
    say("act8 ties")
    mant = torch.arange(128, 256, dtype=torch.float32)
    rows = []
    for a in mant:
        for sh in (1, 2, 4, 8, 64):
            v = mant / sh
            v = torch.where(v > a, -v / 2, v)
            rows += [torch.cat((a[None], v[:63])), torch.cat((a[None], v[63:126])),
                     torch.cat((a[None], v[65:128]))]
    x = torch.stack(rows).to(BF)
    assert torch.equal(x.float(), torch.stack(rows))
    _round_trip(x)


def test_special_blocks():
    say("act8 special blocks")
    x = _acts(9, 35, 256)
    x[0] = 0
    x[1, 3], x[2, 70], x[3, 130], x[34, 255] = float("inf"), float("nan"), float("-inf"), float("nan")
    x[4, :64] = -0.0
    x[5, 64:128] = torch.finfo(BF).max
    x[6, 64:128] = torch.finfo(BF).min
    _round_trip(x)


def test_buffers_and_no_rows():
    say("act8 no rows, given buffers")
    a = q.qlora_act8_quantize(torch.zeros((0, 64), dtype=BF, device=DEV))
    assert q.qlora_act8_dequantize(a).shape == (0, 64)
    x = _acts(1, 40, 128).to(DEV)
    kept = torch.full((40 * 128 + 64,), 77, dtype=torch.int8, device=DEV)
    scale = torch.full((2 * 64 + 16,), 5.0, device=DEV)
    a = q.Act8Tensor(40, 128, codes=kept[:40 * 128].view(40, 128), scale=scale[:128].view(2, 64))
    q.qlora_act8_quantize(x, a)
    assert (kept[40 * 128:] == 77).all() and (scale[128:] == 5.0).all()


# ----------------------------------------------------------------- backward
def _bwd_case(seed, M, N, K, r, groups=None):
    rng = np.random.default_rng(seed)
    G = len(groups) if groups else 1
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    x = _acts(seed + 1, M, K)
    t = lambda v: torch.from_numpy(v.astype(np.float32)).to(BF)  # noqa: E731
    A = t(rng.uniform(-1, 1, (G * r, K)) / np.sqrt(K))
    B = t(rng.standard_normal((N, G * r)) * 0.05)
    if groups:
        at = 0
        for i, n in enumerate(groups):
            B[at:at + n, :i * r] = 0
            B[at:at + n, (i + 1) * r:] = 0
            at += n
    return w, x, A, B, t(rng.standard_normal((M, N))), t(rng.standard_normal((M, G * r)))


def _check_adapters(a, A, B, dY, XA, alpha, r, dA, dB, keep=None, p=0.0, diag=None):
    """dA and dB against float64.  G = dY B adds N float32 terms, dA M of its
    products; scale and product round once each, the two-part split of G scale
    leaves at most 2^-16 of it: every bound is a multiple of the sum of
    absolute terms."""
    f = lambda v: host(v).double().numpy()  # noqa: E731
    codes, scale = host(a.codes).double().numpy(), host(a.scale).double().numpy()
    M, K = codes.shape
    N = dY.shape[1]
    x = (codes.reshape(M, K // 64, 64) * scale[:, :M].T[..., None]).reshape(M, K)
    if keep is not None:
        x = x * keep / (1 - p)
    s = alpha / r
    dy, b, xa = f(dY), f(B), f(XA)
    G = dy @ b
    bound = s * (np.abs(dy) @ np.abs(b)).T @ np.abs(x) * (2.0 ** -16 + (M + N + 16) * U)
    ref = s * G.T @ x
    got = f(dA)
    assert np.all(np.abs(got - ref) <= bound), float(np.max(np.abs(got - ref) - bound))
    # and as a whole to float32 grade
    assert np.linalg.norm(got - ref) <= 2e-5 * np.linalg.norm(ref) + 1e-30
    refB = s * dy.T @ xa
    boundB = s * np.abs(dy).T @ np.abs(xa) * (M + 16) * U
    if diag is not None:
        refB, boundB = refB * diag, boundB * diag
    assert np.all(np.abs(f(dB) - refB) <= boundB)


SHAPES = [  # M, N, K, r, need_dx
    (1, 32, 64, 1, True), (1, 64, 128, 8, False), (5, 72, 64, 3, True), (16, 256, 192, 16, True),
    (33, 100, 128, 16, False), (64, 249, 320, 17, False), (128, 1024, 1024, 8, True),
    (331, 512, 704, 32, True), (700, 320, 448, 64, True), (513, 264, 1088, 128, True),
    (2048, 256, 512, 16, False), (1100, 1000, 128, 40, True), (4100, 64, 64, 4, False),
]


@pytest.mark.parametrize("M,N,K,r,need_dx", SHAPES)
def test_backward(M, N, K, r, need_dx):
    say("bwd act8 M=%d N=%d K=%d r=%d dx=%s" % (M, N, K, r, need_dx))
    w, x, A, B, dY, XA = _bwd_case(M + N + K, M, N, K, r)
    W, _ = q.qlora_quantize_nf4(to_dev(w))
    A, B, dY, XA = (t.to(DEV) for t in (A, B, dY, XA))
    a = q.qlora_act8_quantize(x.to(DEV))
    dX, dA, dB = q.qlora_linear_bwd_act8(W, a, A, B, 16.0, dY, XA, need_dx=need_dx)
    _check_adapters(a, A, B, dY, XA, 16.0, r, dA, dB)
    again = q.qlora_linear_bwd_act8(W, a, A, B, 16.0, dY, XA, need_dx=need_dx)
    assert torch.equal(dA, again[1]) and torch.equal(dB, again[2])
    if need_dx:      # does not read X: the plain backward's, bit for bit
        plain = q.qlora_linear_bwd(W, x.to(DEV), A, B, 16.0, dY, XA_in=XA)[0]
        assert torch.equal(dX, plain)


@pytest.mark.parametrize("M,N,K,r,p,bits", [
    (1, 64, 64, 4, 0.5, True), (37, 96, 128, 8, 0.1, True), (37, 96, 128, 8, 0.1, False),
    (600, 320, 704, 64, 0.05, True), (600, 320, 704, 64, 0.05, False),
    (513, 264, 320, 128, 0.3, False), (64, 64, 192, 16, 0.0, False)])
def test_backward_dropout(M, N, K, r, p, bits):
    say("bwd act8 dropout M=%d N=%d K=%d r=%d p=%g bits=%s" % (M, N, K, r, p, bits))
    w, x, A, B, dY, XA = _bwd_case(M * 3 + K, M, N, K, r)
    W, _ = q.qlora_quantize_nf4(to_dev(w))
    A, B, dY, XA = (t.to(DEV) for t in (A, B, dY, XA))
    drop = (p, 1234567)
    keep = odrop.keep_mask(M, K, p, drop[1]).astype(np.float64)
    kb = None
    if bits:
        kb = to_dev(np.packbits(keep.astype(np.uint8).reshape(-1), bitorder="little"))
    a = q.qlora_act8_quantize(x.to(DEV))
    dX, dA, dB = q.qlora_linear_bwd_act8(W, a, A, B, 16.0, dY, XA, dropout=drop, keep_bits=kb)
    _check_adapters(a, A, B, dY, XA, 16.0, r, dA, dB, keep, p)
    plain = q.qlora_linear_bwd(W, x.to(DEV), A, B, 16.0, dY, XA_in=XA, dropout=drop, keep_bits=kb)
    assert torch.equal(dX, plain[0])


@pytest.mark.parametrize("M,K,groups,r", [(3, 64, (32, 40), 4), (200, 704, (256, 64, 64), 16),
                                          (600, 320, (128, 128), 64), (70, 128, (96,) * 8, 16)])
def test_grouped_backward(M, K, groups, r):
    say("bwd act8 grouped M=%d K=%d groups=%s r=%d" % (M, K, groups, r))
    N, R = sum(groups), r * len(groups)
    w, x, A, B, dY, XA = _bwd_case(M + K, M, N, K, r, groups)
    W, _ = q.qlora_quantize_nf4(to_dev(w))
    A, B, dY, XA = (t.to(DEV) for t in (A, B, dY, XA))
    a = q.qlora_act8_quantize(x.to(DEV))
    dX, dA, dB = q.qlora_grouped_bwd_act8(W, a, A, B, r, groups, 16.0, dY, XA)
    diag, at = np.zeros((N, R)), 0
    for i, n in enumerate(groups):
        diag[at:at + n, i * r:(i + 1) * r] = 1
        at += n
    _check_adapters(a, A, B, dY, XA, 16.0, r, dA, dB, diag=diag)
    assert not host(dB).numpy()[diag == 0].any()
    assert torch.equal(dX, q.qlora_grouped_bwd(W, x.to(DEV), A, B, r, groups, 16.0, dY, XA)[0])


@pytest.mark.parametrize("quant_type,double_quant", [("int4", True), ("nf4", False)])
def test_backward_other_weights(quant_type, double_quant):
    say("bwd act8 %s dq=%s" % (quant_type, double_quant))
    w, x, A, B, dY, XA = _bwd_case(77, 100, 128, 192, 8)
    W, _ = q.qlora_quantize_nf4(to_dev(w), quant_type=quant_type, double_quant=double_quant)
    A, B, dY, XA = (t.to(DEV) for t in (A, B, dY, XA))
    a = q.qlora_act8_quantize(x.to(DEV))
    dX, dA, dB = q.qlora_linear_bwd_act8(W, a, A, B, 16.0, dY, XA)
    _check_adapters(a, A, B, dY, XA, 16.0, 8, dA, dB)
    assert torch.equal(dX, q.qlora_linear_bwd(W, x.to(DEV), A, B, 16.0, dY, XA_in=XA)[0])


def test_a_bad_value_reaches_the_gradient_of_its_block_only():
    say("bwd act8 NaN")
    w, x, A, B, dY, XA = _bwd_case(5, 70, 64, 256, 8)
    x[69, 130] = float("nan")
    W, _ = q.qlora_quantize_nf4(to_dev(w))
    A, B, dY, XA = (t.to(DEV) for t in (A, B, dY, XA))
    a = q.qlora_act8_quantize(x.to(DEV))
    dA = host(q.qlora_linear_bwd_act8(W, a, A, B, 16.0, dY, XA, need_dx=False)[1])
    assert torch.isnan(dA[:, 128:192]).all()
    assert torch.isfinite(dA[:, :128]).all() and torch.isfinite(dA[:, 192:]).all()


def test_another_stream_and_graph_replays():
    say("bwd act8 stream and graph")
    w, x, A, B, dY, XA = _bwd_case(6, 300, 192, 320, 16)
    W, _ = q.qlora_quantize_nf4(to_dev(w))
    x, A, B, dY, XA = (t.to(DEV) for t in (x, A, B, dY, XA))
    a = q.qlora_act8_quantize(x)
    ref = [a.codes.clone(), a.scale.clone()] + list(q.qlora_linear_bwd_act8(W, a, A, B, 8.0, dY, XA))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = q.qlora_act8_quantize(x)
        got = [b.codes, b.scale] + list(q.qlora_linear_bwd_act8(W, b, A, B, 8.0, dY, XA))
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(ref, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = q.qlora_act8_quantize(x)
        out = [c.codes, c.scale] + list(q.qlora_linear_bwd_act8(W, c, A, B, 8.0, dY, XA))
    for _ in range(3):
        for t in out:
            t.view(torch.uint8).fill_(0xA5)
        torch.randn(1 << 18, device=DEV).sum().item()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(ref, out))


@pytest.mark.parametrize("dropout", [None, (0.1, 99)])
def test_autograd_from_a_checkpoint(dropout):
    say("autograd act8 dropout=%s" % (dropout,))
    w, x, A, B, dY, _ = _bwd_case(8, 130, 192, 256, 16)
    W, _ = q.qlora_quantize_nf4(to_dev(w))
    x, A, B, dY = (t.to(DEV) for t in (x, A, B, dY))
    grads = {}
    for mode in (None, True, "shared"):
        X, a, b = (t.clone().requires_grad_() for t in (x, A, B))
        act8 = q.qlora_act8_quantize(x) if mode == "shared" else mode
        Y = q.QLoRALinearFn.apply(X, a, b, W, 16.0, dropout, act8)
        Y.backward(dY)
        grads[mode] = (Y.detach(), X.grad, a.grad, b.grad)
    for u, v in zip(grads[True], grads["shared"]):
        assert torch.equal(u, v)
    plain, kept = grads[None], grads[True]
    assert torch.equal(plain[0], kept[0]) and torch.equal(plain[1], kept[1])
    assert torch.equal(plain[3], kept[3])
    # dA from x^: each value off by at most half a step of its block, a / 254
    keep = odrop.keep_mask(130, 256, *dropout).astype(np.float64) / (1 - dropout[0]) \
        if dropout else 1.0
    xs = bf16_np(x)
    step = np.repeat(np.abs(xs.reshape(130, 4, 64)).max(2) / 254, 64, axis=1) * keep
    G = np.abs(bf16_np(dY) @ bf16_np(B))
    ref = oracle.linear_bwd(oracle.dequantize(oracle.quantize(w)).reshape(w.shape), xs * keep,
                            bf16_np(A), bf16_np(B), 16.0, bf16_np(dY))[1]
    got = bf16_np(kept[2])
    bound = G.T @ step + 2.0 ** -8 * np.abs(ref) + 1e-4 * (G.T @ np.abs(xs * keep))
    assert np.all(np.abs(got - ref) <= bound)


def test_checkpoint_of_another_shape_is_refused():
    say("autograd act8 refusal")
    W, _ = q.qlora_quantize_nf4(torch.zeros((64, 128), device=DEV))
    t = lambda *s: torch.zeros(s, dtype=BF, device=DEV)  # noqa: E731
    with pytest.raises(q.QloraError):
        q.QLoRALinearFn.apply(t(32, 128), t(4, 128), t(64, 4), W, 1.0, None,
                              q.qlora_act8_quantize(t(31, 128)))
