"""The backward from an 8-bit checkpoint at every number of rank tiles, with and
without dX, to float32 accuracy as a whole: what a split of its products into
fewer than three bf16 parts would not reach."""
import numpy as np
import pytest
import torch

from gpu_common import DEV, host, say, to_dev
from oracle import dropout as odrop
from test_gpu_act8 import _bwd_case

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu


def _reference(a, B, dY, XA, s, keep):
    f = lambda v: host(v).double().numpy()  # noqa: E731
    M, K = a.codes.shape
    x = f(a.codes).reshape(M, K // 64, 64) * f(a.scale)[:, :M].T[..., None]
    x = x.reshape(M, K) * keep
    return s * (f(dY) @ f(B)).T @ x, s * f(dY).T @ f(XA)


@pytest.mark.parametrize("need_dx", [False, True])
@pytest.mark.parametrize("M,N,K,r", [
    (300, 128, 192, 65), (257, 512, 320, 96), (700, 1024, 704, 128), (1, 64, 64, 128),
    (1030, 320, 64, 100), (64, 250, 128, 127),        # (250: G not through the staged kernel)
    (700, 512, 448, 64), (513, 256, 704, 33), (640, 1024, 256, 16), (33, 192, 128, 1)])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_adapter_gradients_to_float32_accuracy(M, N, K, r, need_dx, p):
    """In norm: three bf16 parts hold a product's 24 bits, and float32 sums of
    N / 32 and 3 M / 32 matrix instructions round each by 2^-24 at random, under
    1e-6 at these sizes."""
    say("act8 ranks M=%d N=%d K=%d r=%d dx=%s p=%g" % (M, N, K, r, need_dx, p))
    w, x, A, B, dY, XA = _bwd_case(M + N + K + r, M, N, K, r)
    W, _ = q.qlora_quantize_nf4(to_dev(w))
    A, B, dY, XA = (t.to(DEV) for t in (A, B, dY, XA))
    a = q.qlora_act8_quantize(x.to(DEV))
    drop = (p, 77) if p else None
    keep = odrop.keep_mask(M, K, p, 77).astype(np.float64) / (1 - p) if p else 1.0
    dX, dA, dB = q.qlora_linear_bwd_act8(W, a, A, B, 16.0, dY, XA, need_dx=need_dx, dropout=drop)
    refA, refB = _reference(a, B, dY, XA, 16.0 / r, keep)
    for got, ref in ((dA, refA), (dB, refB)):
        err = np.linalg.norm(host(got).double().numpy() - ref)
        assert err <= 1e-6 * np.linalg.norm(ref), err / np.linalg.norm(ref)
    plain = q.qlora_linear_bwd(W, x.to(DEV), A, B, 16.0, dY, XA_in=XA, need_dx=need_dx, dropout=drop)
    assert torch.equal(dB, plain[2])
    assert dX is None or torch.equal(dX, plain[0])


def test_a_bad_block_under_dropout():
    """A block's infinity or NaN is its scale's NaN, which no mask takes out: all of
    its columns of dA are NaN, dropped elements or not, and no others."""
    say("act8 NaN under dropout")
    w, x, A, B, dY, XA = _bwd_case(5, 70, 64, 256, 8)
    x[69, 130] = float("inf")
    W, _ = q.qlora_quantize_nf4(to_dev(w))
    A, B, dY, XA = (t.to(DEV) for t in (A, B, dY, XA))
    a = q.qlora_act8_quantize(x.to(DEV))
    dA = host(q.qlora_linear_bwd_act8(W, a, A, B, 16.0, dY, XA, need_dx=False, dropout=(0.5, 3))[1])
    assert torch.isnan(dA[:, 128:192]).all()
    assert torch.isfinite(dA[:, :128]).all() and torch.isfinite(dA[:, 192:]).all()
