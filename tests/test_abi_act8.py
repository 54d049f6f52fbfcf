"""Refusals of the 8-bit checkpoint calls on the host (no GPU needed): every
bad argument comes back as a status, or raises in the binding, before anything
is launched."""
import ctypes

import pytest
import torch

import bit_quantized_lora_quant_amd as q

P = ctypes.c_void_p
FAKE = 0x100000


def _a8(rows=64, cols=128, codes=FAKE, scale=FAKE):
    return q.Act8Descriptor(rows, cols, codes, scale)


@pytest.mark.parametrize("a,want", [
    (_a8(rows=-1), "INVALID_ARG"), (_a8(cols=0), "INVALID_ARG"), (_a8(codes=0), "INVALID_ARG"),
    (_a8(scale=0), "INVALID_ARG"), (_a8(codes=FAKE + 8), "INVALID_ARG"),
    (_a8(scale=FAKE + 4), "INVALID_ARG"), (_a8(cols=96), "UNSUPPORTED"),
    (_a8(cols=(1 << 26) + 64), "UNSUPPORTED"), (_a8(rows=1 << 62, cols=64), "UNSUPPORTED"),
    (_a8(rows=(1 << 31) + 1, cols=64), "UNSUPPORTED")])
def test_bad_checkpoints(a, want):
    want = getattr(q, "QLORA_ERR_" + want)
    assert q.lib().qlora_act8_quantize(P(FAKE), ctypes.byref(a), None) == want
    assert q.lib().qlora_act8_dequantize(ctypes.byref(a), q.QLORA_BF16, P(FAKE), None) == want


def test_quantize_and_dequantize_pointers():
    lib, a = q.lib(), _a8()
    assert lib.qlora_act8_quantize(None, ctypes.byref(a), None) == q.QLORA_ERR_INVALID_ARG
    assert lib.qlora_act8_quantize(P(FAKE + 2), ctypes.byref(a), None) == q.QLORA_ERR_INVALID_ARG
    assert lib.qlora_act8_quantize(P(FAKE), None, None) == q.QLORA_ERR_INVALID_ARG
    assert lib.qlora_act8_dequantize(ctypes.byref(a), 7, P(FAKE), None) == q.QLORA_ERR_INVALID_ARG
    assert lib.qlora_act8_dequantize(ctypes.byref(a), 0, None, None) == q.QLORA_ERR_INVALID_ARG
    none = _a8(rows=0, codes=0, scale=0)
    assert lib.qlora_act8_quantize(None, ctypes.byref(none), None) == q.QLORA_OK
    assert lib.qlora_act8_dequantize(ctypes.byref(none), 0, None, None) == q.QLORA_OK


def _bwd(W, a, r=8, XA=FAKE, dY=FAKE, ws_bytes=1 << 30, alpha=16.0, p=None, dA=FAKE):
    dr = q.QloraDropout(p, 1) if p is not None else None
    return q.lib().qlora_linear_bwd_act8(
        ctypes.byref(W), ctypes.byref(a), P(FAKE), P(FAKE), r, ctypes.c_float(alpha),
        ctypes.byref(dr) if dr else None, None, P(dY) if dY else None, P(XA) if XA else None,
        P(FAKE), P(dA) if dA else None, P(FAKE), P(FAKE), ws_bytes, None)


def test_linear_backward_refusals():
    W = q.NF4Descriptor(256, 128, 64, 256, FAKE, FAKE, FAKE, FAKE)
    bad = q.QLORA_ERR_INVALID_ARG
    assert _bwd(W, _a8(), XA=None) == bad
    assert _bwd(W, _a8(cols=192)) == bad          # another width than the weight's
    assert _bwd(W, _a8(rows=0)) == bad
    assert _bwd(W, _a8(codes=0)) == bad
    assert _bwd(W, _a8(), r=0) == bad
    assert _bwd(W, _a8(), r=129) == bad
    assert _bwd(W, _a8(), dY=FAKE + 2) == bad
    assert _bwd(W, _a8(), dA=None) == bad
    assert _bwd(W, _a8(), p=1.0) == bad
    assert _bwd(W, _a8(), alpha=float("nan")) == bad
    need = q.qlora_linear_act8_workspace_bytes(64, 256, 128, 8)
    assert need > q.qlora_linear_workspace_bytes(64, 256, 128, 8)
    assert _bwd(W, _a8(), ws_bytes=need - 1) == q.QLORA_ERR_WORKSPACE
    assert q.qlora_linear_act8_workspace_bytes(64, 256, 128, 129) == 0
    assert q.qlora_linear_act8_workspace_bytes(1 << 20, 64, 1 << 12, 8) == 0
    rows = (ctypes.c_int64 * 2)(128, 127)
    a = _a8()
    assert q.lib().qlora_grouped_bwd_act8(
        ctypes.byref(W), ctypes.byref(a), P(FAKE), P(FAKE), 8, 2, rows, ctypes.c_float(1.0),
        P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), 1 << 30, None) == bad


def _raises(fn, *args, **kw):
    with pytest.raises(q.QloraError) as e:
        fn(*args, **kw)
    assert e.value.status == q.QLORA_ERR_INVALID_ARG


def test_binding_refusals():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    _raises(q.qlora_act8_quantize, x)                              # on the host
    _raises(q.qlora_act8_quantize, x.float())
    _raises(q.qlora_act8_quantize, x[:, ::2])
    _raises(q.qlora_act8_quantize, x, q.Act8Tensor(4, 64, "cpu"))
    _raises(q.Act8Tensor, 4, 96, "cpu")
    _raises(q.Act8Tensor, 4, 128, codes=torch.zeros(4, 64, dtype=torch.int8))
    _raises(q.Act8Tensor, 4, 128, "cpu", scale=torch.zeros(2, 4))
    a = q.Act8Tensor(4, 128, "cpu")
    assert a.scale.shape == (2, 32) and a.nbytes() == 4 * 128 + 2 * 32 * 4
    _raises(q.qlora_act8_dequantize, a)
    _raises(q.qlora_act8_dequantize, a, out=torch.zeros(4, 64))
    W = q.NF4Tensor(256, 128, "cpu")
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    good = dict(q=W, a=a, A=b(8, 128), B=b(256, 8), alpha=1.0, dY=b(4, 256), XA_in=b(4, 8))
    _raises(q.qlora_linear_bwd_act8, **good)                       # on the host
    for name, v in (("A", b(8, 64)), ("B", b(256, 4)), ("dY", b(5, 256)), ("XA_in", b(4, 4)),
                    ("dY", b(4, 512)[:, ::2]), ("dA", b(8, 128)), ("dX", torch.zeros(4, 128)),
                    ("keep_bits", torch.zeros(3, dtype=torch.uint8)), ("XA_in", None)):
        _raises(q.qlora_linear_bwd_act8, **{**good, name: v})


@pytest.mark.parametrize("rows,cols", [(1 << 29, 64), ((1 << 29) - 31, 64), (1 << 29, 256),
                                       (1 << 28, 320), (1 << 28, 512), (1 << 31, 64)])
def test_checkpoints_of_more_tiles_than_a_launch_has(rows, cols):
    # below the limit of values, but 2^24 or more tiles of 32 rows x 256 columns,
    # a workgroup of 256 threads each: refused, where a launch would fail
    assert rows * cols <= 1 << 37
    a = _a8(rows=rows, cols=cols)
    assert q.lib().qlora_act8_quantize(P(FAKE), ctypes.byref(a), None) == q.QLORA_ERR_UNSUPPORTED
    for out in (q.QLORA_BF16, q.QLORA_F32):
        assert q.lib().qlora_act8_dequantize(ctypes.byref(a), out, P(FAKE), None) == \
            q.QLORA_ERR_UNSUPPORTED


def test_strided_keep_bits_are_refused():
    W, a = q.NF4Tensor(256, 128, "cpu"), q.Act8Tensor(4, 128, "cpu")
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    for bits in (torch.zeros(128, dtype=torch.uint8)[::2], torch.zeros(1, dtype=torch.uint8).expand(64)):
        with pytest.raises(q.QloraError, match="keep_bits"):
            q.qlora_linear_bwd_act8(W, a, b(8, 128), b(256, 8), 1.0, b(4, 256), b(4, 8),
                                    dropout=(0.1, 1), keep_bits=bits)
