"""What a call of the orthogonalised update writes, it reads as nothing else: refused on the
host (no GPU needed)."""
import contextlib

import pytest
import torch

import bit_quantized_lora_quant_amd as q


def test_outputs_of_the_wrong_shape():
    x = torch.zeros(4, 50)
    for out in (x[0], x.new_zeros(()), x.unsqueeze(0), torch.zeros(4, 50, 1)):
        with pytest.raises(q.QloraError):
            q.qlora_orthogonalize([x], out=[out])


def test_an_output_that_is_another_matrix():
    """Its matrix may still be read when the first one's result is written."""
    x, y, z = (torch.zeros(4, 50) for _ in range(3))
    for ms, out in (([x, y], [y, x]), ([x, y], [y, z]), ([x, y], [z, x]), ([x, x], [x, z]),
                    ([x, x], [z, x]), ([x, y, z], [x, z, y])):
        with pytest.raises(q.QloraError, match="another matrix"):
            q.qlora_orthogonalize(ms, out=out)
    e = torch.zeros(0, 5)
    for ms, out in (([x, y], [x, y]), ([x, x], [y, z]), ([x, y], [x, z]), ([e, x, e], [e, x, e])):
        with pytest.raises(q.QloraError, match="GPU|devices"):       # for the host only
            q.qlora_orthogonalize(ms, out=out)


def test_a_gradient_that_is_written():
    """The update reads gradients again when momenta and parameters are written."""
    x, y, z, w = (torch.zeros(4, 50) for _ in range(4))
    b = x.bfloat16()
    for bad in ([(x, x, z, None)], [(x, z, z, None)], [(x, b, z, b)],
                [(x, y, z, None), (w, z, y.clone(), None)],
                [(x, y, z, None), (w, x, y.clone(), None)]):
        with pytest.raises(q.QloraError, match="gradient"):
            q.MuonPlan(bad)


def test_a_new_gradient_that_is_written(monkeypatch):
    monkeypatch.setattr(q, "_on", lambda *a: contextlib.nullcontext())
    x, y, z, w, e = [torch.zeros(4, 50) for _ in range(4)] + [torch.zeros(0, 5)]
    plan = q.MuonPlan([(x, y, z, None), (e, e, e, None)])
    plan._bind("bind", None)
    plan._bind("bind", [w, e])
    for bad in (x, z):
        with pytest.raises(q.QloraError, match="gradient"):
            plan._bind("bind", [bad, e])
    x.data = w.data                          # the parameter moves to where the gradient lies
    with pytest.raises(q.QloraError, match="gradient"):
        plan._bind("bind", None)
    plan._bind("bind", [y, e])
    assert plan.array[0].grad == y.data_ptr() and plan.array[0].param == w.data_ptr()
