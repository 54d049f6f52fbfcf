"""What a MuonPlan finds anew each step, on the host with the check for a GPU left out
(no GPU needed): a tensor that was laid out otherwise in its place is refused."""
import contextlib

import pytest
import torch

import bit_quantized_lora_quant_amd as q

BF = torch.bfloat16


@pytest.fixture(params=["torch's table", "one by one"])
def plan(request, monkeypatch):
    """A plan of a wide and a tall matrix whose rows lie in wider ones, bound once; its
    tensors looked at through torch's table of functions or from Python."""
    if request.param == "one by one":
        monkeypatch.setattr(q, "_exchange", lambda: None)
    monkeypatch.setattr(q, "_on", lambda *a: contextlib.nullcontext())
    bufs = [torch.zeros(4096) for _ in range(6)] + [torch.zeros(4096, dtype=BF) for _ in range(2)]
    wide, tall = [(b[:16 * 40].view(16, 40)[:8, :20]) for b in bufs[0:6:2] + bufs[6:7]], \
        [(b[:50 * 24].view(50, 24)[:, :8]) for b in bufs[1:6:2] + bufs[7:]]
    p = q.MuonPlan([tuple(wide), tuple(tall)])
    p._bind("bind", None)
    p._bind("bind", None)
    return p


OTHER = {
    "rows": lambda t: t[:-1],
    "columns": lambda t: t[:, :-1],
    "stride": lambda t: torch.as_strided(t, t.shape, (t.stride(0) + 4, 1)),
    "transposed": lambda t: t.t(),
    "shape of as many values": lambda t: torch.as_strided(t, (t.shape[0] * 2, t.shape[1] // 2),
                                                          t.stride()),
    "type": lambda t: torch.as_strided(t.new_empty(0).to(t.dtype).set_(t.untyped_storage())
                                       .view(torch.int32 if t.dtype != BF else torch.float16),
                                       t.shape, t.stride()),
}


@pytest.mark.parametrize("how", OTHER)
@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("tensor", range(2))
def test_laid_out_otherwise_in_its_place(plan, tensor, which, how):
    t = plan.tensors[tensor][which]
    at, was = t.data_ptr(), t.data
    t.data = OTHER[how](t.data)
    assert t.data_ptr() == at
    with pytest.raises(q.QloraError, match="another type, shape, stride or device"):
        plan._bind("bind", None)
    t.data = was                            # and a refusal leaves the plan as it was
    plan._bind("bind", None)


def test_a_gradient_of_another_type_in_its_place(plan):
    """A bf16 gradient read as float32 would be read past its end."""
    g = plan.tensors[1][1]
    half = g.data.untyped_storage()
    g.data = torch.empty(0, dtype=BF).set_(half)[:50 * 24].view(50, 24)[:, :8]
    with pytest.raises(q.QloraError, match="another type"):
        q.qlora_muon_step(plan, 0.1)


def test_moved_memory_is_followed(plan):
    for k in range(3):
        for t in plan.tensors[k % 2]:
            t.data = torch.empty(4096, dtype=t.dtype)[8:8 + 2400].view(-1, t.stride(0))[
                :t.shape[0], :t.shape[1]]
        plan._bind("bind", None)
        for a, (p, g, m, pb) in zip(plan.array, plan.tensors):
            assert (a.param, a.grad, a.momentum, a.param_bf16) == tuple(
                t.data_ptr() for t in (p, g, m, pb))


def test_what_is_no_matrix_is_refused(plan):
    good = [t[1] for t in plan.tensors]
    for bad in (None, 3, [1.0], good[0].unsqueeze(0), good[0][0], good[0].new_zeros(()),
                good[0].to("meta"), torch.zeros((8, 20)).to_sparse()):
        with pytest.raises((q.QloraError, NotImplementedError, RuntimeError)):
            plan._bind("bind", [bad, good[1]])
    plan._bind("bind", good)
    assert [g.data_ptr() for g in good] == [a.grad for a in plan.array]


def test_the_two_looks_agree():
    """Both tell apart what is laid out differently, and nothing else."""
    assert q._exchange() is not None
    x = torch.zeros((12, 20))
    some = [x, x.clone(), x[:, :10], x[:6], x.t(), x.double(), x.bool(), x.to(BF), x[::2], x[:, ::2],
            torch.nn.Parameter(x.clone()), x[:0], x[:, :0]]
    fast = [q._layouts("t", [t]) for t in some]
    assert [int.from_bytes(a, "little") for a, _ in fast] == [t.data_ptr() for t in some]
    key = [(t.dtype, t.device, t.shape, t.stride()) for t in some]
    for i in range(len(some)):
        for j in range(len(some)):
            assert (fast[i][1] == fast[j][1]) == (key[i] == key[j]), (i, j)
    at, layout = q._layouts("t", some)
    assert at == b"".join(a for a, _ in fast) and layout == b"".join(b for _, b in fast)
    with pytest.raises(q.QloraError):
        q._layouts("t", [x, "no tensor"])


@pytest.mark.parametrize("shape,strides", [((1, 30), [(30, 1), (1, 1), (64, 1), (0, 1)]),
                                           ((30, 1), [(1, 1), (1, 30), (1, 64), (1, 0)]),
                                           ((1, 1), [(1, 1), (9, 5), (0, 0)]),
                                           ((30, 1), [(4, 1), (4, 7)]),
                                           ((0, 30), [(30, 1), (1, 1), (7, 3)]),
                                           ((30, 0), [(1, 1), (30, 5), (0, 0)])])
def test_strides_of_single_rows_and_columns(plan, shape, strides):
    """The stride of a dimension of one (or no) element is no part of a layout."""
    buf = torch.arange(256.)
    of = lambda s: torch.as_strided(buf, shape, s)  # noqa: E731
    p, m = torch.zeros(shape), torch.zeros(shape)
    one = q.MuonPlan([(p, of(strides[0]), m, None)])
    for s in strides[::-1]:
        one._bind("bind", [of(s)])
        assert (one.array[0].grad or 0) == of(s).data_ptr()       # (0 reads as None)
    if shape[0] > 1 and shape[1] == 1:          # this one's row stride counts
        with pytest.raises(q.QloraError, match="stride"):
            one._bind("bind", [of((strides[0][0] + 1, 1))])
