"""Steps of more tensors than one launch takes, of every padded rank, both gradient types
and rows in wider ones, each tensor against float64 to its own roundings."""
import numpy as np
import pytest
import torch

from gpu_common import host, say
from test_gpu_muon import BF, F32, _expect, _matrix, _np, _tensors

import bit_quantized_lora_quant_amd as q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [46, 113])
@pytest.mark.parametrize("nesterov", [True, False])
def test_every_tensor_of_a_table(count, nesterov):
    say("%d tensors, nesterov=%s" % (count, nesterov))
    rng = np.random.default_rng(count)
    shapes, grad = [], [(F32, BF)[i % 3 == 1] for i in range(count)]
    for i in range(count):
        r, n = int(rng.integers(1, 129)), int(rng.integers(1, 900))
        shapes.append((r, n) if i % 2 else (n, r))
    pads = [0, 5, 4]
    ts = [(p, g.to(grad[i]), m, pb if i % 4 else None) for i, (p, g, m, pb) in
          enumerate(_tensors(shapes, pads=pads))]
    plan = q.MuonPlan([(p, _matrix(0, *s, grad[i], pad=pads[i % 3]), m, pb)
                       for i, ((p, _, m, pb), s) in enumerate(zip(ts, shapes))])
    for k in range(3):
        grads = [_matrix(7000 * k + i, *s, grad[i], pad=pads[i % 3]) for i, s in enumerate(shapes)]
        lr = 0.01 + 0.2 * k
        # (each step from the tensors as the last one left them)
        ref = [_expect(p, g, m, lr, 0.95, nesterov, 0.01, "shape")
               for (p, _, m, _), g in zip(ts, grads)]
        q.qlora_muon_step(plan, lr, nesterov=nesterov, weight_decay=0.01, grads=grads)
        for (p, _, m, pb), (m_ref, p_ref, tol), s in zip(ts, ref, shapes):
            assert np.array_equal(host(m).numpy(), m_ref), s
            assert np.all(np.abs(_np(p) - p_ref) <= tol), s
            assert pb is None or torch.equal(pb, p.to(BF)), s
