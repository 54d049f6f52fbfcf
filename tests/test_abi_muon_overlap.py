"""What a call of the orthogonalised update writes, it reads as nothing else: refused on the
host (no GPU needed)."""
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
