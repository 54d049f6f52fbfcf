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
