"""CPU check of the binding: a gate is rows, or one row, of the width of y; other shapes of as many elements are not."""
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from test_abi_ragged import L  # noqa: F401


@pytest.mark.parametrize("shape", [(2, 32), (64, 1), (4, 16), (1, 1, 64)])
def test_gate_of_another_shape(L, shape):  # noqa: F811
    y, h = torch.zeros(3, 64), torch.zeros(3, 64)
    with pytest.raises(ValueError, match="gate"):
        k8.block_norm_k8v4(y, None, h, gate=torch.zeros(shape))
    with pytest.raises(ValueError, match="gate"):          # as many elements as all rows
        k8.block_norm_k8v4(y, None, h, gate=torch.zeros(64, 3))
    for good in ((64,), (1, 64), (3, 64)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            k8.block_norm_k8v4(y, None, h, gate=torch.zeros(good))
