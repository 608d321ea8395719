"""block_norm_k8v4 at the ends of its ranges."""
import numpy as np
import pytest
import torch

import quantized_paged_kv_q8_gb300 as k8
from test_gpu_block_norm import F32_HALF

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("dim", [2048, 2051])
def test_fp32_gates_far_from_0(act, dim):
    """fp32 in, fp32 out: the gate's function to a few units at any argument (the exponential 2 units, two more
    operations and the products one half each; the last a subnormal's half)."""
    z = torch.linspace(-86.0, 40.0, 3 * dim, device="cuda").view(3, dim)
    y = torch.from_numpy(np.random.default_rng(dim).uniform(0.5, 2.0, (3, dim)).astype(np.float32)).cuda()
    h = torch.empty_like(y)
    k8.block_norm_k8v4(y, None, h, gate=z, gate_act=act)
    u = torch.sigmoid(z.double())
    want = y.double() * (z.double() * u if act == "silu" else u)
    assert ((h.double() - want).abs() <= 10 * F32_HALF * want.abs() + 2.0 ** -149).all()


def test_most_rows():
    """2^31 - 1 rows of one element, four to a CTA."""
    n = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("9 GB of rows")
    y, h = (torch.empty(n, 1, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    y.fill_(3.0)
    y[-1], h[-4:] = 5.0, 0.0
    k8.block_norm_k8v4(y, None, h, residual_scale=2.0)
    torch.cuda.synchronize()
    assert h[-1].item() == 10.0 and h[0].item() == 6.0 and (h[-1000:-1] == 6.0).all()
