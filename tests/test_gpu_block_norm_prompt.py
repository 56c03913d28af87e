"""The combine of expert rows over a prompt: many rows, long ones, with gates."""
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
from test_gpu_block_norm import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,over", [(2048, 5120, dict(k=8)), (777, 8192, dict(k=8, gate=nv.GATE_SILU)),
                                      (500, 9216, dict(k=8, gate=nv.GATE_SIGMOID)), (400, 17408, dict(k=4, post=17408)),
                                      (310, 18464, dict(k=3, gate=nv.GATE_LINEAR, residual=False))])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_combine_over_a_prompt(M, K, over, dtype):
    check(make(M, K, dtype, **over), dtype)
