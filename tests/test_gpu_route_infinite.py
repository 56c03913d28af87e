"""+inf among the router's logits counts as the largest float, whatever the
logits' type: above every finite bf16, a tie with the largest FP32 number."""
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
from test_gpu_route import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 300])
@pytest.mark.parametrize("norm", [nv.ROUTE_SOFTMAX_ALL, nv.ROUTE_SOFTMAX_TOPK])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinity_beside_the_largest_number(M, norm, dtype):
    x = torch.randn(M, 40, generator=torch.Generator().manual_seed(M)).to(dtype)
    x[:, 3] = torch.finfo(dtype).max
    x[:, 17] = float("inf")
    x[:, 30] = float("inf")
    x[:, 8] = torch.finfo(dtype).min
    b = check(x.cuda(), 4, norm)
    first = [3, 17, 30] if dtype == torch.float32 else [17, 30, 3]
    assert b["expert_ids"][0].tolist()[:3] == first
    w = b["weights"][0].tolist()
    assert w[:2] == pytest.approx([1 / 3] * 2 if dtype == torch.float32 else [0.5] * 2) and w[3] == 0.0
