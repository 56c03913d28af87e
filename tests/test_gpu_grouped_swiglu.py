"""SwiGLU in the grouped quantizer: products that leave FP32."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
import oracle
from gpu_helpers import check_device_error_word
from grouped_helpers import offsets_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_products_beyond_fp32_saturate(dtype):
    """Finite inputs whose product is not: encoded as the largest float is, and never as NaN."""
    K, g = 64, 2.0 ** -120
    x = torch.zeros(3, 2 * K)
    x[0, :K], x[0, K:] = 2.0 ** 100, 2.0 ** 100               # +inf
    x[1, :K], x[1, K:] = 2.0 ** 64, -(2.0 ** 63)              # -2^127, finite
    x[2, 0], x[2, K] = 2.0 ** 100, -(2.0 ** 100)              # one -inf among zeros
    h = (x[:, :K].double() * x[:, K:].double()).clamp(-torch.finfo(torch.float32).max, torch.finfo(torch.float32).max)
    for gs in (g, 1.0, 2.0 ** -140):                          # the last: a scale of zero, codes of signed zeros
        codes, scales = nv.alloc_grouped(3, 1, K, "cuda")
        nv.nvfp4_grouped_quantize(x.to(dtype).cuda(), offsets_of([3]).cuda(), torch.full((1,), gs, device="cuda"), codes,
                                  scales, act=nv.ACT_SWIGLU)
        torch.cuda.synchronize()
        check_device_error_word()
        c, s = oracle.quantize(h.float().numpy(), np.float32(gs))
        assert np.array_equal(codes.cpu().numpy(), c)
        assert np.array_equal(oracle.scales_from_tc(scales.cpu().numpy(), 3, K), s)
