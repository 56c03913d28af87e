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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [[1], [0, 3, 130, 0, 40], [300, 500]])
def test_rows_through_an_index(dtype, rows):
    """The same bytes as for the rows gathered beforehand, rows taken several times among them."""
    K, E, T = 352, len(rows), sum(rows) + 2
    g = torch.Generator().manual_seed(T)
    x = (3 * torch.randn(max(2, T // 3), 2 * K, generator=g)).to(dtype).cuda()
    idx = torch.randint(0, x.shape[0], (T,), generator=g, dtype=torch.int32).cuda()
    gs, offs = (50.0 * (1 + torch.rand(E, generator=g))).cuda(), offsets_of(rows).cuda()
    got = []
    for src, index in ((x, idx), (x[idx.long()].contiguous(), None)):
        codes, scales = nv.alloc_grouped(T, E, K, "cuda")
        codes.fill_(255)
        scales.fill_(255)
        nv.nvfp4_grouped_quantize(src, offs, gs, codes, scales, row_index=index, act=nv.ACT_SWIGLU)
        got.append((codes, scales))
    torch.cuda.synchronize()
    check_device_error_word()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert got[0][0][sum(rows):].eq(255).all()


def test_a_bad_index_is_reported_and_quantized_as_zeros():
    K = 64
    x = torch.ones(4, 2 * K, device="cuda")
    idx = torch.tensor([0, 4, -1, 3], dtype=torch.int32, device="cuda")
    codes, scales = nv.alloc_grouped(4, 1, K, "cuda")
    nv.nvfp4_grouped_quantize(x, offsets_of([4]).cuda(), torch.ones(1, device="cuda"), codes, scales, row_index=idx,
                              act=nv.ACT_SWIGLU)
    assert nv.nvfp4_last_device_error() == nv.ERR_DEVICE
    assert codes[1].eq(0).all() and codes[2].eq(0).all() and not codes[0].eq(0).any() and not codes[3].eq(0).any()
