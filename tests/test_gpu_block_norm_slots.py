"""Slots of the block norm outside [-1, y_rows): each is reported by itself,
skipped, and harms no other row."""
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
from gpu_helpers import check_device_error_word

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.mark.parametrize("slot", [5, 2 ** 31 - 1, -2, -100, -2 ** 31])
@pytest.mark.parametrize("K", [64, 1056, 9216])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_slot_that_y_does_not_have_is_reported(slot, K, dtype):
    y = torch.randn(5, K, generator=torch.Generator().manual_seed(K)).to(dtype).cuda()
    slots = torch.tensor([[0, 4], [slot, 1], [2, -1], [3, slot]], dtype=I32).cuda()
    w = torch.ones(4, 2, device="cuda")
    out = torch.empty(4, K, dtype=dtype, device="cuda")
    nv.nvfp4_block_norm(y, slots=slots, slot_weights=w, out=out)
    assert nv.nvfp4_last_device_error() == nv.ERR_DEVICE
    assert torch.equal(out[0], (y[0].float() + y[4].float()).to(dtype))
    assert all(torch.equal(out[i], y[j]) for i, j in ((1, 1), (2, 2), (3, 3)))
    slots[slots == slot] = -1                            # left empty by the router: nothing to report
    nv.nvfp4_block_norm(y, slots=slots, slot_weights=w, out=out)
    torch.cuda.synchronize()
    check_device_error_word()
