"""Reading the device error word clears it before the call returns: what a
kernel on another stream reports right afterwards is not lost."""
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv

pytestmark = pytest.mark.gpu


def test_a_report_right_after_a_read_is_kept():
    y, w = torch.ones(2, 64, device="cuda"), torch.ones(1, 1, device="cuda")
    slots = torch.tensor([[7]], dtype=torch.int32, device="cuda")       # y has two rows
    out, st = torch.empty(1, 64, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    assert nv.nvfp4_last_device_error() == nv.OK
    with torch.cuda.stream(st):
        for _ in range(200):
            nv.nvfp4_block_norm(y, slots=slots, slot_weights=w, out=out)
            assert nv.nvfp4_last_device_error() == nv.ERR_DEVICE
    assert nv.nvfp4_last_device_error() == nv.OK
