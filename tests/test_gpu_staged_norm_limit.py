"""The staged block norm when a row never arrives: the waits for it run out,
NVFP4_ERR_TIMEOUT is reported, the kernel ends, what arrived is right, and so
is the next call.  Nothing faults: a test entry leaves the copies out."""
import ctypes

import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
from gpu_helpers import check_device_error_word

P = ctypes.c_void_p


@pytest.mark.parametrize("rows", [-1, 301])
def test_the_first_missing_row_lies_in_the_input(rows):
    assert nv.lib().nvfp4_test_block_norm_stalled(P(0x10000), 1, 300, 17408, None, rows, P(0x10000),
                                                  None) == nv.ERR_INVALID_ARG


# rows on each CTA's first, second and third turn; rings of 3 slots (two arrays, so that a row's copies lie on both
# sides of its end), of one array and of one slot
@pytest.mark.gpu
@pytest.mark.parametrize("stalled_from", [0, 1, 147, 200, 319])
@pytest.mark.parametrize("K,dtype,residual", [(17408, torch.float32, True), (32768, torch.float32, False),
                                              (32768, torch.bfloat16, True)])
def test_a_row_that_never_arrives_is_reported(K, dtype, residual, stalled_from):
    M = 320
    g = torch.Generator().manual_seed(K)
    y = torch.randn(M, K, generator=g).to(dtype).cuda()
    r = torch.randn(M, K, generator=g).to(dtype).cuda() if residual else None
    want, out = torch.empty(M, K, dtype=dtype, device="cuda"), torch.empty(M, K, dtype=dtype, device="cuda")
    nv.nvfp4_block_norm(y, residual=r, out=want)
    torch.cuda.synchronize()
    check_device_error_word()
    try:
        nv.nvfp4_set_wait_timeout_ns(1_000_000)
        nv.nvfp4_test_block_norm_stalled(y, stalled_from, out, residual=r)
        status = nv.nvfp4_last_device_error()
    finally:
        nv.nvfp4_set_wait_timeout_ns(0)
    assert status == nv.ERR_TIMEOUT
    assert torch.equal(out[:stalled_from], want[:stalled_from])
    for _ in range(2):
        out.fill_(3.0)
        nv.nvfp4_block_norm(y, residual=r, out=out)
        torch.cuda.synchronize()
        check_device_error_word()
        assert torch.equal(out, want)


@pytest.mark.gpu
def test_nothing_is_reported_when_every_row_arrives():
    y = torch.randn(320, 17408, generator=torch.Generator().manual_seed(1)).cuda()
    out = torch.empty_like(y)
    nv.nvfp4_test_block_norm_stalled(y, 320, out)
    torch.cuda.synchronize()
    check_device_error_word()
    assert torch.equal(out, y)
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.nvfp4_test_block_norm_stalled(y[:100], 10, out[:100])      # too few rows to be staged
    assert e.value.status == nv.ERR_UNSUPPORTED
