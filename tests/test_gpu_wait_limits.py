"""GEMMs whose waits run out: every role gives up together, the call ends and
reports NVFP4_ERR_TIMEOUT, and the next call is right.  No wait here is for
something that never comes: the limit is only shorter than the work."""
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
from gpu_helpers import check_device_error_word, gpu_quantize
from grouped_helpers import experts, offsets_of

pytestmark = pytest.mark.gpu


def grouped(rows, N, K, dtype):
    E, T = len(rows), sum(rows)
    wc, ws, gw, _ = experts(E, N, K, 3)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).cuda()
    ga, offs = torch.full((E,), 200.0, device="cuda"), offsets_of(rows).cuda()
    codes, scales = nv.alloc_grouped(T, E, K, "cuda")
    nv.nvfp4_grouped_quantize(x, offs, ga, codes, scales)
    return lambda out: nv.nvfp4_grouped_gemm(codes, scales, ga, wc, ws, gw, offs, out), (T, N), dtype


def dense(M, N, K, dtype):
    g = torch.Generator().manual_seed(2)
    ac, asc, _ = gpu_quantize(torch.randn(M, K, generator=g).cuda(), 300.0)
    wc, wsc, _ = gpu_quantize(0.02 * torch.randn(N, K, generator=g).cuda(), 20000.0)
    return lambda out: nv.nvfp4_gemm(ac, asc, 300.0, wc, wsc, 20000.0, M, N, K, out), (M, N), dtype


CASES = {
    "grouped small, bf16": lambda: grouped([3, 70, 0, 128, 33], 520, 1024, torch.bfloat16),
    "grouped large, f32, rows not on 16 bytes": lambda: grouped([300, 513, 129], 513, 1024, torch.float32),
    "dense pairs": lambda: dense(600, 1024, 2048, torch.bfloat16),
    "dense, f32, one row block": lambda: dense(129, 250, 1024, torch.float32),
    "dense decode": lambda: dense(8, 4096, 2048, torch.float32),
}


@pytest.mark.parametrize("case", CASES)
def test_a_gemm_whose_waits_run_out_ends_and_the_next_is_right(case):
    call, shape, dtype = CASES[case]()
    want = torch.empty(shape, dtype=dtype, device="cuda")
    call(want)
    torch.cuda.synchronize()
    check_device_error_word()
    try:
        nv.nvfp4_set_wait_timeout_ns(1)
        call(torch.empty_like(want))
        status = nv.nvfp4_last_device_error()
    finally:
        nv.nvfp4_set_wait_timeout_ns(0)
    assert status == nv.ERR_TIMEOUT          # operands come from memory: no first look finds them there
    for _ in range(2):
        out = torch.empty_like(want)
        call(out)
        torch.cuda.synchronize()
        check_device_error_word()
        assert torch.equal(out, want)
