"""The first decode-shaped GEMM on a stream, whose K-split workspace the library
allocates then: it is empty before the kernel reads it, whatever lay in that
memory and whatever the default stream is busy with."""
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
from gpu_helpers import check_device_error_word, gpu_quantize

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(4, 700, 17408), (8, 12288, 5120), (40, 1024, 4096)])
def test_first_call_on_a_stream_while_the_default_stream_is_busy(M, N, K):
    g = torch.Generator().manual_seed(N)
    a, sa, _ = gpu_quantize(torch.randn(M, K, generator=g).cuda(), 300.0)
    w, sw, _ = gpu_quantize(0.02 * torch.randn(N, K, generator=g).cuda(), 20000.0)

    def call(out):
        nv.nvfp4_gemm(a, sa, 300.0, w, sw, 20000.0, M, N, K, out)

    want = torch.empty(M, N, device="cuda")
    call(want)
    torch.cuda.synchronize()
    check_device_error_word()
    for _ in range(6):
        outs = [torch.full((M, N), 9.0, device="cuda") for _ in range(3)]
        nv.nvfp4_release_workspaces()
        # memory that goes back to the driver full of words that look like partial sums
        junk = [torch.full((8 << 20,), (1 << 32) + 0x3F800000, dtype=torch.int64, device="cuda") for _ in range(6)]
        torch.cuda.synchronize()
        del junk
        torch.cuda.empty_cache()
        torch.cuda._sleep(40_000_000)                    # some 20 ms of the default stream
        streams = [torch.cuda.Stream() for _ in outs]
        for st, out in zip(streams, outs):
            with torch.cuda.stream(st):
                call(out)
                call(out)
        torch.cuda.synchronize()
        check_device_error_word()
        assert all(torch.equal(out, want) for out in outs)
    nv.nvfp4_release_workspaces()
