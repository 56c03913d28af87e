"""Calls that follow one another without a pause, on buffers that each call
rewrites: every kernel sees what the one right before it wrote, not what stood
there when it started."""
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
from gpu_helpers import check_device_error_word
from grouped_helpers import I32, experts

pytestmark = pytest.mark.gpu


def buffers(M, E, k):
    return dict(expert_ids=torch.empty(M, k, dtype=I32, device="cuda"), weights=torch.empty(M, k, device="cuda"),
                slots=torch.empty(M, k, dtype=I32, device="cuda"), row_index=torch.empty(M * k, dtype=I32, device="cuda"),
                group_offsets=torch.empty(E + 1, dtype=I32, device="cuda"))


# one launch; a cluster; two launches with few and with many runs of tokens
@pytest.mark.parametrize("M", [8, 200, 600, 5000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_router_calls_share_a_workspace(M, dtype):
    E, k, n = 64, 6, 24
    g = torch.Generator().manual_seed(M)
    x = (torch.randn(n, M, E, generator=g) * 2).to(dtype).cuda()
    x[1::2, :, E // 2:] = float("-inf")                      # counts far from the call before's
    space = torch.empty(nv.nvfp4_route_workspace_bytes(E), dtype=torch.uint8, device="cuda")
    want = []
    for i in range(n):
        b = buffers(M, E, k)
        nv.nvfp4_route(x[i], 0, **b, workspace=space)
        torch.cuda.synchronize()
        want.append(b)
    got = [buffers(M, E, k) for _ in range(n)]
    for _ in range(3):
        torch.cuda.synchronize()
        for i in range(n):
            nv.nvfp4_route(x[i], 0, **got[i], workspace=space)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for name in a:
                assert torch.equal(a[name], b[name]), name
    one = buffers(M, E, k)                                   # and every buffer the same
    for i in range(n):
        nv.nvfp4_route(x[i], 0, **one, workspace=space)
    torch.cuda.synchronize()
    for name in one:
        assert torch.equal(one[name], want[-1][name]), name
    check_device_error_word()


@pytest.mark.parametrize("M", [8, 400])
def test_layers_share_every_buffer(M):
    """Route, gather, multiply, combine, again and again on one set of buffers; only the outputs of a layer are its own."""
    E, k, K, N, n = 16, 4, 256, 192, 16
    g = torch.Generator().manual_seed(M)
    logits = torch.randn(n, M, E, generator=g).cuda()
    logits[1::2, :, E // 2:] = float("-inf")
    x = torch.randn(n, M, K, generator=g).to(torch.bfloat16).cuda()
    scales = (100.0 * (1 + torch.rand(n, E, generator=g))).cuda()
    wc, ws, gw, _ = experts(E, N, K, 1)
    r, space = buffers(M, E, k), torch.empty(nv.nvfp4_route_workspace_bytes(E), dtype=torch.uint8, device="cuda")
    codes, sc = nv.alloc_grouped(M * k, E, K, "cuda")
    y = torch.empty(M * k, N, device="cuda")

    def layer(i, out):
        nv.nvfp4_route(logits[i], 1, **r, workspace=space)
        nv.nvfp4_grouped_quantize(x[i], r["group_offsets"], scales[i], codes, sc, row_index=r["row_index"])
        nv.nvfp4_grouped_gemm(codes, sc, scales[i], wc, ws, gw, r["group_offsets"], y)
        nv.nvfp4_block_norm(y, slots=r["slots"], slot_weights=r["weights"], out=out)

    want = [torch.empty(M, N, device="cuda") for _ in range(n)]
    for i in range(n):
        layer(i, want[i])
        torch.cuda.synchronize()
    got = [torch.empty(M, N, device="cuda") for _ in range(n)]
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=st):
        for i in range(n):
            layer(i, got[i])
    for run in (lambda: [layer(i, got[i]) for i in range(n)], graph.replay, graph.replay):
        for t in got:
            t.fill_(7.0)
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    check_device_error_word()
