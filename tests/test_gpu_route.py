"""Router (nvfp4_route) against a 64-bit host form: ids, slots, row order and
offsets exactly, weights within the FP32 error of their own steps."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
from gpu_helpers import check_device_error_word

pytestmark = pytest.mark.gpu
I32 = torch.int32


def buffers(M, E, k):
    dev = "cuda"
    return dict(expert_ids=torch.full((M, k), 77, dtype=I32, device=dev), weights=torch.full((M, k), 7.0, device=dev),
                slots=torch.full((M, k), 77, dtype=I32, device=dev),
                row_index=torch.full((M * k,), 77, dtype=I32, device=dev),
                group_offsets=torch.full((E + 1,), 77, dtype=I32, device=dev),
                workspace=torch.full((nv.nvfp4_route_workspace_bytes(E),), 255, dtype=torch.uint8, device=dev))


def reference(x, k, all_experts):
    """Plain host form on float64 logits (already the values of the input type)."""
    M, E = x.shape
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    ids = np.argsort(-x, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(x, ids, 1)
    ok = top > -np.inf
    ids = np.where(ok, ids, -1)
    peak = np.where(ok[:, :1], top[:, :1], 0.0)
    e = np.where(ok, np.exp(top - peak), 0.0)
    total = np.exp(x - peak).sum(1, keepdims=True) if all_experts else e.sum(1, keepdims=True)
    w = np.where(ok, e / np.where(total > 0, total, 1.0), 0.0)
    slots = np.full((M, k), -1, dtype=np.int64)
    offsets = np.zeros(E + 1, dtype=np.int64)
    rows = np.full(M * k, -1, dtype=np.int64)
    n = 0
    for g in range(E):
        m, j = np.nonzero(ids == g)
        slots[m, j] = n + np.arange(m.size)
        rows[n:n + m.size] = m
        n += m.size
        offsets[g + 1] = n
    # FP32: each exp argument is off by |x - max| 2^-24, expf by 2 ulp, the sum by one rounding an addend, one division
    tol = (40 + E / 32 + np.where(ok, peak - np.where(ok, top, 0.0), 0.0)) * 2.0 ** -24 * w + 2.0 ** -126
    return ids, w, slots, rows, offsets, tol


def check(x, k, norm):
    M, E = x.shape
    b = buffers(M, E, k)
    nv.nvfp4_route(x, norm, **b)
    torch.cuda.synchronize()
    check_device_error_word()
    ids, w, slots, rows, offsets, tol = reference(x.double().cpu().numpy(), k, norm == nv.ROUTE_SOFTMAX_ALL)
    assert np.array_equal(b["expert_ids"].cpu().numpy(), ids)
    assert np.array_equal(b["group_offsets"].cpu().numpy(), offsets)
    assert np.array_equal(b["slots"].cpu().numpy(), slots)
    assert np.array_equal(b["row_index"].cpu().numpy(), rows)
    assert np.all(np.abs(b["weights"].double().cpu().numpy() - w) <= tol)
    return b


@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 8, 8), (1, 512, 32), (8, 64, 8), (32, 64, 8), (33, 64, 8),
                                   (40, 5, 2), (63, 33, 3), (64, 128, 8),
                                   (65, 64, 6), (129, 31, 5), (700, 160, 8), (2500, 512, 10), (20001, 96, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_matches_host_form(M, E, k, dtype):
    g = torch.Generator().manual_seed(M * 1000 + E * 10 + k)
    x = (2 * torch.randn(M, E, generator=g)).to(dtype).cuda()
    check(x, k, nv.ROUTE_SOFTMAX_ALL)
    check(x, k, nv.ROUTE_SOFTMAX_TOPK)


@pytest.mark.parametrize("M", [5, 300])
def test_ties_go_to_the_lowest_index(M):
    x = torch.zeros(M, 40, device="cuda")
    x[:, 7] = -0.0
    x[:, 20] = 1.0
    b = check(x, 4, nv.ROUTE_SOFTMAX_ALL)
    assert b["expert_ids"][0].tolist() == [20, 0, 1, 2]
    x[:, :8] = 0.0
    x[:, 0] = -0.0                                     # -0 ties with 0
    assert check(x, 3, nv.ROUTE_SOFTMAX_TOPK)["expert_ids"][0].tolist() == [20, 0, 1]


@pytest.mark.parametrize("M", [9, 400])
@pytest.mark.parametrize("norm", [nv.ROUTE_SOFTMAX_ALL, nv.ROUTE_SOFTMAX_TOPK])
def test_masks_infinities_and_nan(M, norm):
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, 48, generator=g)
    x[torch.rand(M, 48, generator=g) < 0.9] = float("-inf")     # rows with fewer than k experts
    x[0] = float("-inf")                                        # none at all
    x[1] = float("nan")
    x[2] = torch.finfo(torch.float32).min                       # a mask of the lowest value is a finite logit
    x[3, 5] = float("inf")
    x[4, 5:7] = float("inf")
    x[5, :] = float("-inf")
    x[5, 47] = torch.finfo(torch.float32).min
    b = check(x.cuda(), 6, norm)
    assert b["expert_ids"][0].tolist() == [-1] * 6 and b["weights"][0].tolist() == [0.0] * 6
    assert b["expert_ids"][5].tolist() == [47] + [-1] * 5 and b["weights"][5, 0].item() == 1.0


def test_every_token_to_one_expert_and_empty_experts():
    x = torch.full((777, 64), -1.0, device="cuda")
    x[:, 63] = 5.0
    b = check(x, 1, nv.ROUTE_SOFTMAX_TOPK)
    assert b["group_offsets"].tolist() == [0] * 64 + [777]


def test_captured_and_replayed_on_new_logits():
    M, E, k = 500, 64, 8
    g = torch.Generator().manual_seed(3)
    x = torch.randn(M, E, generator=g).cuda()
    b = buffers(M, E, k)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        nv.nvfp4_route(x, 0, **b)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        nv.nvfp4_route(x, 0, **b)
    for seed in (4, 5):
        x.copy_(torch.randn(M, E, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        ids, w, slots, rows, offsets, _ = reference(x.double().cpu().numpy(), k, True)
        assert np.array_equal(b["slots"].cpu().numpy(), slots)
        assert np.array_equal(b["row_index"].cpu().numpy(), rows)
        assert np.array_equal(b["group_offsets"].cpu().numpy(), offsets)


# one launch: a CTA up to 32 tokens, then a cluster of 2, 4 or 8; two launches beyond
@pytest.mark.parametrize("M", [31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 160, 255, 256, 257, 511, 512, 513, 1023, 1024,
                               1025])
@pytest.mark.parametrize("E,k,dtype", [(60, 3, torch.float32), (512, 32, torch.bfloat16)])
def test_every_number_of_runs(M, E, k, dtype):
    x = torch.randn(M, E, generator=torch.Generator().manual_seed(M))
    x[M // 2:, E // 3:] = float("-inf")                   # tokens with fewer than k experts
    check(x.to(dtype).cuda(), k, nv.ROUTE_SOFTMAX_ALL)
