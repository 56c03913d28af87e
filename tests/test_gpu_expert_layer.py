"""The expert layer as a model runs it: norm, route, quantize, up projections,
SwiGLU, down projection, combine with the next norm, on one stream and as a
captured graph, against a 64-bit form fed stage by stage."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
import oracle
from gpu_helpers import assert_gemm_close, check_device_error_word
from grouped_helpers import experts, grouped_scales, oracle_rows, product

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Layer:
    def __init__(self, M, K, F, E, k, seed):
        dev, i32 = "cuda", torch.int32
        g = torch.Generator().manual_seed(seed)
        self.M, self.K, self.F, self.E, self.k, T = M, K, F, E, k, M * k
        self.up, self.down = experts(E, 2 * F, K, seed), experts(E, K, F, seed + 1)
        self.stream_in = torch.randn(M, K, generator=g).to(torch.bfloat16).to(dev)
        self.branch = torch.randn(M, K, generator=g).to(torch.bfloat16).to(dev)
        self.w1, self.w2 = torch.ones(K, device=dev), torch.full((K,), 0.5, device=dev)
        self.gate_w = (torch.randn(E, K, generator=g) / K ** 0.5).to(dev)
        self.gs1, self.gs2 = torch.full((E,), 300.0, device=dev), torch.full((E,), 150.0, device=dev)
        self.resid = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
        self.h = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
        self.r = dict(expert_ids=torch.empty(M, k, dtype=i32, device=dev), weights=torch.empty(M, k, device=dev),
                      slots=torch.empty(M, k, dtype=i32, device=dev),
                      row_index=torch.empty(T, dtype=i32, device=dev),
                      group_offsets=torch.empty(E + 1, dtype=i32, device=dev),
                      workspace=torch.empty(nv.nvfp4_route_workspace_bytes(E), dtype=torch.uint8, device=dev))
        self.c1, self.s1 = nv.alloc_grouped(T, E, K, dev)
        self.c2, self.s2 = nv.alloc_grouped(T, E, F, dev)
        self.u = torch.empty(T, 2 * F, dtype=torch.bfloat16, device=dev)
        self.d = torch.empty(T, K, dtype=torch.bfloat16, device=dev)
        self.out_resid = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
        self.out_codes, self.out_scales = nv.alloc_quantized(M, K, dev)
        self.logits = torch.empty(M, E, device=dev)

    def run(self):
        nv.nvfp4_block_norm(self.branch, residual=self.stream_in, residual_out=self.resid, pre_weight=self.w1, out=self.h)
        torch.matmul(self.h.float(), self.gate_w.t(), out=self.logits)
        nv.nvfp4_route(self.logits, nv.ROUTE_SOFTMAX_TOPK, **self.r)
        offs = self.r["group_offsets"]
        nv.nvfp4_grouped_quantize(self.h, offs, self.gs1, self.c1, self.s1, row_index=self.r["row_index"])
        nv.nvfp4_grouped_gemm(self.c1, self.s1, self.gs1, *self.up[:3], offs, self.u)
        nv.nvfp4_grouped_quantize(self.u, offs, self.gs2, self.c2, self.s2, act=nv.ACT_SWIGLU)
        nv.nvfp4_grouped_gemm(self.c2, self.s2, self.gs2, *self.down[:3], offs, self.d)
        nv.nvfp4_block_norm(self.d, slots=self.r["slots"], slot_weights=self.r["weights"], residual=self.resid,
                            residual_out=self.out_resid, pre_weight=self.w2, codes=self.out_codes,
                            block_scales=self.out_scales, global_scale=100.0)

    def outputs(self):
        return [self.r["slots"], self.r["weights"], self.u, self.d, self.out_resid, self.out_codes, self.out_scales]


@pytest.mark.parametrize("M,K,F,E,k", [(1, 256, 128, 8, 2), (8, 512, 256, 16, 4), (333, 384, 160, 8, 3),
                                       (900, 256, 96, 4, 2)])
def test_layer(M, K, F, E, k):
    L = Layer(M, K, F, E, k, M)
    L.run()
    torch.cuda.synchronize()
    check_device_error_word()
    rows = np.diff(L.r["group_offsets"].cpu().numpy())
    T = M * k
    assert rows.sum() == T
    # up projections: the oracle on the rows the router chose
    x = L.h.float().cpu().numpy()[L.r["row_index"].cpu().numpy()]
    codes, per = oracle_rows(x, rows, L.gs1.cpu().numpy(), T, K)
    assert np.array_equal(L.c1.cpu().numpy(), codes)
    u = product(codes, per, L.gs1.cpu().numpy(), L.up[3], rows, 2 * F)
    got = L.u.double().cpu().numpy()
    assert np.all(np.abs(got - u) <= 2.0 ** -8 * np.abs(u) + 1e-5 * np.abs(u).max())
    # down projection on the codes the SwiGLU step wrote (its own test checks them)
    chunk, at, blk, per2 = -(-F // 64) * 512, 0, 0, []
    s2 = L.s2.cpu().numpy()
    for n in rows:
        nb = -(-n // 128)
        keep = oracle.scales_to_tc(np.ones((n, F // 16), dtype=np.uint8), F).astype(bool) if n else None
        per2.append(oracle.scales_from_tc(np.where(keep, s2[blk * chunk:(blk + nb) * chunk], 0).astype(np.uint8), n, F)
                    if n else np.zeros((0, F // 16), dtype=np.uint8))
        blk += nb
    d = product(L.c2.cpu().numpy(), per2, L.gs2.cpu().numpy(), L.down[3], rows, K)
    got = L.d.double().cpu().numpy()
    assert np.all(np.abs(got - d) <= 2.0 ** -8 * np.abs(d) + 1e-5 * np.abs(d).max())
    # combine: every token gets its own experts' rows
    w, slots = L.r["weights"].double().cpu().numpy(), L.r["slots"].cpu().numpy()
    v = L.resid.double().cpu().numpy() + (w[:, :, None] * got[slots]).sum(1)
    tol = 2.0 ** -8 * np.abs(v) + (2 * k + 4) * 2.0 ** -24 * (np.abs(w[:, :, None] * got[slots]).sum(1) + np.abs(v))
    assert np.all(np.abs(L.out_resid.double().cpu().numpy() - v) <= tol)
    # and the next W4A4 GEMM takes the result
    y = torch.empty(M, 2 * F, device="cuda")
    nv.nvfp4_gemm(L.out_codes, L.out_scales, 100.0, L.up[0][0].contiguous(), L.up[1][0].contiguous(),
                  float(L.up[2][0]), M, 2 * F, K, y)
    wc, wsc, gw = L.up[3][0]
    sc = oracle.scales_from_tc(L.out_scales.cpu().numpy(), M, K)
    assert_gemm_close(y.cpu().numpy(), oracle.gemm(L.out_codes.cpu().numpy(), sc, np.float32(100.0), wc, wsc, gw))


@pytest.mark.parametrize("M", [8, 333])
def test_layer_as_a_graph_on_other_inputs(M):
    L = Layer(M, 512, 256, 16, 4, 1)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        L.run()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        L.run()
    for seed in (5, 6):
        L.branch.copy_(torch.randn(M, 512, generator=torch.Generator().manual_seed(seed)))
        L.run()
        torch.cuda.synchronize()
        eager = [t.clone() for t in L.outputs()]
        for t in L.outputs():
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(L.outputs(), eager):
            assert torch.equal(a, b)
    check_device_error_word()


def test_suites_pass_on_the_debug_build():
    """Every address these kernels compute is inside its buffer (bounds-checked build, in a process of its own)."""
    env = dict(os.environ, NVFP4_DEBUG_BOUNDS="1")
    suites = ["-k", "not past and not more_than", "tests/test_gpu_route.py", "tests/test_gpu_grouped.py", "tests/test_gpu_block_norm.py"]
    if nv.DEBUG_BOUNDS:
        pytest.skip("this is the debug build")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider"] + suites,
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1500)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
