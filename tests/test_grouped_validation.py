"""Argument checks of the router, the grouped layer and the block norm: every
refusal happens before anything touches the GPU (CPU only; pointer values are
never dereferenced on a failing check)."""
import ctypes

import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv

P = ctypes.c_void_p
A16, A4, A1 = P(0x10000), P(0x10004), P(0x10001)
BIG = 1 << 40


def route(x=A16, dt=0, M=4, E=8, k=2, norm=0, ids=A16, w=A16, slots=A16, rows=A16, offs=A16, ws=A16, wsb=BIG):
    return nv.lib().nvfp4_route(x, dt, M, E, k, norm, ids, w, slots, rows, offs, ws, wsb, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(ids=None), dict(w=None), dict(slots=None), dict(rows=None),
                                dict(offs=None), dict(ws=None), dict(M=0), dict(E=0), dict(k=0), dict(k=9),
                                dict(dt=2), dict(norm=2), dict(wsb=0),
                                dict(wsb=nv.nvfp4_route_workspace_bytes(8) - 1)])
def test_route_invalid(kw):
    assert route(**kw) == nv.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(E=513, k=1), dict(E=64, k=33), dict(M=1 << 31, k=1), dict(M=1 << 30, k=2)])
def test_route_unsupported(kw):
    assert route(**kw) == nv.ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["x", "ids", "w", "slots", "rows", "offs", "ws"])
def test_route_alignment(name):
    assert route(**{name: A4}) == nv.ERR_ALIGNMENT


def gquant(x=A16, dt=0, act=0, M=8, K=64, rows=A4, offs=A4, E=4, T=8, gs=A4, codes=A16, sc=A16):
    return nv.lib().nvfp4_grouped_quantize(x, dt, act, M, K, rows, offs, E, T, gs, codes, sc, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(offs=None), dict(gs=None), dict(codes=None), dict(sc=None),
                                dict(dt=2), dict(act=2), dict(M=0), dict(T=0), dict(K=0), dict(K=48), dict(E=0),
                                dict(rows=None, M=7)])
def test_grouped_quantize_invalid(kw):
    assert gquant(**kw) == nv.ERR_INVALID_ARG


def test_grouped_quantize_limits_and_alignment():
    assert gquant(E=513) == nv.ERR_UNSUPPORTED
    assert gquant(M=1 << 31) == nv.ERR_UNSUPPORTED
    assert gquant(T=1 << 31) == nv.ERR_UNSUPPORTED
    assert gquant(T=1 << 27, K=256) == nv.ERR_UNSUPPORTED           # T * K / 16 = 2^31
    for name in ("x", "codes", "sc"):
        assert gquant(**{name: A4}) == nv.ERR_ALIGNMENT
    for name in ("rows", "offs", "gs"):
        assert gquant(**{name: A1}) == nv.ERR_ALIGNMENT


def ggemm(a=A16, sa=A16, ga=A4, w=A16, sw=A16, gw=A4, offs=A4, E=4, T=8, N=16, K=64, out=A16, od=0):
    return nv.lib().nvfp4_grouped_gemm(a, sa, ga, w, sw, gw, offs, E, T, N, K, out, od, None)


@pytest.mark.parametrize("kw", [dict(a=None), dict(sa=None), dict(ga=None), dict(w=None), dict(sw=None), dict(gw=None),
                                dict(offs=None), dict(out=None), dict(T=0), dict(N=0), dict(K=0), dict(K=48),
                                dict(E=0), dict(od=2)])
def test_grouped_gemm_invalid(kw):
    assert ggemm(**kw) == nv.ERR_INVALID_ARG


def test_grouped_gemm_limits_and_alignment():
    assert ggemm(E=513) == nv.ERR_UNSUPPORTED
    assert ggemm(T=1 << 31) == nv.ERR_UNSUPPORTED
    assert ggemm(T=1 << 30, N=1 << 20, E=1) == nv.ERR_UNSUPPORTED   # more tiles than a grid has
    assert ggemm(K=1 << 31) == nv.ERR_UNSUPPORTED
    assert ggemm(E=512, N=1 << 23) == nv.ERR_UNSUPPORTED            # 512 N >= 2^31
    assert ggemm(T=(1 << 31) - 65536, K=1 << 16) == nv.ERR_UNSUPPORTED   # scale chunks beyond 32 bits
    for name in ("a", "sa", "w", "sw", "out"):
        assert ggemm(**{name: A4}) == nv.ERR_ALIGNMENT
    for name in ("ga", "gw", "offs"):
        assert ggemm(**{name: A1}) == nv.ERR_ALIGNMENT


def norm(y=A16, dt=0, M=4, K=64, rows=None, slots=None, sw=None, k=0, pw=None, pwid=0, gate=None, kind=0, res=None,
         rs=1.0, ro=None, pre=A16, eps=1e-6, out=A16, codes=None, sc=None, gs=1.0, layout=1):
    return nv.lib().nvfp4_block_norm(y, dt, M, K, M if rows is None else rows, slots, sw, k, pw, pwid, gate, kind, res,
                                     ctypes.c_float(rs), ro, pre, ctypes.c_float(eps), out, codes, sc,
                                     ctypes.c_float(gs), layout, None)


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kw", [dict(y=None), dict(dt=2), dict(M=0), dict(K=0), dict(K=48), dict(rows=5),
                                dict(slots=A4, k=2), dict(sw=A4, k=2), dict(slots=A4, sw=A4, k=0),
                                dict(slots=A4, sw=A4, k=2, rows=0), dict(gate=A16), dict(kind=1), dict(kind=4, gate=A16),
                                dict(kind=-1, gate=A16), dict(codes=A16), dict(sc=A16), dict(out=None), dict(eps=0.0),
                                dict(eps=-1.0), dict(eps=INF), dict(eps=NAN), dict(rs=INF), dict(rs=NAN),
                                dict(codes=A16, sc=A16, gs=0.0), dict(codes=A16, sc=A16, gs=NAN),
                                dict(codes=A16, sc=A16, layout=2), dict(pw=A16, pwid=0), dict(pw=A16, pwid=24),
                                dict(pw=A16, pwid=128), dict(pw=A16, pwid=8), dict(pw=A16, pwid=48, K=96)])
def test_block_norm_invalid(kw):
    assert norm(**kw) == nv.ERR_INVALID_ARG


def test_block_norm_limits_and_alignment():
    assert norm(K=32800) == nv.ERR_UNSUPPORTED
    assert norm(M=1 << 31) == nv.ERR_UNSUPPORTED
    assert norm(pw=A16, pwid=1024, K=2048) == nv.ERR_INVALID_ARG    # heads of at most 512
    for name in ("y", "pre", "out", "res", "ro"):
        assert norm(**{name: A4}) == nv.ERR_ALIGNMENT
    assert norm(gate=A4, kind=2) == nv.ERR_ALIGNMENT
    assert norm(pw=A4, pwid=64) == nv.ERR_ALIGNMENT
    assert norm(codes=A4, sc=A16) == nv.ERR_ALIGNMENT
    assert norm(slots=A1, sw=A4, k=2) == nv.ERR_ALIGNMENT


@pytest.mark.parametrize("T,E,K", [(1, 1, 32), (1, 512, 64), (127, 3, 96), (128, 1, 5120), (129, 2, 5120),
                                   (32768, 64, 5120), (1000, 24, 1056)])
def test_grouped_scale_bytes_holds_every_split(T, E, K):
    got = nv.nvfp4_grouped_scale_bytes(T, E, K)
    chunk = -(-K // 64) * 512
    assert got % chunk == 0
    # the worst split: as many groups as possible one row over a multiple of 128
    n = min(E, T)
    worst = max(sum(-(-r // 128) for r in [1] * (n - 1) + [T - n + 1]), -(-T // 128))
    extra = (T - n) // 128
    worst = max(worst, n + extra)
    assert got // chunk >= worst
    assert got // chunk <= T // 128 + n


def test_size_functions_refuse():
    assert nv.nvfp4_grouped_scale_bytes(0, 1, 64) == 0
    assert nv.nvfp4_grouped_scale_bytes(1, 0, 64) == 0
    assert nv.nvfp4_grouped_scale_bytes(1, 513, 64) == 0
    assert nv.nvfp4_grouped_scale_bytes(1, 1, 24) == 0
    assert nv.nvfp4_route_workspace_bytes(0) == 0
    assert nv.nvfp4_route_workspace_bytes(513) == 0


def test_binding_refuses_host_tensors():
    i32 = torch.int32
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        nv.nvfp4_route(torch.zeros(2, 4), 0, torch.zeros(2, 1, dtype=i32), torch.zeros(2, 1),
                       torch.zeros(2, 1, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(5, dtype=i32),
                       torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        nv.nvfp4_block_norm(torch.zeros(2, 64), out=torch.zeros(2, 64))
