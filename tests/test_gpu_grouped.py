"""Grouped quantizer and grouped GEMM against the oracle, expert by expert."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
import oracle
from gpu_helpers import assert_gemm_close, check_device_error_word
from grouped_helpers import I32, activation, experts, grouped_scales, offsets_of, oracle_rows, product

pytestmark = pytest.mark.gpu

SPLITS = {
    "one row": [1],
    "one group": [37],
    "empty ends": [0, 0, 5, 0, 16, 17, 0],
    "tile edges": [128, 1, 127, 129, 0, 256, 255, 257],
    "all empty": [0, 0, 0],
    "skewed": [0, 700, 3, 0, 1, 64, 33, 2],
}


def alpha_scales(E, base=100.0):
    return torch.tensor([base * (1 + 0.25 * (e % 5)) for e in range(E)], dtype=torch.float32)


# ------------------------------------------------------------------ quantizer

@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("K", [32, 64, 352, 1088])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantizer_is_bitwise_the_oracle(split, K, dtype):
    rows = SPLITS[split]
    E, total = len(rows), sum(rows)
    T = total + 3                                        # three rows behind the last group
    gs = alpha_scales(E)
    src = torch.from_numpy(activation(max(1, total) + 5, K, K + total)).to(dtype)
    idx = torch.from_numpy(np.random.default_rng(1).integers(0, src.shape[0], T).astype(np.int32))
    codes, scales = nv.alloc_grouped(T, E, K, "cuda")
    codes.fill_(255)
    scales.fill_(255)
    nv.nvfp4_grouped_quantize(src.cuda(), offsets_of(rows).cuda(), gs.cuda(), codes, scales, row_index=idx.cuda())
    torch.cuda.synchronize()
    check_device_error_word()
    x = src.float().numpy()[idx.numpy()]
    want, per = oracle_rows(x, rows, gs.numpy(), T, K)
    assert np.array_equal(codes.cpu().numpy(), want)     # rows behind the groups are left as they were
    buf, _ = grouped_scales(per, T, K)
    assert np.array_equal(scales.cpu().numpy(), buf)
    if total:                                            # without an index: row t of x
        codes2, scales2 = torch.full_like(codes, 255), torch.full_like(scales, 255)
        nv.nvfp4_grouped_quantize(src[idx.long()].cuda(), offsets_of(rows).cuda(), gs.cuda(), codes2, scales2)
        assert torch.equal(codes2, codes) and torch.equal(scales2, scales)


def nearest_check(codes, scales, h, g):
    """codes and E4M3 scales are the NVFP4 encoding of values within 16 * 2^-24 of h (relative): each is a nearest
    grid value, or so close to the border that such a difference decides."""
    M, K = h.shape
    rel = 16 * 2.0 ** -24
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    e4 = np.array([oracle.e4m3_decode(b) for b in range(127)])
    s = e4[scales]
    t = np.abs(h).reshape(M, -1, 16).max(2) / 6.0 * g
    t = np.minimum(t, 448.0)
    best = np.abs(t[..., None] - e4).min(-1)
    assert np.all(np.abs(t - s) <= best + 2 * rel * t)
    nib = np.stack([codes & 15, codes >> 4], 2).reshape(M, K)
    mag, sign = grid[nib & 7], np.where(nib & 8, -1.0, 1.0)
    sf = np.repeat(s, 16, 1)
    y = np.where(sf > 0, h * (g / np.where(sf > 0, sf, 1.0)), 0.0)
    d = np.abs(np.minimum(np.abs(y), 6.0) - mag)
    near = np.abs(np.minimum(np.abs(y), 6.0)[..., None] - grid).min(-1)
    assert np.all(d <= near + 2 * rel * np.abs(y))
    assert np.all((mag == 0) | (sign == np.sign(y)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [32, 352])
def test_swiglu(dtype, K):
    rows = [0, 3, 130, 0, 40]
    E, T = len(rows), sum(rows) + 2
    r = np.random.default_rng(K)
    x = torch.from_numpy(r.standard_normal((T, 2 * K)).astype(np.float32) * 3).to(dtype)
    x[0, :4] = torch.tensor([-100.0, 100.0, 0.0, -0.0])          # far ends of the sigmoid
    gs = alpha_scales(E)
    codes, scales = nv.alloc_grouped(T, E, K, "cuda")
    scales.fill_(255)
    nv.nvfp4_grouped_quantize(x.cuda(), offsets_of(rows).cuda(), gs.cuda(), codes, scales, act=nv.ACT_SWIGLU)
    torch.cuda.synchronize()
    check_device_error_word()
    a, b = x.double().numpy()[:, :K], x.double().numpy()[:, K:]
    h = a / (1 + np.exp(-a)) * b
    per = [np.zeros((n, K // 16), dtype=np.uint8) for n in rows]
    _, mask = grouped_scales(per, T, K)
    got, at, blk = scales.cpu().numpy(), 0, 0
    assert np.all(got[~mask] == 255)
    chunk = -(-K // 64) * 512
    for e, n in enumerate(rows):
        if not n:
            continue
        nb = -(-n // 128)
        s = oracle.scales_from_tc(np.where(mask, got, 0)[blk * chunk:(blk + nb) * chunk].copy(), n, K)
        nearest_check(codes.cpu().numpy()[at:at + n], s, h[at:at + n], float(gs[e]))
        at += n
        blk += nb


def test_bad_row_index_is_reported_and_quantized_as_zeros():
    K = 64
    x = torch.ones(4, K, device="cuda")
    idx = torch.tensor([0, 4, -1, 3], dtype=I32, device="cuda")
    codes, scales = nv.alloc_grouped(4, 1, K, "cuda")
    nv.nvfp4_grouped_quantize(x, offsets_of([4]).cuda(), torch.ones(1, device="cuda"), codes, scales, row_index=idx)
    assert nv.nvfp4_last_device_error() == nv.ERR_DEVICE
    assert codes[1].eq(0).all() and codes[2].eq(0).all() and not codes[0].eq(0).any() and not codes[3].eq(0).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", [nv.ACT_NONE, nv.ACT_SWIGLU])
def test_source_on_a_16_byte_boundary(dtype, act):
    rows, K = [3, 0, 40], 96
    E, T = 3, 43
    x = torch.randn(T, K * (2 if act else 1), generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    n = 16 // x.element_size()
    y = torch.empty(x.numel() + 2 * n, dtype=dtype, device="cuda")[n:n + x.numel()].view(x.shape).copy_(x)
    assert y.data_ptr() % 32 == 16
    got = []
    for src in (x, y):
        codes, scales = nv.alloc_grouped(T, E, K, "cuda")
        scales.zero_()
        nv.nvfp4_grouped_quantize(src, offsets_of(rows).cuda(), alpha_scales(E).cuda(), codes, scales, act=act)
        got.append((codes, scales))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_codes_past_4_gib():
    T, K = 1_100_000, 8192                               # 4.5 GB of codes
    x = torch.randn(3, K, generator=torch.Generator().manual_seed(3)).cuda()
    idx = torch.zeros(T, dtype=I32, device="cuda")
    idx[-1], idx[T // 2] = 2, 1
    codes, scales = nv.alloc_grouped(T, 2, K, "cuda")
    g = torch.tensor([200.0, 300.0], device="cuda")
    nv.nvfp4_grouped_quantize(x, offsets_of([5, T - 5]).cuda(), g, codes, scales, row_index=idx)
    torch.cuda.synchronize()
    check_device_error_word()
    for row, src, gs in ((0, 0, 200.0), (5, 0, 300.0), (T // 2, 1, 300.0), (T - 2, 0, 300.0), (T - 1, 2, 300.0)):
        c, s = oracle.quantize(x[src:src + 1].cpu().numpy(), np.float32(gs))
        assert np.array_equal(codes[row].cpu().numpy(), c[0]), row
        pos = row if row < 5 else 128 + row - 5
        j = np.arange(K // 16)
        off = ((pos >> 7) * (K // 64) + (j >> 2)) * 512 + (pos & 31) * 16 + ((pos >> 5) & 3) * 4 + (j & 3)
        assert np.array_equal(scales[torch.from_numpy(off).cuda()].cpu().numpy(), s[0]), row


# ------------------------------------------------------------------ GEMM

def gemm_operands(rows, N, K, seed=0, T=None):
    """Device operands of one grouped product, and its oracle result (computed when asked for)."""
    E, total = len(rows), sum(rows)
    T = max(1, total + 5) if T is None else T
    wc, ws, gw, host = experts(E, N, K, seed + 1)
    ga = alpha_scales(E)
    x = activation(max(1, total), K, seed + 2)
    codes, per = oracle_rows(x, rows, ga.numpy(), T, K)
    buf, _ = grouped_scales(per, T, K)
    a = (torch.from_numpy(codes).cuda(), torch.from_numpy(buf).cuda(), ga.cuda(), wc, ws, gw, offsets_of(rows).cuda())
    return a, T, lambda: product(codes, per, ga.numpy(), host, rows, N)


def run_gemm(rows, N, K, out_dtype, seed=0, T=None):
    a, T, ref = gemm_operands(rows, N, K, seed, T)
    out = torch.full((T, N), 777.0, dtype=out_dtype, device="cuda")
    nv.nvfp4_grouped_gemm(*a, out)
    torch.cuda.synchronize()
    check_device_error_word()
    return out, ref


@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("N,K", [(8, 32), (129, 96), (200, 352), (256, 1088)])
def test_small_tiles_match_the_oracle(split, N, K):
    rows = SPLITS[split]
    T = 128 * len(rows) - 1                              # under 128 rows a group on average
    if sum(rows) > T:
        pytest.skip("this split has more rows a group")
    out, ref = run_gemm(rows, N, K, torch.float32, T=T)
    want, total = ref(), sum(rows)
    if total:
        assert_gemm_close(out[:total].cpu().numpy(), want, split)
    assert out[total:].eq(777.0).all()                   # rows behind the groups are left as they were
    half, _ = run_gemm(rows, N, K, torch.bfloat16, T=T)
    assert torch.equal(half[:total], out[:total].to(torch.bfloat16))


@pytest.mark.parametrize("split", SPLITS)
@pytest.mark.parametrize("N,K", [(8, 32), (129, 96), (200, 352), (512, 1088)])
def test_large_tiles_match_the_oracle(split, N, K):
    rows = SPLITS[split]
    T = max(128 * len(rows), sum(rows) + 5)              # 128 rows a group and more
    out, ref = run_gemm(rows, N, K, torch.float32, T=T)
    want, total = ref(), sum(rows)
    if total:
        assert_gemm_close(out[:total].cpu().numpy(), want, split)
    assert out[total:].eq(777.0).all()
    half, _ = run_gemm(rows, N, K, torch.bfloat16, T=T)
    assert torch.equal(half[:total], out[:total].to(torch.bfloat16))


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [[300, 48, 256, 100, 511, 64, 65, 31], [48, 100, 17, 128, 90, 64, 63, 1]])
@pytest.mark.parametrize("K", [32, 96])
def test_many_ragged_tiles_a_pair(rows, K, out_dtype):
    """Short K and some tens of ragged tiles a CTA pair: every staging buffer is reused behind a TMA store and behind
    masked stores, in every order."""
    rows, N = rows * 5, 4608
    a, T, ref = gemm_operands(rows, N, K)
    want, first = ref(), None
    for _ in range(5):
        out = torch.full((T, N), 777.0, dtype=out_dtype, device="cuda")
        nv.nvfp4_grouped_gemm(*a, out)
        torch.cuda.synchronize()
        check_device_error_word()
        if first is None:
            first = out
            got = out[:sum(rows)].double().cpu().numpy()
            if out_dtype == torch.float32:
                assert_gemm_close(got, want)
            tol = (2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -20) * np.abs(want) + 1e-5 * np.abs(want).max()
            assert np.all(np.abs(got - want) <= tol)
        assert torch.equal(out, first)


@pytest.mark.parametrize("E,N,K", [(512, 40, 64), (130, 136, 160)])
def test_many_groups(E, N, K):
    r = np.random.default_rng(E)
    rows = r.integers(0, 3, E).tolist()
    out, ref = run_gemm(rows, N, K, torch.float32)
    assert_gemm_close(out[:sum(rows)].cpu().numpy(), ref(), f"{E} groups")


@pytest.mark.parametrize("rows", [[8, 0, 3], [40, 0, 60], [300, 700, 200]])
def test_a_group_equals_its_own_gemm(rows):
    """Each group's rows agree with nvfp4_gemm on that expert alone."""
    E, N, K = len(rows), 264, 640
    out, _ = run_gemm(rows, N, K, torch.float32, seed=9)
    wc, ws, gw, _ = experts(E, N, K, 10)
    ga = alpha_scales(E)
    x = activation(sum(rows), K, 11)
    at = 0
    for e, n in enumerate(rows):
        if n:
            c, s = oracle.quantize(np.ascontiguousarray(x[at:at + n]), np.float32(ga[e]))
            one = torch.empty(n, N, device="cuda")
            nv.nvfp4_gemm(torch.from_numpy(c).cuda(), torch.from_numpy(oracle.scales_to_tc(s, K)).cuda(), float(ga[e]),
                          wc[e].contiguous(), ws[e].contiguous(), float(gw[e]), n, N, K, one)
            assert_gemm_close(out[at:at + n].cpu().numpy(), one.double().cpu().numpy(), f"group {e}")
        at += n


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_output_past_2_31_elements(out_dtype):
    rows, N, K = [30_000, 40_000], 32_768, 32
    T = sum(rows)
    wc, ws, gw, host = experts(2, N, K, 3)
    ga = alpha_scales(2)
    x = activation(8, K, 4)
    at = [0, 29_999, 30_000, 30_128, 65_535, 65_537, 69_998, 69_999]
    full = np.zeros((T, K), dtype=np.float32)
    full[at] = x
    codes, per = oracle_rows(full, rows, ga.numpy(), T, K)
    buf, _ = grouped_scales(per, T, K)
    out = torch.empty(T, N, dtype=out_dtype, device="cuda")
    nv.nvfp4_grouped_gemm(torch.from_numpy(codes).cuda(), torch.from_numpy(buf).cuda(), ga.cuda(), wc, ws, gw,
                          offsets_of(rows).cuda(), out)
    torch.cuda.synchronize()
    check_device_error_word()
    for r in at:
        e = 0 if r < rows[0] else 1
        c, s, g = host[e]
        ref = oracle.gemm(codes[r:r + 1], per[e][r - e * rows[0]][None], np.float32(ga[e]), c, s, g)
        got = out[r:r + 1].double().cpu().numpy()
        tol = (2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -20) * np.abs(ref) + 1e-5 * np.abs(ref).max()
        assert np.all(np.abs(got - ref) <= tol), r
    assert out[1].eq(0).all() and out[T - 3].eq(0).all()


def test_result_does_not_depend_on_timing():
    rows = [3, 0, 17, 1, 64, 128, 9, 2]
    first, _ = run_gemm(rows, 512, 2048, torch.float32)
    for _ in range(5):
        again, _ = run_gemm(rows, 512, 2048, torch.float32)
        assert torch.equal(first, again)


BAD = {"start": [1, 4, 8], "decrease": [0, 6, 4], "past T": [0, 4, 9], "negative": [0, -1, 8]}


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("T,E", [(8, 2), (500, 2)])
def test_bad_offsets_are_reported_and_nothing_is_written(bad, T, E):
    N, K = 64, 64
    offs = torch.tensor(BAD[bad], dtype=I32, device="cuda")
    if bad == "past T":
        offs[-1] = T + 1
    codes, scales = nv.alloc_grouped(T, E, K, "cuda")
    codes.fill_(17)
    scales.fill_(17)
    one = torch.ones(E, device="cuda")
    nv.nvfp4_grouped_quantize(torch.ones(T, K, device="cuda"), offs, one, codes, scales)
    assert nv.nvfp4_last_device_error() == nv.ERR_DEVICE
    assert codes.eq(17).all() and scales.eq(17).all()
    wc, ws, gw, _ = experts(E, N, K, 1)
    out = torch.full((T, N), 5.0, device="cuda")
    nv.nvfp4_grouped_gemm(codes, scales, one, wc, ws, gw, offs, out)
    assert nv.nvfp4_last_device_error() == nv.ERR_DEVICE
    assert out.eq(5.0).all()


def test_two_captured_graphs_run_at_once():
    rows, N, K = [5, 0, 30, 2], 384, 2048
    E, T = len(rows), sum(rows)
    wc, wsc, gw, host = experts(E, N, K, 5)
    ga, offs = alpha_scales(E).cuda(), offsets_of(rows).cuda()
    st = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs, refs, keep = [], [], [], []
    for i in range(2):
        codes, per = oracle_rows(activation(T, K, 20 + i), rows, ga.cpu().numpy(), T, K)
        buf, _ = grouped_scales(per, T, K)
        c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(buf).cuda()
        out = torch.empty(T, N, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st[0]):          # captured on one stream, replayed on two
            nv.nvfp4_grouped_gemm(c, s, ga, wc, wsc, gw, offs, out)
        graphs.append(g)
        outs.append(out)
        refs.append(product(codes, per, ga.cpu().numpy(), host, rows, N))
        keep.append((c, s))
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    check_device_error_word()
    for i in range(2):
        assert_gemm_close(outs[i].cpu().numpy(), refs[i], f"graph {i}")


def test_binding_refuses_wrong_shapes_and_types():
    codes, scales = nv.alloc_grouped(4, 2, 64, "cuda")
    one, offs = torch.ones(2, device="cuda"), offsets_of([2, 2]).cuda()
    x = torch.ones(4, 64, device="cuda")
    with pytest.raises(ValueError):
        nv.nvfp4_grouped_quantize(x, offs.long(), one, codes, scales)
    with pytest.raises(ValueError):
        nv.nvfp4_grouped_quantize(x, offs, one, codes, scales, act=nv.ACT_SWIGLU)
    with pytest.raises(ValueError):
        nv.nvfp4_grouped_quantize(x, offs, one, codes, scales[:-1])
    with pytest.raises(ValueError):
        nv.nvfp4_grouped_quantize(x.t(), offs, one, codes, scales)
    wc, ws, gw, _ = experts(2, 64, 64, 1)
    with pytest.raises(ValueError):
        nv.nvfp4_grouped_gemm(codes, scales, one, wc, ws, gw, offs, torch.empty(4, 63, device="cuda"))
    with pytest.raises(ValueError):
        nv.nvfp4_grouped_gemm(codes, scales, one, wc, ws, gw[:1], offs, torch.empty(4, 64, device="cuda"))
