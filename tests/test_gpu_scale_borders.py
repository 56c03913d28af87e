"""Block scales next to an E4M3 border: the format divides the block maximum by
6 with correct rounding, and where a product with 1/6 gives another last bit
the whole block would get the neighbouring scale.  Every quantizer must land
on the divided side, as the oracle does."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
import oracle
from gpu_helpers import check_device_error_word
from grouped_helpers import I32, grouped_scales, offsets_of, oracle_rows

pytestmark = pytest.mark.gpu
F = np.float32
SCALES = np.array([oracle.e4m3_decode(b) for b in range(127)])


def e4m3(t):
    """Nearest E4M3 magnitude (its code), ties to even."""
    t = np.minimum(t.astype(np.float64), 448.0)
    up = np.clip(np.searchsorted(SCALES, t), 1, 126)
    down = up - 1
    du, dd = SCALES[up] - t, t - SCALES[down]
    return np.where((du < dd) | ((du == dd) & (up % 2 == 0)), up, down)


def borders(g, bf16):
    """Block maxima whose scale under global scale g depends on how the sixth is rounded."""
    mid = (SCALES[8:-1] + SCALES[9:]) / 2
    a = (6.0 * mid / float(g)).astype(F)
    if bf16:
        near = (a.view(np.uint32) >> 16).astype(np.int64)[:, None] + np.arange(-1, 2)
        a = np.unique(near << 16).astype(np.uint32).view(F)
    else:
        a = np.unique((a.view(np.uint32).astype(np.int64)[:, None] + np.arange(-8, 9))).astype(np.uint32).view(F)
    divided, product = (a / F(6)).astype(F), (a * (F(1) / F(6))).astype(F)
    return a[e4m3((divided * g).astype(F)) != e4m3((product * g).astype(F))]


def blocks(bf16, K, want):
    """(rows [n, K] on such borders, the global scale of each row): every block's maximum is a border of its row's scale."""
    r = np.random.default_rng(5 + bf16)
    rows, scales = [], []
    while len(rows) < want:
        # bf16 maxima are sparse: scales from a block maximum and a border, so that their products meet
        g = F(r.uniform(20, 400))
        if bf16:
            a0 = (np.array([r.uniform(1, 8)], dtype=F).view(np.uint32) & 0xFFFF0000).view(F)[0]
            m = r.integers(60, 110)
            g = F((SCALES[m] + SCALES[m + 1]) / 2 / float(a0 / F(6)))
        a = borders(g, bf16)
        if not a.size:
            continue
        row = r.uniform(-0.9, 0.9, K).astype(F)
        row[0::16] = r.choice([-1.0, 1.0], K // 16)
        row *= np.repeat(r.choice(a, K // 16), 16)
        rows.append(row)
        scales.append(g)
    x = torch.from_numpy(np.stack(rows))
    if bf16:                                            # maxima stay: they are bf16 values
        x = x.to(torch.bfloat16)
    return x, np.array(scales, dtype=F)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_sixth_is_a_correctly_rounded_quotient(dtype):
    K, n = 96, 40
    x, gs = blocks(dtype == torch.bfloat16, K, n)
    host = x.float().numpy()
    # grouped quantizer: a group a row, each with its own scale; block norm without norms: h = y
    codes, scales = nv.alloc_grouped(n, n, K, "cuda")
    scales.fill_(255)
    nv.nvfp4_grouped_quantize(x.cuda(), offsets_of([1] * n).cuda(), torch.from_numpy(gs).cuda(), codes, scales,
                              row_index=torch.arange(n, dtype=I32, device="cuda"))
    want, per = oracle_rows(host, [1] * n, gs, n, K)
    assert np.array_equal(codes.cpu().numpy(), want)
    assert np.array_equal(scales.cpu().numpy(), grouped_scales(per, n, K)[0])
    for i in range(n):
        c, s = oracle.quantize(host[i:i + 1], gs[i])
        for call in (nv.nvfp4_quantize, None):
            codes, scales = nv.alloc_quantized(1, K, "cuda", nv.SF_ROWMAJOR)
            if call:
                call(x[i:i + 1].cuda(), float(gs[i]), codes, scales, nv.SF_ROWMAJOR)
            else:
                nv.nvfp4_block_norm(x[i:i + 1].cuda(), codes=codes, block_scales=scales, global_scale=float(gs[i]),
                                    layout=nv.SF_ROWMAJOR)
            assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy().reshape(s.shape), s)
    torch.cuda.synchronize()
    check_device_error_word()
