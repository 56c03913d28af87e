"""Block norm against a 64-bit form, with tolerances counted from its FP32
steps, and its codes against the oracle's encoding of its own dense output."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_10_b200 as nv
import oracle
from gpu_helpers import check_device_error_word

pytestmark = pytest.mark.gpu
EPS = 1e-6
ULP = 2.0 ** -24


def make(M, K, dtype, k=0, post=0, gate=nv.GATE_NONE, residual=True, pre=True, seed=0):
    g = torch.Generator().manual_seed(seed + M * 7 + K)
    rn = lambda *s: torch.randn(*s, generator=g)                                   # noqa: E731
    rows = M if not k else 2 * M + 1
    a = dict(y=(3 * rn(rows, K)).to(dtype).cuda())
    if k:
        a["slots"] = torch.randint(-1, rows, (M, k), generator=g, dtype=torch.int32).cuda()
        a["slot_weights"] = torch.rand(M, k, generator=g).cuda()
    if post:
        a["post_weight"] = (1 + 0.3 * rn(post)).cuda()
    if gate != nv.GATE_NONE:
        a["gate"], a["gate_kind"] = (4 * rn(M, K)).to(dtype).cuda(), gate
    if residual:
        a["residual"], a["residual_scale"] = rn(M, K).to(dtype).cuda(), 0.7
    if pre:
        a["pre_weight"] = (1 + 0.3 * rn(K)).cuda()
    return a


def reference(a):
    """(v, bound of v's FP32 error, h, bound of h's) in float64."""
    d = lambda t: t.double().cpu().numpy()                                         # noqa: E731
    y = d(a["y"])
    K = y.shape[1]
    k = 0
    mag = np.abs(y)
    if "slots" in a:
        s, w = a["slots"].cpu().numpy(), d(a["slot_weights"])
        k = s.shape[1]
        b, mag = np.zeros((s.shape[0], K)), np.zeros((s.shape[0], K))
        for j in range(k):
            t = np.where(s[:, j:j + 1] >= 0, w[:, j:j + 1], 0.0) * y[np.maximum(s[:, j], 0)]
            b += t
            mag += np.abs(t)
    else:
        b = y
    err = k * ULP * mag                                # one rounding an addend
    # a norm: the mean of squares sums 16 a thread, then trees (some 30 roundings, halved by the square root), rsqrt 2
    # ulp, three products; an error of its input moves each value and the norm
    N = 32 * ULP
    if "post_weight" in a:
        width = a["post_weight"].numel()
        hb, he = b.reshape(-1, width), err.reshape(-1, width)
        r = 1 / np.sqrt((hb ** 2).mean(1, keepdims=True) + EPS)
        pw = d(a["post_weight"])
        rel = np.sqrt((he ** 2).mean(1, keepdims=True)) * r
        out = hb * r * pw
        err = (he * r * np.abs(pw) + (N + rel) * np.abs(out)).reshape(b.shape)
        b = out.reshape(b.shape)
    if "gate" in a:
        z = d(a["gate"])
        sg = 1 / (1 + np.exp(-z))
        f = {nv.GATE_LINEAR: z, nv.GATE_SIGMOID: sg, nv.GATE_SILU: z * sg}[a["gate_kind"]]
        err = err * np.abs(f) + 8 * ULP * np.abs(b * f)
        b = b * f
    sc = float(np.float32(a.get("residual_scale", 1.0)))
    r0 = d(a["residual"]) if "residual" in a else 0.0
    v = r0 + sc * b
    verr = abs(sc) * err + 2 * ULP * (np.abs(v) + np.abs(sc * b))
    if "pre_weight" not in a:
        return v, verr, v, verr
    r = 1 / np.sqrt((v ** 2).mean(1, keepdims=True) + EPS)
    w = d(a["pre_weight"])
    h = v * r * w
    rel = np.sqrt((verr ** 2).mean(1, keepdims=True)) * r
    return v, verr, h, verr * r * np.abs(w) + (N + rel) * np.abs(h)


def close(got, want, err, dtype, what):
    half = torch.finfo(dtype).eps / 2
    tol = err + half * (np.abs(want) + err) + 1e-38
    bad = np.abs(got.double().cpu().numpy() - want) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} beyond the bound"


def check(a, dtype, quant=True, layout=nv.SF_TCGEN05, g=30.0):
    M = a["slots"].shape[0] if "slots" in a else a["y"].shape[0]
    K = a["y"].shape[1]
    v, verr, h, herr = reference(a)
    ro, out = torch.empty(M, K, dtype=dtype, device="cuda"), torch.empty(M, K, dtype=dtype, device="cuda")
    codes, scales = nv.alloc_quantized(M, K, "cuda", layout)
    codes.fill_(255)
    scales.fill_(255)
    nv.nvfp4_block_norm(**a, eps=EPS, residual_out=ro, out=out, codes=codes, block_scales=scales, global_scale=g,
                        layout=layout)
    torch.cuda.synchronize()
    check_device_error_word()
    close(ro, v, verr, dtype, "residual")
    close(out, h, herr, dtype, "out")
    # the unrounded h: the same call on the FP32 copies of the inputs gives it as its output
    f = {n: t.float() if torch.is_tensor(t) and t.dtype == torch.bfloat16 else t for n, t in a.items()}
    h32 = torch.empty(M, K, device="cuda")
    nv.nvfp4_block_norm(**f, eps=EPS, out=h32)
    torch.cuda.synchronize()
    assert torch.equal(out, h32.to(dtype))
    c, s = oracle.quantize(h32.cpu().numpy(), np.float32(g))
    assert np.array_equal(codes.cpu().numpy(), c)
    want = oracle.scales_to_tc(s, K) if layout == nv.SF_TCGEN05 else s.reshape(-1)
    assert np.array_equal(scales.cpu().numpy(), want)


SIZES = [(1, 32), (3, 96), (130, 64), (7, 512), (5, 544), (9, 1024), (4, 1056), (2, 5120), (200, 4096), (3, 8192),
         (2, 8224), (3, 17408), (2, 32768)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_residual_and_norm(M, K, dtype):
    check(make(M, K, dtype), dtype)


@pytest.mark.parametrize("M,K", [(1, 32), (6, 1024), (11, 5120), (3, 17408)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", [nv.GATE_LINEAR, nv.GATE_SIGMOID, nv.GATE_SILU])
def test_sandwich_with_gate(M, K, dtype, gate):
    check(make(M, K, dtype, post=K, gate=gate), dtype, layout=nv.SF_ROWMAJOR)


# long rows, more than two an SM: staged through shared memory, several to a CTA, in rings of 1 to 3 rows
@pytest.mark.parametrize("M,K", [(297, 16384), (460, 17408), (300, 18464), (300, 18944), (300, 32768)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_long_rows(M, K, dtype):
    check(make(M, K, dtype, post=K, gate=nv.GATE_SILU), dtype)


@pytest.mark.parametrize("M,K,over", [(600, 16384, dict()), (460, 16416, dict(residual=False)),
                                      (460, 16384, dict(post=512, gate=nv.GATE_SILU, residual=False, pre=False)),
                                      (460, 17408, dict(post=256)), (460, 18944, dict(residual=False, pre=False)),
                                      (300, 24576, dict(post=24576, pre=False, gate=nv.GATE_LINEAR, residual=False)),
                                      (300, 32768, dict(post=32768, residual=False)), (330, 32768, dict(pre=False))])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_long_rows_with_fewer_inputs(M, K, over, dtype):
    check(make(M, K, dtype, **over), dtype, layout=nv.SF_ROWMAJOR)


@pytest.mark.parametrize("K", [5120, 17408])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_row_does_not_depend_on_how_many_there_are(K, dtype):
    a = make(310, K, dtype, post=K, gate=nv.GATE_SIGMOID)
    out, few = (torch.empty(310, K, dtype=dtype, device="cuda") for _ in range(2))
    nv.nvfp4_block_norm(**a, out=out)
    for i in range(0, 310, 31):
        part = {n: t[i:i + 31] if torch.is_tensor(t) and t.dim() == 2 else t for n, t in a.items()}
        nv.nvfp4_block_norm(**part, out=few[i:i + 31])
    assert torch.equal(out, few)
    torch.cuda.synchronize()
    check_device_error_word()


@pytest.mark.parametrize("into", ["residual", "gate", "y"])
def test_many_long_rows_in_place(into):
    M, K = 320, 17408
    a = make(M, K, torch.float32, post=K, gate=nv.GATE_SILU)
    want_r, want = torch.empty(M, K, device="cuda"), torch.empty(M, K, device="cuda")
    nv.nvfp4_block_norm(**a, residual_out=want_r, out=want)
    other = torch.empty(M, K, device="cuda")
    b = {n: t.clone() if torch.is_tensor(t) else t for n, t in a.items()}
    nv.nvfp4_block_norm(**b, residual_out=b[into], out=other)
    assert torch.equal(b[into], want_r) and torch.equal(other, want)
    b = {n: t.clone() if torch.is_tensor(t) else t for n, t in a.items()}
    nv.nvfp4_block_norm(**b, residual_out=other, out=b[into])
    assert torch.equal(other, want_r) and torch.equal(b[into], want)


@pytest.mark.parametrize("K,width", [(32, 16), (64, 32), (512, 64), (768, 256), (1024, 512), (4096, 128), (5120, 256),
                                     (8704, 512), (512, 512)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_heads(K, width, dtype):
    check(make(37, K, dtype, post=width, gate=nv.GATE_SILU, residual=False, pre=False), dtype)


@pytest.mark.parametrize("k", [1, 3, 8, 11])
@pytest.mark.parametrize("K", [64, 1056, 9216])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_combine(k, K, dtype):
    check(make(19, K, dtype, k=k, post=K if k == 3 else 0), dtype)


def test_rows_of_zeros_and_empty_slots():
    K = 256
    a = make(4, K, torch.float32, k=2)
    a["slots"].fill_(-1)
    a["slot_weights"].fill_(float("nan"))               # a weight at -1 is not read into the sum
    a["residual"].zero_()
    out = torch.full((4, K), 9.0, device="cuda")
    codes, scales = nv.alloc_quantized(4, K, "cuda")
    nv.nvfp4_block_norm(**a, out=out, codes=codes, block_scales=scales)
    assert out.eq(0).all() and scales.eq(0).all() and codes.eq(0).all()


def test_slot_outside_y_is_reported_and_skipped():
    K = 64
    a = make(2, K, torch.float32, k=2, residual=False, pre=False)
    a["slots"].copy_(torch.tensor([[0, 5], [-2, 1]], dtype=torch.int32))     # y has 5 rows
    a["slot_weights"].fill_(1.0)
    out = torch.empty(2, K, device="cuda")
    nv.nvfp4_block_norm(**a, out=out)
    assert nv.nvfp4_last_device_error() == nv.ERR_DEVICE
    assert torch.equal(out[0], a["y"][0]) and torch.equal(out[1], a["y"][1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_outputs_in_place_of_inputs(dtype):
    a = make(33, 1088, dtype, post=1088, gate=nv.GATE_SIGMOID)
    ro, out = torch.empty_like(a["y"]), torch.empty_like(a["y"])
    nv.nvfp4_block_norm(**a, residual_out=ro, out=out)
    nv.nvfp4_block_norm(**a, residual_out=a["residual"], out=a["y"])
    assert torch.equal(a["residual"], ro) and torch.equal(a["y"], out)


def test_on_another_stream_and_captured():
    a = make(64, 5120, torch.bfloat16, k=4)
    want, out = torch.empty(64, 5120, dtype=torch.bfloat16, device="cuda"), torch.empty(64, 5120, dtype=torch.bfloat16,
                                                                                       device="cuda")
    nv.nvfp4_block_norm(**a, out=want)
    torch.cuda.synchronize()
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        nv.nvfp4_block_norm(**a, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def shifted(t):
    """A copy of t that starts 16 bytes past a 32-byte boundary."""
    n = 16 // t.element_size()
    buf = torch.empty(t.numel() + 2 * n, dtype=t.dtype, device="cuda")
    out = buf[n:n + t.numel()].view(t.shape).copy_(t)
    assert out.data_ptr() % 32 == 16
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [96, 1056, 9216])
def test_buffers_on_16_byte_boundaries(K, dtype):
    a = make(9, K, dtype, k=3, post=K, gate=nv.GATE_SILU)
    b = {n: shifted(t) if torch.is_tensor(t) and t.is_floating_point() and n != "slot_weights" else t
         for n, t in a.items()}
    want, out = torch.empty(9, K, dtype=dtype, device="cuda"), shifted(torch.zeros(9, K, dtype=dtype, device="cuda"))
    nv.nvfp4_block_norm(**a, out=want)
    nv.nvfp4_block_norm(**b, out=out)
    assert torch.equal(out, want)


def test_gate_far_out_on_both_sides():
    K = 64
    y = torch.ones(1, K, device="cuda")
    z = torch.linspace(-120.0, 120.0, K, device="cuda").view(1, K)
    for kind in (nv.GATE_SIGMOID, nv.GATE_SILU):
        out = torch.empty(1, K, device="cuda")
        nv.nvfp4_block_norm(y, gate=z, gate_kind=kind, out=out)
        d = z.double()
        want = torch.sigmoid(d) * (d if kind == nv.GATE_SILU else 1.0)
        # exp 2 ulp, quotient 2 ulp, a product; the exponent's own rounding is expf's; below 2^-126 flushed
        assert ((out.double() - want).abs() <= 8 * ULP * want.abs() + 2.0 ** -125 * (1 + d.abs())).all()


def test_more_than_2_31_elements():
    M, K = 140_000, 16_384
    y = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(4, K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    at = torch.tensor([0, 1, 131_073, M - 1], device="cuda")          # row 131072 starts at element 2^31
    y.zero_()
    y[at] = rows
    w = torch.ones(K, device="cuda")
    small = torch.empty(4, K, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_block_norm(rows, pre_weight=w, out=small)
    nv.nvfp4_block_norm(y, pre_weight=w, out=y)
    assert torch.equal(y[at], small)
    assert y[2].eq(0).all() and y[M - 2].eq(0).all()


def test_staged_rows_survive_a_wait_that_runs_out():
    M, K = 320, 17408
    a = make(M, K, torch.float32, post=K, gate=nv.GATE_SILU)
    want, out = torch.empty(M, K, device="cuda"), torch.empty(M, K, device="cuda")
    nv.nvfp4_block_norm(**a, out=want)
    torch.cuda.synchronize()
    try:
        nv.nvfp4_set_wait_timeout_ns(1)
        nv.nvfp4_block_norm(**a, out=out)
        # (a copy may have landed at the first look)
        assert nv.nvfp4_last_device_error() in (nv.OK, nv.ERR_TIMEOUT)
    finally:
        nv.nvfp4_set_wait_timeout_ns(0)
    nv.nvfp4_block_norm(**a, out=out)
    torch.cuda.synchronize()
    check_device_error_word()
    assert torch.equal(out, want)
