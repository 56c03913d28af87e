"""The plain torch forms of the expert-grouped workloads against the kernels,
number by number.  The one step in which they part is the sixth of a block's
maximum: the format divides, and torch's division of a GPU tensor by a host
number is a product with the reciprocal, which puts a block next to an E4M3
border on the other side once in some 100000 to a million blocks."""
import pytest
import torch

import perf.operators as forms
from gpu_helpers import check_device_error_word

pytestmark = pytest.mark.gpu


def divided(x, gs):
    """forms._quantize with the quotient taken on the device."""
    b = x.view(x.shape[0], -1, 16)
    amax = b.abs().amax(2)
    s = (amax / torch.full_like(amax, 6.0) * gs).clamp(max=forms.E4M3_MAX).to(torch.float8_e4m3fn)
    sf = s.float()
    y = b * torch.where(sf > 0, gs / sf, torch.zeros_like(sf)).unsqueeze(2)
    return (forms._round_e2m1(y.abs()) | (torch.signbit(b).to(torch.uint8) << 3)).view(x.shape), s


def both(case, seed, monkeypatch):
    """(kernel's output, plain form's, the sum of magnitudes that each number is made of)"""
    s = forms.prepare(case, seed)
    monkeypatch.setattr(forms, "own", False)
    want = forms.run(s).double()
    m = dict(s, w_codes=s["w_codes"] & 0x77)               # without signs: the codes of magnitudes
    if "x" in s:
        m["x"] = s["x"].abs()
    else:
        m["a_codes"] = s["a_codes"] & 0x77
    size = forms.run(m).double()
    monkeypatch.setattr(forms, "own", True)
    got = forms.run(s).double()
    torch.cuda.synchronize()
    check_device_error_word()
    return got, want, size


# each of K additions rounds once on either side, FP32: 2^-24 of at most the sum of magnitudes
@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("case", [dict(M=1574, k=5, E=29, N=72, K=128, x="bf16"), dict(M=655, k=6, E=17, N=131, K=160, x="f32"),
                                  dict(M=3, k=4, E=40, N=264, K=1056, x="f32"), dict(M=2186, k=2, E=2, N=64, K=96, x="f32")])
def test_linear(case, seed, monkeypatch):
    monkeypatch.setattr(forms, "_quantize", divided)
    got, want, size = both(dict(op="linear", act="none", out="f32", **case), seed, monkeypatch)
    assert ((got - want).abs() <= 2 * case["K"] * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("case", [dict(T=7, spare=3, E=12, N=72, K=96), dict(T=900, spare=0, E=5, N=300, K=544)])
def test_gemm(case, monkeypatch):
    got, want, size = both(dict(op="gemm", out="f32", skew=1.0, **case), 1, monkeypatch)
    assert ((got - want).abs() <= 2 * case["K"] * 2.0 ** -24 * size).all()
